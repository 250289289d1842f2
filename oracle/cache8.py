"""fp64 oracle of the rotary positions and of the 8-bit paged cache: plain
definitions in NumPy, sharing nothing with the CUDA path."""

from __future__ import annotations

import numpy as np

from .attention import fp8_e4m3_decode, gather_paged_kv, paged_decode

E_MIN, E_MAX = -100, 119

# The finite e4m3 magnitudes in order: code c has value _MAGNITUDES[c].
_MAGNITUDES = fp8_e4m3_decode(np.arange(127, dtype=np.uint8))


def rope(x, positions, inv_freq, axis, rot_dim: int, adjacent: bool = False, inverse: bool = False):
    """Turns the pairs of the first rot_dim values of every row of x [..., d]
    by positions[axis[j]] * inv_freq[j]; positions [axes, ...] broadcast
    against x's leading dimensions."""
    x = np.asarray(x, dtype=np.float64)
    half = rot_dim // 2
    out = x.copy()
    for j in range(half):
        a, b = (2 * j, 2 * j + 1) if adjacent else (j, j + half)
        angle = np.asarray(positions[axis[j]], dtype=np.float64) * float(inv_freq[j]) * (-1.0 if inverse else 1.0)
        c, s = np.cos(angle), np.sin(angle)
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., b] * c + x[..., a] * s
    return out


def quantise_rows(x):
    """(codes uint8 [..., d], exponents int [...]) of rows x [..., d].

    e is the smallest exponent in E_MIN .. E_MAX with max|x| <= 448 * 2^e (NaN
    aside); the code is the nearest e4m3 value of x * 2^-e, ties to the even
    code, magnitudes beyond 448 to 448, NaN to 0x7F."""
    x = np.asarray(x, dtype=np.float64)
    mag = np.where(np.isnan(x), 0.0, np.abs(x))
    amax = mag.max(axis=-1)
    e = np.full(amax.shape, E_MAX, dtype=np.int64)
    for k in range(E_MAX, E_MIN - 1, -1):
        e = np.where(amax <= 448.0 * 2.0 ** k, k, e)
    y = np.minimum(mag * np.exp2(-e.astype(np.float64))[..., None], 448.0)
    hi = np.searchsorted(_MAGNITUDES, y).clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    dh, dl = _MAGNITUDES[hi] - y, y - _MAGNITUDES[lo]
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    code = code | (np.signbit(x).astype(np.uint8) << 7)
    return np.where(np.isnan(x), np.uint8(0x7F), code).astype(np.uint8), e


def dequantise(codes, scale_bytes):
    """Values code * 2^(byte - 127) of codes [..., d] and bytes [...]."""
    return fp8_e4m3_decode(codes) * np.exp2(np.asarray(scale_bytes, dtype=np.float64) - 127.0)[..., None]


def pool_values(pool_codes, kv_scales, which: int):
    """The values of a whole pool [num_pages, page_size, Hkv, d]; which: 0 for K, 1 for V."""
    scales = np.asarray(kv_scales)[..., which].transpose(0, 2, 1)  # [num_pages, page_size, Hkv]
    return dequantise(pool_codes, scales)


def paged_append8(k_pool, v_pool, kv_scales, k_new, v_new, block_table, cu_seqlens_q, seq_lens, page_size: int):
    """New (k_pool, v_pool, kv_scales) after writing each sequence's rows
    quantised; rows behind cu_seqlens_q[-1] are ignored."""
    kp, vp, sc = (np.array(a, copy=True) for a in (k_pool, v_pool, kv_scales))
    for s in range(len(seq_lens)):
        q0, q1 = int(cu_seqlens_q[s]), int(cu_seqlens_q[s + 1])
        if q1 == q0:
            continue
        rows = [quantise_rows(np.asarray(new)[q0:q1]) for new in (k_new, v_new)]
        for i in range(q1 - q0):
            t = int(seq_lens[s]) - (q1 - q0) + i
            page, slot = int(block_table[s, t // page_size]), t % page_size
            for j, (pool, (codes, e)) in enumerate(zip((kp, vp), rows)):
                pool[page, slot] = codes[i]
                sc[page, :, slot, j] = e[i] + 127
    return kp, vp, sc


def paged_gather8(k_pool, v_pool, kv_scales, block_table, seq_lens, page_size: int):
    """Per sequence: the K and V values [seq_len, Hkv, d] in logical order."""
    k, v = pool_values(k_pool, kv_scales, 0), pool_values(v_pool, kv_scales, 1)
    return [(gather_paged_kv(k, block_table[s], int(n), page_size), gather_paged_kv(v, block_table[s], int(n), page_size))
            for s, n in enumerate(seq_lens)]


def paged_decode8(q, k_pool, v_pool, kv_scales, block_table, seq_lens, page_size: int, scale: float):
    """(O, LSE) of one query a sequence over the cached values; an empty
    sequence gives O = 0 and LSE = -inf."""
    k, v = pool_values(k_pool, kv_scales, 0), pool_values(v_pool, kv_scales, 1)
    q = np.asarray(q, dtype=np.float64)
    o, lse = np.zeros(q.shape), np.full(q.shape[:2], -np.inf)
    live = [s for s in range(len(seq_lens)) if int(seq_lens[s]) > 0]
    if live:
        o[live], lse[live] = paged_decode(q[live], k, v, np.asarray(block_table)[live], np.asarray(seq_lens)[live], page_size,
                                          scale)
    return o, lse
