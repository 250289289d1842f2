"""Rotary positions and the 8-bit cache without a GPU: the oracle's pins, the
rotation's description, and every refusal (made before any CUDA call)."""

import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
from attention_flashattention_fwd_04_b200 import api
from attention_flashattention_fwd_04_b200.build import build

FAKE = 1 << 20  # a 16-byte aligned non-null value; never dereferenced


@pytest.fixture(scope="module")
def lib():
    build()
    return api.lib()


# ------------------------------------------------------------------ the oracle

def test_quantise_rows_by_hand():
    x = np.zeros((5, 8))
    x[0, :3] = [448.0, 1.0, -17.0]       # e = 0: 17 lies between 16 and 18 -> the even code, 16
    x[1, :3] = [449.0, 2.0, 3.0]         # e = 1
    x[2, :3] = [3.5, 0.21875, -0.0]      # e = -7 (3.5 = 448 * 2^-7): 0.21875 * 128 = 28
    x[3, :3] = [np.nan, np.inf, 1.0]     # e = 119, inf -> 448, 1 -> 0, NaN stays
    codes, e = oracle.quantise_rows(x)
    assert e.tolist() == [0, 1, -7, 119, -100]
    v = oracle.dequantise(codes, e + 127)
    assert v[0, :3].tolist() == [448.0, 1.0, -16.0]
    assert v[1, :3].tolist() == [448.0, 2.0, 3.0]  # 449 / 2 = 224.5 -> 224
    assert v[2, :3].tolist() == [3.5, 0.21875, 0.0] and np.signbit(v[2, 2])
    assert np.isnan(v[3, 0]) and v[3, 1] == 448.0 * 2.0 ** 119 and v[3, 2] == 0.0
    assert not v[4].any()


def test_quantise_rows_matches_torch_codes():
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((400, 64)) * np.exp2(rng.integers(-60, 60, (400, 1)))).astype(np.float32)
    x = torch.from_numpy(x).to(torch.bfloat16)
    codes, e = oracle.quantise_rows(x.double().numpy())
    y = x.double() * torch.from_numpy(np.exp2(-e.astype(np.float64)))[:, None]
    assert np.array_equal(y.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy(), codes)
    amax = x.double().abs().amax(-1).numpy()
    assert np.all(amax <= 448 * np.exp2(e.astype(np.float64))) and np.all(amax > 448 * np.exp2(e - 1.0))
    # every value is exact in bf16
    v = oracle.dequantise(codes, e + 127)
    assert np.array_equal(torch.from_numpy(v).to(torch.bfloat16).double().numpy(), v)


def test_rope_is_the_complex_rotation_and_its_inverse_the_gradient():
    rng = np.random.default_rng(2)
    x, g = rng.standard_normal((2, 5, 3, 16))
    pos = rng.integers(-50, 50, (2, 5, 1))
    freq, axis = [1.0, 0.3, 0.1, 0.03], [0, 1, 1, 0]
    y = oracle.rope(x, pos, freq, axis, 8)
    for j in range(4):
        z = (x[..., j] + 1j * x[..., j + 4]) * np.exp(1j * pos[axis[j]] * freq[j])
        assert np.allclose(y[..., j], z.real) and np.allclose(y[..., j + 4], z.imag)
    assert np.array_equal(y[..., 8:], x[..., 8:])
    # d/dx of sum(g * rope(x)) by differences, against the inverse rotation of g
    for adjacent in (False, True):
        grad = oracle.rope(g, pos, freq, axis, 8, adjacent, inverse=True)
        for at in [(0, 0, 0), (4, 2, 5), (2, 1, 3), (1, 0, 12)]:
            h = np.zeros_like(x)
            h[at] = 1e-5
            up, down = (np.sum(g * oracle.rope(x + d, pos, freq, axis, 8, adjacent)) for d in (h, -h))
            assert abs((up - down) / 2e-5 - grad[at]) < 1e-8
        assert np.allclose(oracle.rope(oracle.rope(x, pos, freq, axis, 8, adjacent), pos, freq, axis, 8, adjacent, True), x)


def test_oracle_gather_and_decode_read_what_the_append_wrote():
    rng = np.random.default_rng(3)
    kp, vp, sc = np.zeros((4, 16, 2, 64), np.uint8), np.zeros((4, 16, 2, 64), np.uint8), np.zeros((4, 2, 16, 2), np.uint8)
    table, cu, lens = np.array([[2, 0], [3, -1]]), np.array([0, 20, 25]), np.array([20, 5])
    k, v = rng.standard_normal((2, 26, 2, 64))
    kp, vp, sc = oracle.paged_append8(kp, vp, sc, k, v, table, cu, lens, 16)
    got = oracle.paged_gather8(kp, vp, sc, table, lens, 16)
    for s in range(2):
        want = oracle.dequantise(*(lambda c, e: (c, e + 127))(*oracle.quantise_rows(k[cu[s]:cu[s + 1]])))
        assert np.array_equal(got[s][0], want)
    q = rng.standard_normal((3, 4, 64))
    o, lse = oracle.paged_decode8(q, kp, vp, sc, np.array([[2, 0], [3, -1], [0, 0]]), [20, 5, 0], 16, 0.125)
    z = np.einsum("hd,td->ht", q[0, 2:], got[0][0][:, 1]) * 0.125
    assert np.allclose(lse[0, 2:], np.log(np.exp(z).sum(-1)))
    assert not o[2].any() and np.all(lse[2] == -np.inf)


# --------------------------------------------------------- the rotation's spec

def test_rope_spec_layouts():
    s = api.rope_spec(128, [20, 22, 22])
    assert (s.rot_dim, s.num_axes, s.adjacent_pairs) == (128, 3, 0)
    assert list(s.axis) == [0] * 20 + [1] * 22 + [2] * 22
    assert all(s.inv_freq[j] == 10000.0 ** (-2.0 * j / 128) for j in range(64))
    s = api.rope_spec(64, [2, 10, 4], rot_dim=32, interleaved_sections=True, adjacent_pairs=True)
    assert list(s.axis[:16]) == [0, 1, 2, 0, 1, 2, 1, 2, 1, 2, 1, 1, 1, 1, 1, 1]
    assert s.adjacent_pairs == 1
    s = api.rope_spec(64, inv_freq=[1.0 / (j + 1) for j in range(32)])
    assert s.num_axes == 1 and s.inv_freq[31] == 1.0 / 32


@pytest.mark.parametrize("kw", [dict(d=96), dict(d=64, rot_dim=128), dict(d=64, rot_dim=24), dict(d=64, rot_dim=0),
                                dict(d=64, sections=[16, 15]), dict(d=64, sections=[33, -1]), dict(d=64, sections=[]),
                                dict(d=64, inv_freq=[1.0])])
def test_rope_spec_refuses(kw):
    with pytest.raises(ValueError):
        api.rope_spec(**kw)


# ------------------------------------------------------------------- refusals

def _strides(b=0, h=128, n=1024):
    return (ctypes.c_longlong * 3)(b, h, n)


def _rope(lib, q=FAKE, qo=FAKE, qs=None, qos=None, Hq=8, k=FAKE, ko=FAKE, ks=None, kos=None, Hkv=2, B=1, N=5, d=128,
          pos=FAKE, spec=None, inverse=0):
    spec = api.rope_spec(d if d in (64, 128) else 128) if spec is None else spec
    return lib.attn_rope(q, qo, qs or _strides(), qos or _strides(), Hq, k, ko, ks or _strides(), kos or _strides(), Hkv, B, N,
                         d, pos, ctypes.byref(spec) if spec else None, inverse, None)


def _bad_spec(**kw):
    s = api.rope_spec(128, [30, 34])
    for name, v in kw.items():
        if name in ("inv_freq", "axis"):
            getattr(s, name)[3] = v
        else:
            setattr(s, name, v)
    return s


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(qo=None), 1), (dict(pos=None), 1), (dict(spec=False), 1), (dict(ko=None), 1), (dict(k=None), 1),
    (dict(B=-1), 2), (dict(N=-1), 2), (dict(d=96), 2), (dict(Hq=0), 2), (dict(Hkv=0), 2), (dict(inverse=2), 2),
    (dict(B=1 << 16, N=1 << 16), 2), (dict(qs=_strides(n=-8)), 2), (dict(qos=_strides(n=0)), 2), (dict(kos=_strides(h=0)), 2),
    (dict(spec=_bad_spec(rot_dim=24)), 2), (dict(spec=_bad_spec(rot_dim=144)), 2), (dict(spec=_bad_spec(num_axes=0)), 2),
    (dict(spec=_bad_spec(adjacent_pairs=2)), 2), (dict(spec=_bad_spec(axis=2)), 2), (dict(spec=_bad_spec(inv_freq=math.inf)), 2),
    (dict(spec=_bad_spec(inv_freq=math.nan)), 2),
    (dict(q=FAKE + 8), 3), (dict(ko=FAKE + 2), 3), (dict(qs=_strides(n=1020)), 3), (dict(pos=FAKE + 2), 3),
])
def test_attn_rope_rejects(lib, kw, code):
    assert _rope(lib, **kw) == code


def test_attn_rope_with_no_tokens_is_a_no_op(lib):
    assert _rope(lib, N=0, q=None, pos=None) == 0 and _rope(lib, B=0) == 0


def _cache(**kw):
    a = dict(q=FAKE, kn=FAKE, vn=FAKE, qo=FAKE, pos=FAKE, spec=None, kp=FAKE, vp=FAKE, sc=FAKE, cu=FAKE, sl=FAKE, bt=FAKE, ko=FAKE,
             vo=FAKE, o=FAKE, lse=FAKE, S=2, T=5, Hq=8, Hkv=2, d=128, ps=16, mp=4, np=8, scale=0.1, ws=FAKE, wb=1 << 40)
    a.update(kw)
    return a


def _call(lib, fn, **kw):
    a = _cache(**kw)
    end = [a["S"], a["T"]]
    if fn == "append":
        return lib.paged_kv_append_fp8(a["kn"], a["vn"], a["kp"], a["vp"], a["sc"], a["cu"], a["sl"], a["bt"], *end, a["Hkv"],
                                       a["d"], a["ps"], a["mp"], a["np"], None)
    if fn == "step":
        spec = api.rope_spec(128) if a["spec"] is None else a["spec"]
        return lib.paged_rope_append_fp8(a["q"], a["kn"], a["vn"], a["qo"], a["pos"], ctypes.byref(spec), a["kp"], a["vp"],
                                         a["sc"], a["cu"], a["sl"], a["bt"], *end, a["Hq"], a["Hkv"], a["d"], a["ps"], a["mp"],
                                         a["np"], None)
    if fn == "gather":
        return lib.paged_kv_gather_fp8(a["kp"], a["vp"], a["sc"], a["bt"], a["sl"], a["cu"], a["ko"], a["vo"], *end, a["Hkv"],
                                       a["d"], a["ps"], a["mp"], a["np"], None)
    return lib.paged_attn_decode_fp8(a["q"], a["kp"], a["vp"], a["sc"], a["bt"], a["sl"], a["ps"], a["o"], a["lse"], a["S"],
                                     a["Hq"], a["Hkv"], a["d"], a["mp"], a["np"], a["scale"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("fn", ["append", "step", "gather", "decode"])
@pytest.mark.parametrize("kw,code", [
    (dict(kp=None), 1), (dict(vp=None), 1), (dict(sc=None), 1), (dict(sl=None), 1), (dict(bt=None), 1),
    (dict(S=0), 2), (dict(Hkv=0), 2), (dict(d=96), 2), (dict(ps=0), 2), (dict(mp=0), 2), (dict(np=0), 2),
    (dict(S=70000), 2), (dict(np=1 << 28), 2), (dict(mp=1 << 28), 2),
    (dict(ps=8), 5), (dict(ps=24), 5), (dict(ps=272), 5),
    (dict(kp=FAKE + 8), 3), (dict(sc=FAKE + 2), 3), (dict(sl=FAKE + 2), 3), (dict(bt=FAKE + 1), 3),
])
def test_8bit_cache_calls_reject(lib, fn, kw, code):
    assert _call(lib, fn, **kw) == code


@pytest.mark.parametrize("fn,kw,code", [
    *[(f, dict(kn=None), 1) for f in ("append", "step")], *[(f, dict(vn=None), 1) for f in ("append", "step")],
    *[(f, dict(cu=None), 1) for f in ("append", "step", "gather")], *[(f, dict(T=-1), 2) for f in ("append", "step", "gather")],
    *[(f, dict(cu=FAKE + 2), 3) for f in ("append", "step", "gather")],
    ("append", dict(vn=FAKE + 8), 3), ("step", dict(q=None), 1), ("step", dict(qo=None), 1), ("step", dict(pos=None), 1),
    ("step", dict(Hq=0), 2), ("step", dict(spec=_bad_spec(rot_dim=8)), 2), ("step", dict(qo=FAKE + 8), 3),
    ("step", dict(d=64, spec=_bad_spec(rot_dim=128)), 2),
    ("gather", dict(ko=None), 1), ("gather", dict(vo=None), 1), ("gather", dict(ko=FAKE + 8), 3), ("gather", dict(vo=FAKE + 16), 3),
    ("decode", dict(q=None), 1), ("decode", dict(o=None), 1), ("decode", dict(lse=None), 1), ("decode", dict(Hq=7), 2),
    ("decode", dict(scale=0.0), 2), ("decode", dict(scale=math.nan), 2), ("decode", dict(Hq=34), 5),
    ("decode", dict(ws=None, mp=512), 4), ("decode", dict(wb=16, mp=512), 4), ("decode", dict(ws=FAKE + 8, mp=512), 3), ("decode", dict(q=FAKE + 2), 3),
    ("decode", dict(lse=FAKE + 2), 3),
])
def test_8bit_cache_calls_reject_their_own(lib, fn, kw, code):
    assert _call(lib, fn, **kw) == code


@pytest.mark.parametrize("fn", ["append", "step", "gather"])
def test_8bit_cache_calls_with_no_rows_are_no_ops(lib, fn):
    assert _call(lib, fn, T=0, kn=None, vn=None, ko=None, vo=None, q=None, qo=None, pos=None) == 0


def test_decode_fp8_workspace(lib):
    w = lib.paged_attn_decode_fp8_workspace_bytes
    assert w(64, 32, 8, 128, 512, 16) > 0 and w(64, 32, 8, 128, 512, 16) % 16 == 0
    assert w(4, 32, 8, 128, 64, 16) == 0  # few and short sequences need none
    assert w(0, 32, 8, 128, 64, 16) == 0 and w(4, 32, 8, 96, 64, 16) == 0 and w(4, 32, 0, 128, 64, 16) == 0


# ------------------------------------------------- refusals of the Python calls

def _tensors(**bad):
    k, v, sc = api.kv_cache_fp8(6, 16, 2, 64, device="cpu")
    t = dict(q=torch.zeros(5, 8, 64, dtype=torch.bfloat16), k_new=torch.zeros(5, 2, 64, dtype=torch.bfloat16),
             v_new=torch.zeros(5, 2, 64, dtype=torch.bfloat16), positions=torch.zeros(1, 5, dtype=torch.int32),
             spec=api.rope_spec(64), k_pool=k, v_pool=v, kv_scales=sc, block_table=torch.zeros(3, 2, dtype=torch.int32),
             cu=torch.zeros(4, dtype=torch.int32), seq_lens=torch.zeros(3, dtype=torch.int32), total_rows=4)
    t.update(bad)
    return t


def _python(fn, t):
    cache = (t["k_pool"], t["v_pool"], t["kv_scales"], t["block_table"])
    if fn == "append":
        return api.paged_kv_append_fp8(t["k_new"], t["v_new"], *cache, t["cu"], t["seq_lens"])
    if fn == "step":
        return api.paged_rope_append_fp8(t["q"], t["k_new"], t["v_new"], t["positions"], t["spec"], *cache, t["cu"], t["seq_lens"])
    if fn == "gather":
        return api.paged_kv_gather_fp8(*cache, t["seq_lens"], t["cu"], t["total_rows"])
    return api.paged_attn_decode_fp8(t["q"][:3], *cache, t["seq_lens"])


@pytest.mark.parametrize("fn", ["append", "step", "gather", "decode"])
def test_python_calls_check_shapes_then_types_then_devices(fn):
    t = _tensors()
    with pytest.raises(ValueError, match="CUDA tensor"):
        _python(fn, t)
    for bad, what in ((dict(v_pool=t["v_pool"][:-1]), "v_pool"), (dict(kv_scales=t["kv_scales"][:, :, :8].contiguous()), "kv_scales"),
                      (dict(kv_scales=t["kv_scales"].view(torch.uint8).float()), "kv_scales"), (dict(k_pool=t["k_pool"].float()), "k_pool"),
                      (dict(block_table=t["block_table"][:2]), "block_table"), (dict(block_table=t["block_table"].long()), "block_table"),
                      (dict(k_pool=t["k_pool"].transpose(1, 2)), "k_pool")):
        with pytest.raises(ValueError, match=what):
            _python(fn, _tensors(**bad))


@pytest.mark.parametrize("fn,bad,what", [
    ("append", dict(v_new=torch.zeros(4, 2, 64, dtype=torch.bfloat16)), "do not match"),
    ("append", dict(cu=torch.zeros(3, dtype=torch.int32)), "number of sequences"),
    ("step", dict(q=torch.zeros(4, 8, 64, dtype=torch.bfloat16)), "do not match"),
    ("step", dict(positions=torch.zeros(2, 5, dtype=torch.int32)), "positions"),
    ("gather", dict(total_rows=None), "total_rows"), ("gather", dict(cu=torch.zeros(3, dtype=torch.int32)), "number of sequences"),
    ("decode", dict(q=torch.zeros(5, 8, 128, dtype=torch.bfloat16)), "q must be"),
])
def test_python_calls_refuse_mismatched_shapes(fn, bad, what):
    with pytest.raises(ValueError, match=what):
        _python(fn, _tensors(**bad))


def test_python_rope_refusals():
    q, pos, spec = torch.zeros(2, 4, 6, 64, dtype=torch.bfloat16), torch.zeros(1, 2, 6, dtype=torch.int32), api.rope_spec(64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.attn_rope(q, None, pos, spec)
    with pytest.raises(ValueError, match="positions"):
        api.attn_rope(q, None, pos[:, :, :5].contiguous(), spec)
    with pytest.raises(ValueError, match="contiguous"):
        api.attn_rope(q.transpose(2, 3), None, pos, spec)
    with pytest.raises(ValueError, match="k shape"):
        api.attn_rope(q, q[:1], pos, spec)
    with pytest.raises(ValueError, match="k_out"):
        api.attn_rope(q, None, pos, spec, k_out=q)
    with pytest.raises(ValueError, match="bfloat16"):
        api.attn_rope(q.float(), None, pos, spec)
    with pytest.raises(TypeError):
        api.attn_rope(q, None, pos, object())


# ------------------------------------------------- the decode's share-out of work

@pytest.mark.parametrize("seed", range(6))
def test_decode_share_out(seed):
    """The split pass's runs and the merge's pieces, in their own arithmetic: every tile falls to one run, a CTA writes at most
    one partial result to each of its two slots, and the merge reads exactly the slots that were written."""
    rng = np.random.default_rng(seed)
    for case in range(80):
        S, groups = int(rng.integers(1, 20)), int(rng.integers(1, 5))
        n = (rng.integers(0, 300 if case % 2 else 30, S) * (rng.random(S) < 0.8)).astype(int)
        tiles, live = int(n.sum()), int((n > 0).sum())
        ctas = min(int(rng.integers(1, 60)), tiles * groups)
        extra = min(3, tiles * groups // (8 * ctas)) if ctas else 0
        first = np.concatenate([[0], np.cumsum(n + extra * (n > 0))]).astype(int)
        total = (tiles + extra * live) * groups
        each, more = divmod(total, ctas) if ctas else (0, 0)

        def begin(c):
            return c * each + min(c, more)

        def owner(t):
            cut = more * (each + 1)
            return t // (each + 1) if t < cut else more + (t - cut) // each

        seen, slots = set(), {}
        for c in range(ctas):
            at, end = begin(c), begin(c + 1)
            assert at < end
            while at < end:
                lo, hi = 0, S
                while hi - lo > 1:
                    mid = (lo + hi) // 2
                    lo, hi = (mid, hi) if first[mid] * groups <= at else (lo, mid)
                units = int(first[lo + 1] - first[lo])
                assert units > extra
                hg, u = divmod(at - int(first[lo]) * groups, units)
                v = min(units, u + end - at)
                at += v - u
                a, b = max(u - extra, 0), max(v - extra, 0)
                for t in range(a, b):
                    assert (lo, hg, t) not in seen
                    seen.add((lo, hg, t))
                if a < b and not (a == 0 and b == units - extra):
                    slot = 2 * c + (1 if a == 0 else 0)
                    assert slot not in slots
                    slots[slot] = (lo, hg)
        assert len(seen) == tiles * groups
        read = {}
        for s in range(S):
            for hg in range(groups if n[s] else 0):
                at = int(first[s]) * groups + hg * int(n[s] + extra) + extra
                c0, c1 = owner(at), owner(at + int(n[s]) - 1)
                if c1 > c0:
                    read.update({2 * (c0 + i) + (1 if i == 0 else 0): (s, hg) for i in range(c1 - c0 + 1)})
        assert read == slots
