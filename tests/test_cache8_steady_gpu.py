"""The 8-bit cache's kernels where they run longest: many tiles a CTA of the
decode (ring places used again and again, the next part of the block table
fetched, shares weighted by the sequences' begins), clusters whose CTAs go round
their ring, several tokens a block of the rotation, many rows a warp of the
append.  That the sizes reach these is worked out from them and asserted.

Sequences share pages, so that caches stay small, and the 64-bit values of the
decode are computed by plain torch products on the GPU.  Tolerances: those of
test_cache8_gpu."""

import numpy as np
import pytest
import torch

import oracle
from attention_flashattention_fwd_04_b200 import api

from .test_cache8_gpu import ERR_TABLE, assert_turned, cache_case, codes, f64, gpu_cache, make_spec, oracle_append, oracle_rope, rows

pytestmark = pytest.mark.gpu


def filled_pools(seed, pages, ps, Hkv, d):
    """Pools of quantised rows and, for the checks, their values in 64 bits."""
    kv = []
    scales = np.zeros((pages, Hkv, ps, 2), np.uint8)
    for i in range(2):
        x = f64(rows(seed + i, pages * ps, Hkv, d)).reshape(pages, ps, Hkv, d)
        c, e = oracle.quantise_rows(x)
        scales[..., i] = (e + 127).transpose(0, 2, 1)
        kv.append((torch.from_numpy(c).cuda(), torch.from_numpy(oracle.dequantise(c, e + 127)).cuda()))
    return kv[0][0], kv[1][0], torch.from_numpy(scales).cuda(), kv[0][1], kv[1][1]


def assert_close_to_64_bits(q, K, V, table, lens, scale, o, lse):
    ps, Hkv, d = K.shape[1:]
    group = q.shape[1] // Hkv
    for s, n in enumerate(lens):
        if n == 0:
            assert not o[s].any() and bool((lse[s] == -float("inf")).all())
            continue
        pages = table[s, :-(-n // ps)].long()
        k, v = (x[pages].reshape(-1, Hkv, d)[:n] for x in (K, V))
        qs = q[s].double().view(Hkv, group, d)
        z = scale * torch.einsum("hgd,lhd->hgl", qs, k)
        slip = 2.0 ** -17 * scale * torch.einsum("hgd,lhd->hgl", qs.abs(), k.abs()).amax(-1)
        wl = torch.logsumexp(z, -1)
        p = torch.exp(z - wl[..., None])
        wo = torch.einsum("hgl,lhd->hgd", p, v)
        bound = 2.0 ** -8 * wo.abs() + (2 * slip[..., None] + 2.0 ** -11 + 2.0 ** -12) * torch.einsum("hgl,lhd->hgd", p, v.abs()) + 1e-30
        err = (o[s].double().view(Hkv, group, d) - wo).abs()
        assert bool((err <= bound).all()), (s, float((err / bound).max()))
        off = (lse[s].double().view(Hkv, group) - wl).abs()
        assert bool((off <= slip + 2.0 ** -21 * (wl.abs() + 20)).all()), (s, float(off.max()))


LONG = [
    # Hq, Hkv, d, page, ring places, heads of a tile, lengths
    (32, 8, 128, 16, 3, 8, [4000 + 731 * i % 4000 for i in range(32)] + [0, 1, 17, 5999]),
    (8, 2, 128, 48, 3, 2, [30011, 1, 0, 60001, 129, 47999, 64, 90000]),
    (16, 1, 128, 64, 6, 1, [100000, 0, 70001, 128, 90063, 1, 33333]),
    (48, 3, 128, 16, 6, 1, [20011, 17, 0, 40001, 1300, 33]),
    (8, 8, 64, 16, 6, 8, [4000 + 977 * i % 5000 for i in range(30)] + [0, 15]),
    (7, 1, 64, 256, 6, 1, [131072, 131071, 5, 0, 100000, 77777, 128]),
    (32, 2, 64, 64, 6, 2, [65537, 1, 64, 0, 90001, 80000, 63]),
    (64, 4, 64, 32, 6, 4, [60000, 70011, 0, 31, 55555]),
    (16, 16, 128, 32, 3, 8, [20000 + 777 * i % 9000 for i in range(5)] + [1, 0]),
    (36, 12, 64, 48, 6, 4, [23000, 30011, 47, 0, 25555, 1]),
]


@pytest.mark.parametrize("Hq,Hkv,d,ps,stages,hb,lens", LONG)
def test_decode_many_tiles_a_cta(Hq, Hkv, d, ps, stages, hb, lens):
    S, group, width = len(lens), Hq // Hkv, -(-max(lens) // ps)
    # A CTA's share, from the sizes: two partial results a CTA, hb * group rows of d + 1 floats each, are the workspace.
    ctas = api.paged_attn_decode_fp8_workspace_bytes(S, Hq, Hkv, d, width, ps) // (2 * hb * group * (d + 1) * 4)
    tokens = 128 // hb
    tiles = sum(-(-n // tokens) for n in lens) * (Hkv // hb)
    assert ctas in (148, 296)
    assert tiles // ctas > stages + 1, "the ring goes round"
    assert tiles // ctas >= 8, "the begin of a sequence has a weight"
    assert max(lens) // tokens > tiles // ctas and tiles // ctas * tokens > 512 + tokens, "a run goes past 32 chunks of its table"
    pages = min(sum(-(-n // ps) for n in lens), max(8, 6000 // ps))
    kp, vp, sc, K, V = filled_pools(400, pages, ps, Hkv, d)
    g = torch.Generator().manual_seed(401)
    table = torch.randint(0, pages, (S, width), generator=g, dtype=torch.int32).cuda()
    for s, n in enumerate(lens):
        table[s, -(-n // ps):] = -1
    q = rows(402, S, Hq, d).cuda()
    scale = float(np.float32(d ** -0.5))
    seq_lens = torch.tensor(lens, dtype=torch.int32).cuda()
    args = (q, kp, vp, sc, table, seq_lens, scale)
    o, lse = api.paged_attn_decode_fp8(*args)
    again = [api.paged_attn_decode_fp8(*args) for _ in range(8)]
    assert api.device_status() == 0
    assert all(torch.equal(o, a) and torch.equal(lse, b) for a, b in again)  # the same sums in the same order
    assert_close_to_64_bits(q, K, V, table, lens, scale, o, lse)


@pytest.mark.parametrize("Hq,Hkv,d,lens", [
    (32, 8, 128, [2048 - 57 * i for i in range(16)]), (16, 1, 128, [1000 + i for i in range(8)]), (32, 8, 64, [1900, 3, 0, 2048] * 4),
    (16, 1, 64, [4096, 4000, 1, 3333, 0, 129])])
def test_decode_clusters_go_round_their_ring(Hq, Hkv, d, lens):
    """Up to 8 tiles of 128 tokens a CTA of a cluster, with 3 or 6 places in its ring."""
    ps, S = 16, len(lens)
    width = -(-max(lens) // ps)
    assert api.paged_attn_decode_fp8_workspace_bytes(S, Hq, Hkv, d, width, ps) == 0, "clusters"
    kp, vp, sc, K, V = filled_pools(410, 300, ps, Hkv, d)
    g = torch.Generator().manual_seed(411)
    table = torch.randint(0, 300, (S, width), generator=g, dtype=torch.int32).cuda()
    q = rows(412, S, Hq, d).cuda()
    scale = float(np.float32(d ** -0.5))
    args = (q, kp, vp, sc, table, torch.tensor(lens, dtype=torch.int32).cuda(), scale)
    o, lse = api.paged_attn_decode_fp8(*args)
    again = [api.paged_attn_decode_fp8(*args) for _ in range(8)]
    assert api.device_status() == 0
    assert all(torch.equal(o, a) and torch.equal(lse, b) for a, b in again)
    assert_close_to_64_bits(q, K, V, table, lens, scale, o, lse)


# ------------------------------------------------------- several tokens a block

def tokens_of_a_block(tokens):
    n = 4
    while n > 0 and tokens >> n < 2 * 148:
        n -= 1
    return 1 << n


@pytest.mark.parametrize("layout", ["bhnd", "bnhd"])
@pytest.mark.parametrize("B,N,Hq,Hkv,d,rot,adjacent", [
    (1, 601, 33, 3, 128, None, False), (3, 421, 32, 8, 128, 48, True), (5, 997, 16, 1, 64, None, False), (2, 2501, 40, 4, 64, 32, True),
    (7, 703, 9, 9, 128, None, False), (1, 4747, 70, 2, 128, 64, False)])
def test_rope_many_tokens_a_block(B, N, Hq, Hkv, d, rot, adjacent, layout):
    per = tokens_of_a_block(B * N)
    assert per > 1 and B * N % per, "several tokens a block, the last block cut"
    assert B == 1 or N % per, "blocks across two batch entries"
    spec = make_spec(d, 3, rot, adjacent, True)
    shape = (lambda h: (B, h, N, d)) if layout == "bhnd" else (lambda h: (B, N, h, d))
    q, k = rows(420, *shape(Hq)), rows(421, *shape(Hkv))
    if layout == "bnhd":
        q, k = q.transpose(1, 2), k.transpose(1, 2)
    pos = torch.randint(0, 100000, (3, B, N), generator=torch.Generator().manual_seed(422), dtype=torch.int32)
    qo, ko = api.attn_rope(q.cuda(), k.cuda(), pos.cuda(), spec)
    assert_turned(qo, q, oracle_rope(spec, f64(q), pos.numpy()[:, :, None]))
    assert_turned(ko, k, oracle_rope(spec, f64(k), pos.numpy()[:, :, None]))
    qi, ki = q.cuda(), k.cuda()
    api.attn_rope(qi, ki, pos.cuda(), spec, q_out=qi, k_out=ki)
    assert torch.equal(qi, qo) and torch.equal(ki, ko)


def uneven(seed, total, S):
    """S numbers of new rows, some none, that make `total`."""
    g = np.random.default_rng(seed)
    new = (g.random(S) ** 3 * (g.random(S) < 0.8) * 2 * total / S).astype(int)
    new[-1] += max(0, total - int(new.sum()))
    return [int(n) for n in new]


@pytest.mark.parametrize("T,S,Hq,Hkv,d,ps,rot,adjacent", [
    (1100, 40, 32, 8, 128, 16, None, False), (2700, 90, 12, 3, 64, 48, 32, True), (4999, 30, 16, 1, 128, 256, None, False),
    (5003, 300, 33, 2, 64, 16, None, False)])
def test_rope_append_many_tokens_a_block(T, S, Hq, Hkv, d, ps, rot, adjacent):
    """Blocks with tokens of several sequences, of a sequence whose page is bad, and of the padding."""
    new = uneven(430, T, S)
    ctx = [(37 * i) % 90 for i in range(S)]
    c = cache_case(431, ctx, new, Hkv, d, ps, pad=5)
    T = c["T"]
    assert tokens_of_a_block(T + 5) > 1
    spec = make_spec(d, 3, rot, adjacent, True)
    q = rows(432, T + 5, Hq, d)
    pos = torch.randint(0, 70000, (3, T + 5), generator=torch.Generator().manual_seed(433), dtype=torch.int32)
    bad = next(s for s in range(S // 2, S) if new[s] > 0)  # its last page lies outside the pool
    page_at = (int(c["lens"][bad]) - 1) // ps
    kept = int(c["table"][bad, page_at])
    lost = [i for i in range(int(c["cu"][bad]), int(c["cu"][bad + 1])) if (int(c["lens"][bad]) - (int(c["cu"][bad + 1]) - i)) // ps == page_at]
    table = c["table"].clone()
    table[bad, page_at] = c["pages"] + 3
    kp, vp, sc = gpu_cache(c)
    q_out = torch.full_like(q, 7.0).cuda()
    api.paged_rope_append_fp8(q.cuda(), c["k"].cuda(), c["v"].cuda(), pos.cuda(), spec, kp, vp, sc, table.cuda(), c["cu"].cuda(),
                              c["lens"].cuda(), q_out=q_out)
    assert api.device_status() == ERR_TABLE and api.device_status() == 0
    there = np.setdiff1d(np.arange(T), lost)
    assert_turned(q_out[there], q[there], oracle_rope(spec, f64(q), pos.numpy()[:, :, None])[there])
    assert torch.all(q_out[T:] == 7.0) and torch.all(q_out[lost] == 7.0)
    turned = oracle_rope(spec, f64(c["k"]), pos.numpy()[:, :, None])
    wk, wv, ws = oracle_append(c, turned)
    wv[kept], ws[kept] = c["vp"].numpy()[kept], c["sc"].numpy()[kept]
    assert np.array_equal(codes(vp), wv) and np.array_equal(codes(sc)[..., 1], ws[..., 1])
    # The keys: half a step of the row's scale, and every slot that no row went to as it was.
    seq = np.searchsorted(c["cu"].numpy(), there, side="right") - 1
    t = c["lens"].numpy()[seq] - (c["cu"].numpy()[seq + 1] - there)
    page, slot = c["table"].numpy()[seq, t // ps], t % ps
    gk, gs = codes(kp), codes(sc)[page, :, slot, 0]
    two = np.exp2(gs.astype(np.float64) - 127)
    got, size = oracle.dequantise(gk[page, slot], gs), np.abs(f64(c["k"])[there]).max(-1)
    slack = 2.0 ** -20 * size
    assert np.all(np.abs(got - turned[there]) <= 2.0 ** -4 * np.abs(turned[there]) + 2.0 ** -10 * two[..., None] + slack[..., None])
    top = np.abs(turned[there]).max(-1)
    assert np.all(top <= 448 * two + slack) and np.all(top > 224 * two - slack)
    untouched = np.ones((c["pages"], ps), bool)
    untouched[page, slot] = False
    assert np.array_equal(gk[untouched], c["kp"].numpy()[untouched])
    assert np.array_equal(codes(sc).transpose(0, 2, 1, 3)[untouched], c["sc"].numpy().transpose(0, 2, 1, 3)[untouched])


@pytest.mark.parametrize("T,S,Hkv,d,ps", [(12001, 60, 8, 128, 16), (20011, 700, 1, 64, 32), (10007, 9, 9, 128, 256)])
def test_append_many_rows_a_warp(T, S, Hkv, d, ps):
    """More items than the warps of 16 blocks an SM: each warp goes on to others, of the same sequence and of another."""
    groups = -(-Hkv * d // 512)
    new = uneven(440, T, S)
    c = cache_case(441, [(11 * i) % 70 for i in range(S)], new, Hkv, d, ps, pad=9)
    assert (c["T"] + 9) * groups > 16 * 148 * 4, "a warp has several items"
    kp, vp, sc = gpu_cache(c)
    api.paged_kv_append_fp8(c["k"].cuda(), c["v"].cuda(), kp, vp, sc, c["table"].cuda(), c["cu"].cuda(), c["lens"].cuda())
    assert api.device_status() == 0
    wk, wv, ws = oracle_append(c)
    assert np.array_equal(codes(kp), wk) and np.array_equal(codes(vp), wv) and np.array_equal(codes(sc), ws)
