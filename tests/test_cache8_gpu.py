"""Rotary positions and the 8-bit paged cache on the GPU, against the fp64
oracle, with tolerances counted in roundings:

* a rounding to t is off by at most finfo(t).eps / 2 of the value (bf16 2^-8,
  e4m3 2^-4, or half of the smallest step, 2^-10 of the row's scale);
* the rotation in fp32 adds a few 2^-24 of |x| + |y|: 2^-21 is allowed;
* decode: a score is a sum of d products in fp32, off by at most 2^-17 of the
  sum of their magnitudes; that moves LSE by as much and a weight by twice as
  much; a weight is rounded once to 11 bits or better before P V (2^-11), and the
  sums over tokens in fp32 and exp2 add less than 2^-12 together; o itself is
  rounded to bf16.
"""

import numpy as np
import pytest
import torch

import oracle
from attention_flashattention_fwd_04_b200 import api

pytestmark = pytest.mark.gpu

ERR_TABLE = 1 << 14
MARK = 9.0625  # exact in bf16, and no value of the 8-bit cache (5 fraction bits)


def f64(t):
    return t.detach().double().cpu().numpy()


def codes(t):
    return t.detach().cpu().view(torch.uint8).numpy()


def rows(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g) * torch.exp(torch.randn(*shape[:-1], 1, generator=g))
    return x.to(torch.bfloat16)


def make_spec(d, axes=3, rot=None, adjacent=False, spread=False):
    half = (rot or d) // 2
    rest = half // axes
    return api.rope_spec(d, [half - rest * (axes - 1)] + [rest] * (axes - 1), rot_dim=rot, adjacent_pairs=adjacent,
                         interleaved_sections=spread)


def oracle_rope(spec, x, pos, inverse=False):
    half = spec.rot_dim // 2
    return oracle.rope(x, pos, list(spec.inv_freq[:half]), list(spec.axis[:half]), spec.rot_dim, bool(spec.adjacent_pairs), inverse)


def assert_turned(out, x, want):
    """bf16 outputs against the fp64 rotation of x."""
    size = np.abs(f64(x)).max(axis=-1, keepdims=True)
    err = np.abs(f64(out) - want)
    assert np.all(err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * size), err.max()


# ------------------------------------------------------------------- rotation

@pytest.mark.parametrize("d,axes,rot,adjacent,spread", [
    (128, 3, None, False, False), (128, 3, None, True, True), (128, 1, None, False, False), (128, 2, 64, False, False),
    (128, 4, 48, True, False), (128, 3, 16, False, True), (64, 3, None, False, True), (64, 2, 32, True, False),
    (64, 1, 48, False, False), (64, 2, 16, True, True)])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_packed(d, axes, rot, adjacent, spread, inverse):
    spec = make_spec(d, axes, rot, adjacent, spread)
    T, Hq, Hkv = 67, 5, 3
    q, k = rows(1, T, Hq, d), rows(2, T, Hkv, d)
    g = torch.Generator().manual_seed(3)
    pos = torch.randint(-3000, 3000, (axes, T), generator=g, dtype=torch.int32)
    qo, ko = api.attn_rope(q.cuda(), k.cuda(), pos.cuda(), spec, inverse=inverse)
    for out, x in ((qo, q), (ko, k)):
        assert_turned(out, x, oracle_rope(spec, f64(x), pos.numpy()[:, :, None], inverse))
    # values behind rot pass through bit for bit
    assert torch.equal(qo.cpu()[..., spec.rot_dim:], q[..., spec.rot_dim:])


@pytest.mark.parametrize("B,Hq,Hkv,N", [(1, 1, 1, 1), (2, 3, 1, 33), (3, 16, 2, 5), (1, 40, 8, 130)])
def test_rope_batched_layout_and_none(B, Hq, Hkv, N):
    spec = make_spec(128)
    q, k = rows(4, B, Hq, N, 128), rows(5, B, Hkv, N, 128)
    pos = torch.randint(0, 100000, (3, B, N), generator=torch.Generator().manual_seed(6), dtype=torch.int32)
    qo, ko = api.attn_rope(q.cuda(), k.cuda(), pos.cuda(), spec)
    assert_turned(qo, q, oracle_rope(spec, f64(q), pos.numpy()[:, :, None]))
    assert_turned(ko, k, oracle_rope(spec, f64(k), pos.numpy()[:, :, None]))
    alone, none = api.attn_rope(q.cuda(), None, pos.cuda(), spec)
    assert none is None and torch.equal(alone, qo)


def test_rope_strided_in_place_and_expanded():
    """Slices of a fused QKV projection, outputs in place, broadcast inputs."""
    spec = make_spec(128)
    B, N, Hq, Hkv, d = 2, 37, 6, 2, 128
    qkv = rows(7, B, N, (Hq + 2 * Hkv), d).cuda()
    before = qkv.clone()
    q, k = qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
    pos = torch.randint(0, 5000, (3, B, N), generator=torch.Generator().manual_seed(8), dtype=torch.int32).cuda()
    want = api.attn_rope(q.contiguous(), k.contiguous(), pos, spec)
    got = api.attn_rope(q, k, pos, spec)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(qkv, before)
    api.attn_rope(q, k, pos, spec, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(qkv[:, :, Hq + Hkv:], before[:, :, Hq + Hkv:])  # V untouched
    one = rows(9, 1, 1, 1, d).cuda()
    wide = one.expand(B, 4, N, d)
    assert torch.equal(api.attn_rope(wide, None, pos, spec)[0], api.attn_rope(wide.contiguous(), None, pos, spec)[0])
    with pytest.raises(api.AttnError) as e:
        api.attn_rope(wide, None, pos, spec, q_out=wide)  # rows of the output would fall together
    assert e.value.status == 2


@pytest.mark.parametrize("far", [2 ** 31 - 1, -2 ** 31, 16777217, 123456789])
def test_rope_far_positions(far):
    """Angles of far positions, where a product in 32 bits would be off by whole turns (in 64 bits it is off by 2^-22 rad at most)."""
    spec = make_spec(64, 1)
    q = rows(10, 3, 2, 64)
    pos = torch.tensor([[far, far - (1 if far > 0 else -1), 0]], dtype=torch.int32)
    out, _ = api.attn_rope(q.cuda(), None, pos.cuda(), spec)
    assert_turned(out, q, oracle_rope(spec, f64(q), pos.numpy()[:, :, None]))
    assert torch.equal(out.cpu()[2], q[2])  # position 0 turns nothing


def test_rope_gradient_by_differences_and_round_trip():
    spec = make_spec(64, 2, 48, True)
    x, g = rows(11, 9, 2, 64), rows(12, 9, 2, 64)
    pos = torch.randint(0, 900, (2, 9), generator=torch.Generator().manual_seed(13), dtype=torch.int32)
    grad, _ = api.attn_rope(g.cuda(), None, pos.cuda(), spec, inverse=True)
    xs, gs, p = f64(x), f64(g), pos.numpy()[:, :, None]
    for at in [(0, 0, 0), (3, 1, 7), (8, 0, 47), (5, 1, 50)]:
        h = np.zeros_like(xs)
        h[at] = 1e-4
        want = (np.sum(gs * oracle_rope(spec, xs + h, p)) - np.sum(gs * oracle_rope(spec, xs - h, p))) / 2e-4
        size = np.abs(gs[at[:2]]).max()
        assert abs(float(grad[at]) - want) <= 2.0 ** -8 * abs(want) + 2.0 ** -20 * size + 1e-7 * size
    # rope then its inverse: one rounding on the way (of values up to sqrt(2) |pair|), one at the end
    there, _ = api.attn_rope(x.cuda(), None, pos.cuda(), spec)
    back, _ = api.attn_rope(there, None, pos.cuda(), spec, inverse=True)
    pairs = np.abs(xs).max(axis=-1, keepdims=True)
    assert np.all(np.abs(f64(back) - xs) <= 2.0 ** -8 * np.abs(xs) + 2.0 ** -7 * 1.5 * pairs)


# --------------------------------------------------------------------- append

def cache_case(seed, ctx, new, Hkv, d, ps, pad=0, spare=2, width_more=1):
    """A cache whose slots all hold marked codes, a table over a permutation,
    the packed new rows (with `pad` rows behind the last sequence)."""
    g = torch.Generator().manual_seed(seed)
    S = len(new)
    lens = [c + n for c, n in zip(ctx, new)]
    need = [-(-n // ps) for n in lens]
    pages = sum(need) + spare
    perm = torch.randperm(pages, generator=g)
    table = torch.full((S, max(need + [1]) + width_more), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = perm[at:at + n].to(torch.int32)
        at += n
    shape = (pages, ps, Hkv, d)
    kp, vp = (torch.randint(0, 256, shape, generator=g, dtype=torch.uint8) for _ in range(2))
    sc = torch.randint(0, 256, (pages, Hkv, ps, 2), generator=g, dtype=torch.uint8)
    T = sum(new)
    cu = torch.tensor([sum(new[:i]) for i in range(S + 1)], dtype=torch.int32)
    return dict(kp=kp, vp=vp, sc=sc, table=table, cu=cu, lens=torch.tensor(lens, dtype=torch.int32), T=T,
                k=rows(seed + 1, T + pad, Hkv, d), v=rows(seed + 2, T + pad, Hkv, d), ps=ps, d=d, Hkv=Hkv, pages=pages)


def gpu_cache(c):
    return c["kp"].cuda().view(torch.float8_e4m3fn), c["vp"].cuda().view(torch.float8_e4m3fn), c["sc"].cuda().view(torch.float8_e8m0fnu)


def oracle_append(c, k=None):
    return oracle.paged_append8(c["kp"].numpy(), c["vp"].numpy(), c["sc"].numpy(), f64(c["k"]) if k is None else k, f64(c["v"]),
                                c["table"].numpy(), c["cu"].numpy(), c["lens"].numpy(), c["ps"])


APPENDS = [
    # ctx, new, Hkv, d, page
    ([0], [1], 1, 64, 16), ([0, 15, 16, 17], [1, 1, 1, 1], 8, 128, 16), ([3, 0, 31], [0, 40, 2], 2, 64, 32),
    ([100, 7], [61, 130], 3, 128, 48), ([0, 250], [256, 9], 5, 64, 256), ([5] * 70, [1] * 35 + [0] * 10 + [3] * 25, 2, 128, 16),
]


@pytest.mark.parametrize("ctx,new,Hkv,d,ps", APPENDS)
def test_append_is_the_oracle_bit_for_bit(ctx, new, Hkv, d, ps):
    c = cache_case(20, ctx, new, Hkv, d, ps, pad=3)
    kp, vp, sc = gpu_cache(c)
    api.paged_kv_append_fp8(c["k"].cuda(), c["v"].cuda(), kp, vp, sc, c["table"].cuda(), c["cu"].cuda(), c["lens"].cuda())
    assert api.device_status() == 0
    wk, wv, ws = oracle_append(c)
    assert np.array_equal(codes(kp), wk) and np.array_equal(codes(vp), wv) and np.array_equal(codes(sc), ws)


def test_append_edge_values():
    """Zero rows, borders of the scale, ties, subnormals, the largest and smallest magnitudes, infinities and NaN."""
    d = 64
    c = cache_case(21, [0], [16], 1, d, 16)
    k = torch.zeros(16, 1, d)
    k[1] = 448.0
    k[2, 0, 0], k[2, 0, 1:] = 450.0, 1.0
    k[3] = torch.linspace(-17, 17, d)
    k[4] = 3.3e38
    k[5] = 1e-38
    k[6] = 1e-30
    k[7, 0, :3] = torch.tensor([float("inf"), -float("inf"), 1.0])
    k[8, 0, :3] = torch.tensor([float("nan"), 2.0, -3.0])
    k[9, 0, :2] = torch.tensor([448.0, 2.0 ** -10])   # a tie between 0 and the smallest code
    k[10, 0, :2] = torch.tensor([448.0, 3 * 2.0 ** -10])
    k[11] = -0.0
    k[12, 0, 5] = 2.0 ** -126
    k[13] = torch.full((d,), float("nan"))
    k[14, 0] = torch.arange(d) * 0.25 + 8
    k[15, 0] = 2.0 ** 127
    c["k"], c["v"] = k.to(torch.bfloat16), (-k).to(torch.bfloat16)
    kp, vp, sc = gpu_cache(c)
    api.paged_kv_append_fp8(c["k"].cuda(), c["v"].cuda(), kp, vp, sc, c["table"].cuda(), c["cu"].cuda(), c["lens"].cuda())
    wk, wv, ws = oracle_append(c)
    assert np.array_equal(codes(sc), ws)
    nan = (wk & 0x7F) == 0x7F  # a NaN's sign says nothing
    assert np.array_equal(codes(kp) | (nan * 0x80).astype(np.uint8), wk | (nan * 0x80).astype(np.uint8))
    assert np.array_equal(codes(vp) | (nan * 0x80).astype(np.uint8), wv | (nan * 0x80).astype(np.uint8))


@pytest.mark.parametrize("ctx,new,Hkv,d,ps", APPENDS)
@pytest.mark.parametrize("rot,adjacent", [(None, False), (48, True)])
def test_rope_append(ctx, new, Hkv, d, ps, rot, adjacent):
    c = cache_case(22, ctx, new, Hkv, d, ps, pad=2)
    spec = make_spec(d, 3, rot, adjacent, True)
    Hq, T = 2 * Hkv + 1, c["T"]
    q = rows(23, T + 2, Hq, d)
    pos = torch.randint(0, 70000, (3, T + 2), generator=torch.Generator().manual_seed(24), dtype=torch.int32)
    kp, vp, sc = gpu_cache(c)
    q_out = torch.full_like(q, 7.0).cuda()
    got = api.paged_rope_append_fp8(q.cuda(), c["k"].cuda(), c["v"].cuda(), pos.cuda(), spec, kp, vp, sc, c["table"].cuda(),
                                    c["cu"].cuda(), c["lens"].cuda(), q_out=q_out)
    assert got is q_out and api.device_status() == 0
    assert_turned(q_out[:T], q[:T], oracle_rope(spec, f64(q), pos.numpy()[:, :, None])[:T])
    assert torch.all(q_out[T:] == 7.0)
    turned = oracle_rope(spec, f64(c["k"]), pos.numpy()[:, :, None])
    wk, wv, ws = oracle_append(c, turned)
    assert np.array_equal(codes(vp), wv) and np.array_equal(codes(sc)[..., 1], ws[..., 1])
    # untouched slots keep their codes; the new keys are within half a step of the rotated ones
    written = np.zeros((c["pages"], ps), bool)
    cu, lens, table = c["cu"].tolist(), c["lens"].tolist(), c["table"].numpy()
    gk, gs = codes(kp), codes(sc)
    for s in range(len(lens)):
        for i in range(cu[s], cu[s + 1]):
            t = lens[s] - (cu[s + 1] - i)
            page, slot = table[s, t // ps], t % ps
            written[page, slot] = True
            two = np.exp2(gs[page, :, slot, 0].astype(np.float64) - 127)[:, None]
            got_k, size = oracle.dequantise(gk[page, slot], gs[page, :, slot, 0]), np.abs(f64(c["k"])[i]).max(-1, keepdims=True)
            slack = 2.0 ** -20 * size
            assert np.all(np.abs(got_k - turned[i]) <= 2.0 ** -4 * np.abs(turned[i]) + 2.0 ** -10 * two + slack)
            top = np.abs(turned[i]).max(-1)
            e = gs[page, :, slot, 0].astype(np.float64) - 127
            assert np.all(top <= 448 * np.exp2(e) + slack[:, 0]) and np.all(top > 448 * np.exp2(e - 1) - slack[:, 0])
    assert np.array_equal(gk[~written], c["kp"].numpy()[~written])
    assert np.array_equal(gs.transpose(0, 2, 1, 3)[~written], c["sc"].numpy().transpose(0, 2, 1, 3)[~written])
    # without rounding between: the same as attn_rope for q, in place too
    qi = q.cuda()
    api.paged_rope_append_fp8(qi, c["k"].cuda(), c["v"].cuda(), pos.cuda(), spec, kp, vp, sc, c["table"].cuda(), c["cu"].cuda(),
                              c["lens"].cuda(), q_out=qi)
    assert torch.equal(qi[:T], q_out[:T]) and torch.equal(qi[T:].cpu(), q[T:])
    assert torch.equal(qi[:T], api.attn_rope(q[:T].cuda(), None, pos[:, :T].contiguous().cuda(), spec)[0])


def test_append_reports_bad_lengths_and_pages():
    c = cache_case(25, [4, 30, 2], [3, 20, 5], 2, 64, 16)
    c["table"][1, 2] = c["pages"]     # tokens 32.. of sequence 1
    c["lens"][2] = 4                  # more new tokens than tokens
    kp, vp, sc = gpu_cache(c)
    api.paged_kv_append_fp8(c["k"].cuda(), c["v"].cuda(), kp, vp, sc, c["table"].cuda(), c["cu"].cuda(), c["lens"].cuda())
    assert api.device_status() == ERR_TABLE and api.device_status() == 0
    c["cu"] = torch.tensor([0, 3, 5, 5], dtype=torch.int32)  # what is left: sequence 0, and sequence 1 up to token 31
    c["lens"] = torch.tensor([7, 32, 2], dtype=torch.int32)
    wk, wv, ws = oracle_append(c)
    wk, wv, ws = oracle.paged_append8(wk, wv, ws, f64(c["k"])[21:], f64(c["v"])[21:], c["table"].numpy(), [0, 0, 2, 2],
                                      [7, 50, 2], 16)  # tokens 48 and 49 of sequence 1, on the page behind the bad one
    assert np.array_equal(codes(kp), wk) and np.array_equal(codes(vp), wv) and np.array_equal(codes(sc), ws)
    c["lens"][0] = c["table"].shape[1] * 16 + 1
    before = codes(kp).copy()
    api.paged_kv_append_fp8(c["k"][:3].cuda(), c["v"][:3].cuda(), kp, vp, sc, c["table"].cuda(),
                            torch.tensor([0, 3, 3, 3], dtype=torch.int32).cuda(), c["lens"].cuda())
    assert api.device_status() == ERR_TABLE and np.array_equal(codes(kp), before)


# --------------------------------------------------------------------- gather

def filled_case(seed, lens, Hkv, d, ps):
    """A cache whose sequences are quantised rows, every other slot NaN codes and wild scales."""
    c = cache_case(seed, [0] * len(lens), list(lens), Hkv, d, ps)
    c["kp"].fill_(0x7F)
    c["vp"].fill_(0xFF)
    c["sc"].fill_(255)
    wk, wv, ws = oracle_append(c)
    c["kp"], c["vp"], c["sc"] = (torch.from_numpy(np.ascontiguousarray(a)) for a in (wk, wv, ws))
    return c


LENGTHS = [[1], [0, 16, 15, 17, 0], [300, 1, 64, 0], [33] * 40]


@pytest.mark.parametrize("lens", LENGTHS)
@pytest.mark.parametrize("Hkv,d,ps", [(1, 64, 16), (8, 128, 16), (3, 128, 48), (2, 64, 256)])
def test_gather_is_exact_and_leaves_the_rest(lens, Hkv, d, ps):
    c = filled_case(30, lens, Hkv, d, ps)
    kp, vp, sc = gpu_cache(c)
    room = [n + (i % 3) * 5 for i, n in enumerate(lens)]
    cu = [sum(room[:i]) for i in range(len(lens) + 1)]
    total = cu[-1] + 4
    ko, vo = (torch.full((total, Hkv, d), MARK, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    api.paged_kv_gather_fp8(kp, vp, sc, c["table"].cuda(), c["lens"].cuda(), torch.tensor(cu, dtype=torch.int32).cuda(),
                            k_out=ko, v_out=vo)
    assert api.device_status() == 0
    want = [np.full((total, Hkv, d), MARK) for _ in range(2)]
    for s, (k, v) in enumerate(oracle.paged_gather8(codes(kp), codes(vp), codes(sc), c["table"].numpy(), lens, ps)):
        want[0][cu[s]:cu[s] + lens[s]], want[1][cu[s]:cu[s] + lens[s]] = k, v
    assert np.array_equal(f64(ko), want[0]) and np.array_equal(f64(vo), want[1])


def test_gather_every_code_and_scale():
    """All 256 codes under the smallest, a middle and the largest scale (NaN codes give NaN)."""
    kp = torch.arange(256, dtype=torch.uint8).repeat(16 * 64 // 256 * 3).view(3, 16, 1, 64).contiguous()
    sc = torch.tensor([27, 127, 246], dtype=torch.uint8).view(3, 1, 1, 1).repeat(1, 1, 16, 2).contiguous()
    table, lens = torch.tensor([[0, 1, 2]], dtype=torch.int32), torch.tensor([48], dtype=torch.int32)
    k, v = api.paged_kv_gather_fp8(kp.cuda(), kp.cuda(), sc.cuda(), table.cuda(), lens.cuda(),
                                   torch.tensor([0, 48], dtype=torch.int32).cuda(), 48)
    want = oracle.dequantise(kp.numpy(), np.broadcast_to(sc[:, :, :, 0].numpy().transpose(0, 2, 1), (3, 16, 1))).reshape(48, 1, 64)
    assert np.array_equal(f64(k), want, equal_nan=True) and torch.equal(k.view(torch.int16), v.view(torch.int16))


def test_gather_reports_bad_input():
    c = filled_case(31, [20, 40, 5], 2, 64, 16)
    kp, vp, sc = gpu_cache(c)
    cu = torch.tensor([0, 20, 50, 55], dtype=torch.int32)  # sequence 1 has room for 30 of its 40
    ko, vo = (torch.full((55, 2, 64), MARK, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    api.paged_kv_gather_fp8(kp, vp, sc, c["table"].cuda(), c["lens"].cuda(), cu.cuda(), k_out=ko, v_out=vo)
    assert api.device_status() == ERR_TABLE
    assert torch.all(ko[20:50] == MARK) and not torch.any(ko[:20] == MARK)
    table = c["table"].clone()
    table[0, 1] = -1
    lens = torch.tensor([20, -3, 5], dtype=torch.int32)
    ko.fill_(MARK)
    api.paged_kv_gather_fp8(kp, vp, sc, table.cuda(), lens.cuda(), cu.cuda(), k_out=ko, v_out=vo)
    assert api.device_status() == ERR_TABLE
    assert torch.all(ko[16:50] == MARK) and not torch.any(ko[:16] == MARK) and not torch.any(ko[50:] == MARK)


# --------------------------------------------------------------------- decode

def run_decode(c, q, scale, **kw):
    kp, vp, sc = gpu_cache(c)
    return api.paged_attn_decode_fp8(q.cuda(), kp, vp, sc, c["table"].cuda(), c["lens"].cuda(), scale, **kw)


def assert_decoded(c, q, scale, o, lse):
    lens = c["lens"].tolist()
    wo, wl = oracle.paged_decode8(f64(q), c["kp"].numpy(), c["vp"].numpy(), c["sc"].numpy(), c["table"].numpy(), lens, c["ps"], scale)
    o, lse = f64(o), f64(lse)
    cached = oracle.paged_gather8(c["kp"].numpy(), c["vp"].numpy(), c["sc"].numpy(), c["table"].numpy(), lens, c["ps"])
    group = q.shape[1] // c["Hkv"]
    for s, n in enumerate(lens):
        if n == 0:
            assert not o[s].any() and np.all(lse[s] == -np.inf)
            continue
        for h in range(q.shape[1]):
            k, v = cached[s][0][:, h // group], cached[s][1][:, h // group]
            qs = f64(q)[s, h]
            z = scale * (k @ qs)
            slip = 2.0 ** -17 * (scale * (np.abs(k) @ np.abs(qs))).max()
            p = np.exp(z - wl[s, h])
            bound = 2.0 ** -8 * np.abs(wo[s, h]) + (2 * slip + 2.0 ** -11 + 2.0 ** -12) * (p @ np.abs(v)) + 1e-30
            err = np.abs(o[s, h] - wo[s, h])
            assert np.all(err <= bound), (s, h, (err / bound).max())
            assert abs(lse[s, h] - wl[s, h]) <= slip + 2.0 ** -21 * (abs(wl[s, h]) + 20), (s, h, lse[s, h], wl[s, h])


DECODES = [
    # Hq, Hkv, d, page, lens
    (32, 8, 128, 16, [1, 15, 16, 17, 0, 255, 256, 257, 1000]), (8, 8, 128, 32, [1, 31, 33, 700]),
    (16, 1, 64, 64, [63, 64, 65, 1500]), (12, 3, 128, 48, [513, 2, 0, 2100]), (4, 2, 64, 16, [16, 48, 80, 777]),
    (64, 4, 128, 256, [255, 3000]), (7, 1, 128, 16, [129]), (9, 1, 64, 16, [40, 1]), (10, 10, 64, 16, [70]),
    (24, 6, 128, 128, [5, 333]), (2, 1, 128, 16, [20000]), (32, 2, 64, 64, [9000, 4097]),
    (16, 1, 128, 32, [4096, 0, 3000, 129]), (32, 4, 64, 16, [500, 128, 127]), (8, 8, 128, 16, [1, 100] * 16),
]


def widen(c, tokens=16384):
    """A table for longer sequences (room for `tokens`): the calls that do not fit a cluster's CTAs, by the sizes alone."""
    S, width = c["table"].shape
    room = -(-tokens // c["ps"])
    c["table"] = torch.cat([c["table"], torch.full((S, max(0, room - width)), -1, dtype=torch.int32)], 1).contiguous()
    return c


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d,ps,lens", DECODES)
def test_decode(Hq, Hkv, d, ps, lens, wide):
    c = filled_case(40, lens, Hkv, d, ps)
    if wide:
        widen(c)
    q = rows(41, len(lens), Hq, d)
    scale = float(np.float32(d ** -0.5))
    o, lse = run_decode(c, q, scale)
    assert api.device_status() == 0
    assert_decoded(c, q, scale, o, lse)


@pytest.mark.parametrize("Hq,Hkv,d,lens", [
    (32, 8, 128, [2000]),               # more than 100 partial rows a head
    (16, 8, 128, [1200, 0, 900, 1, 700]),
    (32, 8, 128, [300] * 13 + [0, 17, 4000]),  # about 18
    (8, 2, 64, [1500, 1490, 64, 0, 1, 2000, 777]),
    (8, 8, 128, [100] * 46 + [1, 2500]),       # about 6
    (16, 2, 64, [300] * 60),
    (8, 8, 128, [30] * 199 + [1600]),          # at most a few
])
def test_decode_joins_any_number_of_partial_rows(Hq, Hkv, d, lens):
    """Sequences and heads from 1 to 200, so that each has from over a hundred partial rows down to one."""
    c = widen(filled_case(44, lens, Hkv, d, 16))
    q = rows(45, len(lens), Hq, d)
    scale = float(np.float32(d ** -0.5))
    o, lse = run_decode(c, q, scale)
    assert api.device_status() == 0
    assert_decoded(c, q, scale, o, lse)


@pytest.mark.parametrize("S,Hq,Hkv,d", [(13, 16, 1, 128), (14, 16, 1, 128), (16, 16, 1, 128), (32, 8, 1, 128), (33, 2, 1, 64), (64, 4, 1, 64)])
def test_decode_clusters_more_than_fit_at_once(S, Hq, Hkv, d):
    """One KV head and up to 64 sequences of up to 1024 tokens: as many clusters as the SMs hold, and more."""
    lens = [1 + (s * 331) % 1024 for s in range(S)]
    c = filled_case(46, lens, Hkv, d, 16)
    q = rows(47, S, Hq, d)
    scale = float(np.float32(d ** -0.5))
    o, lse = run_decode(c, q, scale)
    assert api.device_status() == 0
    assert_decoded(c, q, scale, o, lse)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("t_star", [0, 15, 16, 63, 64, 255, 256, 999, 1000])
def test_decode_reads_the_right_slot(t_star, wide):
    """One token outweighs all others: O is its value row, bit for bit."""
    L, Hkv, d, ps = 1001, 2, 128, 16
    c = cache_case(42, [0, 0], [L, 37], Hkv, d, ps)
    c["kp"].fill_(0x7F), c["vp"].fill_(0x7F), c["sc"].fill_(255)
    c["k"] = (c["k"].float().clamp(-1, 1) * 0.01).to(torch.bfloat16)
    c["k"][t_star, :, 0] = 2048.0
    wk, wv, ws = oracle_append(c)
    c["kp"], c["vp"], c["sc"] = (torch.from_numpy(np.ascontiguousarray(a)) for a in (wk, wv, ws))
    q = torch.zeros(2, 8, d)
    q[..., 0] = 1.0
    o, lse = run_decode(widen(c) if wide else c, q.to(torch.bfloat16), 0.125)
    page, slot = int(c["table"][0, t_star // ps]), t_star % ps
    want = oracle.dequantise(wv[page, slot], ws[page, :, slot, 1])
    assert np.array_equal(f64(o)[0], np.repeat(want, 4, axis=0))
    assert np.allclose(f64(lse)[0], 256.0, atol=2.0 ** -12)


@pytest.mark.parametrize("wide", [False, True])
def test_decode_scales_far_apart(wide):
    """Values whose scales span the whole range: the largest must not drown the weights of the others, nor overflow."""
    d, ps, L = 64, 16, 96
    for seed, (lo, hi) in enumerate([(-90, 110), (-60, 60), (-100, -80), (90, 119)]):
        c = cache_case(50 + seed, [0], [L], 1, d, ps)
        rng = np.random.default_rng(seed)
        size = np.exp2(rng.uniform(lo, hi, (L, 1, 1)))
        c["v"] = torch.from_numpy(rng.standard_normal((L, 1, d)) * size).to(torch.bfloat16)
        c["k"] = torch.from_numpy(rng.standard_normal((L, 1, d)) * 3).to(torch.bfloat16)
        if seed == 0:
            c["v"][10:20] = 0.0
        c["kp"].fill_(0x7F), c["vp"].fill_(0x7F), c["sc"].fill_(0)
        wk, wv, ws = oracle_append(c)
        c["kp"], c["vp"], c["sc"] = (torch.from_numpy(np.ascontiguousarray(a)) for a in (wk, wv, ws))
        q = rows(60 + seed, 1, 4, d)
        if wide:
            widen(c)
        o, lse = run_decode(c, q, 0.125)
        assert_decoded(c, q, 0.125, o, lse)


@pytest.mark.parametrize("size", [1e-30, 1e-6, 1e6, 1e18])
def test_decode_queries_of_any_size(size):
    """Queries far from 1 (the scale brings the scores back), with keys the other way."""
    c = filled_case(70, [200], 2, 128, 16)
    q = (rows(71, 1, 8, 128).float() * size).to(torch.bfloat16)
    scale = float(np.float32(0.1 / size))
    o, lse = run_decode(c, q, scale)
    assert_decoded(c, q, scale, o, lse)


@pytest.mark.parametrize("wide", [False, True])
def test_decode_reports_bad_input_and_goes_on(wide):
    c = filled_case(72, [100, 50, 30, 20], 2, 128, 16)
    if wide:
        widen(c)
    q = rows(73, 4, 8, 128)
    good, good_lse = run_decode(c, q, 0.1)
    assert api.device_status() == 0
    c["table"][0, 2] = c["pages"] + 7
    c["lens"][1], c["lens"][2] = -1, c["table"].shape[1] * 16 + 1
    o, lse = run_decode(c, q, 0.1)
    assert api.device_status() == ERR_TABLE and api.device_status() == 0
    assert not o[1:3].any() and torch.all(lse[1:3] == -float("inf"))
    assert torch.equal(o[3], good[3]) and torch.equal(lse[3], good_lse[3])


def test_decode_garbage_workspace_shared_pages_and_repeat():
    c = widen(filled_case(74, [400, 390, 64], 2, 128, 16))
    c["table"][1, :20], c["table"][2, :4] = c["table"][0, :20].clone(), c["table"][0, :4].clone()
    q = rows(75, 3, 8, 128)
    need = api.paged_attn_decode_fp8_workspace_bytes(3, 8, 2, 128, c["table"].shape[1], 16)
    assert need > 0
    ws = torch.full((need // 4 + 1,), float("nan"), device="cuda")
    o, lse = run_decode(c, q, 0.1, workspace=ws)
    assert_decoded(c, q, 0.1, o, lse)
    again = run_decode(c, q, 0.1)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])  # the same sums in the same order


@pytest.mark.parametrize("wide", [False, True])
def test_decode_empty_batch_and_single_token(wide):
    c = filled_case(76, [0, 0, 0], 2, 64, 16)
    if wide:
        widen(c)
    o, lse = run_decode(c, rows(77, 3, 4, 64), 0.1)
    assert api.device_status() == 0 and not o.any() and torch.all(lse == -float("inf"))
    c = widen(filled_case(78, [1], 1, 64, 16), 16384 if wide else 16)  # one token: its value row, and its score
    q = rows(79, 1, 1, 64)
    o, lse = run_decode(c, q, 0.1)
    page = int(c["table"][0, 0])
    want = oracle.dequantise(c["vp"][page, 0].numpy(), c["sc"][page, :, 0, 1].numpy())
    assert np.array_equal(f64(o)[0], want)
    assert_decoded(c, q, 0.1, o, lse)


def test_decode_more_sequences_than_one_launch_takes():
    """1500 sequences (1024 a launch), sharing pages, some empty."""
    c = filled_case(100, [40, 17, 0, 33], 2, 64, 16)
    S = 1500
    pick = torch.arange(S) % 4
    c["table"], c["lens"] = c["table"][pick].contiguous(), c["lens"][pick].contiguous()
    q = rows(101, 4, 4, 64)[pick].contiguous()
    q[1300:1304] = rows(102, 4, 4, 64)
    o, lse = run_decode(c, q, 0.1)
    assert api.device_status() == 0
    for s0 in (0, 1020, 1300, 1496):
        part = dict(c, table=c["table"][s0:s0 + 4], lens=c["lens"][s0:s0 + 4])
        assert_decoded(part, q[s0:s0 + 4], 0.1, o[s0:s0 + 4], lse[s0:s0 + 4])
    # runs begin elsewhere in other sequences, so sums group differently: equal but for roundings
    assert torch.allclose(lse[:1024:4], lse[0].expand(256, -1), atol=1e-5, rtol=0)


def test_pages_behind_two_gigabytes():
    """Pools of more than 2^31 bytes: append to, read back from and attend to their last pages."""
    num_pages, ps, Hkv, d = 140000, 16, 8, 128
    kp, vp = (torch.empty(num_pages, ps, Hkv, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    sc = torch.empty(num_pages, Hkv, ps, 2, dtype=torch.uint8, device="cuda")
    assert kp.numel() > 2 ** 31
    last = torch.tensor([[num_pages - 1, num_pages - 5, num_pages - 2]], dtype=torch.int32)
    k, v = rows(110, 40, Hkv, d), rows(111, 40, Hkv, d)
    cu, lens = torch.tensor([0, 40], dtype=torch.int32), torch.tensor([40], dtype=torch.int32)
    cache = kp, vp, sc, last.cuda()
    api.paged_kv_append_fp8(k.cuda(), v.cuda(), *cache, cu.cuda(), lens.cuda())
    at = [num_pages - 5, num_pages - 2, num_pages - 1]
    small = dict(kp=kp[at].cpu(), vp=vp[at].cpu(), sc=sc[at].cpu(), table=torch.tensor([[2, 0, 1]], dtype=torch.int32), lens=lens, ps=ps,
                 Hkv=Hkv)
    ko, vo = api.paged_kv_gather_fp8(*cache, lens.cuda(), cu.cuda(), 40)
    (wk, wv), = oracle.paged_gather8(small["kp"].numpy(), small["vp"].numpy(), small["sc"].numpy(), [[2, 0, 1]], [40], ps)
    codes_k, e = oracle.quantise_rows(f64(k))
    assert np.array_equal(wk, oracle.dequantise(codes_k, e + 127))
    assert np.array_equal(f64(ko), wk) and np.array_equal(f64(vo), wv)
    q = rows(112, 1, 32, d)
    o, lse = api.paged_attn_decode_fp8(q.cuda(), *cache, lens.cuda(), 0.1)
    assert api.device_status() == 0
    assert_decoded(small, q, 0.1, o, lse)


def test_gather_rows_behind_two_to_the_27():
    """Outputs of more rows than 2^32 threads of 32 a row: the last sequence's rows lie behind them, the room before is left."""
    Hkv, d, ps, far = 1, 64, 16, 2 ** 27
    if torch.cuda.mem_get_info()[0] < 50 * 2 ** 30:
        pytest.skip("needs 34 GB of outputs")
    c = filled_case(48, [20, 33], Hkv, d, ps)
    kp, vp, sc = gpu_cache(c)
    ko, vo = (torch.empty(far + 64, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for x in (ko, vo):
        x[:64], x[far - 8:] = MARK, MARK
    cu = torch.tensor([0, far + 4, far + 40], dtype=torch.int32).cuda()
    api.paged_kv_gather_fp8(kp, vp, sc, c["table"].cuda(), c["lens"].cuda(), cu, k_out=ko, v_out=vo)
    assert api.device_status() == 0
    (k0, v0), (k1, v1) = oracle.paged_gather8(codes(kp), codes(vp), codes(sc), c["table"].numpy(), [20, 33], ps)
    for x, a, b in ((ko, k0, k1), (vo, v0, v1)):
        assert np.array_equal(f64(x[:20]), a) and np.array_equal(f64(x[far + 4:far + 37]), b)
        assert bool((x[20:64] == MARK).all()) and bool((x[far - 8:far + 4] == MARK).all()) and bool((x[far + 37:] == MARK).all())


# ------------------------------------------------------- as they are used, together

def test_serving_steps_together():
    """Prompt chunks appended (rotated), read back and attended to with paged_prefill; then decode steps over the cache,
    the first of them a captured graph."""
    S, Hq, Hkv, d, ps = 3, 8, 2, 128, 16
    spec = make_spec(d)
    prompt, steps = [37, 5, 130], 3
    width = max(-(-(n + steps) // ps) for n in prompt)
    table = torch.randperm(S * width, generator=torch.Generator().manual_seed(80)).to(torch.int32).view(S, width).cuda()
    kp, vp, sc = api.kv_cache_fp8(S * width, ps, Hkv, d)
    T = sum(prompt)
    cu = torch.tensor([sum(prompt[:i]) for i in range(S + 1)], dtype=torch.int32).cuda()
    lens = torch.tensor(prompt, dtype=torch.int32).cuda()
    q, k, v = (x.cuda() for x in (rows(81, T, Hq, d), rows(82, T, Hkv, d), rows(83, T, Hkv, d)))
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in prompt]).repeat(3, 1).contiguous().cuda()
    qr = api.paged_rope_append_fp8(q, k, v, pos, spec, kp, vp, sc, table, cu, lens)
    # read back into a bf16 pool (starts rounded up to pages) and prefill over it
    room = [-(-n // ps) * ps for n in prompt]
    start = torch.tensor([sum(room[:i]) for i in range(S + 1)], dtype=torch.int32)
    ko, vo = api.paged_kv_gather_fp8(kp, vp, sc, table, lens, start.cuda(), total_rows=sum(room))
    bt = torch.full((S, max(room) // ps), -1, dtype=torch.int32)
    for s in range(S):
        bt[s, :room[s] // ps] = torch.arange(int(start[s]) // ps, int(start[s + 1]) // ps, dtype=torch.int32)
    o, lse = api.paged_prefill(qr, ko.view(-1, ps, Hkv, d), vo.view(-1, ps, Hkv, d), bt.cuda(), cu, lens, True, 0.1)
    assert api.device_status() == 0
    kv = oracle.paged_gather8(codes(kp), codes(vp), codes(sc), table.cpu().numpy(), prompt, ps)
    for s in range(S):
        a, b = int(cu[s]), int(cu[s + 1])
        kk, vv = (np.repeat(x, Hq // Hkv, axis=1).transpose(1, 0, 2)[None] for x in kv[s])
        wo, wl = oracle.attention_forward(f64(qr[a:b]).transpose(1, 0, 2)[None], kk, vv, True, 0.1)
        assert np.abs(f64(o[a:b]) - wo[0].transpose(1, 0, 2)).max() <= 2e-2 * max(1, np.abs(wo).max())
        assert np.abs(f64(lse[a:b]) - wl[0].T).max() <= 1e-3
    # decode steps on buffers that a graph holds
    one = torch.arange(S + 1, dtype=torch.int32).cuda()
    qs, ks, vs = (torch.zeros(S, h, d, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv))
    ps1, qo = torch.zeros(3, S, dtype=torch.int32, device="cuda"), torch.empty(S, Hq, d, dtype=torch.bfloat16, device="cuda")
    out, ol = torch.empty_like(qo), torch.empty(S, Hq, device="cuda")
    ws = torch.empty(api.paged_attn_decode_fp8_workspace_bytes(S, Hq, Hkv, d, width, ps), dtype=torch.uint8, device="cuda")

    def step():
        api.paged_rope_append_fp8(qs, ks, vs, ps1, spec, kp, vp, sc, table, one, lens, q_out=qo)
        api.paged_attn_decode_fp8(qo, kp, vp, sc, table, lens, 0.1, workspace=ws, out=out, lse=ol)

    graph = torch.cuda.CUDAGraph()
    saved = kp.view(torch.uint8).clone(), vp.view(torch.uint8).clone(), sc.view(torch.uint8).clone()
    lens += 1
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    assert all(torch.equal(a, b.view(torch.uint8)) for a, b in zip(saved, (kp, vp, sc)))  # captured, not run
    for i in range(steps):
        for buf, seed in ((qs, 90), (ks, 91), (vs, 92)):
            buf.copy_(rows(seed + 10 * i, *buf.shape).cuda())
        ps1.copy_((lens - 1).repeat(3, 1))
        if i == 1:
            step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        c = dict(kp=kp.view(torch.uint8).cpu(), vp=vp.view(torch.uint8).cpu(), sc=sc.view(torch.uint8).cpu(), table=table.cpu(),
                 lens=lens.cpu(), ps=ps, Hkv=Hkv)
        assert_turned(qo, qs, oracle_rope(spec, f64(qs), f64(ps1)[:, :, None]))
        assert_decoded(c, qo, 0.1, out, ol)
        lens += 1
    assert api.device_status() == 0


def test_calls_on_another_stream():
    """Everything a call makes for itself lives on the stream it runs on."""
    c = widen(filled_case(84, [3000, 2500], 2, 128, 16))
    q = rows(85, 2, 8, 128)
    want = run_decode(c, q, 0.1)
    kp, vp, sc = gpu_cache(c)
    table, lens, qc = c["table"].cuda(), c["lens"].cuda(), q.cuda()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got.append(api.paged_attn_decode_fp8(qc, kp, vp, sc, table, lens, 0.1, stream=side))
        torch.full((1 << 16,), float("nan"), device="cuda")  # current stream: must not fall on the call's workspace
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[0]) and torch.equal(l, want[1]) for o, l in got)
    with torch.cuda.stream(side):
        spec = make_spec(128)
        qo, _ = api.attn_rope(qc, None, torch.zeros(3, 2, dtype=torch.int32, device="cuda"), spec)
    side.synchronize()
    assert torch.equal(qo, qc)


@pytest.mark.parametrize("short", [False, True])
def test_steps_back_to_back_equal_steps_apart(short):
    """A chain of steps whose kernels may begin while the ones before them end gives, bit for bit, what the same steps give with
    the device idle between them."""
    S, Hq, Hkv, d, ps, width = 5, 16, 4, 128, 16, 40 if short else 400
    spec = make_spec(d)
    table = torch.randperm(S * width, generator=torch.Generator().manual_seed(120)).to(torch.int32).view(S, width).cuda()
    one = torch.arange(S + 1, dtype=torch.int32).cuda()
    steps = [tuple(rows(130 + 7 * i + j, S, h, d).cuda() for j, h in enumerate((Hq, Hkv, Hkv))) for i in range(40)]
    start = torch.tensor([0, 15, 200, 555, 31], dtype=torch.int32).cuda()
    results = []
    for apart in (False, True):
        kp, vp, sc = api.kv_cache_fp8(S * width, ps, Hkv, d)
        lens, got = start.clone(), []
        torch.cuda.synchronize()
        for q, k, v in steps:
            lens += 1
            if apart:
                torch.cuda.synchronize()
            qo = api.paged_rope_append_fp8(q, k, v, lens.repeat(3, 1), spec, kp, vp, sc, table, one, lens)
            if apart:
                torch.cuda.synchronize()
            got.append((qo, *api.paged_attn_decode_fp8(qo, kp, vp, sc, table, lens, 0.1)))
            if apart:
                torch.cuda.synchronize()
            got.append(api.paged_attn_decode_fp8(got[-1][1], kp, vp, sc, table, lens, 0.1))  # reads what the merge wrote
        torch.cuda.synchronize()
        results.append(got)
    assert api.device_status() == 0
    for a, b in zip(*results):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_graphs_of_one_memory_pool_and_two_streams():
    c, c2 = widen(filled_case(140, [700, 33], 2, 128, 16)), widen(filled_case(141, [5, 900], 2, 128, 16))
    args = []
    for x, seed in ((c, 142), (c2, 143)):
        kp, vp, sc = gpu_cache(x)
        args.append((rows(seed, 2, 8, 128).cuda(), kp, vp, sc, x["table"].cuda(), x["lens"].cuda(), 0.1))
    want = [api.paged_attn_decode_fp8(*a) for a in args]
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    torch.cuda.synchronize()
    for g, a in zip(graphs, args):
        with torch.cuda.graph(g, pool=graphs[0].pool() if outs else None):
            outs.append(api.paged_attn_decode_fp8(*a))
    for _ in range(5):
        for g, w, o in zip(graphs, want, outs):
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[api.paged_attn_decode_fp8(*a, stream=s) for s, a in zip(streams, args)] for _ in range(20)]
    torch.cuda.synchronize()
    for pair in got:
        for o, w in zip(pair, want):
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])


def test_unaligned_outputs_are_refused():
    c = filled_case(144, [20], 1, 64, 16)
    kp, vp, sc = gpu_cache(c)
    buf = torch.empty(20 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    off = buf[8:].view(20, 1, 64)  # 16-byte aligned only
    with pytest.raises(api.AttnError) as e:
        api.paged_kv_gather_fp8(kp, vp, sc, c["table"].cuda(), c["lens"].cuda(), torch.tensor([0, 20], dtype=torch.int32).cuda(),
                                k_out=off, v_out=torch.empty_like(off))
    assert e.value.status == 3
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.paged_attn_decode_fp8(rows(1, 1, 2, 64), kp, vp, sc, c["table"].cuda(), c["lens"].cuda())
