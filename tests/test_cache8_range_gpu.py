"""The decode over the 8-bit cache at the ends of its range: keys, queries and
values as large and as small as the types hold, against the fp64 oracle.  The
tolerances are those of test_cache8_gpu: its counts of roundings are relative
and hold at any magnitude."""

import numpy as np
import pytest
import torch

import oracle
from attention_flashattention_fwd_04_b200 import api

from .test_cache8_gpu import assert_decoded, cache_case, f64, oracle_append, rows, run_decode, widen

pytestmark = pytest.mark.gpu

TOP = 448.0 * 2.0 ** 119  # the cache's largest value


def stored(c, k, v):
    """The case with the rows k and v [T, Hkv, d] quantised in its cache, every other slot NaN codes under the scale 255."""
    c["k"], c["v"] = k.to(torch.bfloat16), v.to(torch.bfloat16)
    c["kp"].fill_(0x7F), c["vp"].fill_(0xFF), c["sc"].fill_(255)
    c["kp"], c["vp"], c["sc"] = (torch.from_numpy(np.ascontiguousarray(a)) for a in oracle_append(c))
    return c


def one_hot(c, L, d, Hkv, scores, v):
    """Scores of the caller's choice: q is the first unit vector, the scale 1, and k's first value the score."""
    k = torch.zeros(L, Hkv, d)
    k[:, :, 0] = scores[:, None]
    assert torch.equal(k.to(torch.bfloat16).float(), k)
    c = stored(c, k, v)
    q = torch.zeros(1, 4 * Hkv, d)
    q[..., 0] = 1.0
    return c, q.to(torch.bfloat16)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("d,group", [(64, 4), (128, 4), (64, 16), (128, 16)])
@pytest.mark.parametrize("key,query", [(112, 0), (120, 0), (126, -1), (120, -110), (126, -125), (126, -40), (-90, 100), (-95, 120), (0, 119),
                                       (100, 20), (0, -110)])
def test_keys_and_queries_of_any_size(key, query, d, group, wide):
    """Keys about 2^key, queries about 2^query, and the scale that makes their scores a few."""
    lens = [300, 5, 40]
    c = cache_case(200, [0] * 3, lens, 2, d, 16)
    T = sum(lens)
    k = torch.ldexp(rows(201, T, 2, d).float().clamp(-4, 4), torch.tensor(key)).clamp(-3.3e38, 3.3e38)
    c = stored(c, k, rows(202, T, 2, d).float())
    q = torch.ldexp(rows(203, 3, 2 * group, d).float().clamp(-4, 4), torch.tensor(query)).to(torch.bfloat16)
    assert torch.isfinite(q).all()
    scale = float(np.float32(2.0 ** min(-(key + query) - 3, 3)))
    o, lse = run_decode(widen(c) if wide else c, q, scale)
    assert api.device_status() == 0
    assert_decoded(c, q, scale, o, lse)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("key,query,scale", [(-85, 70, 2.0 ** 16), (-85, 0, 2.0 ** 86), (-70, 100, 2.0 ** 40), (-85, 120, 2.0 ** 60), (-85, -30, 2.0 ** 120)])
def test_scores_far_from_zero_under_small_keys(key, query, scale, wide):
    """Queries times scale near fp32's range and beyond it, where the keys bring the scores back: finite, and LSE the largest score."""
    L = 300
    c, q = one_hot(cache_case(209, [0], [L], 2, 64, 16), L, 64, 2, torch.ldexp(torch.arange(L) % 7 - 3.0, torch.tensor(key)),
                   rows(210, L, 2, 64).float())
    q = torch.ldexp(q.float(), torch.tensor(query)).to(torch.bfloat16)
    o, lse = run_decode(widen(c) if wide else c, q, scale)
    assert_decoded(c, q, scale, o, lse)
    top = 3.0 * 2.0 ** (key + query) * scale
    assert torch.isfinite(o).all() and (top < 2.0 ** 20 or np.allclose(f64(lse), top, rtol=2.0 ** -22, atol=0))


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("key,query", [(120, 17), (70, 66), (30, 110)])
def test_scales_below_the_normal_floats(key, query, wide):
    """A scale of few bits is what it is, not what is left of its product with log2(e)."""
    c = cache_case(205, [0] * 2, [200, 33], 2, 64, 16)
    c = stored(c, torch.ldexp(rows(206, 233, 2, 64).float().clamp(-4, 4), torch.tensor(key)), rows(207, 233, 2, 64).float())
    q = torch.ldexp(rows(208, 2, 8, 64).float().clamp(-4, 4), torch.tensor(query)).to(torch.bfloat16)
    scale = float(np.float32(5 * 2.0 ** (-(key + query) - 5)))
    assert 0 < scale < 2.0 ** -126
    o, lse = run_decode(widen(c) if wide else c, q, scale)
    assert_decoded(c, q, scale, o, lse)


@pytest.mark.parametrize("wide", [False, True])
def test_saturated_keys(wide):
    """Rows with an infinity are saturated: a legal cache, and finite scores."""
    c = cache_case(210, [0, 0], [90, 700], 2, 128, 16)
    k = rows(211, 790, 2, 128).float()
    k[::7, :, 3] = float("inf")
    k[5::9, :, 8] = -float("inf")
    c = stored(c, k, rows(212, 790, 2, 128).float())
    q = rows(213, 2, 8, 128)
    scale = float(np.float32(2.0 ** -126))
    o, lse = run_decode(widen(c) if wide else c, q, scale)
    assert api.device_status() == 0 and torch.isfinite(o).all() and torch.isfinite(lse).all()
    assert_decoded(c, q, scale, o, lse)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("d,ps", [(64, 16), (128, 32)])
@pytest.mark.parametrize("exponent", [-120, -95, 0, 90, 119, 126])
def test_many_small_weights_under_any_value_scale(exponent, d, ps, wide):
    """One token 9 above thousands: together they weigh as much as a third of it, however large or small the values are."""
    L = 3000
    c = cache_case(220, [0], [L], 2, d, ps)
    g = torch.Generator().manual_seed(221)
    v = torch.ldexp(torch.randn(L, 2, d, generator=g).clamp(-1.9, 1.9), torch.tensor(exponent))
    scores = torch.zeros(L)
    scores[1234] = 9.0
    c, q = one_hot(c, L, d, 2, scores, v)
    o, lse = run_decode(widen(c) if wide else c, q, 1.0)
    assert_decoded(c, q, 1.0, o, lse)
    assert np.allclose(f64(lse), np.log(np.exp(9.0) + L - 1), atol=2.0 ** -17)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("first,last", [(119, -100), (-100, 119), (119, 0), (0, -100), (-100, 0)])
@pytest.mark.parametrize("rise", [0.0, 60.0, -60.0, -80.0, 240.0])
def test_value_scales_and_scores_that_change_along_the_sequence(first, last, rise, wide):
    """Values of one scale under scores of one height, then of another under another."""
    L, half, d = 1500, 700, 64
    c = cache_case(230, [0], [L], 2, d, 16)
    g = torch.Generator().manual_seed(231)
    v = torch.randn(L, 2, d, generator=g).clamp(-1.9, 1.9)
    v = torch.cat([torch.ldexp(v[:half], torch.tensor(first)), torch.ldexp(v[half:], torch.tensor(last))])
    scores = torch.randint(-2, 3, (L,), generator=g).float()
    scores[half:] += rise
    scores = scores.to(torch.bfloat16).float()
    c, q = one_hot(c, L, d, 2, scores, v)
    o, lse = run_decode(widen(c) if wide else c, q, 1.0)
    assert_decoded(c, q, 1.0, o, lse)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("d,L", [(64, 1000), (128, 2000), (128, 30)])
def test_the_largest_values_and_none(d, L, wide):
    """Every value the largest there is: so is O, not an infinity on the way.  Values of zero: O is zero, LSE that of the scores."""
    c = cache_case(240, [0], [L], 2, d, 16)
    g = torch.Generator().manual_seed(241)
    scores = torch.randint(-8, 9, (L,), generator=g).float()
    v = torch.full((L, 2, d), float("inf"))
    v[:, :, 1::2] = -float("inf")
    v[:, 1] = 0.0
    c, q = one_hot(c, L, d, 2, scores, v)
    o, lse = run_decode(widen(c) if wide else c, q, 1.0)
    o, lse = f64(o), f64(lse)
    want = np.log(np.exp(scores.double().numpy()).sum())
    assert np.allclose(lse, want, atol=2.0 ** -17)
    assert np.all(np.abs(o[0, :4, ::2] / TOP - 1) <= 2.0 ** -8) and np.all(np.abs(o[0, :4, 1::2] / -TOP - 1) <= 2.0 ** -8)
    assert not o[0, 4:].any()


def oracle_values(c, L):
    """The values of the case's first sequence [L, Hkv, d]."""
    return oracle.paged_gather8(c["kp"].numpy(), c["vp"].numpy(), c["sc"].numpy(), c["table"].numpy(), [L], c["ps"])[0][1]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** 13, 2.0 ** 16, 2.0 ** 20, 2.0 ** 24, 2.0 ** 28, 2.0 ** 40, 2.0 ** 60, 2.0 ** 100, 2.0 ** 124])
def test_scores_of_any_size(size, d, wide):
    """A token at 1.5 * size, the others at most at 1.25 * size: O is its value row and LSE its score.  Thousands at the same score:
    O is a mean of their values and LSE log n above it.  Parts of a sequence are joined by their LSEs, whose rounding, 2^-24 of them,
    is that of the parts' weights (twice, for two LSEs): until it counts, O is the mean with equal weights."""
    L = 2500
    c = cache_case(250, [0], [L], 2, d, 16)
    g = torch.Generator().manual_seed(251)
    v = torch.randn(L, 2, d, generator=g)
    scores = torch.tensor([1.25, 1.0, -1.5, 0.0])[torch.randint(0, 4, (L,), generator=g)] * size
    scores[777] = 1.5 * size
    alone, q = one_hot(c, L, d, 2, scores, v)
    o, lse = run_decode(widen(alone) if wide else alone, q, 1.0)
    page, slot = int(alone["table"][0, 777 // 16]), 777 % 16
    want = alone["vp"][page, slot].view(torch.float8_e4m3fn).double() * torch.exp2(alone["sc"][page, :, slot, 1].double() - 127)[:, None]
    # a weight, a sum and their quotient: none is off by more than a few 2^-11, which the rounding to bf16 of a value of 4 bits takes back
    assert np.array_equal(f64(o)[0], np.repeat(want.numpy(), 4, axis=0))
    assert np.allclose(f64(lse), 1.5 * size, rtol=2.0 ** -22, atol=0)
    same, q = one_hot(cache_case(252, [0], [L], 2, d, 16), L, d, 2, torch.full((L,), 1.5 * size), v)
    o, lse = run_decode(widen(same) if wide else same, q, 1.0)
    cached = np.repeat(oracle_values(same, L), 4, axis=1)
    o, mean = f64(o)[0], cached.mean(0)
    off = 2.0 ** -11 + 2.0 ** -12 + 2 * 2.0 ** -24 * 1.5 * size
    assert np.all(np.abs(o - mean) <= 2.0 ** -8 * np.abs(mean) + off * np.abs(cached).mean(0)) or off > 0.1
    slack = 2.0 ** -8 * np.abs(o)
    assert np.all(o <= cached.max(0) + slack) and np.all(o >= cached.min(0) - slack)
    assert np.allclose(f64(lse), 1.5 * size + np.log(L), rtol=2.0 ** -22, atol=2.0 ** -17)
