"""The decode over the 8-bit cache at the ends of its range: keys, queries and
values as large and as small as the types hold, against the fp64 oracle.  The
tolerances are those of test_cache8_gpu: its counts of roundings are relative
and hold at any magnitude."""

import numpy as np
import pytest
import torch

from attention_flashattention_fwd_04_b200 import api

from .test_cache8_gpu import assert_decoded, cache_case, oracle_append, rows, run_decode, widen

pytestmark = pytest.mark.gpu


def stored(c, k, v):
    """The case with the rows k and v [T, Hkv, d] quantised in its cache, every other slot NaN codes under the scale 255."""
    c["k"], c["v"] = k.to(torch.bfloat16), v.to(torch.bfloat16)
    c["kp"].fill_(0x7F), c["vp"].fill_(0xFF), c["sc"].fill_(255)
    c["kp"], c["vp"], c["sc"] = (torch.from_numpy(np.ascontiguousarray(a)) for a in oracle_append(c))
    return c


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
