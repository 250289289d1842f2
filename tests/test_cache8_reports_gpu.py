"""What the 8-bit cache's calls report, where no row of a step's own runs into it."""

import numpy as np
import pytest
import torch

import oracle
from attention_flashattention_fwd_04_b200 import api

from .test_cache8_gpu import ERR_TABLE, MARK, codes, f64, filled_case, gpu_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("at", [0, 2, 699])
@pytest.mark.parametrize("n", [5, -3, 1 << 20])
def test_gather_reports_a_sequence_without_room(at, n):
    """A sequence with tokens (or a bad length) and no row of the output: reported; the others are read."""
    S = 700
    lens = [(3 * i) % 4 for i in range(S)]
    lens[at] = 6
    c = filled_case(300, lens, 2, 64, 16)
    kp, vp, sc = gpu_cache(c)
    room = list(lens)
    room[at] = 0
    cu = [sum(room[:i]) for i in range(S + 1)]
    told = c["lens"].clone()
    told[at] = n
    ko, vo = (torch.full((cu[-1] + 3, 2, 64), MARK, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    call = lambda: api.paged_kv_gather_fp8(kp, vp, sc, c["table"].cuda(), told.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(),  # noqa: E731
                                           k_out=ko, v_out=vo)
    call()
    assert api.device_status() == ERR_TABLE and api.device_status() == 0
    want = np.full((cu[-1] + 3, 2, 64), MARK)
    for s, (k, _) in enumerate(oracle.paged_gather8(codes(kp), codes(vp), codes(sc), c["table"].numpy(), lens, 16)):
        if s != at:
            want[cu[s]:cu[s + 1]] = k
    assert np.array_equal(f64(ko), want)
    told[at] = 0  # no tokens need no room
    call()
    assert api.device_status() == 0


@pytest.mark.parametrize("rows,status", [(60, 0), (52, 0), (51, ERR_TABLE), (30, ERR_TABLE), (10, ERR_TABLE)])
def test_gather_reports_tokens_behind_the_outputs(rows, status):
    """The last sequence's tokens take rows 40 to 51: fewer rows cut tokens off, of it or of those before it."""
    lens, cu = [13, 7, 12], [0, 20, 40, 60]
    c = filled_case(310, lens, 2, 64, 16)
    kp, vp, sc = gpu_cache(c)
    buf = [torch.full((60, 2, 64), MARK, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    api.paged_kv_gather_fp8(kp, vp, sc, c["table"].cuda(), c["lens"].cuda(), torch.tensor(cu, dtype=torch.int32).cuda(),
                            k_out=buf[0][:rows], v_out=buf[1][:rows])
    assert api.device_status() == status and api.device_status() == 0
    want = np.full((60, 2, 64), MARK)
    for s, (k, _) in enumerate(oracle.paged_gather8(codes(kp), codes(vp), codes(sc), c["table"].numpy(), lens, 16)):
        want[cu[s]:cu[s] + lens[s]] = k
    want[rows:] = MARK
    assert np.array_equal(f64(buf[0]), want)
