"""Which frequencies the rotation takes (checked before any CUDA call)."""

import ctypes

import pytest

from attention_flashattention_fwd_04_b200 import api
from attention_flashattention_fwd_04_b200.build import build


@pytest.mark.parametrize("freq,status", [(2.0 ** 62, 2), (-2.0 ** 62, 2), (1e300, 2), (float("inf"), 2), (float("nan"), 2),
                                         (2.0 ** 62 - 2.0 ** 9, 0), (-1e18, 0), (0.0, 0), (5e-324, 0)])
def test_frequencies_that_the_call_takes(freq, status):
    build()
    spec = api.rope_spec(64, inv_freq=[1.0] * 31 + [freq])
    assert api.lib().attn_rope(None, None, None, None, 1, None, None, None, None, 0, 1, 0, 64, None, ctypes.byref(spec), 0, None) == status
