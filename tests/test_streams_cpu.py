"""A call's stream has to be on its tensors' device, however they are given."""

import types

import pytest
import torch

from attention_flashattention_fwd_04_b200 import api


class OnDevice(torch.Tensor):
    """A tensor that says it is on a GPU (none is touched: the call is refused before)."""

    where = torch.device("cuda", 1)
    is_cuda = property(lambda self: True)
    device = property(lambda self: self.where)


@pytest.mark.parametrize("call", [
    lambda t, s: api.paged_attn_decode_fp8(t, t, t, t, t, t, stream=s),
    lambda t, s: api.paged_attn_decode_fp8(q=t, k_pool=t, v_pool=t, kv_scales=t, block_table=t, seq_lens=t, stream=s),
    lambda t, s: api.paged_kv_append_fp8(k_new=t, v_new=t, k_pool=t, v_pool=t, kv_scales=t, block_table=t, cu_seqlens_q=t, seq_lens=t,
                                         stream=s),
    lambda t, s: api.attn_rope(q=t, k=None, positions=t, spec=api.rope_spec(64), stream=s),
    lambda t, s: api.paged_kv_gather_fp8(k_pool=t, v_pool=t, kv_scales=t, block_table=t, seq_lens=t, cu_seqlens_k=t, stream=s),
])
def test_a_stream_of_another_device_is_refused(call):
    t = torch.zeros(1).as_subclass(OnDevice)
    with pytest.raises(ValueError, match="stream is on cuda:0, the tensors on cuda:1"):
        call(t, types.SimpleNamespace(device=torch.device("cuda", 0)))
