"""The splits that attention behind a shared prefix takes when none are given."""
import pytest
import torch

import paged_kv_attention_20_gb300 as pka
from test_shared_prefix_gpu import setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,hq,hkv,d,ps", [(torch.float32, 8, 2, 128, 16), (torch.bfloat16, 8, 2, 64, 16), (torch.float16, 8, 2, 96, 16),
                                            (torch.bfloat16, 8, 2, 128, 8), (torch.bfloat16, 130, 1, 128, 16)])
def test_shapes_without_a_prefix_kernel_are_split_as_always(cuda_device, dt, hq, hkv, d, ps):
    """They attend to all keys of every sequence: with the split heuristic's count, the same bits as the call that does just that."""
    shared, own = 4096, [30, 500, 7]
    plan, (q, k, v), _ = setup(shared, own, [(s, shared + n - 1) for s, n in enumerate(own)], hq, hkv, d, ps, dt)
    n = pka.paged_attn_split_heuristic(plan, hq, hkv)
    assert n > 2
    assert torch.equal(pka.paged_attn_forward_shared(plan, q, k, v, 0.1, shared), pka.paged_attn_forward_split(plan, q, k, v, 0.1, n))
    assert pka.device_status() == 0
