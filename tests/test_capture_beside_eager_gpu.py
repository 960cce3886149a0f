"""A thread that captures a call with a second stream and meanwhile makes others on other streams."""
import pytest
import torch

import paged_kv_attention_20_gb300 as pka
from test_q8_gpu import big_mixed
from test_shared_prefix_gpu import setup as shared_setup

pytestmark = pytest.mark.gpu


def eight_bit():
    plan, dev, _ = big_mixed()

    def call(ws=None, out=None):
        return pka.paged_attn_forward_q8(plan, *dev, 0.09, splits=1, workspace=ws, out=out)
    return call, lambda: pka.make_q8_workspace(plan, 32, 8, 128, 128, 1), dev[0]


def sixteen_bit():
    plan, (q, kc, vc, _, _), _ = big_mixed()
    k, v = kc.float().bfloat16() / 64, vc.float().bfloat16() / 64

    def call(ws=None, out=None):
        return pka.paged_attn_forward_split(plan, q, k, v, 0.09, 2, workspace=ws, out=out)
    return call, lambda: pka.make_workspace(plan, 32, 128, 2), q


def shared():
    own = [900 - 3 * i for i in range(48)]
    plan, (q, k, v), _ = shared_setup(8192, own, [(s, 8192 + n - 1) for s, n in enumerate(own)], 16, 4, 128, 16, torch.bfloat16)

    def call(ws=None, out=None):
        return pka.paged_attn_forward_shared(plan, q, k, v, 0.09, 8192, splits=(4, 1), workspace=ws, out=out)
    return call, lambda: pka.make_workspace(plan, 16, 128, 5), q


@pytest.mark.parametrize("kind", [eight_bit, sixteen_bit, shared])
def test_eager_calls_beside_a_capture(cuda_device, kind):
    call, workspace, q = kind()
    ref = call()                                              # (and the thread's second stream is there)
    ws, outs = [workspace() for _ in range(3)], [torch.zeros_like(q) for _ in range(3)]
    captured, eager, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=captured, capture_error_mode="relaxed"):
        call(ws[0], outs[0])
        with torch.cuda.stream(eager):
            call(ws[1], outs[1])
        call(ws[2], outs[2])
    torch.cuda.synchronize()
    assert torch.equal(outs[1], ref) and not bool(outs[0].any()) and not bool(outs[2].any())
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], ref) and torch.equal(outs[2], ref)
    assert torch.equal(call(), ref) and pka.device_status() == 0
