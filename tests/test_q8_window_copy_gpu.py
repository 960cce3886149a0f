"""Prompt chunks over the 8-bit cache under a window, in a workspace of just what the window needs."""
import pytest
import torch

import paged_kv_attention_20_gb300 as pka
from q8_reference import attend
from test_q8_gpu import DT, check, setup

pytestmark = pytest.mark.gpu


def call(plan, dev, window, splits, causal=True, max_keys=0):
    q = dev[0]
    ws = pka.make_q8_workspace(plan, q.shape[1], dev[1].shape[2], 128, 128, splits, q.dtype, max_keys=max_keys, window=window)
    guard = torch.cat([ws, torch.full((4096,), 3.0, device="cuda")])
    guard[:ws.numel()] = float("nan")
    out = pka.paged_attn_forward_q8(plan, *dev, 128 ** -0.5, splits=splits, window=window, causal=causal, workspace=guard[:ws.numel()])
    torch.cuda.synchronize()
    assert bool((guard[ws.numel():] == 3.0).all())                # nothing past the workspace
    return out


# chunks that begin on, before and behind a block of 128 keys, and windows that reach there; several chunks of one sequence
@pytest.mark.parametrize("window", [1, 16, 100, 128, 129, 300, 5000])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_window(cuda_device, dt, window):
    lens = [1500, 700, 129, 40, 900]
    queries = [(0, i) for i in range(1280, 1500)] + [(1, i) for i in range(511, 700)] + [(2, i) for i in range(0, 129)] + [(3, 39)] \
        + [(4, i) for i in range(140, 160)] + [(4, i) for i in range(640, 900)]
    plan, dev, args = setup(lens, queries, 4, 2, 128, 128, 16, DT[dt])
    ref = attend(*args, 128 ** -0.5, True, window)
    for splits in (1, 3):
        check(call(plan, dev, window, splits), ref, DT[dt], f"splits {splits}")
    if window in (100, 300):
        check(call(plan, dev, window, 2, causal=False), attend(*args, 128 ** -0.5, False, window), DT[dt], "not causal")
    assert pka.device_status() == 0


def test_more_sequences_than_threads(cuda_device):
    """Places in more than one round of the block that works them out; most sequences have no chunk."""
    lens = [300] * 1100
    with_chunk = [0, 3, 500, 1023, 1024, 1099]
    queries = [(s, i) for s in with_chunk for i in range(280, 300)] + [(7, 299), (1050, 100)]
    plan, dev, args = setup(lens, queries, 2, 1, 128, 128, 16, torch.bfloat16, poison=False)
    for window in (0, 50):
        check(call(plan, dev, window, 1), attend(*args, 128 ** -0.5, True, window), torch.bfloat16, f"window {window}")
    assert pka.device_status() == 0


def test_staged_plans(cuda_device):
    """A captured windowed call, replayed for histories of other lengths: in bounds, and right while the blocks fit."""
    ps, h, window = 16, 2, 150
    lens = {n: [n, 64] for n in (200, 640, 1000)}
    queries = {n: [(0, i) for i in range(n - 20, n)] + [(1, 63)] for n in lens}
    plan, dev, args = setup([1000, 64], queries[1000], 4, h, 128, 128, ps, torch.bfloat16)
    table = args[4]
    plans = {n: pka.paged_attn_plan(lens[n], table, [s for s, _ in queries[n]], [p for _, p in queries[n]], ps, dev[1].shape[0], upload=False)
             for n in lens}
    words = torch.empty(plans[200].device_bytes(), dtype=torch.uint8, device="cuda")
    host = {n: torch.empty(p.device_bytes(), dtype=torch.uint8).pin_memory() for n, p in plans.items()}
    for n, p in plans.items():
        p.stage(host[n], words)
    ws, out = pka.make_q8_workspace(plans[200], 4, h, 128, 128, 1, max_keys=window + 20 + 128, window=window), torch.empty_like(dev[0])
    words.copy_(host[200])
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        pka.paged_attn_forward_q8(plans[200], *dev, 0.1, splits=1, workspace=ws, out=out, window=window)
    for n in (200, 640, 1000, 200):
        words.copy_(host[n])
        graph.replay()
        torch.cuda.synchronize()
        assert pka.device_status() == 0
        check(out, attend(*args[:3], lens[n], table, ps, [s for s, _ in queries[n]], [p for _, p in queries[n]], 0.1, True, window),
              torch.bfloat16, f"{n}")
