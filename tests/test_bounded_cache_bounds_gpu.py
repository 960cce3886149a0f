"""The operators around a bounded cache at lengths that only the device's copy of a plan knows, and at other bounds."""
import numpy as np
import pytest
import torch

import paged_kv_attention_20_gb300 as pka
from cache_ops_reference import kept_keys, slots

pytestmark = pytest.mark.gpu

PS, HKV, D, PAGES = 16, 2, 16, 16
TABLE = np.array([[0, 1, 2, 3], [4, 5, 6, -1]])
TRUE = [45, 40]


def advanced(seed=1):
    """Two sequences planned at 20 and 15 keys whose device copy stands at TRUE (the host's at 21 and 16)."""
    plan = pka.paged_attn_plan([20, 15], TABLE, [0, 1], [19, 14], PS, PAGES, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        pka.paged_attn_plan_advance(plan)
    for _ in range(25):
        g.replay()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    k, v = (torch.randn(PAGES, PS, HKV, D, generator=gen, device="cuda") for _ in range(2))
    return plan, torch.rand(PAGES, HKV, PS, generator=gen, device="cuda"), k, v


def evict_and_check(kept_lens, table, sink, recent, status):
    plan, mass, k, v = advanced()
    kept_plan = pka.paged_attn_plan(kept_lens, table, [], [], PS, PAGES, device="cuda")
    flat = lambda t: t.transpose(1, 2).reshape(-1, HKV).clone() if t is mass else t.reshape(-1, HKV, D).clone()   # noqa: E731
    want = [flat(t) for t in (mass, k, v)]
    old = [t.clone() for t in want]
    kept = pka.paged_kv_evict(plan, kept_plan, mass, k, v, sink=sink, recent=recent).cpu().numpy()
    assert pka.device_status() == status
    host = old[0].cpu().numpy()
    for s, (n, m) in enumerate(zip(TRUE, kept_lens)):
        m = min(n, m)
        at, to = slots(TABLE, PS, s, n), slots(table, PS, s, m)
        for h in range(HKV):
            first = min(sink, m)
            ids = kept_keys(host[at, h], m, first, min(recent, m - first))
            assert np.array_equal(kept[s, h, :m], ids) and (kept[s, h, m:] == -1).all()
            for new, was in zip(want, old):
                new[torch.from_numpy(to).cuda(), h] = was[torch.from_numpy(at[ids]).cuda(), h]
    for t, new in zip((mass, k, v), want):
        assert torch.equal(flat(t), new)


@pytest.mark.parametrize("kept_lens,table", [
    ([30, 20], [[0, 1, 2, 3], [4, 5, 6, -1]]),       # in place, between the host's length and the device's
    ([40, 40], [[0, 1, 2, 3], [4, 5, 6, -1]]),       # onto pages past the host's; all of the second
    ([30, 20], [[8, 9], [10, 11]]),                  # fresh pages
    ([40, 35], [[0, 12, 2], [4, 13, 6]])])           # page by page
def test_evict_at_the_device_length(cuda_device, kept_lens, table):
    evict_and_check(kept_lens, np.array(table), 2, 5, 0)


def test_evict_budget_above_the_device_length(cuda_device):
    """64 and 41 keys of 45 and 40: every key stays, and PA_DEVICE_RANGE says that the budgets are not filled."""
    evict_and_check([64, 41], np.array([[8, 9, 10, 11], [12, 13, 14, -1]]), 2, 5, 4)


def test_evict_device_length_makes_a_budget_too_small(cuda_device):
    """The host sees 21 of 21 keys stay; of the device's 45, 21 are fewer than the sink and the recent keys."""
    evict_and_check([21, 16], TABLE, 18, 6, 4)
