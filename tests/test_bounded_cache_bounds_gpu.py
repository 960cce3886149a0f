"""The operators around a bounded cache at lengths that only the device's copy of a plan knows, and at other bounds."""
import numpy as np
import pytest
import torch

import paged_kv_attention_20_gb300 as pka
from cache_ops_reference import kept_keys, key_mass, slots, weight_tolerance
from test_evict_gpu import verify as verify_eviction
from test_key_mass_gpu import decode_case as mass_case, run_case, verify as verify_mass
from workloads import build_case

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


def test_page_facts_follow_an_eager_advance(cuda_device):
    """What a plan has found out about its pages is found again once it has advanced: totals of a page that two used
    entries name by then, and an eviction onto a page that another sequence has reached, are refused."""
    k, v = (torch.zeros(4, PS, HKV, 64, device="cuda") for _ in range(2))
    mass, q = torch.zeros(4, HKV, PS, device="cuda"), torch.zeros(1, 2 * HKV, 64, device="cuda")
    plan = pka.paged_attn_plan([16], [[0, 0]], [0], [15], PS, 4, device="cuda")
    call = lambda: pka.paged_attn_forward_mass(plan, q, k, v, mass, 0.125, splits=1)   # noqa: E731
    call()
    pka.paged_attn_plan_advance(plan)
    with pytest.raises(pka.PagedAttentionError) as e:
        call()
    assert e.value.status == 5
    # the first row's second entry names the second's page: padding, until the first row has come to it
    plan = pka.paged_attn_plan([16, 14], [[0, 3], [3, 1]], [0, 1], [15, 13], PS, 4, device="cuda")
    kept_plan = pka.paged_attn_plan([8, 8], [[0], [3]], [], [], PS, 4, device="cuda")
    pka.paged_kv_evict(plan, kept_plan, mass, k, v)
    pka.paged_attn_plan_advance(plan)
    with pytest.raises(pka.PagedAttentionError) as e:
        pka.paged_kv_evict(plan, kept_plan, mass, k, v)
    assert e.value.status == 5
    assert pka.device_status() == 0


def test_large_scores_key_by_key(cuda_device):
    """Scores in the hundreds: weights near 1 and near 0, each key against its float64 sum.  Beside the relative tolerance a
    weight below the smallest normal number may be lost, one a head."""
    case = mass_case(8, 2, 128, 128, 16, torch.bfloat16)
    case.scale = 4.0
    _, mass, before, dc, _ = run_case(case)
    added, seen = key_mass(case, dc.k_cache)
    b, got = before.double().cpu().numpy(), mass.double().cpu().numpy()
    tol = weight_tolerance(case, dc.k_cache) * added + 2.0 ** -24 * (b + added) + 4 * 2.0 ** -126
    assert (np.abs(got - b - added)[seen] <= tol[seen]).all() and np.array_equal(got[~seen], b[~seen])


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_long_lists_of_full_width(cuda_device, dt, in_place):
    """Several long histories with eight heads of 128: every column slice walks its ranks to the end."""
    verify_eviction([30000, 41111, 777, 20000], [7001, 40000, 777, 513], hkv=8, d=128, dv=128, dt=dt, in_place=in_place,
                    sink=4, recent=100)


@pytest.mark.parametrize("splits", [1, 2])
@pytest.mark.parametrize("d,ps,dt", [(256, 16, torch.bfloat16), (256, 32, torch.float32), (128, 16, torch.float32)])
def test_prompt_chunks_of_wide_heads(cuda_device, d, ps, dt, splits):
    """Chunks with totals where the tiles have no tensor-core kernel: wide heads and fp32, beside decode items."""
    lens = [200, 90, 300]
    queries = [(0, 150 + i) for i in range(40)] + [(1, i) for i in range(90)] + [(2, 299)]
    verify_mass(build_case("mass", 31, lens, queries, 4, 2, d, d, ps, dt, d ** -0.5), splits)
