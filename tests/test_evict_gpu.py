"""Eviction by accumulated weight: the kept indices, rows and totals, exactly."""
import numpy as np
import pytest
import torch

import paged_kv_attention_20_gb300 as pka
from cache_ops_reference import kept_keys, slots

pytestmark = pytest.mark.gpu


def bits(t):
    return t.contiguous().view(torch.uint8)


def setup(lens, kept_lens, ps, hkv, d, dv, dt, in_place, seed=1, totals=None, spare=3):
    rng = np.random.default_rng(seed)
    used = [-(-n // ps) for n in lens]
    fresh = [0 if in_place else -(-m // ps) for m in kept_lens]
    pool = sum(used) + sum(fresh) + spare
    order = list(rng.permutation(pool))
    take = lambda n: [int(order.pop()) for _ in range(n)]               # noqa: E731
    pad = lambda rows: [r + [-1] * (max(map(len, rows), default=0) - len(r)) for r in rows]   # noqa: E731
    src = [take(n) for n in used]
    dst = src if in_place else [take(n) for n in fresh]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    k = torch.randn(pool, ps, hkv, d, generator=gen, device="cuda").to(dt)
    v = torch.randn(pool, ps, hkv, dv, generator=gen, device="cuda").to(dt)
    mass = torch.full((pool, hkv, ps), float("nan"), device="cuda")     # slots past a sequence's end are not read
    host = np.full((pool * ps, hkv), np.nan, dtype=np.float32)
    for s, n in enumerate(lens):
        t = np.exp(2 * rng.standard_normal((n, hkv))).astype(np.float32) if totals is None else totals(rng, n, hkv)
        host[slots(np.array(pad(src)), ps, s, n)] = t
    mass.copy_(torch.from_numpy(host.reshape(pool, ps, hkv).transpose(0, 2, 1).copy()))
    plan = pka.paged_attn_plan(lens, np.array(pad(src)).reshape(len(lens), -1), [], [], ps, pool, device="cuda")
    kept_plan = pka.paged_attn_plan(kept_lens, np.array(pad(dst)).reshape(len(lens), -1), [], [], ps, pool, device="cuda")
    return plan, kept_plan, mass, k, v, np.array(pad(src)), np.array(pad(dst)), host


def verify(lens, kept_lens, ps=16, hkv=2, d=128, dv=128, dt=torch.bfloat16, in_place=True, sink=0, recent=0, **kw):
    plan, kept_plan, mass, k, v, src, dst, host = setup(lens, kept_lens, ps, hkv, d, dv, dt, in_place, **kw)
    want_k, want_v, want_m = k.clone().view(-1, hkv, d), v.clone().view(-1, hkv, dv), torch.from_numpy(host).cuda()
    k0, v0, m0 = want_k.clone(), want_v.clone(), want_m.clone()
    want = np.full((len(lens), hkv, max(kept_lens, default=0)), -1, dtype=np.int64)
    for s, (n, m) in enumerate(zip(lens, kept_lens)):
        at, to = slots(src, ps, s, n), slots(dst, ps, s, m)
        for h in range(hkv):
            ids = kept_keys(host[at, h], m, sink, recent)
            want[s, h, :m] = ids
            i, o = torch.from_numpy(at[ids]).cuda(), torch.from_numpy(to).cuda()
            want_k[o, h], want_v[o, h], want_m[o, h] = k0[i, h], v0[i, h], m0[i, h]
    kept = pka.paged_kv_evict(plan, kept_plan, mass, k, v, sink=sink, recent=recent)
    torch.cuda.synchronize()
    assert pka.device_status() == 0
    assert np.array_equal(kept.cpu().numpy(), want)
    assert torch.equal(bits(k.view(-1, hkv, d)), bits(want_k)) and torch.equal(bits(v.view(-1, hkv, dv)), bits(want_v))
    assert torch.equal(bits(mass), bits(want_m.view(-1, ps, hkv).transpose(1, 2)))


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("ps,hkv,d,dv", [(16, 8, 128, 128), (24, 2, 64, 96), (1, 1, 40, 24), (3, 3, 7, 5), (64, 1, 1024, 8)])
def test_shapes(cuda_device, ps, hkv, d, dv, dt, in_place):
    verify([300, 1, 77, 513], [100, 1, 76, 513], ps, hkv, d, dv, dt, in_place, sink=4, recent=16)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("n,m,sink,recent", [
    (2, 1, 0, 0), (2, 1, 1, 0), (2, 1, 0, 1), (17, 16, 4, 12), (100, 8, 4, 4), (1000, 999, 0, 0), (1025, 1024, 1, 1),
    (5000, 64, 4, 32), (9, 0, 0, 0), (40000, 20001, 4, 1000), (16, 16, 3, 3)])
def test_lengths_and_budgets(cuda_device, n, m, sink, recent, in_place):
    verify([n], [m], hkv=2, d=16, dv=8, in_place=in_place, sink=sink, recent=recent)


@pytest.mark.parametrize("name", ["equal", "two", "zeros", "signs", "odd"])
def test_ties_and_odd_totals(cuda_device, name):
    """Equal totals (the lower index stays), two values, signed zeros, negative totals, infinities and NaN."""
    def totals(rng, n, hkv):
        if name == "equal":
            return np.full((n, hkv), 0.25, np.float32)
        if name == "two":
            return rng.choice([0.5, 0.75], size=(n, hkv)).astype(np.float32)
        if name == "zeros":
            return rng.choice([0.0, -0.0], size=(n, hkv)).astype(np.float32)
        if name == "signs":
            return rng.standard_normal((n, hkv)).astype(np.float32)
        return rng.choice([np.nan, np.inf, -np.inf, 0.0, 1e-45, 3e38, -3e38], size=(n, hkv)).astype(np.float32)
    verify([700, 90], [333, 20], sink=2, recent=5, totals=totals)


@pytest.mark.parametrize("n,m", [(3000, 1500), (200000, 60000)])
@pytest.mark.parametrize("spread", [1e-6, 1.0, 30.0])
@pytest.mark.parametrize("levels", [0, 3, 900, 5000])
def test_crowded_and_wide_totals(cuda_device, n, m, spread, levels):
    """Totals that crowd into a sliver, or span most of the exponents, with up to thousands of equal values around the
    threshold: the choice takes from one to three rounds."""
    def totals(rng, k, hkv):
        x = np.exp(np.clip(spread * rng.standard_normal((k, hkv)), -80, 80))
        if levels:
            x = np.round(x / x.max() * levels) / levels if spread < 5 else np.exp(np.round(np.log(x) * levels / 900) * 900 / levels)
        return np.clip(x, 0, 3e38).astype(np.float32)
    verify([n], [m], hkv=2, d=8, dv=8, sink=4, recent=7, totals=totals)


@pytest.mark.parametrize("seqs,hkv,n", [(1, 1, 4500), (2, 4, 12000), (4, 8, 32768), (3, 8, 60000), (2, 8, 100001), (1, 8, 60000),
                                        (1, 2, 200000), (16, 8, 9000)])
@pytest.mark.parametrize("ties", [False, True])
def test_lists_over_any_number_of_ctas(cuda_device, seqs, hkv, n, ties):
    """Lists so many and so long that one to eight CTAs share one, some much shorter than the longest; with few
    different totals the threshold's equals lie in every CTA's part."""
    def totals(rng, k, heads):
        x = rng.random((k, heads)).astype(np.float32)
        return np.round(x * 7) / 7 if ties else x
    lens = [n // (1 + 2 * (s % 3)) + s for s in range(seqs)]
    verify(lens, [m // 4 + 7 for m in lens], hkv=hkv, d=8, dv=8, in_place=False, sink=3, recent=10, totals=totals)


def test_many_sequences(cuda_device):
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(30, 900, size=70)]
    verify(lens, [max(20, n // 3) for n in lens], hkv=4, d=64, dv=64, sink=4, recent=8, in_place=False)


def test_long_history(cuda_device):
    verify([300000], [70001], hkv=1, d=8, dv=8, sink=4, recent=100, in_place=True)


def test_empty_sequences(cuda_device):
    verify([0, 50, 0], [0, 20, 0], in_place=True)
    plan = pka.paged_attn_plan([], np.zeros((0, 0), np.int32), [], [], 16, 1, device="cuda")
    kept = pka.paged_kv_evict(plan, plan, torch.zeros(1, 2, 16, device="cuda"), torch.zeros(1, 16, 2, 8, device="cuda"),
                              torch.zeros(1, 16, 2, 8, device="cuda"))
    assert kept.shape == (0, 2, 0)


def test_shared_prefix_inside_the_sink(cuda_device):
    """Two sequences share their first page, which lies within the sink: it stays, the rest is evicted."""
    ps, hkv, d = 16, 2, 32
    k = torch.randn(6, ps, hkv, d, device="cuda")
    v, mass = torch.randn_like(k), torch.rand(6, hkv, ps, device="cuda")
    plan = pka.paged_attn_plan([48, 40], [[0, 1, 2], [0, 3, 4]], [], [], ps, 6, device="cuda")
    kept_plan = pka.paged_attn_plan([24, 24], [[0, 1, 2], [0, 3, 4]], [], [], ps, 6, device="cuda")
    k0, m0 = k.clone(), mass.cpu().numpy()
    kept = pka.paged_kv_evict(plan, kept_plan, mass, k, v, sink=16, recent=4).cpu().numpy()
    assert torch.equal(k[0], k0[0])
    for s, pages in enumerate(([0, 1, 2], [0, 3, 4])):
        for h in range(hkv):
            assert np.array_equal(kept[s, h], kept_keys(m0[pages, h].reshape(-1)[:[48, 40][s]], 24, 16, 4))
    with pytest.raises(pka.PagedAttentionError) as e:      # one row of the shared page would be written
        pka.paged_kv_evict(plan, kept_plan, mass, k, v, sink=15, recent=4)
    assert e.value.status == 5


def test_pages_partly_in_place(cuda_device):
    """Each kept page is the source's own or a fresh one, entry by entry; a third sequence only moves house."""
    ps, hkv, d = 16, 2, 64
    lens, kept_lens = [100, 64, 40], [50, 40, 40]
    src = np.array([[0, 1, 2, 3, 4, 5, 6], [7, 8, 9, 10, -1, -1, -1], [11, 12, 13, -1, -1, -1, -1]])
    dst = np.array([[0, 20, 2, 21], [22, 8, 9, -1], [23, 24, 25, -1]])
    gen = torch.Generator(device="cuda").manual_seed(4)
    k = torch.randn(26, ps, hkv, d, generator=gen, device="cuda").half()
    v, mass = torch.randn_like(k), torch.rand(26, hkv, ps, generator=gen, device="cuda")
    plan = pka.paged_attn_plan(lens, src, [], [], ps, 26, device="cuda")
    kept_plan = pka.paged_attn_plan(kept_lens, dst, [], [], ps, 26, device="cuda")
    rows = lambda t: t.view(-1, hkv, d)                                     # noqa: E731
    want_k, want_v = rows(k.clone()), rows(v.clone())
    host = mass.cpu().numpy().transpose(0, 2, 1).reshape(-1, hkv)
    want_m = host.copy()
    ids = [[kept_keys(host[slots(src, ps, s, n), h], m, 3, 9) for h in range(hkv)]
           for s, (n, m) in enumerate(zip(lens, kept_lens))]
    for s, (n, m) in enumerate(zip(lens, kept_lens)):
        for h in range(hkv):
            at, to = slots(src, ps, s, n)[ids[s][h]], slots(dst, ps, s, m)
            want_k[torch.from_numpy(to).cuda(), h] = rows(k)[torch.from_numpy(at).cuda(), h]
            want_v[torch.from_numpy(to).cuda(), h] = rows(v)[torch.from_numpy(at).cuda(), h]
            want_m[to, h] = host[at, h]
    kept = pka.paged_kv_evict(plan, kept_plan, mass, k, v, sink=3, recent=9).cpu().numpy()
    assert pka.device_status() == 0
    for s in range(3):
        for h in range(hkv):
            assert np.array_equal(kept[s, h, :kept_lens[s]], ids[s][h])
    assert torch.equal(bits(rows(k)), bits(want_k)) and torch.equal(bits(rows(v)), bits(want_v))
    assert np.array_equal(mass.cpu().numpy().transpose(0, 2, 1).reshape(-1, hkv), want_m)


def test_source_advanced_on_the_device(cuda_device):
    """Lengths are the device copy's: a plan advanced by graph replays is evicted at its true length."""
    ps, hkv, d = 16, 1, 16
    plan = pka.paged_attn_plan([20], [[0, 1, 2, 3]], [0], [19], ps, 4, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        pka.paged_attn_plan_advance(plan)          # the host copy is at 21, the device copy at 20
    for _ in range(25):
        g.replay()                                 # device: 45
    k = torch.randn(4, ps, hkv, d, device="cuda")
    v, mass = torch.randn_like(k), torch.rand(4, hkv, ps, device="cuda")
    m0 = mass.cpu().numpy().reshape(-1)[:45]
    kept_plan = pka.paged_attn_plan([12], [[0, 1, 2, 3]], [], [], ps, 4, device="cuda")
    kept = pka.paged_kv_evict(plan, kept_plan, mass, k, v, sink=1, recent=2)
    assert np.array_equal(kept[0, 0].cpu().numpy(), kept_keys(m0, 12, 1, 2))


def test_captured_eviction(cuda_device):
    plan, kept_plan, mass, k, v, *_ = setup([500, 200], [128, 64], 16, 2, 64, 64, torch.bfloat16, False)
    want = pka.paged_kv_evict(plan, kept_plan, mass, k, v, sink=4, recent=16)
    k1, v1, m1 = k.clone(), v.clone(), mass.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = pka.paged_kv_evict(plan, kept_plan, mass, k, v, sink=4, recent=16)
    kept.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(kept, want) and torch.equal(bits(k), bits(k1)) and torch.equal(bits(v), bits(v1)) \
        and torch.equal(bits(mass), bits(m1))
