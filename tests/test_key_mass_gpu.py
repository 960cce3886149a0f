"""Attention with per-key weight totals: the output against the oracle, the totals against float64 sums.

The totals' tolerance is weight_tolerance() of what the call added, plus half a
step of fp32 of the total that was there for every addition to it.
"""
import numpy as np
import pytest
import torch

import paged_kv_attention_20_gb300 as pka
from cache_ops_reference import key_mass, weight_tolerance
from helpers import assert_close, oracle_after_store, plan_for
from workloads import build_case, decode_queries

pytestmark = pytest.mark.gpu

BF, HF, SF = torch.bfloat16, torch.float16, torch.float32


def run_case(case, splits=1, causal=True, window=0, workspace=None, calls=1):
    dc = case.to("cuda")
    plan = plan_for(case)
    pka.paged_kv_store(plan, dc.new_k, dc.new_v, dc.k_cache, dc.v_cache)
    gen = torch.Generator(device="cuda").manual_seed(1)
    mass = torch.rand(case.num_pages, case.hkv, case.page_size, generator=gen, device="cuda")
    before = mass.clone()
    for _ in range(calls):
        out = pka.paged_attn_forward_mass(plan, dc.q, dc.k_cache, dc.v_cache, mass, case.scale, splits=splits,
                                          workspace=workspace, causal=causal, window=window)
    torch.cuda.synchronize()
    assert pka.device_status() == 0
    return out, mass, before, dc, plan


def verify(case, splits=1, causal=True, window=0):
    out, mass, before, dc, plan = run_case(case, splits, causal, window)
    ref, _, _, _ = oracle_after_store(case, causal=causal, window=window)
    assert_close(out.double().cpu().numpy(), ref, case.dtype, "out")
    added, seen = key_mass(case, dc.k_cache, causal, window)
    b, got = before.double().cpu().numpy(), mass.double().cpu().numpy()
    steps = max(np.bincount(np.asarray(case.query_seq)).max(), 1)
    tol = weight_tolerance(case, dc.k_cache) * added + 2.0 ** -24 * steps * (b + added)
    err = np.abs(got - b - added)
    assert (err[seen] <= tol[seen]).all(), f"worst {np.max(err[seen] / tol[seen]):.2f} tolerances"
    assert np.array_equal(got[~seen], b[~seen])             # slots no query sees are left alone
    # the same call on the same inputs: the same bits
    out2, mass2, _, _, _ = run_case(case, splits, causal, window)
    assert torch.equal(mass, mass2) and torch.equal(out, out2)
    # and the output is the plain call's
    plain = pka.paged_attn_forward_split(plan, dc.q, dc.k_cache, dc.v_cache, case.scale, splits, causal=causal,
                                         window=window)
    assert torch.equal(out, plain)


def decode_case(hq, hkv, d, dv, ps, dt, lens=(1, 17, 64, 333), seed=3):
    lens = list(lens)
    return build_case("mass", seed, lens, decode_queries(lens), hq, hkv, d, dv, ps, dt, 1 / np.sqrt(d), pool_pages=None)


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("hq,hkv,d,dv,ps,dt", [
    (4, 4, 64, 64, 16, SF), (8, 2, 128, 128, 16, BF), (4, 4, 128, 128, 16, HF), (2, 1, 256, 256, 32, BF),
    (12, 2, 64, 64, 64, HF), (16, 2, 128, 128, 16, BF), (64, 1, 128, 128, 32, HF), (128, 1, 128, 128, 16, BF),
    (40, 1, 128, 128, 8, BF), (8, 2, 64, 64, 24, BF), (8, 1, 128, 128, 5, HF), (6, 2, 40, 24, 5, HF), (3, 1, 7, 9, 1, SF),
    (2, 2, 1024, 1, 3, SF), (8, 2, 96, 96, 16, BF), (130, 1, 16, 16, 16, HF)])
def test_decode(cuda_device, hq, hkv, d, dv, ps, dt, splits):
    verify(decode_case(hq, hkv, d, dv, ps, dt), splits)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [1, 37, 200])
@pytest.mark.parametrize("hq,hkv,d,ps,dt", [(8, 2, 128, 16, BF), (16, 2, 128, 16, HF), (4, 2, 64, 24, BF), (4, 2, 40, 5, SF)])
def test_decode_windows(cuda_device, hq, hkv, d, ps, dt, window, causal):
    lens = [1, 17, 64, 333]
    queries = decode_queries(lens[:3]) + [(3, 150)]
    case = build_case("mass", 4, lens, queries, hq, hkv, d, d, ps, dt, 1 / np.sqrt(d))
    verify(case, 2, causal, window)


@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("hq,hkv,d,ps,dt", [(8, 2, 128, 16, BF), (32, 2, 128, 16, BF), (4, 2, 64, 16, SF)])
def test_several_queries_of_a_sequence(cuda_device, hq, hkv, d, ps, dt, window):
    """Short runs, scattered positions, and queries of one sequence apart in the packing; one sequence unread."""
    queries = [(2, 299), (0, 5), (1, 90), (2, 10), (0, 6), (1, 91), (0, 7), (2, 298), (1, 0)]
    case = build_case("mass", 6, [8, 100, 300, 40], queries, hq, hkv, d, d, ps, dt, 1 / np.sqrt(d))
    verify(case, 1, True, window)
    verify(case, 4, True, window)


def test_many_items_in_few_sequences(cuda_device):
    """More decode items than a CTA scans for its sequence (they come from a grouped list), every second position."""
    lens = [1500, 1300, 40]
    queries = [(s, p) for s, n in enumerate(lens) for p in range(0, n, 2)]
    case = build_case("mass", 17, lens, queries, 4, 2, 64, 64, 16, BF, 0.125)
    assert case.num_queries > 1024
    verify(case, 1)
    verify(case, 2, True, 300)


def test_drafted_tokens_under_a_window(cuda_device):
    """Queries a few positions apart see ranges a few keys apart: every key still has one owner."""
    lens = [2000, 1111, 700]
    queries = [(s, n - 5 + i) for s, n in enumerate(lens) for i in range(5)]
    case = build_case("mass", 7, lens, queries, 4, 2, 64, 64, 32, HF, 0.125)
    verify(case, 3, True, 1000)


@pytest.mark.parametrize("hq,hkv,d,ps,dt", [(8, 2, 128, 16, BF), (16, 2, 128, 16, BF), (4, 2, 64, 24, HF), (4, 2, 40, 5, SF)])
@pytest.mark.parametrize("window", [32, 64])
def test_window_starts_at_any_key(cuda_device, hq, hkv, d, ps, dt, window):
    """Score rows start up to three keys before a window that fills them, and both of its ends fall inside a four of
    keys; sequences of one item, and of four items a key apart.  The last item's row ends with the workspace."""
    lens = [200, 201, 202, 203]
    for queries in (decode_queries(lens), [(s, n - 4 + i) for s, n in enumerate(lens) for i in range(4)]):
        case = build_case("mass", 21, lens, queries, hq, hkv, d, d, ps, dt, 1 / np.sqrt(d))
        verify(case, 1, True, window)
        verify(case, 2, True, window)


@pytest.mark.parametrize("window", [0, 70])
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("hq,hkv,d,ps,dt", [
    (4, 1, 128, 16, BF), (4, 4, 128, 32, HF), (8, 2, 128, 64, BF), (2, 1, 128, 128, BF),   # tensor-core tiles
    (4, 2, 64, 16, BF), (2, 1, 32, 24, SF), (2, 2, 128, 8, HF), (2, 1, 128, 48, BF)])      # tiles on the decode kernels
def test_prompt_chunks(cuda_device, hq, hkv, d, ps, dt, splits, window):
    """A chunk over cached context, a whole prompt, one of a tile's length + 1, decode items beside them; one of the
    sequences has a chunk and a separate early query."""
    lens = [260, 150, 129, 400, 33, 90]
    queries = [(0, 100 + i) for i in range(160)] + [(1, i) for i in range(150)] + [(4, 32)] + \
              [(2, i) for i in range(129)] + [(3, 399), (0, 3)] + [(5, 60 + i) for i in range(16)]
    case = build_case("mass", 8, lens, queries, hq, hkv, d, d, ps, dt, 1 / np.sqrt(d))
    verify(case, splits, True, window)


def test_mixed_step_beside_and_in_turn(cuda_device):
    """A step large enough to run its decode items on the thread's second stream, and the same step captured on a
    thread that has none: the same bits, weights that add to one per query and head, and float64 sums for a sequence
    of each kind.  Also with a sequence that has a chunk and an early query (its totals then wait for each other)."""
    import threading
    from workloads import mixed_prefill_decode_bf16
    base = mixed_prefill_decode_bf16(n_prefill=8, chunk=512, off_hi=4096, n_decode=120)
    for extra in ([], [(0, 0)]):
        if extra and base.meta["prefill_offsets"][0] == 0:
            continue
        case = mixed_prefill_decode_bf16(n_prefill=8, chunk=512, off_hi=4096, n_decode=120)
        if extra:
            case.query_seq = np.append(case.query_seq, np.int32(0))
            case.query_pos = np.append(case.query_pos, np.int32(0))
            case.q = torch.cat([case.q, case.q[:1]])
            case.new_k, case.new_v = torch.cat([case.new_k, case.new_k[:1]]), torch.cat([case.new_v, case.new_v[:1]])
        dc, plan = case.to("cuda"), plan_for(case)
        pka.paged_kv_store(plan, dc.new_k, dc.new_v, dc.k_cache, dc.v_cache)
        assert pka.paged_attn_decode_sms_beside_prefill(plan, case.hq, case.hkv, 128, 128) > 0
        mass = torch.zeros(case.num_pages, case.hkv, 16, device="cuda")
        ws = pka.make_mass_workspace(plan, case.hq, case.hkv, 128, 1)
        call = lambda m: pka.paged_attn_forward_mass(plan, dc.q, dc.k_cache, dc.v_cache, m, case.scale, splits=1,   # noqa: E731
                                                     workspace=ws)
        out = call(mass)
        torch.cuda.synchronize()
        assert pka.device_status() == 0
        serial, box = torch.zeros_like(mass), {}

        def captured():
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                box["out"] = call(serial)
            g.replay()
            torch.cuda.synchronize()
            box["graph"] = g
        t = threading.Thread(target=captured)
        t.start()
        t.join()
        assert pka.device_status() == 0
        assert torch.equal(out, box["out"]) and torch.equal(mass, serial)
        got = mass.double().cpu().numpy()
        k = dc.k_cache.double()
        for s, n in enumerate(case.seq_lens):
            used = np.asarray(case.block_table)[s][: -(-int(n) // 16)]
            mine = np.nonzero(np.asarray(case.query_seq) == s)[0]
            assert np.allclose(got[used].sum((0, 2)), 4.0 * len(mine), rtol=1e-4)
            if s not in (0, 3, 8, 127):
                continue
            keys = k[torch.as_tensor(used).cuda().long()].reshape(-1, 8, 128)[:n]
            q = dc.q[torch.as_tensor(mine).cuda()].double().view(len(mine), 8, 4, 128)
            logit = torch.einsum("qhgd,nhd->hgqn", q, keys) * case.scale
            pos = torch.as_tensor(np.asarray(case.query_pos)[mine]).cuda()[:, None]
            logit.masked_fill_(torch.arange(int(n), device="cuda") > pos, -np.inf)
            want = logit.softmax(-1).sum((1, 2)).cpu().numpy()            # [Hkv, n]
            have = got[used].transpose(1, 0, 2).reshape(8, -1)[:, :n]
            assert np.max(np.abs(have - want) / want) < weight_tolerance(case, torch.nan_to_num(dc.k_cache.cpu())) + len(mine) * 2.0 ** -23


@pytest.mark.parametrize("window", [0, 40])
def test_prompt_chunks_not_causal(cuda_device, window):
    queries = [(0, 100 + i) for i in range(60)] + [(1, 40)]
    case = build_case("mass", 9, [260, 50], queries, 4, 2, 128, 128, 16, BF, 0.09)
    verify(case, 1, False, window)


def test_large_scores(cuda_device):
    """Weights of one key near 1 and of the others near 0; scores in the hundreds."""
    case = decode_case(8, 2, 128, 128, 16, BF)
    case.scale = 4.0
    out, mass, before, dc, _ = run_case(case)
    added, seen = key_mass(case, dc.k_cache)
    got = (mass - before).double().cpu().numpy()
    # the weights of a row add to 1 whatever their errors: compare totals per sequence and head
    for s, n in enumerate(case.seq_lens):
        used = np.asarray(case.block_table)[s][: -(-int(n) // 16)]
        assert np.allclose(got[used].sum((0, 2)), 4.0, atol=4e-4)
    assert np.isfinite(got).all()


def test_nan_query_reaches_only_its_own_sequence(cuda_device):
    case = decode_case(8, 2, 128, 128, 16, BF)
    case.q[1] = float("nan")
    _, mass, before, _, _ = run_case(case)
    used = lambda s: torch.as_tensor(np.asarray(case.block_table)[s][: -(-int(case.seq_lens[s]) // 16)]).cuda()  # noqa: E731
    assert torch.isnan(mass[used(1)]).any()
    for s in (0, 2, 3):
        assert torch.isfinite(mass[used(s)]).all()


def test_reused_workspace_and_two_calls(cuda_device):
    """A workspace of another plan's leftovers; two calls add twice."""
    case = decode_case(16, 2, 128, 128, 16, BF)
    big = torch.full((1 << 20,), float("nan"), device="cuda")
    out, once, before, _, _ = run_case(case, 2, workspace=big)
    _, twice, _, _, _ = run_case(case, 2, workspace=big, calls=2)
    assert torch.allclose(twice - before, 2 * (once - before), rtol=1e-4, atol=1e-6)


def test_captured_decode_loop(cuda_device):
    """advance + append + attend captured once; the replays add at growing lengths.  A workspace with room for them is
    enough; one sized for the captured length alone reports PA_DEVICE_RANGE and leaves the totals."""
    steps = 20
    lens = [40, 5]
    table = [[0, 1, 2, 3], [4, 5, 6, 7]]
    gen = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.bfloat16)   # noqa: E731
    q, nk, nv = rnd(2, 8, 128), rnd(2, 2, 128), rnd(2, 2, 128)
    k0, v0 = rnd(8, 16, 2, 128), rnd(8, 16, 2, 128)

    def loop(max_keys, captured):
        plan = pka.paged_attn_plan(lens, table, [0, 1], [n - 1 for n in lens], 16, 8, device="cuda")
        k, v, mass = k0.clone(), v0.clone(), torch.zeros(8, 2, 16, device="cuda")
        ws = pka.make_mass_workspace(plan, 8, 2, 128, 2, max_keys=max_keys)

        def one():
            pka.paged_attn_plan_advance(plan)
            pka.paged_kv_store(plan, nk, nv, k, v)
            return pka.paged_attn_forward_mass(plan, q, k, v, mass, 0.09, splits=2, workspace=ws)
        if not captured:
            for _ in range(steps):
                out = one()
        else:
            out = one()
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                out = one()
            for _ in range(steps - 1):
                g.replay()
        torch.cuda.synchronize()
        return out.clone(), mass.clone()

    want, total = loop(64, False)
    assert pka.device_status() == 0
    got, mass = loop(64, True)
    assert pka.device_status() == 0
    assert torch.equal(got, want) and torch.equal(mass, total)
    got, mass = loop(0, True)            # rows of 64 keys (41 rounded up): the replays stay within
    assert pka.device_status() == 0 and torch.equal(mass, total)
    lens = [30, 5]                       # rows of 32 keys; the replays reach 50
    got, mass = loop(0, True)
    assert pka.device_status() == 4
    want, total = loop(64, True)
    assert pka.device_status() == 0
    assert torch.equal(got, want)        # the outputs are right all the same
    assert torch.equal(mass[4:], total[4:]) and not torch.equal(mass[:4], total[:4])


def test_two_streams_at_once(cuda_device):
    """Calls on two streams with a workspace and totals each, on one plan and cache: the bits of calls in turn."""
    lens = [700, 350, 300]
    queries = [(0, i) for i in range(300, 700)] + [(1, 349), (2, 298), (2, 299)]
    case = build_case("mass", 12, lens, queries, 8, 2, 128, 128, 16, BF, 0.088)
    dc, plan = case.to("cuda"), plan_for(case)
    pka.paged_kv_store(plan, dc.new_k, dc.new_v, dc.k_cache, dc.v_cache)
    call = lambda m, ws: pka.paged_attn_forward_mass(plan, dc.q, dc.k_cache, dc.v_cache, m, case.scale, splits=2,   # noqa: E731
                                                     workspace=ws)
    new = lambda: (torch.zeros(case.num_pages, 2, 16, device="cuda"), pka.make_mass_workspace(plan, 8, 2, 128, 2))   # noqa: E731
    want, (m0, ws) = None, new()
    for _ in range(3):
        want = call(m0, ws)
    torch.cuda.synchronize()
    both = [(torch.cuda.Stream(), *new()) for _ in range(2)]
    torch.cuda.synchronize()
    outs = [None, None]
    for _ in range(3):
        for i, (st, m, w) in enumerate(both):
            with torch.cuda.stream(st):
                outs[i] = call(m, w)
    torch.cuda.synchronize()
    assert pka.device_status() == 0
    for i, (_, m, _) in enumerate(both):
        assert torch.equal(outs[i], want) and torch.equal(m, m0)


def test_refusals(cuda_device):
    case = decode_case(4, 2, 64, 64, 16, BF, lens=(20, 20))
    dc, plan = case.to("cuda"), plan_for(case)
    mass = torch.zeros(case.num_pages, 2, 16, device="cuda")
    call = lambda m=mass, p=plan, **k: pka.paged_attn_forward_mass(p, dc.q, dc.k_cache, dc.v_cache, m, 0.1, **k)  # noqa: E731
    for m in (mass[:1], mass.transpose(1, 2).contiguous(), mass[:, :, None]):
        with pytest.raises(ValueError):
            call(m)
    with pytest.raises(TypeError):
        call(mass.half())
    with pytest.raises(ValueError):
        call(mass.cpu())
    with pytest.raises(pka.PagedAttentionError, match="overlaps"):
        call(torch.zeros(mass.numel() + 64, device="cuda")[:mass.numel()].view(mass.shape), splits=1,
             workspace=dc.v_cache.view(-1).view(torch.float32))
    with pytest.raises(pka.PagedAttentionError, match="overlaps"):
        call(dc.k_cache.view(-1).view(torch.float32)[:mass.numel()].view(mass.shape))
    status = lambda **k: pytest.raises(pka.PagedAttentionError, call, **k).value.status   # noqa: E731
    assert status(splits=0) == 7 and status(splits=65) == 7
    assert status(splits=2, workspace=torch.empty(64, device="cuda")) == 6
    assert status(window=-1, splits=1, workspace=torch.empty(1 << 16, device="cuda")) == 1
    shared = pka.paged_attn_plan([40, 40], [[0, 1, 2], [0, 3, 1]], [0, 1], [39, 39], 16, case.num_pages, device="cuda")
    assert status(p=shared, splits=1) == 5
    assert torch.all(mass == 0)
