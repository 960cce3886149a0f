"""Per-head norm + rotation + append against the float64 formulas, and its refusals.

Tolerance: the fp32 arithmetic of an element is off by less than 32 roundings of
2^-24 of its pair's magnitude |a| + |b| (sum of squares <= 38 terms in a row,
halved by the root; root, three products, one addition), then one rounding of
half a step of the operand type.
"""
import numpy as np
import pytest
import torch

import paged_kv_attention_20_gb300 as pka
from cache_ops_reference import norm_rope
from helpers import bits_equal, plan_for
from workloads import build_case, decode_queries

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}


def table(far, rot, base=10000.0):
    angle = np.arange(far)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1)).float()


def check(got, ref, size, dt, what):
    got = got.detach().cpu().double().numpy()
    fp32 = 32 * 2.0 ** -24 * size
    tol = HALF_STEP[dt] * (np.abs(ref) + fp32) + fp32 + TINY[dt]
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} elements off, worst {np.max(np.abs(got - ref) / tol):.2f} tolerances"


def step(seq_lens, queries, hq, hkv, d, dv, ps, dt, rot, interleaved=False, norms="qk", positions=None, far=500,
         fused=False, reset=True, eps=1e-6, alias=False, seed=5):
    case = build_case("rope", seed, seq_lens, queries, hq, hkv, d, dv, ps, dt, 0.1, pool_pages=None if sum(seq_lens) > 140 else 140)
    dc = case.to("cuda")
    plan = plan_for(case)
    gen = torch.Generator().manual_seed(seed)
    qw = (1 + 0.2 * torch.randn(d, generator=gen)).to(dt) if "q" in norms else None
    kw = (1 + 0.2 * torch.randn(d, generator=gen)).to(dt) if "k" in norms else None
    tab = table(far, rot) if rot else None
    q, nk, nv = dc.q, dc.new_k, dc.new_v
    if fused:   # three views of one projection output
        n = case.num_queries
        rows = torch.cat([q.reshape(n, -1), nk.reshape(n, -1), nv.reshape(n, -1)], 1).contiguous()
        q = rows[:, :hq * d].view(n, hq, d)
        nk = rows[:, hq * d:(hq + hkv) * d].view(n, hkv, d)
        nv = rows[:, (hq + hkv) * d:].view(n, hkv, dv)
    mass = torch.rand(case.num_pages, hkv, ps, device="cuda") + 1 if reset else None
    before = None if mass is None else mass.clone()
    k0, v0 = dc.k_cache.clone(), dc.v_cache.clone()
    pos = None if positions is None else torch.tensor(positions, dtype=torch.int32, device="cuda")
    cu = lambda t: None if t is None else t.cuda()                     # noqa: E731
    out = pka.paged_qk_norm_rope_store(plan, q, nk, nv, dc.k_cache, dc.v_cache, rope_table=cu(tab), q_weight=cu(qw),
                                       k_weight=cu(kw), eps=eps, interleaved=interleaved, positions=pos, key_mass=mass,
                                       q_out=q if alias else None)
    torch.cuda.synchronize()
    assert pka.device_status() == 0
    at = np.asarray(case.query_pos if positions is None else positions)
    cos = sin = None
    if rot:
        t = tab.double().numpy()
        cos, sin = t[at, :rot // 2], t[at, rot // 2:]
    ref, size = norm_rope(case.q, qw, eps, cos, sin, interleaved)
    check(out, ref, size, dt, "q")
    ref, size = norm_rope(case.new_k, kw, eps, cos, sin, interleaved)
    page = np.asarray(case.block_table)[case.query_seq, np.asarray(case.query_pos) // ps]
    row = np.asarray(case.query_pos) % ps
    check(dc.k_cache[page, row], ref, size, dt, "k")
    assert bits_equal(dc.v_cache[page, row].cpu(), case.new_v)
    # nothing else of the caches moved
    k0[page, row], v0[page, row] = dc.k_cache[page, row], dc.v_cache[page, row]
    assert bits_equal(dc.k_cache, k0) and bits_equal(dc.v_cache, v0)
    if reset:
        before[page, :, row] = 0
        assert torch.equal(mass, before)
    return out


LENS = [1, 17, 64, 40]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("hq,hkv,d,dv,ps,rot,inter", [
    (32, 8, 128, 128, 16, 128, False), (4, 4, 64, 64, 16, 32, True), (12, 4, 96, 96, 24, 32, False),
    (6, 2, 80, 64, 5, 80, True), (8, 1, 256, 128, 16, 64, False), (3, 3, 16, 16, 1, 16, False),
    (4, 2, 512, 512, 16, 512, False), (2, 1, 1024, 1024, 16, 1024, True), (5, 5, 40, 24, 3, 20, False),
    (2, 2, 7, 5, 4, 6, True), (2, 1, 1, 3, 4, 0, False), (2, 2, 130, 6, 4, 2, False)])
def test_shapes(cuda_device, dt, hq, hkv, d, dv, ps, rot, inter):
    step(LENS, decode_queries(LENS) + [(3, 0), (2, 5)], hq, hkv, d, dv, ps, dt, rot, inter)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [128, 40])
@pytest.mark.parametrize("norms", ["", "q", "k", "qk"])
@pytest.mark.parametrize("rot", [0, 40])
def test_optional_parts(cuda_device, dt, d, norms, rot):
    step(LENS, decode_queries(LENS), 4, 2, d, d, 16, dt, rot if d == 40 else (rot and 64), norms=norms, reset=False)


@pytest.mark.parametrize("d,dv", [(128, 128), (96, 64), (30, 30)])
def test_views_of_one_projection(cuda_device, d, dv):
    step(LENS, decode_queries(LENS), 8, 2, d, dv, 16, torch.bfloat16, 30 if d == 30 else 96 if d == 96 else 128, fused=True)


@pytest.mark.parametrize("d", [128, 36])
def test_queries_in_place(cuda_device, d):
    step(LENS, decode_queries(LENS), 8, 2, d, d, 16, torch.float16, 36 if d == 36 else 64, alias=True)


def test_positions_ahead_of_the_slots(cuda_device):
    """After an eviction a key's place in the text is ahead of its cache row."""
    step(LENS, decode_queries(LENS), 8, 2, 128, 128, 16, torch.bfloat16, 128, positions=[130000, 7, 131071, 0], far=131072)


def test_one_query(cuda_device):
    step([33], [(0, 32)], 32, 8, 128, 128, 16, torch.bfloat16, 128)


def test_prompt_chunk(cuda_device):
    step([700], [(0, i) for i in range(3, 700)], 16, 4, 128, 128, 16, torch.bfloat16, 128, far=700)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("hq,hkv,d,dv,ps,rot,inter,kw", [
    (8, 2, 128, 128, 16, 128, False, dict(fused=True)), (3, 1, 64, 32, 16, 32, True, {}), (4, 4, 96, 64, 24, 64, False, {}),
    (2, 2, 256, 256, 64, 128, True, dict(alias=True, norms="q")), (5, 1, 512, 8, 16, 512, False, dict(norms="k")),
    (2, 1, 16, 16, 16, 16, False, dict(norms="", reset=False)), (6, 2, 128, 128, 16, 0, False, {})])
def test_many_tokens(cuda_device, dt, hq, hkv, d, dv, ps, rot, inter, kw):
    """Prompts long enough for the streaming kernel: every shape it takes, its last tokens ragged over the warps."""
    lens = [1500, 801, 33]
    queries = [(s, i) for s, n in enumerate(lens) for i in range(n) if (s, i) != (0, 5)]
    step(lens, queries, hq, hkv, d, dv, ps, dt, rot, inter, far=1500, **kw)


def test_many_tokens_with_positions_outside_the_table(cuda_device):
    lens = [2500]
    case = build_case("rope", 9, lens, [(0, i) for i in range(2500)], 4, 2, 64, 64, 16, torch.bfloat16, 0.1)
    dc, plan = case.to("cuda"), plan_for(case)
    pos = torch.arange(2500, dtype=torch.int32, device="cuda")
    bad = [0, 1, 700, 2499]
    pos[bad] = torch.tensor([-5, 2500, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    good = torch.ones(2500, dtype=torch.bool, device="cuda")
    good[bad] = False
    k0, v0 = dc.k_cache.clone(), dc.v_cache.clone()
    out = torch.full_like(dc.q, 7.0)
    tab = table(2500, 64)
    pka.paged_qk_norm_rope_store(plan, dc.q, dc.new_k, dc.new_v, dc.k_cache, dc.v_cache, rope_table=tab.cuda(),
                                 positions=pos, q_out=out)
    torch.cuda.synchronize()
    assert pka.device_status() == 4
    t = tab.double().numpy()
    ref, size = norm_rope(case.q, None, 0, t[np.arange(2500), :32], t[np.arange(2500), 32:], False)
    check(out[good], ref[good.cpu().numpy()], size[good.cpu().numpy()], torch.bfloat16, "q")
    assert torch.all(out[~good] == 7)
    page = np.asarray(case.block_table)[0, np.arange(2500) // 16]
    row = np.arange(2500) % 16
    assert bits_equal(dc.k_cache[page, row][~good], k0[page, row][~good])
    assert bits_equal(dc.v_cache[page, row][~good], v0[page, row][~good])
    assert bits_equal(dc.v_cache[page, row][good].cpu(), case.new_v[good.cpu()])


def test_zero_and_large_rows(cuda_device):
    """A row of zeros stays zero (eps > 0); rows of the type's largest values keep their direction."""
    case = build_case("rope", 3, [4], [(0, 3)], 2, 2, 64, 64, 4, torch.float16, 0.1)
    dc = case.to("cuda")
    q = torch.zeros_like(dc.q)
    q[0, 1] = 65504.0
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    out = pka.paged_qk_norm_rope_store(plan_for(case), q, dc.new_k, dc.new_v, dc.k_cache, dc.v_cache, q_weight=w)
    assert torch.all(out[0, 0] == 0) and torch.all(out[0, 1] == 1)


def test_position_outside_the_table(cuda_device):
    """That query's rows stay as they were, the others are written, and the status word says so."""
    case = build_case("rope", 4, [9, 20], decode_queries([9, 20]), 4, 2, 64, 64, 16, torch.bfloat16, 0.1)
    for bad in (-1, 50, 2 ** 31 - 1):
        dc = case.to("cuda")
        k0 = dc.k_cache.clone()
        out = torch.full_like(dc.q, 7.0)
        pos = torch.tensor([bad, 49], dtype=torch.int32, device="cuda")
        pka.paged_qk_norm_rope_store(plan_for(case), dc.q, dc.new_k, dc.new_v, dc.k_cache, dc.v_cache,
                                     rope_table=table(50, 64).cuda(), positions=pos, q_out=out)
        torch.cuda.synchronize()
        assert pka.device_status() == 4
        assert torch.all(out[0] == 7) and not torch.any(out[1] == 7)
        page = np.asarray(case.block_table)[0, 0]
        assert bits_equal(dc.k_cache[page, 8], k0[page, 8])
    assert pka.device_status() == 0


def test_empty_plan_and_refusals(cuda_device):
    plan = pka.paged_attn_plan([3], [[0]], [], [], 4, 1, device="cuda")
    kc = torch.ones(1, 4, 1, 8, device="cuda")
    e = torch.empty(0, 1, 8, device="cuda")
    assert pka.paged_qk_norm_rope_store(plan, e, e, e, kc, kc.clone()).shape == (0, 1, 8)
    plan = pka.paged_attn_plan([3], [[0]], [0], [2], 4, 1, device="cuda")
    x = torch.ones(1, 1, 8, device="cuda")
    call = lambda **k: pka.paged_qk_norm_rope_store(plan, k.pop("q", x), k.pop("nk", x), x, kc, kc.clone(), **k)  # noqa: E731
    tab = torch.zeros(4, 8, device="cuda")
    big = torch.ones(40, device="cuda")
    for kw in (dict(q_out=kc.view(4, 1, 8)[:1]), dict(q_out=x), dict(q=big[:8].view(1, 1, 8), q_out=big[4:12].view(1, 1, 8)),
               dict(q=kc.view(4, 1, 8)[:1]), dict(nk=kc.view(4, 1, 8)[3:]), dict(key_mass=kc.view(-1)[:4].view(1, 1, 4)),
               dict(q_weight=kc.view(-1)[24:]), dict(rope_table=kc.view(4, 8)), dict(rope_table=tab[:, :7].contiguous()), dict(rope_table=torch.zeros(4, 10, device="cuda")),
               dict(positions=torch.zeros(1, dtype=torch.int32, device="cuda")),
               dict(q_weight=torch.ones(8, device="cuda"), eps=float("nan")),
               dict(q_weight=torch.ones(8, device="cuda"), eps=-1.0)):
        with pytest.raises(pka.PagedAttentionError):
            call(**kw)
    for kw in (dict(rope_table=tab[:0]), dict(q_weight=torch.ones(7, device="cuda")), dict(rope_table=tab, positions=torch.zeros(2, dtype=torch.int32, device="cuda")),
               dict(key_mass=torch.zeros(1, 4, 1, device="cuda")), dict(q=torch.ones(1, 1, 9, device="cuda")),
               dict(q=torch.ones(1, 8, 2, device="cuda").transpose(1, 2)), dict(nk=torch.ones(1, 2, 8, device="cuda")),
               dict(rope_table=tab.cpu())):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(rope_table=tab.double()), dict(q=x.half())):
        with pytest.raises(TypeError):
            call(**kw)
    assert pka.device_status() == 0


def test_captured_and_replayed_on_another_stream(cuda_device):
    case = build_case("rope", 6, LENS, decode_queries(LENS), 8, 2, 128, 128, 16, torch.bfloat16, 0.1)
    dc, eager = case.to("cuda"), case.to("cuda")
    plan, tab = plan_for(case), table(100, 128).cuda()
    w = torch.rand(128, device="cuda").to(torch.bfloat16)
    args = dict(rope_table=tab, q_weight=w, k_weight=w)
    want = pka.paged_qk_norm_rope_store(plan, eager.q, eager.new_k, eager.new_v, eager.k_cache, eager.v_cache, **args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        out = pka.paged_qk_norm_rope_store(plan, dc.q, dc.new_k, dc.new_v, dc.k_cache, dc.v_cache, **args)
    with torch.cuda.stream(side):
        g.replay()
        g.replay()
    torch.cuda.synchronize()
    assert bits_equal(out, want) and bits_equal(dc.k_cache, eager.k_cache) and bits_equal(dc.v_cache, eager.v_cache)
