"""NaN and infinity among a prompt chunk's values reach the queries that see them and no others.

Rows that some queries of a tile see and others do not: the chunk's own tokens (the diagonal) and, under a window, the
keys that leave it.  The float64 form sees each query's keys alone.
"""
import numpy as np
import pytest
import torch

import paged_kv_attention_20_gb300 as pka
from q8_reference import E4M3, HALF_STEP, TINY, attend, quantise, slots

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
P_ERROR = {torch.float16: 2.0 ** -10, torch.bfloat16: 2.0 ** -8}      # of a weight, in the coarser of the kernels
HQ, HKV, D = 4, 2, 128
KINDS = (float("nan"), float("inf"), float("-inf"))


def case(lens, runs, ps, dt, bad, bad_keys=(), seed=31):
    """Caches of paged 16-bit rows with bad[(s, key)] = (head, dim, value); the queries are `runs` of positions."""
    gen = torch.Generator().manual_seed(seed)
    used = [-(-n // ps) for n in lens]
    pool = sum(used) + 1
    order = torch.randperm(pool, generator=gen).tolist()
    table, at = np.full((len(lens), max(used)), -1, dtype=np.int64), 0
    for s, n in enumerate(used):
        table[s, :n] = order[at:at + n]
        at += n
    k, v = (torch.randn(pool * ps, HKV, D, generator=gen).to(dt) for _ in "kv")
    for (s, j), (h, e, x) in bad.items():
        v[slots(table, ps, s, lens[s])[j], h, e] = x
    for s, j, h in bad_keys:
        k[slots(table, ps, s, lens[s])[j], h, 9] = float("nan")
    queries = [(s, p) for s, r in runs for p in r]
    seq, pos = [s for s, _ in queries], [p for _, p in queries]
    plan = pka.paged_attn_plan(lens, table, seq, pos, ps, pool, device="cuda")
    q = (torch.randn(len(queries), HQ, D, generator=gen) / 2).to(dt)
    return plan, q, k, v, (lens, table, ps, seq, pos), pool


def check(got, q, k, v, rest, dt, causal, window, what):
    """Bits that are not finite where the formula's are, the others within their tolerance."""
    with np.errstate(invalid="ignore"):
        want = attend(q, k, v, *rest, D ** -0.5, causal, window)[0]
        kept = np.nan_to_num(k, nan=0.0), np.nan_to_num(v, nan=0.0, posinf=0.0, neginf=0.0)
        clean, size, off, most = attend(q, *kept, *rest, D ** -0.5, causal, window)
    got = got.cpu().double().numpy()
    odd = ~np.isfinite(want)
    assert np.array_equal(np.isfinite(got), ~odd), (what, int((np.isfinite(got) == odd).sum()))
    # A key of another split in a tile that a split loads weighs 0 there, and 0 * inf is NaN, as is NaN + inf in the
    # merge: an infinite output of a split call may come as NaN.  Neither reaches a query that does not see the key.
    split = "split" in what or what == "shared"
    same = (got == want) | np.isnan(got) if split else (got == want) | (np.isnan(got) & np.isnan(want))
    assert same[odd].all() and not (np.isnan(want) & ~np.isnan(got)).any(), what
    err = (off + P_ERROR[dt]) * size + 2.0 ** -30 * most
    tol = HALF_STEP[dt] * (np.abs(clean) + err) + err + TINY[dt]
    assert (np.abs(got - clean) <= tol)[~odd].all(), what
    return odd


def some(keys, seed):
    """A few elements a key, in turn NaN, +inf and -inf."""
    r = np.random.default_rng(seed)
    return {k: (int(r.integers(HKV)), int(r.integers(D)), KINDS[i % 3]) for i, k in enumerate(keys)}


# (lens, runs, keys whose values are not finite): one tile, tiles off and on a tile's border, several tiles, two chunks
CASES = [
    ([300], [(0, range(260, 300))], [(0, 299), (0, 270), (0, 241), (0, 260)]),
    ([256], [(0, range(128, 256))], [(0, 255), (0, 128), (0, 200), (0, 127), (0, 64)]),
    ([700], [(0, range(333, 700))], [(0, 699), (0, 420), (0, 500), (0, 501), (0, 340), (0, 250), (0, 300)]),
    ([150, 40, 90], [(0, range(16)), (1, range(40)), (2, range(60, 90))], [(0, 15), (0, 149), (1, 39), (1, 0), (1, 20), (2, 89), (2, 55)]),
    ([130], [(0, range(100, 116)), (0, range(129, 130))], [(0, 129), (0, 120), (0, 115), (0, 114)]),
]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("case_at", range(len(CASES)))
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1), (True, 20), (True, 150), (False, 0), (False, 30)])
def test_values(cuda_device, dt, case_at, causal, window):
    lens, runs, keys = CASES[case_at]
    for ps in (16, 128):
        plan, q, k, v, rest, pool = case(lens, runs, ps, DT[dt], some(keys, case_at))
        dev = q.cuda(), k.cuda().view(pool, ps, HKV, D), v.cuda().view(pool, ps, HKV, D)
        f64 = k.double().numpy(), v.double().numpy()
        outs = {"whole": pka.paged_attn_forward(plan, *dev, D ** -0.5, causal=causal, window=window)}
        for n in (2, 5):
            outs[f"{n} splits"] = pka.paged_attn_forward_split(plan, *dev, D ** -0.5, n, causal=causal, window=window)
        if window == 0:
            outs["shared"] = pka.paged_attn_forward_shared(plan, *dev, D ** -0.5, 0, splits=(1, 2), causal=causal)
        for what, out in outs.items():
            odd = check(out, q, *f64, rest, DT[dt], causal, window, what)
            assert odd.any() or window == 1
    assert pka.device_status() == 0


@pytest.mark.parametrize("window", [0, 20, 150])
def test_every_element_of_some_rows(cuda_device, window):
    """Whole rows, and NaN keys beside them; the totals of the keys' weights are taken in the same call."""
    lens, ps, dt = [300], 16, torch.bfloat16
    plan, q, k, v, rest, pool = case(lens, [(0, range(210, 300))], ps, dt, {}, bad_keys=[(0, 298, 1)])
    at = slots(rest[1], ps, 0, 300)
    v[at[[215, 255, 256, 290]]] = torch.tensor(KINDS + (float("nan"),)).to(dt)[:, None, None]
    dev = q.cuda(), k.cuda().view(pool, ps, HKV, D), v.cuda().view(pool, ps, HKV, D)
    f64 = k.double().numpy(), v.double().numpy()
    check(pka.paged_attn_forward(plan, *dev, D ** -0.5, window=window), q, *f64, rest, dt, True, window, "whole")
    mass = torch.zeros(pool, HKV, ps, device="cuda")
    out = pka.paged_attn_forward_mass(plan, *dev, mass, D ** -0.5, window=window)
    check(out, q, *f64, rest, dt, True, window, "with totals")
    assert pka.device_status() == 0


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("case_at", range(len(CASES)))
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 20), (True, 150), (False, 0)])
def test_8_bit_cache(cuda_device, dt, case_at, causal, window):
    """What is not finite is NaN there, in chunks as among drafted tokens."""
    lens, runs, keys = CASES[case_at]
    plan, q, k, v, rest, pool = case(lens, runs, 16, DT[dt], some(keys, case_at))
    dev, f64 = [q.cuda()], []
    scales = []
    for x in (k, v):
        c, b = quantise(x)
        f64.append(c * 2.0 ** (b - 127.0)[..., None])
        dev.append(torch.from_numpy(c).float().to(E4M3).cuda().view(pool, 16, HKV, D))
        scales.append(torch.from_numpy(b).to(torch.uint8).view(pool, 16, HKV).transpose(1, 2).contiguous().cuda())
    for n in (1, 3):
        out = pka.paged_attn_forward_q8(plan, *dev, *scales, D ** -0.5, splits=n, causal=causal, window=window)
        check(out, q, *f64, rest, DT[dt], causal, window, f"{n} splits")
    assert pka.device_status() == 0
