"""A bounded-cache serving loop: norm + rotation + append, attention with key totals, eviction, over and over.

Two sequences start with a prompt chunk each and decode past their budgets; every few steps the cache is cut back, in
place or into fresh pages, and the loop goes on with positions ahead of the cache rows.  Each step is followed in
float64 on the host: the stored rows against the formulas, the output and the totals against the keys that are really
there (read back from the cache, so that roundings do not pile up), the eviction's choice against the totals on the
device.
"""
import numpy as np
import pytest
import torch

import paged_kv_attention_20_gb300 as pka
from cache_ops_reference import kept_keys, norm_rope, slots

pytestmark = pytest.mark.gpu

HQ, HKV, D, PS, POOL, ROT = 4, 2, 128, 16, 40, 64
G = HQ // HKV
SINK, RECENT, BUDGET, EVERY = 4, 8, 40, 6


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_loop(cuda_device, dt, in_place):
    gen = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=gen).to(dt)                  # noqa: E731
    scale = D ** -0.5
    angle = np.arange(300)[:, None] * 10000.0 ** (-np.arange(0, ROT, 2) / ROT)
    table = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1)).float()
    tab64, dtable = table.double().numpy(), table.cuda()
    qw, kw = (1 + 0.1 * rnd(D).float()).to(dt), (1 + 0.1 * rnd(D).float()).to(dt)
    k_cache = torch.full((POOL, PS, HKV, D), float("nan"), dtype=dt, device="cuda")
    v_cache, mass = k_cache.clone(), torch.full((POOL, HKV, PS), float("nan"), device="cuda")
    free = list(range(POOL))
    pages = [[free.pop() for _ in range(5)] for _ in range(2)]
    lens, text = [0, 0], [0, 0]                                             # keys in the cache, tokens so far
    total = [np.zeros((0, HKV)), np.zeros((0, HKV))]                        # float64 totals
    half = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}[dt]

    for step in range(26):
        new = [50, 33] if step == 0 else [1, 1 + step % 2]                  # prompt chunks, then one or two tokens
        seq = [s for s in range(2) for _ in range(new[s])]
        row = [lens[s] + i for s in range(2) for i in range(new[s])]
        at = [text[s] + i for s in range(2) for i in range(new[s])]
        n = len(seq)
        lens = [lens[s] + new[s] for s in range(2)]
        text = [text[s] + new[s] for s in range(2)]
        for s in range(2):
            while len(pages[s]) * PS < lens[s]:
                pages[s].append(free.pop())
        width = max(map(len, pages))
        bt = np.array([p + [-1] * (width - len(p)) for p in pages])
        plan = pka.paged_attn_plan(lens, bt, seq, row, PS, POOL, device="cuda")
        qkv = rnd(n, (HQ + 2 * HKV) * D)
        dev = qkv.cuda()
        q = pka.paged_qk_norm_rope_store(
            plan, dev[:, :HQ * D].view(n, HQ, D), dev[:, HQ * D:(HQ + HKV) * D].view(n, HKV, D),
            dev[:, (HQ + HKV) * D:].view(n, HKV, D), k_cache, v_cache, rope_table=dtable, q_weight=qw.cuda(),
            k_weight=kw.cuda(), positions=torch.tensor(at, dtype=torch.int32, device="cuda"), key_mass=mass)
        out = pka.paged_attn_forward_mass(plan, q, k_cache, v_cache, mass, scale)
        torch.cuda.synchronize()
        assert pka.device_status() == 0
        # what was stored
        cos, sin = tab64[at, :ROT // 2], tab64[at, ROT // 2:]
        want_q, size_q = norm_rope(qkv[:, :HQ * D].reshape(n, HQ, D), qw, 1e-6, cos, sin, False)
        want_k, size_k = norm_rope(qkv[:, HQ * D:(HQ + HKV) * D].reshape(n, HKV, D), kw, 1e-6, cos, sin, False)
        kc, vc = k_cache.cpu().double().numpy().reshape(-1, HKV, D), v_cache.cpu().double().numpy().reshape(-1, HKV, D)
        where = np.array([slots(bt, PS, s, r + 1)[r] for s, r in zip(seq, row)])
        fp32 = 32 * 2.0 ** -24
        for got, want, size in ((q.cpu().double().numpy(), want_q, size_q), (kc[where], want_k, size_k)):
            assert (np.abs(got - want) <= half * (np.abs(want) + fp32 * size) + fp32 * size).all()
        # attention and totals over the keys that are there
        qs, o = q.cpu().double().numpy(), out.cpu().double().numpy()
        m = mass.cpu().double().numpy().transpose(0, 2, 1).reshape(-1, HKV)
        for s in range(2):
            keys = slots(bt, PS, s, lens[s])
            total[s] = np.concatenate([total[s], np.zeros((new[s], HKV))])
            for i in [i for i in range(n) if seq[i] == s]:
                for h in range(HQ):
                    x = kc[keys[:row[i] + 1], h // G] @ qs[i, h] * scale
                    w = np.exp(x - x.max())
                    w /= w.sum()
                    total[s][:row[i] + 1, h // G] += w
                    ref = w @ vc[keys[:row[i] + 1], h // G]
                    assert np.max(np.abs(o[i, h] - ref)) <= (2e-2 if dt != torch.float32 else 1e-5 * np.sqrt(np.mean(ref ** 2)) + 2e-6)
            # weights are off by their scores' errors (2 * D * 2^-23 * |q||k| scale), totals by a rounding a step
            off = 2 * D * 2.0 ** -23 * np.linalg.norm(qs[[i for i in range(n) if seq[i] == s]], axis=-1).max() \
                * np.linalg.norm(kc[keys], axis=-1).max() * scale + 2.0 ** -19
            assert (np.abs(m[keys] - total[s]) <= (off + 2.0 ** -23 * (step + 52)) * total[s]).all()
        # cut the cache back
        if step % EVERY == EVERY - 1:
            kept_lens = [min(n_, BUDGET - 7 * s) for s, n_ in enumerate(lens)]
            new_pages = [p[:-(-k // PS)] if in_place else [free.pop() for _ in range(-(-k // PS))]
                         for p, k in zip(pages, kept_lens)]
            w2 = max(map(len, new_pages))
            kept_plan = pka.paged_attn_plan(kept_lens, np.array([p + [-1] * (w2 - len(p)) for p in new_pages]), [], [], PS,
                                            POOL, device="cuda")
            kept = pka.paged_kv_evict(plan, kept_plan, mass, k_cache, v_cache, sink=SINK, recent=RECENT).cpu().numpy()
            assert pka.device_status() == 0
            k2 = k_cache.cpu().double().numpy().reshape(-1, HKV, D)
            for s in range(2):
                keys, to = slots(bt, PS, s, lens[s]), slots(kept_plan_table(new_pages), PS, s, kept_lens[s])
                new_total = np.zeros((kept_lens[s], HKV))
                for h in range(HKV):
                    ids = kept_keys(m[keys, h].astype(np.float32), kept_lens[s], SINK, RECENT)
                    assert np.array_equal(kept[s, h, :kept_lens[s]], ids) and (kept[s, h, kept_lens[s]:] == -1).all()
                    assert np.array_equal(k2[to, h], kc[keys[ids], h])
                    new_total[:, h] = total[s][ids, h]
                total[s] = new_total
                free.extend(p for p in pages[s] if p not in new_pages[s])
            pages, lens = new_pages, kept_lens
    assert text[0] > 70 and lens[0] < 50


def kept_plan_table(pages):
    w = max(map(len, pages))
    return np.array([p + [-1] * (w - len(p)) for p in pages])


def test_offsets_past_32_bits(cuda_device):
    """The same step on a pool of 12 pages and on the last pages of one with 4.6 G elements a cache: the same bits."""
    hq, hkv, d, ps, dt = 8, 8, 256, 16, torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(8)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=dt)        # noqa: E731
    k0, v0, m0 = rnd(12, ps, hkv, d), rnd(12, ps, hkv, d), torch.rand(12, hkv, ps, generator=gen, device="cuda")
    q, nk, nv, w = rnd(3, hq, d), rnd(3, hkv, d), rnd(3, hkv, d), rnd(d)
    table = torch.rand(200, 128, generator=gen, device="cuda")
    lens, rows = [100, 50], np.array([[0, 1, 2, 3, 4, 5, 6], [7, 8, 9, 10, -1, -1, -1]])

    def step(pool, first):
        k, v = torch.empty(pool, ps, hkv, d, dtype=dt, device="cuda"), torch.empty(pool, ps, hkv, d, dtype=dt, device="cuda")
        mass = torch.empty(pool, hkv, ps, device="cuda")
        here = slice(first, first + 12)
        k[here], v[here], mass[here] = k0, v0, m0
        bt = np.where(rows >= 0, rows + first, -1)
        plan = pka.paged_attn_plan(lens, bt, [0, 0, 1], [98, 99, 49], ps, pool, device="cuda")
        kept_plan = pka.paged_attn_plan([40, 20], bt, [], [], ps, pool, device="cuda")
        got = [pka.paged_qk_norm_rope_store(plan, q, nk, nv, k, v, rope_table=table, q_weight=w, k_weight=w, key_mass=mass)]
        got.append(pka.paged_attn_forward_mass(plan, got[0], k, v, mass, d ** -0.5, splits=2))
        got.append(mass[here].clone())
        got.append(pka.paged_kv_evict(plan, kept_plan, mass, k, v, sink=2, recent=4))
        torch.cuda.synchronize()
        assert pka.device_status() == 0
        return got + [k[here].clone(), v[here].clone(), mass[here].clone()]

    small, large = step(12, 0), step(140_012, 140_000)
    for a, b in zip(small, large):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
