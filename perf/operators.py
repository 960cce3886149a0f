"""Measured cases of the serving-loop operators around the paged cache.

Three operators of one decode loop over a bounded paged cache:

  rope   per-head RMS norm of Q and new K, position rotation, and the append of K and V into the cache
  mass   paged attention that also adds every key's softmax weight to a per-key fp32 total
  evict  the keys with the smallest totals leave the cache, the others move up (into fresh pages here, so a pass
         can be repeated on the same state)

A case's sequence lengths follow from its `layout` number alone; everything else is drawn from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one new token of one sequence: what a single chat user's decode step pays per layer
        dict(name="rope-one-token", op="rope", dtype="bf16", hq=32, hkv=8, d=128, rot=128, interleaved=False,
             seqs=1, chunk=1, page=16, far=8192, moved=False, reset=False, layout=11),
        # the decode batch of the benchmark's GQA layer, positions that ran ahead of the slots after evictions,
        # far positions, totals of the new keys reset
        dict(name="rope-decode-batch", op="rope", dtype="bf16", hq=32, hkv=8, d=128, rot=128, interleaved=False,
             seqs=64, chunk=1, page=16, far=131072, moved=True, reset=True, layout=12),
        # prompt chunks of a prefill step
        dict(name="rope-prompt-chunks", op="rope", dtype="bf16", hq=32, hkv=8, d=128, rot=128, interleaved=False,
             seqs=8, chunk=2048, page=16, far=16384, moved=False, reset=True, layout=13),
        # odd sizes: 96-wide heads, a partial rotation of neighbouring pairs, pages of 24 rows, fp16
        dict(name="rope-odd-f16", op="rope", dtype="f16", hq=12, hkv=4, d=96, rot=32, interleaved=True,
             seqs=5, chunk=333, page=24, far=5000, moved=True, reset=False, layout=14),
        # the smallest attention call: a few short fp32 histories, no head groups
        dict(name="mass-tiny-f32", op="mass", dtype="f32", hq=4, hkv=4, d=64, page=16, n_pre=0, chunk=0, off=0,
             n_dec=4, run=1, lo=1, hi=200, window=0, layout=21),
        # the GQA decode layer
        dict(name="mass-decode", op="mass", dtype="bf16", hq=32, hkv=8, d=128, page=16, n_pre=0, chunk=0, off=0,
             n_dec=64, run=1, lo=512, hi=8192, window=0, layout=22),
        # few long histories, groups of eight query heads
        dict(name="mass-decode-long", op="mass", dtype="bf16", hq=64, hkv=8, d=128, page=16, n_pre=0, chunk=0, off=0,
             n_dec=4, run=1, lo=32768, hi=131072, window=0, layout=23),
        # a continuous-batching step: prompt chunks over cached context beside decode queries
        dict(name="mass-mixed", op="mass", dtype="bf16", hq=32, hkv=8, d=128, page=16, n_pre=8, chunk=512, off=4096,
             n_dec=120, run=1, lo=1024, hi=4096, window=0, layout=24),
        # four drafted tokens per sequence checked at once, 64-wide heads, a sliding window, fp16
        dict(name="mass-verify-window-f16", op="mass", dtype="f16", hq=16, hkv=8, d=64, page=32, n_pre=0, chunk=0,
             off=0, n_dec=24, run=4, lo=300, hi=5000, window=1000, layout=25),
        # one history passing its budget
        dict(name="evict-one", op="evict", dtype="bf16", hkv=8, d=128, page=16, seqs=1, lo=600, hi=600, share=0.85,
             sink=4, recent=64, layout=31),
        # a decode batch cut to half
        dict(name="evict-batch", op="evict", dtype="bf16", hkv=8, d=128, page=16, seqs=64, lo=512, hi=8192, share=0.5,
             sink=4, recent=128, layout=32),
        # two very long prompts cut to a quarter
        dict(name="evict-long", op="evict", dtype="bf16", hkv=8, d=128, page=16, seqs=2, lo=100000, hi=131072,
             share=0.25, sink=4, recent=1024, layout=33),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "mass", "evict"])
    layout = rng.randrange(1 << 20)
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "rope":
        d = rng.choice([64, 80, 96, 128, 128, 256])
        hkv = rng.choice([1, 2, 4, 8])
        chunk = rng.choice([1, 1, _log(rng, 2, 700)])
        return dict(op=op, dtype=dtype, hq=hkv * rng.choice([1, 2, 4, 8]), hkv=hkv, d=d,
                    rot=rng.choice([d, d, d // 2]), interleaved=rng.random() < 0.3,
                    seqs=_log(rng, 1, 200 if chunk == 1 else 8), chunk=chunk, page=rng.choice([16, 16, 24, 64]),
                    far=_log(rng, 2000, 131072), moved=rng.random() < 0.5, reset=rng.random() < 0.5, layout=layout)
    if op == "mass":
        kind = rng.choice(["decode", "long", "mixed", "verify", "f32"])
        hkv = rng.choice([1, 2, 4, 8])
        if kind == "f32":
            return dict(op=op, dtype="f32", hq=hkv * rng.choice([1, 2, 4]), hkv=hkv, d=rng.choice([64, 128]),
                        page=rng.choice([16, 24]), n_pre=0, chunk=0, off=0, n_dec=_log(rng, 1, 16), run=1, lo=1,
                        hi=_log(rng, 50, 2000), window=0, layout=layout)
        half = rng.choice(["bf16", "bf16", "f16"])
        if kind == "mixed":
            return dict(op=op, dtype=half, hq=hkv * rng.choice([1, 2, 4]), hkv=hkv, d=128, page=rng.choice([16, 32, 64]),
                        n_pre=_log(rng, 1, 6), chunk=_log(rng, 17, 700), off=_log(rng, 1, 3000),
                        n_dec=_log(rng, 1, 60), run=1, lo=1, hi=_log(rng, 100, 4000),
                        window=rng.choice([0, 0, _log(rng, 100, 2000)]), layout=layout)
        if kind == "long":
            return dict(op=op, dtype=half, hq=hkv * rng.choice([4, 8, 16]), hkv=hkv, d=128, page=rng.choice([16, 64]),
                        n_pre=0, chunk=0, off=0, n_dec=rng.randint(1, 2), run=1, lo=20000, hi=_log(rng, 30000, 131072),
                        window=0, layout=layout)
        return dict(op=op, dtype=half, hq=hkv * rng.choice([1, 2, 4, 8]), hkv=hkv, d=rng.choice([64, 128, 128]),
                    page=rng.choice([16, 32]), n_pre=0, chunk=0, off=0, n_dec=_log(rng, 1, 48),
                    run=1 if kind == "decode" else rng.randint(2, 6), lo=10, hi=_log(rng, 100, 8000),
                    window=rng.choice([0, 0, _log(rng, 64, 4000)]), layout=layout)
    hkv = rng.choice([1, 2, 4, 8])
    hi = _log(rng, 300, 131072)
    return dict(op=op, dtype=dtype, hkv=hkv, d=rng.choice([40, 64, 128, 128]), page=rng.choice([16, 24, 64]),
                seqs=max(1, min(64, 160000 // hi // (2 if dtype == "f32" else 1))), lo=max(200, hi // 3), hi=hi,
                share=rng.choice([0.1, 0.25, 0.5, 0.9]), sink=rng.randint(0, 8), recent=rng.randint(0, 64), layout=layout)


# ------------------------------------------------------------------ layouts --
def _lens(case):
    """Sequence lengths of a case: the longest first, the others uniform in the case's range."""
    r = random.Random(case["layout"])
    if case["op"] == "rope":
        return [r.randint(case["chunk"], case["chunk"] + 400) for _ in range(case["seqs"])]
    if case["op"] == "evict":
        return [case["hi"]] + [r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"] - 1)]
    pre = [r.randint(0, case["off"]) + case["chunk"] for _ in range(case["n_pre"])]
    dec = [max(case["run"], r.randint(case["lo"], case["hi"])) for _ in range(case["n_dec"])]
    if dec:
        dec[0] = max(case["run"], case["hi"])
    return pre + dec


def _kept_lens(case):
    floor = case["sink"] + case["recent"]
    return [min(n, max(floor, int(n * case["share"]))) for n in _lens(case)]


def _queries(case):
    """(sequence, position) of every packed query, sequence by sequence."""
    lens = _lens(case)
    if case["op"] == "rope":
        counts = [case["chunk"]] * case["seqs"]
    else:
        counts = [case["chunk"]] * case["n_pre"] + [case["run"]] * case["n_dec"]
    seq = [s for s, c in enumerate(counts) for _ in range(c)]
    pos = [lens[s] - c + i for s, c in enumerate(counts) for i in range(c)]
    return seq, pos


def _pages(lens, page):
    return [-(-n // page) for n in lens]


def prepare(case, seed):
    """The caches, the schedule and the step's rows, on the GPU."""
    dev, dt, ps = torch.device("cuda"), DTYPES[case["dtype"]], case["page"]
    gen = torch.Generator(device=dev).manual_seed(seed)
    host = random.Random(seed)
    lens = _lens(case)
    hkv, d = case["hkv"], case["d"]

    def randn(*shape, dtype=dt):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dtype) if dtype == torch.float32 \
            else torch.randn(shape, generator=gen, device=dev, dtype=dtype)

    used = _pages(lens, ps)
    fresh = _pages(_kept_lens(case), ps) if case["op"] == "evict" else []
    pool = sum(used) + sum(fresh) + 3
    order = list(range(pool))
    host.shuffle(order)
    width, at = max(used), 0
    table, dst_table = [], []
    for n in used:
        table.append(order[at:at + n] + [-1] * (width - n))
        at += n
    for n in fresh:
        dst_table.append(order[at:at + n] + [-1] * (max(fresh) - n))
        at += n
    state = {"case": case, "k_cache": randn(pool, ps, hkv, d), "v_cache": randn(pool, ps, hkv, d),
             "table": torch.tensor(table, device=dev), "lens": torch.tensor(lens, device=dev)}

    if case["op"] == "evict":
        # totals as they come from many steps: spread over decades, some equal, new keys at zero
        mass = torch.exp(2.0 * randn(pool, hkv, ps, dtype=torch.float32))
        state["mass"] = torch.where(mass < 0.2, torch.round(mass * 64) / 64, mass)
        state["dst_table"] = torch.tensor(dst_table, device=dev)
        state["kept_lens"] = torch.tensor(_kept_lens(case), device=dev)
        state["kept_max"] = max(_kept_lens(case))
        if own:  # the schedules that a serving loop has built for this step, before and after the eviction
            import paged_kv_attention_20_gb300 as pka
            state["plan"] = pka.paged_attn_plan(lens, table, [], [], ps, pool, device=dev)
            state["kept_plan"] = pka.paged_attn_plan(_kept_lens(case), dst_table, [], [], ps, pool, device=dev)
        return state

    seq, pos = _queries(case)
    nq, hq = len(seq), case["hq"]
    state["seq"], state["pos"] = torch.tensor(seq, device=dev), torch.tensor(pos, device=dev)
    if own:  # the schedule that a serving loop builds once a step and uses in every layer
        import paged_kv_attention_20_gb300 as pka
        state["plan"] = pka.paged_attn_plan(lens, table, seq, pos, ps, pool, device=dev)
    if case["op"] == "mass":
        state["q"] = randn(nq, hq, d)
        state["scale"] = 1.0 / math.sqrt(d)
        # totals of about one step's weights, so that what this step adds counts in full
        state["mass"] = 1e-3 * torch.rand(pool, hkv, ps, generator=gen, device=dev)
        if own:  # the split count and the workspace, kept from step to step
            state["splits"] = pka.paged_attn_split_heuristic(state["plan"], hq, hkv, window=case["window"])
            state["workspace"] = pka.make_mass_workspace(state["plan"], hq, hkv, d, state["splits"], case["window"])
        return state

    # rope: one fused projection row per token; q, k, v are views of it
    qkv = randn(nq, (hq + 2 * hkv) * d)
    state["q"] = qkv[:, :hq * d].view(nq, hq, d)
    state["new_k"] = qkv[:, hq * d:(hq + hkv) * d].view(nq, hkv, d)
    state["new_v"] = qkv[:, (hq + hkv) * d:].view(nq, hkv, d)
    state["q_weight"] = (1.0 + 0.1 * randn(d, dtype=torch.float32)).to(dt)
    state["k_weight"] = (1.0 + 0.1 * randn(d, dtype=torch.float32)).to(dt)
    rot = case["rot"]
    angle = torch.arange(case["far"], device=dev, dtype=torch.float64)[:, None] \
        * torch.pow(10000.0, -torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)
    state["rope_table"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    state["positions"] = None
    if case["moved"]:  # the positions in the text, ahead of the cache rows
        ahead = [host.randint(0, case["far"] - n) for n in lens]
        state["positions"] = torch.tensor([p + ahead[s] for s, p in zip(seq, pos)], device=dev, dtype=torch.int32)
    state["mass"] = torch.rand(pool, hkv, ps, generator=gen, device=dev) if case["reset"] else None
    return state


# --------------------------------------------------------------- plain forms --
def _norm_rope(x, w, cos, sin, interleaved):
    """x [T, H, D] in fp32: RMS norm of each head row, then the rotation of its first 2 * cos.shape[-1] dims."""
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
    half = cos.shape[-1]
    c, s = cos[:, None], sin[:, None]
    if interleaved:
        a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half:2 * half]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([turned, y[..., 2 * half:]], -1)


def _plain_rope(s):
    case, dt, ps = s["case"], s["q"].dtype, s["case"]["page"]
    rows = s["rope_table"][s["pos"] if s["positions"] is None else s["positions"].long()]
    half = case["rot"] // 2
    cos, sin = rows[:, :half], rows[:, half:]
    page = s["table"][s["seq"], s["pos"] // ps]
    s["k_cache"][page, s["pos"] % ps] = _norm_rope(s["new_k"].float(), s["k_weight"].float(), cos, sin,
                                                   case["interleaved"]).to(dt)
    s["v_cache"][page, s["pos"] % ps] = s["new_v"]
    if s["mass"] is not None:
        s["mass"][page, :, s["pos"] % ps] = 0.0
    return _norm_rope(s["q"].float(), s["q_weight"].float(), cos, sin, case["interleaved"]).to(dt)


def _plain_attend(s, first_seq, n_seqs, first_query, per_seq):
    """Attention of `n_seqs` sequences of `per_seq` queries each, and what it adds to the totals."""
    case, ps, hkv = s["case"], s["case"]["page"], s["case"]["hkv"]
    lens = s["lens"][first_seq:first_seq + n_seqs]
    table = s["table"][first_seq:first_seq + n_seqs].clamp(min=0)
    n_max = max(_lens(case)[first_seq:first_seq + n_seqs])
    j = torch.arange(n_max, device=lens.device)
    page, row = table[:, j // ps], (j % ps).expand(n_seqs, n_max)
    k, v = s["k_cache"][page, row].float(), s["v_cache"][page, row].float()      # [B, n, Hkv, D]
    nq = n_seqs * per_seq
    q = s["q"][first_query:first_query + nq].float().view(n_seqs, per_seq, hkv, -1, case["d"])
    pos = s["pos"][first_query:first_query + nq].view(n_seqs, per_seq, 1)
    seen = j <= pos
    if case["window"]:
        seen = seen & (j > pos - case["window"])
    w = torch.einsum("bqhgd,bnhd->bhgqn", q, k) * s["scale"]
    w = w.masked_fill_(~seen[:, None, None], -math.inf)
    w = torch.exp_(w.sub_(w.amax(-1, keepdim=True)))
    w = w.div_(w.sum(-1, keepdim=True))
    out = torch.einsum("bhgqn,bnhd->bqhgd", w, v).reshape(nq, case["hq"], case["d"])
    live = (j < lens[:, None])[:, None]
    at = (page[:, None] * hkv + torch.arange(hkv, device=j.device)[:, None]) * ps + row[:, None]
    added = w.sum((2, 3))                                                          # [B, Hkv, n]
    s["mass"].view(-1).index_add_(0, torch.where(live, at, 0).reshape(-1), torch.where(live, added, 0.0).reshape(-1))
    return out.to(s["q"].dtype)


def _plain_mass(s):
    c = s["case"]
    pre = [_plain_attend(s, 0, c["n_pre"], 0, c["chunk"])] if c["n_pre"] else []
    dec = [_plain_attend(s, c["n_pre"], c["n_dec"], c["n_pre"] * c["chunk"], c["run"])] if c["n_dec"] else []
    return torch.cat(pre + dec)


def _plain_evict(s):
    case, ps, hkv = s["case"], s["case"]["page"], s["case"]["hkv"]
    n, keep = s["lens"][:, None, None], s["kept_lens"][:, None, None]
    j = torch.arange(max(_lens(case)), device=n.device)
    page, row = s["table"].clamp(min=0)[:, j // ps], j % ps
    mass = s["mass"][page, :, row].transpose(1, 2)                                # [S, Hkv, n]
    # 2: always kept, 1: by total, 0: past the sequence's end
    kind = torch.where(j < n, torch.where((j < case["sink"]) | (j >= n - case["recent"]), 2, 1), 0).expand_as(mass)
    order = torch.sort(mass, dim=-1, descending=True, stable=True).indices
    order = order.gather(-1, torch.sort(kind.gather(-1, order), dim=-1, descending=True, stable=True).indices)
    rank = torch.arange(s["kept_max"], device=n.device)
    kept = torch.where(rank < keep, order[..., :s["kept_max"]], j.numel()).sort(-1).values
    live = rank < keep                                                            # [S, 1, K]
    src = torch.where(live, kept, 0)
    seq = torch.arange(src.shape[0], device=n.device)[:, None, None]
    head = torch.arange(hkv, device=n.device)[None, :, None]
    sp, sr = s["table"].clamp(min=0)[seq, src // ps], src % ps
    # rows of shorter sequences past their kept length go back where they came from
    dp = torch.where(live, s["dst_table"].clamp(min=0)[seq, rank // ps], sp)
    dr = torch.where(live, (rank % ps).expand_as(src), sr)
    k, v, m = s["k_cache"][sp, sr, head], s["v_cache"][sp, sr, head], s["mass"][sp, head, sr]
    s["k_cache"][dp, dr, head] = k
    s["v_cache"][dp, dr, head] = v
    s["mass"][dp, head, dr] = m
    return torch.where(live, kept, -1).to(torch.int32)


def run(state):
    op = state["case"]["op"]
    if own:
        import paged_kv_attention_20_gb300 as pka
        if op == "rope":
            q = pka.paged_qk_norm_rope_store(
                state["plan"], state["q"], state["new_k"], state["new_v"], state["k_cache"], state["v_cache"],
                rope_table=state["rope_table"], q_weight=state["q_weight"], k_weight=state["k_weight"], eps=1e-6,
                interleaved=state["case"]["interleaved"], positions=state["positions"], key_mass=state["mass"])
            return {"q": q, "k_cache": state["k_cache"], "v_cache": state["v_cache"], "mass": state["mass"]}
        if op == "mass":
            out = pka.paged_attn_forward_mass(
                state["plan"], state["q"], state["k_cache"], state["v_cache"], state["mass"], state["scale"],
                splits=state["splits"], workspace=state["workspace"], window=state["case"]["window"])
            return {"out": out, "mass": state["mass"]}
        kept = pka.paged_kv_evict(state["plan"], state["kept_plan"], state["mass"], state["k_cache"], state["v_cache"],
                                  sink=state["case"]["sink"], recent=state["case"]["recent"])
    elif op == "rope":
        q = _plain_rope(state)
        return {"q": q, "k_cache": state["k_cache"], "v_cache": state["v_cache"], "mass": state["mass"]}
    elif op == "mass":
        return {"out": _plain_mass(state), "mass": state["mass"]}
    else:
        kept = _plain_evict(state)
    return {"kept": kept, "k_cache": state["k_cache"], "v_cache": state["v_cache"], "mass": state["mass"]}


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    hkv, d, lens = case["hkv"], case["d"], _lens(case)
    if case["op"] == "rope":
        t = case["seqs"] * case["chunk"]
        row = case["hq"] * d + 2 * hkv * d
        table = min(t, case["far"]) * case["rot"] * 4
        return {"bytes": 2 * t * row * size + table + 2 * d * size + (4 * t * hkv if case["reset"] else 0),
                "flops": t * (case["hq"] + hkv) * (4 * d + 3 * case["rot"])}
    if case["op"] == "evict":
        kept = sum(_kept_lens(case))
        return {"bytes": 4 * hkv * sum(lens) + kept * hkv * (4 + 8 + 4 * d * size), "flops": hkv * sum(lens)}
    seq, pos = _queries(case)
    w = case["window"]
    pairs = sum(min(p + 1, w) if w else p + 1 for p in pos)
    reach = {}
    for s, p in zip(seq, pos):
        lo = max(0, p + 1 - w) if w else 0
        a, b = reach.get(s, (lo, p + 1))
        reach[s] = (min(a, lo), max(b, p + 1))
    keys = sum(b - a for a, b in reach.values())
    rows = len(seq) * case["hq"] * d
    return {"bytes": keys * hkv * (2 * d * size + 8) + 2 * rows * size, "flops": pairs * case["hq"] * (4 * d + 4)}


# ------------------------------------------------------------------- 64 bits --
def exact(case, seed):
    """The operators from their definitions in 64 bits, one sequence after another."""
    s = prepare(case, seed)
    ps, hkv, d = case["page"], case["hkv"], case["d"]
    lens, table = _lens(case), s["table"].tolist()

    def slots_of(rows, n):
        at = torch.tensor([p * ps for p in rows if p >= 0], device="cuda")
        return (at[:, None] + torch.arange(ps, device="cuda")).reshape(-1)[:n]

    if case["op"] == "evict":
        kept = torch.full((len(lens), hkv, s["kept_max"]), -1, dtype=torch.int32, device="cuda")
        k, v = s["k_cache"].view(-1, hkv, d), s["v_cache"].view(-1, hkv, d)
        mass = s["mass"].transpose(1, 2).reshape(-1, hkv).clone()
        src_k, src_v, src_m = k.clone(), v.clone(), mass.clone()
        for i, (n, m) in enumerate(zip(lens, _kept_lens(case))):
            src, dst = slots_of(table[i], n), slots_of(s["dst_table"].tolist()[i], m)
            totals = src_m[src].double().cpu().numpy()
            first, last = min(case["sink"], n), n - case["recent"]
            for h in range(hkv):
                by_total = np.lexsort((np.arange(first, last), -totals[first:last, h]))[:m - first - (n - last)]
                ids = np.sort(np.concatenate([np.arange(first), first + by_total, np.arange(last, n)]))
                ids = torch.from_numpy(ids).to("cuda")
                kept[i, h, :m] = ids.int()
                k[dst, h], v[dst, h], mass[dst, h] = src_k[src[ids], h], src_v[src[ids], h], src_m[src[ids], h]
        return {"kept": kept, "k_cache": s["k_cache"], "v_cache": s["v_cache"],
                "mass": mass.view(-1, ps, hkv).transpose(1, 2).double()}

    seq, pos = _queries(case)
    if case["op"] == "rope":
        at = s["positions"].long() if case["moved"] else s["pos"]
        half = case["rot"] // 2
        turn = torch.complex(s["rope_table"][at, :half].double(), s["rope_table"][at, half:].double())
        out = []
        for x, w in ((s["q"], s["q_weight"]), (s["new_k"], s["k_weight"])):
            x = x.double()
            y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + 1e-6) * w.double()
            r = y[..., :2 * half].reshape(*y.shape[:2], half, 2) if case["interleaved"] \
                else y[..., :2 * half].reshape(*y.shape[:2], 2, half).transpose(-1, -2)
            z = torch.view_as_real(torch.complex(r[..., 0].contiguous(), r[..., 1].contiguous()) * turn[:, None])
            z = z if case["interleaved"] else z.transpose(-1, -2)
            out.append(torch.cat([z.reshape(*y.shape[:2], 2 * half), y[..., 2 * half:]], -1))
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        mass = s["mass"].double() if case["reset"] else None
        for t, (i, p) in enumerate(zip(seq, pos)):
            kc[table[i][p // ps], p % ps] = out[1][t]
            vc[table[i][p // ps], p % ps] = s["new_v"][t].double()
            if mass is not None:
                mass[table[i][p // ps], :, p % ps] = 0.0
        return {"q": out[0], "k_cache": kc, "v_cache": vc, "mass": mass}

    out = torch.empty(len(seq), case["hq"], d, dtype=torch.float64, device="cuda")
    total = s["mass"].transpose(1, 2).reshape(-1, hkv).double()
    group, first = case["hq"] // hkv, 0
    for i, n in enumerate(lens):
        count = case["chunk"] if i < case["n_pre"] else case["run"]
        src = slots_of(table[i], n)
        key, value = s["k_cache"].view(-1, hkv, d)[src].double(), s["v_cache"].view(-1, hkv, d)[src].double()
        p = torch.tensor(pos[first:first + count], device="cuda")[:, None]
        j = torch.arange(n, device="cuda")
        hidden = (j > p) | (j <= p - case["window"]) if case["window"] else j > p
        for h in range(hkv):
            q = s["q"][first:first + count, h * group:(h + 1) * group].double().transpose(0, 1)  # [G, count, D]
            logit = (q @ key[:, h].T) * s["scale"]
            logit[:, hidden] = -math.inf
            w = torch.exp(logit - torch.logsumexp(logit, -1, keepdim=True))
            out[first:first + count, h * group:(h + 1) * group] = (w @ value[:, h]).transpose(0, 1)
            total[src, h] += w.sum((0, 1))
        first += count
    return {"out": out, "mass": total.view(-1, ps, hkv).transpose(1, 2)}
