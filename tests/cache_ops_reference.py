"""Plain float64 forms of the operators around the attention of a bounded cache.

Written from the formulas, one row or one sequence at a time, on the CPU: the
per-head RMS norm and rotation, the per-key sums of the softmax weights, and the
choice of the keys an eviction keeps.
"""
from __future__ import annotations

import numpy as np
import torch


def norm_rope(x, weight, eps, cos, sin, interleaved):
    """x [T, H, D] -> (y, bound): normed and rotated rows, and per element the magnitude |a| + |b| its pair had."""
    x = x.detach().cpu().double().numpy()
    y = x.copy()
    if weight is not None:
        w = weight.detach().cpu().double().numpy()
        y = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * w
    size = np.abs(y)
    if cos is None:
        return y, size
    out = y.copy()
    half = cos.shape[-1]
    for i in range(half):
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        a, b, c, s = y[..., ia], y[..., ib], cos[:, None, i], sin[:, None, i]
        out[..., ia] = a * c - b * s
        out[..., ib] = b * c + a * s
        size[..., ia] = size[..., ib] = np.abs(a) + np.abs(b)
    return out, size


def slots(case_table, ps, seq, n):
    """Physical rows of keys 0..n-1 of a sequence."""
    j = np.arange(n)
    return np.asarray(case_table)[seq][j // ps].astype(np.int64) * ps + j % ps


def key_mass(case, k_cache, causal=True, window=0):
    """What one call adds: [pages, Hkv, ps] float64, and per (page, head, row) whether any query saw the key."""
    ps, hkv = case.page_size, case.hkv
    group = case.hq // hkv
    total = np.zeros((case.num_pages * ps, hkv))
    seen = np.zeros((case.num_pages * ps,), dtype=bool)
    k = k_cache.detach().cpu().double().numpy().reshape(-1, hkv, case.d)
    q = case.q.detach().cpu().double().numpy()
    for i, (s, pos) in enumerate(zip(case.query_seq, case.query_pos)):
        n = int(case.seq_lens[s])
        lo = max(0, int(pos) - window + 1) if window else 0
        hi = int(pos) + 1 if causal else n
        at = slots(case.block_table, ps, s, n)[lo:hi]
        for h in range(case.hq):
            logit = k[at, h // group] @ q[i, h] * case.scale
            w = np.exp(logit - logit.max())
            total[at, h // group] += w / w.sum()
        seen[at] = True
    return (total.reshape(case.num_pages, ps, hkv).transpose(0, 2, 1),
            np.broadcast_to(seen.reshape(case.num_pages, 1, ps), (case.num_pages, hkv, ps)))


def weight_tolerance(case, k_cache):
    """Relative error a softmax weight may have.

    A score is a sum of D products in fp32; each addition is off by at most 2^-23 of the running magnitude
    (a tensor core may truncate), so a score is off by D * 2^-23 * max|q||k| * scale in the worst order.  A
    weight e^(s - lse) carries its own score's error and the log-sum-exp's, which is no larger, and the
    exponentials' and the sum's few units of 2^-22.
    """
    k = torch.nan_to_num(k_cache.detach().cpu().double())
    size = float(case.q.double().norm(dim=-1).max() * k.norm(dim=-1).max()) * case.scale
    return 2.0 * case.d * 2.0 ** -23 * size + 2.0 ** -19


def kept_keys(totals, keep, sink, recent):
    """Indices (ascending) that stay of a history with these totals [n]."""
    n = len(totals)
    if keep >= n:
        return np.arange(n)
    first, last = sink, n - recent
    # largest total first, then lowest index; NaN after every number
    middle = sorted(range(first, last), key=lambda j: (np.isnan(totals[j]), -totals[j] if not np.isnan(totals[j]) else 0.0, j))
    return np.array(sorted(list(range(first)) + middle[:keep - sink - recent] + list(range(last, n))), dtype=np.int64)
