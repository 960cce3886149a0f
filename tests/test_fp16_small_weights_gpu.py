"""A long tail of small softmax weights in fp16, on every tensor-core path: no weight may vanish or lose its bits there.

One key has the row's largest score and a value of 0; the others weigh 2^-t of it and hold 1.  The output is
N 2^-t / (1 + N 2^-t): off by as much as a weight is, since all the tail's weights are the same number.
"""
import math

import pytest
import torch

import paged_kv_attention_20_gb300 as pka

pytestmark = pytest.mark.gpu

# half a step of the output and of a weight (2^-11 each); a score below 2^4 is off by 2^-20 and the exponential by 2^-21; sums
# in fp32, of up to 1500 addends one after the other, by 2^-24 each
TOL = 2.0 ** -11 + 2.0 ** -11 + 2.0 ** -20 + 2.0 ** -21 + 1500 * 2.0 ** -24


def caches(n, hkv, d, logit, peak, ps=16):
    pages = -(-n // ps)
    k, v = (torch.zeros(pages * ps, hkv, d, dtype=torch.float16, device="cuda") for _ in "kv")
    k[:n, :, 0], v[:n] = logit, 1.0
    k[peak, :, 0], v[peak] = 0.0, 0.0
    return k.view(pages, ps, hkv, d), v.view(pages, ps, hkv, d), pages


def check(out, n, logit):
    w = (n - 1) * math.exp(logit)
    want = w / (1 + w)
    off = (out.double() - want).abs().max().item() / want
    assert off <= TOL, (off / TOL, want)
    assert pka.device_status() == 0


@pytest.mark.parametrize("peak", [0, 100, 2990])
@pytest.mark.parametrize("logit", [-8.0, -12.484375, -14.28125])           # 2^-11.5, 2^-18, 2^-20.6
@pytest.mark.parametrize("hq,hkv", [(4, 2), (8, 1), (40, 1)])
def test_chunks_and_decode(cuda_device, hq, hkv, logit, peak):
    n, d = 3000, 128
    k, v, pages = caches(n, hkv, d, logit, peak)
    table = [list(range(pages))]
    for run in (1, 3, 20):                                  # decode items, among them groups of 8 and more; a tile
        plan = pka.paged_attn_plan([n], table, [0] * run, list(range(n - run, n)), 16, pages, device="cuda")
        q = torch.zeros(run, hq, d, dtype=torch.float16, device="cuda")
        q[:, :, 0] = 1.0
        for splits in (1, 3):
            check(pka.paged_attn_forward_split(plan, q, k, v, 1.0, splits, causal=False), n, logit)
        if run == 20:
            kc, vc = (t.to(torch.float8_e4m3fn) for t in (torch.zeros_like(k), v))
            ks, vs = (torch.full((pages, hkv, 16), 127, dtype=torch.uint8, device="cuda") for _ in "kv")
            stored = float(torch.tensor(logit).to(torch.float8_e4m3fn).float())
            kc.view(-1, hkv, d)[:n, :, 0] = torch.tensor(stored, device="cuda").to(torch.float8_e4m3fn)
            kc.view(-1, hkv, d)[peak, :, 0] = torch.tensor(0.0, device="cuda").to(torch.float8_e4m3fn)
            check(pka.paged_attn_forward_q8(plan, q, kc, vc, ks, vs, 1.0, causal=False, splits=1), n, stored)


@pytest.mark.parametrize("logit", [-12.484375, -14.28125])
def test_behind_a_prefix(cuda_device, logit):
    shared, own, hq, hkv, d, ps = 2048, 40, 8, 2, 128, 16
    k, v, pages = caches(shared + 3 * 48, hkv, d, logit, 5)
    table = [list(range(128)) + list(range(128 + 3 * s, 131 + 3 * s)) for s in range(3)]
    plan = pka.paged_attn_plan([shared + own] * 3, table, [0, 1, 2], [shared + own - 1] * 3, ps, pages, device="cuda")
    q = torch.zeros(3, hq, d, dtype=torch.float16, device="cuda")
    q[:, :, 0] = 1.0
    for splits in ((1, 1), (3, 2)):
        check(pka.paged_attn_forward_shared(plan, q, k, v, 1.0, shared, splits=splits), shared + own, logit)


@pytest.mark.parametrize("logit", [-12.484375, -14.28125])
def test_latent_cache(cuda_device, logit):
    """MLA: the latent is key and value; the score comes from the position part."""
    n, r, p, heads, ps = 3000, 512, 64, 128, 64
    pages = -(-n // ps)
    latent = torch.zeros(pages * ps, 1, r, dtype=torch.float16, device="cuda")
    pos = torch.zeros(pages * ps, 1, p, dtype=torch.float16, device="cuda")
    latent[:n], pos[:n, :, 0] = 1.0, logit
    latent[7], pos[7, :, 0] = 0.0, 0.0
    plan = pka.paged_attn_plan([n], [list(range(pages))], [0], [n - 1], ps, pages, device="cuda")
    q = torch.zeros(1, heads, r, dtype=torch.float16, device="cuda")
    qp = torch.zeros(1, heads, p, dtype=torch.float16, device="cuda")
    qp[:, :, 0] = 1.0
    check(pka.paged_mla_forward(plan, q, qp, latent.view(pages, ps, 1, r), pos.view(pages, ps, 1, p), 1.0), n, logit)
