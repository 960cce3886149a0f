"""Attention over 8-bit values so small that their scale is next to fp32's smallest normal number."""
import pytest
import torch

import paged_kv_attention_20_gb300 as pka

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
HALF_STEP, TINY = 2.0 ** -8, 2.0 ** -134          # of bf16
P_ERROR = 2.0 ** -10                              # of a weight in three e5m2 pieces; the sums of 2^16 keys at most in fp32 are below that


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (16, 1, 128), (4, 2, 64), (4, 2, 96)])
@pytest.mark.parametrize("n,splits", [(40, 1), (50000, 1), (50000, 3)])
@pytest.mark.parametrize("low", [-109, -116, -120])
def test_long_history_of_tiny_values(cuda_device, hq, hkv, d, n, splits, low):
    """Equal scores: the output is the values' mean, a normal number of bf16, whatever the history's length."""
    ps = 64
    pages = -(-n // ps)
    gen = torch.Generator(device="cuda").manual_seed(12)
    plan = pka.paged_attn_plan([n], [list(range(pages))], [0], [n - 1], ps, pages, device="cuda")
    kc = torch.zeros(pages, ps, hkv, d, dtype=E4M3, device="cuda")
    vc = (256 * (1 + torch.rand(pages, ps, hkv, d, generator=gen, device="cuda") / 2)).to(E4M3)
    ks = torch.ones(pages, hkv, ps, dtype=torch.uint8, device="cuda")
    vs = torch.full_like(ks, low - 8 + 127 if low > -119 else 1)
    q = torch.randn(1, hq, d, generator=gen, device="cuda").bfloat16()
    out = pka.paged_attn_forward_q8(plan, q, kc, vc, ks, vs, d ** -0.5, splits=splits)[0].double().cpu()
    mean = vc.view(-1, hkv, d)[:n].float().double().mean(0) * 2.0 ** (int(vs[0, 0, 0]) - 127)
    ref = mean.repeat_interleave(hq // hkv, 0).cpu()
    tol = HALF_STEP * ref * (1 + P_ERROR) + P_ERROR * ref + TINY
    assert bool(((out - ref).abs() <= tol).all()), float(((out - ref).abs() / tol).max())
    assert pka.device_status() == 0
