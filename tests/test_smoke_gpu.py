"""The smoke run reaches the kernel that reads a shared prefix once."""
import pytest

import paged_kv_attention_20_gb300 as pka

pytestmark = pytest.mark.gpu


def test_prefix_is_read_once(cuda_device, monkeypatch):
    import __graft_entry__
    taken, forward = [], pka.paged_attn_forward_shared

    def seen(plan, q, k, v, scale, shared, splits=None, **kw):
        taken.append(splits or pka.paged_attn_shared_splits(plan, q.shape[1], k.shape[2], shared))
        return forward(plan, q, k, v, scale, shared, splits=splits, **kw)

    monkeypatch.setattr(pka, "paged_attn_forward_shared", seen)
    __graft_entry__.eight_bit_step(cuda_device)
    assert any(prefix > 0 for prefix, _ in taken), taken
