"""CPU: DeltaStack, Q8Pools and Rotary refuse what they cannot run (before anything touches a GPU)."""
import pytest
import torch


def make(**kw):
    from long_context_layer_b200.stack import DeltaStack
    a = dict(kinds=["full", "delta", "sparse"], num_q_heads=4, num_kv_heads=2, head_dim=64, dtype=torch.bfloat16,
             indptr=torch.zeros(2, dtype=torch.int32), indices=torch.zeros(1, dtype=torch.int32),
             kv_len=torch.zeros(1, dtype=torch.int32), max_pages_per_seq=1, num_phys_pages=1)
    a.update(kw)
    return DeltaStack(**a)


@pytest.mark.parametrize("kw", [
    dict(kinds=["full", "wide"]), dict(cache="fp4"), dict(kinds=["window"]), dict(kinds=["window"], window_tokens=-1),
    dict(kinds=["window"], window_tokens=5, window_sinks=-2), dict(dtype=torch.float16),
])
def test_stack_refusals(kw):
    with pytest.raises(ValueError):
        make(**kw)


def test_pools_and_rotary_refusals():
    from long_context_layer_b200 import DeltaError
    from long_context_layer_b200.stack import Q8Pools, Rotary
    with pytest.raises(ValueError):
        Q8Pools(1, 1, 64, "bf16", device="cpu")
    with pytest.raises(ValueError):
        Rotary(64, layout="rows", device="cpu")
    with pytest.raises(ValueError):
        Rotary(64, scaling="other", device="cpu")
    with pytest.raises(DeltaError):
        Rotary(63, device="cpu")
    r = Rotary(64, device="cpu")
    assert r.turns.dtype == torch.float64 and r.turns.shape == (32,)
