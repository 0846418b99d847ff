"""GPU: a step from host buffers equals step() where the second group of layers starts with a sparse layer."""
import pytest
import torch

from tests.operator_helpers import PAGE, Paged
from tests.test_gpu_operator_step import BUDGET, HKV, HQ, REC, SINK, SINKS, WINDOW, D, Loop

pytestmark = pytest.mark.gpu

ORDERS = [(["delta", "window", "sparse", "sparse"], 2), (["delta", "sparse", "sparse"], 2),
          (["full", "full", "delta", "sparse", "sparse"], 4)]


def host_step(stack, inputs, pools, out, early):
    pin = [x.cpu().pin_memory() for x in inputs]
    got = torch.empty(out.shape, dtype=out.dtype).pin_memory()
    dev = [torch.empty_like(x) for x in inputs]
    torch.cuda.synchronize()
    stack.step_host(*pin, *pools, got, *dev, out, early_layers=early)
    torch.cuda.synchronize()
    return got


@pytest.mark.parametrize("kinds,early", ORDERS)
@pytest.mark.parametrize("cache", ["e4m3", "int8"])
def test_over_the_8_bit_cache(cache, kinds, early):
    steps = 24          # every slot of a page, and into the next one
    a, b = (Loop(cache, [700, 90], steps, seed=31, kinds=kinds) for _ in "ab")
    for t in range(steps):
        a.paged.set_lens(a.lens(t))
        b.paged.set_lens(b.lens(t))
        got = host_step(a.stack, a.inputs[t], (a.pools, None), a.out, early)
        b.stack.step(*b.inputs[t], b.pools, None, b.out)
        assert torch.equal(got, b.out.cpu()), t


@pytest.mark.parametrize("kinds,early", ORDERS)
def test_over_the_plain_cache(kinds, early):
    from long_context_layer_b200.stack import DeltaStack
    steps, prompt = 24, [700, 90]
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    paged = Paged(prompt, seed=2, room=max(prompt) + steps)
    first = [[rand(paged.pages, HKV, PAGE, D) for _ in kinds] for _ in "kv"]
    sides = []
    for _ in "ab":
        st = DeltaStack(kinds, HQ, HKV, D, torch.bfloat16, paged.indptr, paged.indices, paged.kv_len, paged.longest, paged.pages,
                        BUDGET, SINK, REC, window_tokens=WINDOW, window_sinks=SINKS)
        sides.append((st, [[x.clone() for x in p] for p in first], torch.zeros(len(kinds), 2, HQ, D, device="cuda").bfloat16()))
    for t in range(steps):
        paged.set_lens([n + t + 1 for n in prompt])
        x = (rand(len(kinds), 2, HQ, D), rand(len(kinds), 2, HKV, D), rand(len(kinds), 2, HKV, D))
        (sa, pa, oa), (sb, pb, ob) = sides
        got = host_step(sa, x, pa, oa, early)
        sb.step(*x, *pb, ob)
        assert torch.equal(got, ob.cpu()), t
