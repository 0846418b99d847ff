"""GPU: the operators together as a decode loop uses them (rotary prompt and steps, 8-bit cache, full, delta,
sparse and window layers of a DeltaStack), eagerly, captured, on other streams, from host buffers."""
import numpy as np
import pytest
import torch

from oracle import operators as R
from oracle.checks import selection_ok
from tests.operator_helpers import PAGE, Paged, assert_within, attention_tolerance, host, lib, logical, stream
from tests.test_gpu_cache_q8 import Model, counts
from tests.test_gpu_rope import tolerance

pytestmark = pytest.mark.gpu

KINDS = ["full", "window", "delta", "sparse", "window", "sparse", "sparse"]
HQ, HKV, D = 8, 2, 64
BUDGET, SINK, REC = 4, 16, 32
WINDOW, SINKS = 50, 5


class Loop:
    """A stack, its prompt already in the cache, and inputs of further steps."""

    def __init__(self, cache, prompt, steps, seed=0, kinds=KINDS, dtype=torch.bfloat16, **kw):
        from long_context_layer_b200.stack import DeltaStack, Q8Pools, Rotary
        L = lib()
        self.kinds, self.prompt, self.steps, self.cache = kinds, prompt, steps, cache
        self.paged = Paged(prompt, seed=seed, room=max(prompt) + steps)
        self.B, self.n_layers = len(prompt), len(kinds)
        self.rotary = Rotary(D, layout="half", scaling="bands", factor=4.0, original_len=256.0, low_turns=1.0,
                             high_turns=16.0, magnitude=1.1)
        self.stack = DeltaStack(kinds, HQ, HKV, D, dtype, self.paged.indptr, self.paged.indices, self.paged.kv_len,
                                self.paged.longest, self.paged.pages, BUDGET, SINK, REC, keep_scores=True, cache=cache,
                                window_tokens=WINDOW, window_sinks=SINKS, rotary=self.rotary, **kw)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dtype)  # noqa: E731
        T = sum(prompt)
        pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in prompt]).cuda()
        self.pools, self.model = [], []
        for _ in kinds:
            pool = Q8Pools(self.paged.pages, HKV, D, cache)
            k, v = rand(T, HKV, D), rand(T, HKV, D)
            L.rope(self.stack.desc, self.rotary.plan(pos), T, None, None, k, k, stream=stream())     # in place
            L.kv_write_q8(self.stack.desc, self.stack.pt, counts(prompt), max(prompt), k, v, pool.c, stream=stream())
            model = {"k": Model(prompt, HKV, D, cache), "v": Model(prompt, HKV, D, cache)}
            at = np.concatenate([[0], np.cumsum(prompt)])
            for b, n in enumerate(prompt):
                model["k"].write(b, 0, host(k)[at[b]:at[b + 1]])
                model["v"].write(b, 0, host(v)[at[b]:at[b + 1]])
            self.pools.append(pool)
            self.model.append(model)
        self.inputs = [(rand(self.n_layers, self.B, HQ, D), rand(self.n_layers, self.B, HKV, D),
                        rand(self.n_layers, self.B, HKV, D)) for _ in range(steps)]
        self.out = torch.zeros(self.n_layers, self.B, HQ, D, dtype=dtype, device="cuda")

    def lens(self, t):
        return [n + t + 1 for n in self.prompt]

    def check(self, t, out):
        """Every layer's output, cache and selection after step t."""
        q, k, v = self.inputs[t]
        turns = self.rotary.turns.cpu().numpy()
        dtype = "bf16" if q.dtype == torch.bfloat16 else "f32"
        selected = None
        for l, kind in enumerate(self.kinds):
            pos = [n - 1 for n in self.lens(t)]
            for x, rot in ((q, self.stack.q_rot), (k, self.stack.k_rot)):
                ref = R.rope(host(x)[l], pos, turns, "half", float(np.float32(1.1)))
                assert_within(host(rot)[l], ref, tolerance(host(x)[l], ref, turns, "half", 1.1, dtype), f"rotary layer {l}")
            qr, kr = host(self.stack.q_rot)[l], host(self.stack.k_rot)[l]
            if kind == "delta":
                got_sel = self.stack.selection(self.stack.delta_layers.index(l))
                selected = got_sel
            for b, n in enumerate(self.lens(t)):
                m = self.model[l]
                m["k"].write(b, n - 1, kr[b:b + 1])
                m["v"].write(b, n - 1, host(v)[l, b:b + 1])
                K, V = (m[w].values(b, n).transpose(1, 0, 2) for w in "kv")
                seen = list(range(n))
                if kind == "window":
                    seen = R.visible(n, WINDOW, SINKS)
                elif kind == "sparse":
                    seen = [x for j in selected[b] for x in range(j * PAGE, min(n, (j + 1) * PAGE))]
                ref = R.attention(qr[b], K, V, seen)
                tol = attention_tolerance(qr[b], K[:, seen], V[:, seen], ref, dtype, fmt=self.cache)
                assert_within(host(out)[l, b], ref, tol, f"step {t} layer {l} {kind} b={b}")
                if kind == "delta":
                    s = np.stack([K[h * HKV // HQ] @ qr[b, h] for h in range(HQ)]) / np.sqrt(D)
                    p = np.exp(s - s.max(1, keepdims=True))
                    S = np.zeros(-(-n // PAGE))
                    np.add.at(S, np.arange(n) // PAGE, (p / p.sum(1, keepdims=True)).sum(0))
                    assert selection_ok(got_sel[b], S, n, BUDGET, SINK, REC)[0]
        status, bits = lib().read_device_error(self.stack.workspace, stream())
        assert status == 0 and bits == 0


@pytest.mark.parametrize("cache,dtype", [("e4m3", torch.bfloat16), ("int8", torch.bfloat16), ("int8", torch.float32)])
def test_decode_loop(cache, dtype):
    loop = Loop(cache, [130, 1, 47], 20, dtype=dtype)
    for t in range(20):
        loop.paged.set_lens(loop.lens(t))
        loop.stack.step(*loop.inputs[t], loop.pools, None, loop.out)
        loop.check(t, loop.out)
    assert loop.stack.launches_per_step() == 9      # rotary, append, 7 layers


def test_captured_steps_equal_eager_steps():
    # one graph replayed with new inputs and lengths; inputs and outputs on another stream
    a, b = Loop("int8", [90, 33], 6, seed=5), Loop("int8", [90, 33], 6, seed=5)
    q, k, v = (torch.empty_like(x) for x in a.inputs[0])
    side = torch.cuda.Stream()
    graph = None
    for t in range(6):
        a.paged.set_lens(a.lens(t))
        b.paged.set_lens(b.lens(t))
        for x, y in zip((q, k, v), a.inputs[t]):
            x.copy_(y)
        if graph is None:
            graph = a.stack.capture(q, k, v, a.pools, None, a.out)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.current_stream().wait_stream(side)
        b.stack.step(*b.inputs[t], b.pools, None, b.out)
        assert torch.equal(a.out, b.out), t
        for x, y in zip(a.pools, b.pools):
            assert torch.equal(x.k, y.k) and torch.equal(x.v_scale, y.v_scale)


def test_two_graphs_that_share_a_workspace():
    # two captured calls on one workspace, replayed in turn on one stream, many times
    loop = Loop("e4m3", [700, 300], 1, seed=7, kinds=["delta", "sparse"])
    st, (q, k, v) = loop.stack, loop.inputs[0]
    first, second = torch.empty_like(loop.out), torch.empty_like(loop.out)
    st.step(q, k, v, loop.pools, None, loop.out, append=False)
    ref = loop.out.clone()
    st.step(-q, k, v, loop.pools, None, loop.out, append=False)
    ref_neg = loop.out.clone()
    neg = -q
    g1 = st.capture(q, k, v, loop.pools, None, first, append=False)
    g2 = st.capture(neg, k, v, loop.pools, None, second, append=False)
    for _ in range(10):
        g1.replay()
        g2.replay()
    assert torch.equal(first, ref) and torch.equal(second, ref_neg)


def test_step_from_host_buffers():
    a, b = Loop("e4m3", [64, 90], 3, seed=9), Loop("e4m3", [64, 90], 3, seed=9)
    pin = [x.cpu().pin_memory() for x in a.inputs[0]]
    out_host = torch.empty(a.out.shape, dtype=a.out.dtype).pin_memory()
    dev = [torch.empty_like(x) for x in a.inputs[0]]
    for t in range(3):
        a.paged.set_lens(a.lens(t))
        b.paged.set_lens(b.lens(t))
        for x, y in zip(pin, a.inputs[t]):
            x.copy_(y)
        torch.cuda.synchronize()
        a.stack.step_host(*pin, a.pools, None, out_host, *dev, a.out)
        b.stack.step(*b.inputs[t], b.pools, None, b.out)
        torch.cuda.synchronize()
        assert torch.equal(out_host, b.out.cpu()), t


def test_window_layers_over_the_plain_cache():
    from long_context_layer_b200.stack import DeltaStack
    paged = Paged([200, 33, 2], seed=11)
    g = torch.Generator(device="cuda").manual_seed(1)
    kinds = ["window", "full", "delta", "window", "sparse"]
    pools = [[torch.randn(paged.pages, HKV, PAGE, D, generator=g, device="cuda").bfloat16() for _ in kinds] for _ in "kv"]
    st = DeltaStack(kinds, HQ, HKV, D, torch.bfloat16, paged.indptr, paged.indices, paged.kv_len, paged.longest, paged.pages,
                    BUDGET, SINK, REC, window_tokens=WINDOW, window_sinks=SINKS)
    q = torch.randn(5, 3, HQ, D, generator=g, device="cuda").bfloat16()
    k, v = (torch.randn(5, 3, HKV, D, generator=g, device="cuda").bfloat16() for _ in "kv")
    out = torch.zeros_like(q)
    st.step(q, k, v, *pools, out)
    for l in (0, 3):
        for b, n in enumerate(paged.lens):
            seen = R.visible(n, WINDOW, SINKS)
            K, V = (logical(host(p[l]), paged, b) for p in pools)
            qq = host(q)[l, b]
            ref = R.attention(qq, K, V, seen)
            assert_within(host(out)[l, b], ref, attention_tolerance(qq, K, V, ref, "bf16", 2.0 ** -16), f"layer {l} b={b}")
    assert np.array_equal(host(k)[3, 0], host(pools[0][3])[paged.phys(0, 12), :, 7])     # the appended token


def test_calibration_over_the_8_bit_cache():
    loop = Loop("int8", [300, 120], 1, seed=13, kinds=["full", "full", "delta", "sparse"])
    q, k, v = loop.inputs[0]
    shift = loop.stack.calibration_shifts(q, loop.pools, None, loop.out)
    assert torch.equal(shift[:2], torch.zeros_like(shift[:2]))
    assert bool((shift[2:] > 0).all()) and bool((shift[2:] <= 1).all())


def test_other_streams_and_concurrent_calls():
    # calls with workspaces of their own on two streams at once give what they give alone
    loops = [Loop("int8", [900, 411], 1, seed=s) for s in (21, 22)]
    refs = []
    for lp in loops:
        lp.stack.step(*lp.inputs[0], lp.pools, None, lp.out, append=False)
        refs.append(lp.out.clone())
        lp.out.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in loops]
    for _ in range(20):
        for lp, s in zip(loops, streams):
            with torch.cuda.stream(s):
                lp.stack.step(*lp.inputs[0], lp.pools, None, lp.out, append=False)
    torch.cuda.synchronize()
    for lp, ref in zip(loops, refs):
        assert torch.equal(lp.out, ref)
