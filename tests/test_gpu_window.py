"""GPU: window attention with sinks over the bf16 / fp32 cache against fp64."""
import numpy as np
import pytest
import torch

from oracle import operators as R
from tests.operator_helpers import (DT, PAGE, Paged, assert_within, attention_tolerance, desc, flags, host, lib, logical,
                                    stream, workspace)

pytestmark = pytest.mark.gpu
# p as the sum of two bf16 values leaves at most 2^-8 * 2^-8 of it (bf16), nothing is rounded for fp32 (2^-24: the
# product's own rounding)
ROUND = {"bf16": 2.0 ** -16, "f32": 2.0 ** -24}


class Case:
    def __init__(self, dtype, G, hkv, d, lens, seed=0):
        L = lib()
        self.L, self.dtype, self.lens = L, dtype, lens
        self.paged = Paged(lens, seed=seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        shape = (self.paged.pages, hkv, PAGE, d)
        self.k, self.v = (torch.randn(shape, generator=gen, device="cuda").to(DT[dtype]) for _ in range(2))
        self.q = torch.randn(len(lens), G * hkv, d, generator=gen, device="cuda").to(DT[dtype])
        self.o = torch.full_like(self.q, 99.0)
        self.desc = desc(G * hkv, hkv, d, dtype, self.paged.pages)
        self.pt = self.paged.table()
        self.bytes = L.workspace_size(self.desc, len(lens), self.paged.longest)
        self.ws = workspace(self.bytes)

    def run(self, window, sink):
        self.L.window_attn(self.desc, self.pt, window, sink, self.q, self.k, self.v, self.o, self.ws, self.bytes, stream())
        assert flags(self.ws) == 0

    def check(self, window, sink, k=None, v=None):
        k, v = host(self.k) if k is None else k, host(self.v) if v is None else v
        got = host(self.o)
        for b, n in enumerate(self.lens):
            seen = R.visible(n, window, sink)
            K, V = logical(k, self.paged, b), logical(v, self.paged, b)
            q = host(self.q)[b]
            ref = R.attention(q, K, V, seen)
            tol = attention_tolerance(q, K[:, seen], V[:, seen], ref, self.dtype, ROUND[self.dtype])
            assert_within(got[b], ref, tol, f"b={b} n={n}")


LENS = [0, 1, 15, 16, 17, 31, 130, 1003]
WINDOWS = [(1, 0), (16, 0), (15, 1), (17, 4), (100, 16), (33, 37), (512, 128), (5000, 3), (0, 20), (0, 0), (40, 0),
           (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31 - 1, 0)]


@pytest.mark.parametrize("window,sink", WINDOWS)
@pytest.mark.parametrize("dtype,G,hkv,d", [("bf16", 7, 2, 128), ("bf16", 4, 1, 64), ("f32", 8, 1, 64), ("f32", 3, 2, 128)])
def test_window(dtype, G, hkv, d, window, sink):
    c = Case(dtype, G, hkv, d, LENS, seed=window % 1000 + sink % 1000)
    c.run(window, sink)
    c.check(window, sink)


@pytest.mark.parametrize("dtype,G,hkv,d,lens,window,sink", [
    ("bf16", 7, 4, 128, [8192], 4096, 16),                       # one sequence: 8-warp CTAs
    ("bf16", 5, 8, 128, [3000 + 97 * i for i in range(16)], 1024, 16),     # many units
    ("bf16", 1, 1, 64, [60000], 40000, 100),                     # a long window: several clusters a unit
    ("f32", 2, 2, 64, [9000, 20], 8000, 7),
    ("bf16", 8, 8, 128, [2000] * 8, 500, 33),
])
def test_plans(dtype, G, hkv, d, lens, window, sink):
    c = Case(dtype, G, hkv, d, lens, seed=sum(lens))
    c.run(window, sink)
    c.check(window, sink)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_hidden_tokens_and_stale_slots_may_hold_anything(dtype, bad):
    # every hidden token, on listed pages and on others, and every slot past the end
    window, sink = 37, 5
    c = Case(dtype, 4, 2, 64, [200, 43, 70], seed=3)
    k0, v0 = host(c.k), host(c.v)
    hide = torch.ones(c.k.shape[:1] + (PAGE,), dtype=torch.bool)
    for b, n in enumerate(c.lens):
        for t in R.visible(n, window, sink):
            hide[c.paged.phys(b, t // PAGE), t % PAGE] = False
    mask = hide[:, None, :, None].expand(c.k.shape).cuda()
    c.k[mask] = bad
    c.v[mask] = bad
    c.run(window, sink)
    c.check(window, sink, k0, v0)


def test_window_over_everything_equals_full_attention():
    c = Case("f32", 4, 2, 64, [300, 77], seed=4)
    c.run(300, 0)
    full = torch.empty_like(c.o)
    c.L.full_attn(c.desc, c.pt, c.q, c.k, c.v, full, c.ws, c.bytes, stream())
    assert torch.equal(full, c.o)


def test_bad_page_and_length_are_flagged():
    c = Case("bf16", 4, 2, 64, [100, 40], seed=5)
    c.paged.indices[0] = -1
    c.L.window_attn(c.desc, c.pt, 20, 4, c.q, c.k, c.v, c.o, c.ws, c.bytes, stream())
    assert flags(c.ws) == 1
    c.paged.indices[0] = 1
    c.paged.kv_len[0] = 100000
    c.L.window_attn(c.desc, c.pt, 20, 4, c.q, c.k, c.v, c.o, c.ws, c.bytes, stream())
    assert flags(c.ws) == 2
