"""GPU: decode attention over the 8-bit cache (full, delta, sparse, window) against fp64 over the values the
cache stands for."""
import numpy as np
import pytest
import torch

from oracle import delta_oracle as O
from oracle import operators as R
from oracle.checks import selection_ok
from tests.operator_helpers import (DT, PAGE, Q_PART, Paged, Pool8, assert_within, attention_tolerance, desc, flags, host, lib,
                                    logical, stream, workspace)

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, fmt, dtype, G, hkv, d, lens, seed=0, spread=0.5, stale=None, qscale=1.0):
        L = lib()
        self.L, self.dtype, self.lens = L, dtype, lens
        self.paged = Paged(lens, seed=seed)
        self.hq = G * hkv
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.pool = Pool8(self.paged.pages, hkv, d, fmt).fill(gen, spread)
        self.q = (torch.randn(len(lens), self.hq, d, generator=gen, device="cuda") * qscale).to(DT[dtype])
        if stale is not None:        # what slots behind the last token hold
            for b, n in enumerate(lens):
                if n % PAGE:
                    for p in (self.pool.k, self.pool.v):
                        p[self.paged.phys(b, n // PAGE), :, n % PAGE:] = stale
        self.o = torch.full_like(self.q, 99.0)
        self.desc = desc(self.hq, hkv, d, dtype, self.paged.pages)
        self.pt = self.paged.table()
        self.bytes = L.workspace_size_q8(self.desc, len(lens), self.paged.longest)
        self.ws = workspace(self.bytes)

    def kv(self, b):
        if not hasattr(self, "_num"):
            self._num = {w: self.pool.numbers(w) for w in "kv"}
        return logical(self._num["k"], self.paged, b), logical(self._num["v"], self.paged, b)

    def check(self, tokens=lambda b, n: range(n), what=""):
        got = host(self.o)
        for b, n in enumerate(self.lens):
            K, V = self.kv(b)
            seen = list(tokens(b, n))
            q = host(self.q)[b]
            ref = R.attention(q, K, V, seen)
            tol = attention_tolerance(q, K[:, seen], V[:, seen], ref, self.dtype, fmt=self.pool.fmt)
            assert_within(got[b], ref, tol, f"{what} b={b} n={n}")


FULL = [
    # fmt, dtype, G, Hkv, D, lengths
    ("e4m3", "bf16", 7, 4, 128, [8192]),
    ("int8", "bf16", 4, 8, 128, [1, 0, 16, 17, 333, 4097]),
    ("e4m3", "bf16", 1, 2, 64, [31, 2, 15]),
    ("int8", "bf16", 8, 1, 64, [1000, 1]),
    ("e4m3", "bf16", 5, 8, 128, [700] * 16),            # many units: 8-warp CTAs, two an SM
    ("int8", "bf16", 3, 3, 128, [2500, 40]),
    ("e4m3", "bf16", 2, 5, 64, [513, 64, 8]),
    ("int8", "bf16", 6, 1, 128, [20000, 5]),             # several clusters a unit: merged in the workspace
    ("e4m3", "f32", 8, 1, 64, [1024, 3]),
    ("int8", "f32", 7, 2, 128, [600, 1, 0]),
    ("e4m3", "f32", 1, 1, 128, [17000]),
    ("int8", "f32", 5, 4, 64, [90, 1501]),
]


@pytest.mark.parametrize("fmt,dtype,G,hkv,d,lens", FULL)
def test_full(fmt, dtype, G, hkv, d, lens):
    c = Case(fmt, dtype, G, hkv, d, lens, seed=sum(lens), stale=0x7f)
    c.L.full_attn_q8(c.desc, c.pt, c.q, c.pool.cache, c.o, c.ws, c.bytes, stream())
    assert flags(c.ws) == 0
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_blocks_of_very_different_scales(fmt, dtype):
    # block sizes over about 2^-24 .. 2^24 (neighbouring pages differ), large and small queries
    for seed, qscale in ((1, 1e-3), (2, 1e4 if dtype == "f32" else 100.0)):
        c = Case(fmt, dtype, 4, 2, 64, [400, 37], seed=seed, spread=0.0, qscale=qscale)
        r = torch.Generator(device="cuda").manual_seed(seed)
        c.pool.vs *= torch.exp2(torch.randint(-24, 25, c.pool.vs.shape, generator=r, device="cuda").float())
        c.pool.ks *= torch.exp2(torch.randint(-3, 1, c.pool.ks.shape, generator=r, device="cuda").float()) / qscale ** 0.9
        c.L.full_attn_q8(c.desc, c.pt, c.q, c.pool.cache, c.o, c.ws, c.bytes, stream())
        c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_queries_with_an_outlying_dimension(fmt, dtype):
    # one dimension 3000 times the others, which the keys hardly have: the logits hang on the small ones
    c = Case(fmt, dtype, 4, 2, 128, [500, 90], seed=21)
    c.q[..., 7] *= 3000
    c.pool.k[..., 7] = 0
    c.L.full_attn_q8(c.desc, c.pt, c.q, c.pool.cache, c.o, c.ws, c.bytes, stream())
    c.check()


def test_scales_need_not_be_powers_of_two():
    # a cache written elsewhere with the same layout: any finite scale
    c = Case("int8", "bf16", 4, 2, 128, [300, 65], seed=8)
    c.pool.ks *= 0.7
    c.pool.vs *= 1.3
    c.L.full_attn_q8(c.desc, c.pt, c.q, c.pool.cache, c.o, c.ws, c.bytes, stream())
    c.check()


@pytest.mark.parametrize("which", ["k", "v"])
def test_nan_scale_shows_in_its_head_only(which):
    c = Case("int8", "bf16", 2, 3, 64, [100, 50], seed=9)
    (c.pool.ks if which == "k" else c.pool.vs)[c.paged.phys(0, 2), 1] = float("nan")
    c.L.full_attn_q8(c.desc, c.pt, c.q, c.pool.cache, c.o, c.ws, c.bytes, stream())
    nan = np.isnan(host(c.o))
    assert nan[0, 2:4].all() and not nan[0, :2].any() and not nan[0, 4:].any() and not nan[1].any()


def test_every_block_nan_gives_nan_not_zero():
    c = Case("e4m3", "bf16", 4, 1, 64, [40], seed=10)
    c.pool.ks.fill_(float("nan"))
    c.L.full_attn_q8(c.desc, c.pt, c.q, c.pool.cache, c.o, c.ws, c.bytes, stream())
    assert np.isnan(host(c.o)).all()


def test_non_finite_query_shows_in_its_head_only():
    c = Case("e4m3", "bf16", 4, 2, 128, [70], seed=11)
    c.q[0, 5, 17] = float("inf")
    c.L.full_attn_q8(c.desc, c.pt, c.q, c.pool.cache, c.o, c.ws, c.bytes, stream())
    nan = np.isnan(host(c.o))[0]
    assert nan[5].all() and not nan[[0, 1, 2, 3, 4, 6, 7]].any()


def test_zero_queries_and_zero_blocks():
    c = Case("int8", "f32", 2, 2, 64, [33, 16], seed=12)
    c.q[0].zero_()
    c.pool.k.zero_()
    c.pool.ks.fill_(2.0 ** -100)
    c.L.full_attn_q8(c.desc, c.pt, c.q, c.pool.cache, c.o, c.ws, c.bytes, stream())
    c.check()


# ------------------------------------------------------------------ delta- and sparse layers
SELECT = [
    # fmt, dtype, G, Hkv, D, lengths, budget, sink, recency, reduce
    ("e4m3", "bf16", 7, 4, 128, [8192], 64, 16, 256, "sum"),
    ("int8", "bf16", 4, 2, 128, [3000, 1500, 17, 0, 1], 16, 16, 100, "sum"),
    ("int8", "f32", 8, 1, 64, [1024], 8, 16, 64, "sum"),
    ("e4m3", "f32", 5, 2, 128, [400, 50], 100, 16, 64, "sum"),       # budget above the candidates
    ("e4m3", "bf16", 2, 2, 64, [700], 1, 0, 0, "sum"),
    ("int8", "bf16", 5, 8, 128, [1200 + 61 * i for i in range(16)], 16, 16, 64, "sum"),
    ("e4m3", "bf16", 2, 8, 64, [200000, 90000], 200, 16, 512, "sum"),
    ("int8", "bf16", 7, 4, 128, [2048, 33], 16, 16, 64, "max"),
    ("e4m3", "f32", 1, 2, 64, [777], 5, 16, 32, "max"),
]


def select(c, budget, sink, rec, reduce):
    L = c.L
    mode = L.DELTA_HEAD_SUM if reduce == "sum" else L.DELTA_HEAD_MAX
    sp = L.DeltaSelectParams(budget, sink, rec, mode)
    nb = L.workspace_size_q8(c.desc, len(c.lens), c.paged.longest, mode)
    ws = workspace(nb)
    stride = max(1, L.sel_capacity(sp)) + 2
    cnt = torch.full((len(c.lens),), -1, dtype=torch.int32, device="cuda")
    pages = torch.full((len(c.lens), stride), -1, dtype=torch.int32, device="cuda")
    scores = torch.full((len(c.lens), c.paged.longest), -1.0, device="cuda")
    for _ in range(2):     # the workspace's counters are back at zero: the second call gives the same
        L.select_attn_q8(c.desc, c.pt, sp, c.q, c.pool.cache, c.o, cnt, pages, stride, scores, ws, nb, stream())
    assert flags(ws) == 0
    return cnt.cpu().numpy(), pages.cpu().numpy(), scores.cpu().numpy(), (cnt, pages, stride)


def probabilities(q, K):
    G = q.shape[0] // K.shape[0]
    s = np.stack([K[h // G] @ q[h] for h in range(q.shape[0])]) / np.sqrt(q.shape[1])
    p = np.exp(s - s.max(1, keepdims=True))
    return p / p.sum(1, keepdims=True)


@pytest.mark.parametrize("fmt,dtype,G,hkv,d,lens,budget,sink,rec,reduce", SELECT)
def test_select_then_sparse(fmt, dtype, G, hkv, d, lens, budget, sink, rec, reduce):
    c = Case(fmt, dtype, G, hkv, d, lens, seed=sum(lens) + budget, stale=0xff)
    cnt, pages, scores, dev = select(c, budget, sink, rec, reduce)
    c.check(what="delta")
    picked = []
    for b, n in enumerate(lens):
        N = -(-n // PAGE)
        if n == 0:
            assert cnt[b] == 0
            picked.append([])
            continue
        K, _ = c.kv(b)
        p = probabilities(host(c.q)[b], K)
        w = p.sum(0) if reduce == "sum" else p.max(0)
        S = np.zeros(N)
        np.add.at(S, np.arange(n) // PAGE, w)
        # a page's share is 2^(lse - c): the logits' error (attention_tolerance), log2, exp2 and the rounding of
        # values up to 64 in base 2, each on both sides of the difference
        A = np.abs(K).max() * np.abs(host(c.q)[b]).sum(1).max() / np.sqrt(d) * 1.4427
        rel = 2 * ((d + 8) * 2.0 ** -24 * A + 4 * 2.0 ** -22 + 64 * 2.0 ** -24)
        if dtype == "bf16":
            rel += 2 * Q_PART[fmt] * np.abs(host(c.q)[b]).max() * np.abs(K).sum(2).max() / np.sqrt(d)
        assert np.all(np.abs(scores[b, :N] - S) <= rel * S + hkv * 2.0 ** -55), b
        assert np.all(scores[b, N:] == -1.0)
        sel = pages[b, :cnt[b]].tolist()
        ok, _, _ = selection_ok(sel, S, n, budget, sink, rec)
        assert ok, f"selection b={b}"
        assert np.all(pages[b, cnt[b]:] == -1)
        picked.append(sel)
    L = c.L
    seen = lambda b, n: [t for j in picked[b] for t in range(j * PAGE, min(n, (j + 1) * PAGE))]  # noqa: E731
    for fn in (L.sparse_attn_q8, L.sparse_attn_settled_q8):
        c.o.fill_(99.0)
        fn(c.desc, c.pt, dev[0], dev[1], dev[2], c.q, c.pool.cache, c.o, c.ws, c.bytes, stream())
        assert flags(c.ws) == 0
        c.check(seen, fn.__name__)


def test_selection_entries_outside_the_context_are_flagged_and_skipped():
    c = Case("int8", "bf16", 4, 2, 64, [100, 60], seed=13)
    sel = torch.tensor([[0, 3, 9, 2], [1, -4, 0, 0]], dtype=torch.int32, device="cuda")
    cnt = torch.tensor([3, 2], dtype=torch.int32, device="cuda")
    seen = {0: [*range(16), *range(48, 64)], 1: list(range(16, 32))}
    for fn in (c.L.sparse_attn_q8, c.L.sparse_attn_settled_q8):
        fn(c.desc, c.pt, cnt, sel, 4, c.q, c.pool.cache, c.o, c.ws, c.bytes, stream())
        assert flags(c.ws) == 4
        c.check(lambda b, n: seen[b], fn.__name__)


def test_bad_page_and_length_are_flagged():
    c = Case("e4m3", "bf16", 4, 2, 128, [100, 40], seed=14)
    keep = c.paged.indices.clone()
    c.paged.indices[1] = c.paged.pages
    c.L.full_attn_q8(c.desc, c.pt, c.q, c.pool.cache, c.o, c.ws, c.bytes, stream())
    assert flags(c.ws) == 1
    c.check(lambda b, n: [t for t in range(n) if b or not 16 <= t < 32])
    c.paged.indices.copy_(keep)
    c.paged.kv_len[1] = 5000
    c.L.full_attn_q8(c.desc, c.pt, c.q, c.pool.cache, c.o, c.ws, c.bytes, stream())
    assert flags(c.ws) == 2


# ------------------------------------------------------------------ window layers
WINDOWS = [(1, 0), (16, 0), (17, 4), (100, 16), (33, 37), (5000, 3), (0, 20), (0, 0), (2 ** 31 - 1, 2 ** 31 - 1)]


@pytest.mark.parametrize("window,sink", WINDOWS)
@pytest.mark.parametrize("fmt,dtype,G,hkv,d", [("e4m3", "bf16", 7, 2, 128), ("int8", "f32", 4, 1, 64)])
def test_window(fmt, dtype, G, hkv, d, window, sink):
    c = Case(fmt, dtype, G, hkv, d, [0, 1, 15, 16, 17, 130, 1003], seed=window % 1000 + sink % 1000, stale=0x7f)
    c.L.window_attn_q8(c.desc, c.pt, window, sink, c.q, c.pool.cache, c.o, c.ws, c.bytes, stream())
    assert flags(c.ws) == 0
    c.check(lambda b, n: R.visible(n, window, sink))


def test_window_reads_no_hidden_page():
    # blocks of hidden pages hold NaN scales
    c = Case("int8", "bf16", 4, 2, 128, [600, 90], seed=15)
    seen = {b: R.visible(n, 50, 20) for b, n in enumerate(c.lens)}
    for b, n in enumerate(c.lens):
        for j in sorted(set(range(-(-n // PAGE))) - {t // PAGE for t in seen[b]}):
            c.pool.ks[c.paged.phys(b, j)] = float("nan")
            c.pool.vs[c.paged.phys(b, j)] = float("nan")
    c.L.window_attn_q8(c.desc, c.pt, 50, 20, c.q, c.pool.cache, c.o, c.ws, c.bytes, stream())
    assert np.isfinite(host(c.o)).all()
    num = {w: np.nan_to_num(c.pool.numbers(w)) for w in "kv"}
    c._num = num
    c.check(lambda b, n: seen[b])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_hidden_tokens_may_hold_nan_payloads(dtype):
    # e4m3's NaN code in every token of the listed pages that the window does not show
    c = Case("e4m3", dtype, 4, 2, 64, [200, 43], seed=17)
    k0, v0 = c.pool.numbers("k"), c.pool.numbers("v")
    for b, n in enumerate(c.lens):
        seen = set(R.visible(n, 37, 5))
        for j in sorted({t // PAGE for t in seen}):
            for s in range(PAGE):
                if j * PAGE + s not in seen:
                    c.pool.k[c.paged.phys(b, j), :, s] = 0x7f
                    c.pool.v[c.paged.phys(b, j), :, s] = 0xff
    c.L.window_attn_q8(c.desc, c.pt, 37, 5, c.q, c.pool.cache, c.o, c.ws, c.bytes, stream())
    c._num = {"k": k0, "v": v0}
    c.check(lambda b, n: R.visible(n, 37, 5))


def test_stale_selection_is_replaced_after_the_wait():
    # the kernel guesses that the selection buffer already holds this call's selection: buffers that hold another,
    # a shorter, a longer and a garbage list when the launch before it (a delta-layer) writes the real one
    c = Case("int8", "bf16", 4, 2, 128, [3000, 700, 90], seed=18)
    L, sp = c.L, c.L.DeltaSelectParams(20, 16, 64, c.L.DELTA_HEAD_SUM)
    stride = L.sel_capacity(sp)
    cnt0 = torch.zeros(3, dtype=torch.int32, device="cuda")
    sel0 = torch.zeros(3, stride, dtype=torch.int32, device="cuda")
    st = stream()
    L.select_attn_q8(c.desc, c.pt, sp, c.q, c.pool.cache, c.o, cnt0, sel0, stride, None, c.ws, c.bytes, st)
    torch.cuda.synchronize()          # the settled entry's own condition
    L.sparse_attn_settled_q8(c.desc, c.pt, cnt0, sel0, stride, c.q, c.pool.cache, c.o, c.ws, c.bytes, st)
    want = c.o.clone()
    other = torch.empty_like(c.o)
    for cnt_was, sel_was in ((1, 0), (stride, 3), (0, 7), (-5, -1), (2 ** 30, 2 ** 30), (7, 1)):
        for _ in range(3):
            cnt = torch.full_like(cnt0, cnt_was)
            sel = torch.full_like(sel0, sel_was)
            torch.cuda.synchronize()
            L.select_attn_q8(c.desc, c.pt, sp, c.q, c.pool.cache, other, cnt, sel, stride, None, c.ws, c.bytes, st)
            L.sparse_attn_q8(c.desc, c.pt, cnt, sel, stride, c.q, c.pool.cache, c.o, c.ws, c.bytes, st)
            assert torch.equal(c.o, want), (cnt_was, sel_was)
            assert torch.equal(cnt, cnt0)
    assert flags(c.ws) == 0


def test_write_then_attention_at_once():
    # attention launched right behind the bulk write reads the pages it wrote (over and over, other values each time)
    L = lib()
    hkv, d, n = 4, 128, 4000
    paged = Paged([n, n - 7], seed=19)
    pool = Pool8(paged.pages, hkv, d, "int8")
    dd = desc(4 * hkv, hkv, d, "bf16", paged.pages)
    gen = torch.Generator(device="cuda").manual_seed(20)
    q = torch.randn(2, 4 * hkv, d, generator=gen, device="cuda").bfloat16()
    rows = torch.tensor([0, n, 2 * n - 7], dtype=torch.int32, device="cuda")
    nb = L.workspace_size_q8(dd, 2, paged.longest)
    ws = workspace(nb)
    xs = [[torch.randn(2 * n - 7, hkv, d, generator=gen, device="cuda").bfloat16() for _ in "kv"] for _ in range(4)]
    outs, alone = [], []
    for quiet in (True, False):
        for i in range(12):
            o = torch.empty_like(q)
            k, v = xs[i % 4]
            L.kv_write_q8(dd, paged.table(), rows, n, k, v, pool.cache, stream=stream())
            if quiet:
                torch.cuda.synchronize()
            L.full_attn_q8(dd, paged.table(), q, pool.cache, o, ws, nb, stream())
            (alone if quiet else outs).append(o)
    for a, b in zip(alone, outs):
        assert torch.equal(a, b)


def test_offsets_past_32_bits():
    # pools whose pages lie behind 2^32 bytes
    L = lib()
    hkv, d, pages = 64, 128, 32800
    pool = Pool8(pages, hkv, d, "e4m3")
    idx = torch.tensor([pages - 1, 5, 32790], dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(16)
    small = Pool8(3, hkv, d, "e4m3").fill(gen)
    for x, y in ((pool.k, small.k), (pool.v, small.v), (pool.ks, small.ks), (pool.vs, small.vs)):
        x[idx.long()] = y
    ptr = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    near = torch.arange(3, dtype=torch.int32, device="cuda")
    n = torch.tensor([43], dtype=torch.int32, device="cuda")
    q = torch.randn(1, 64, d, generator=gen, device="cuda").bfloat16()
    got = []
    for pages_, p, i in ((pages, pool, idx), (3, small, near)):
        o = torch.empty_like(q)
        dd = desc(64, hkv, d, "bf16", pages_)
        pt = L.DeltaPageTable(ptr.data_ptr(), i.data_ptr(), n.data_ptr(), 1, 3)
        nb = L.workspace_size_q8(dd, 1, 3)
        L.full_attn_q8(dd, pt, q, p.cache, o, workspace(nb), nb, stream())
        got.append(o)
    assert torch.equal(*got)
