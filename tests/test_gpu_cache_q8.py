"""GPU: writing the 8-bit block cache and reading it back, bit for bit what the fp64 definition stores."""
import numpy as np
import pytest
import torch

from oracle import operators as R
from tests.operator_helpers import DT, PAGE, Paged, Pool8, desc, host, lib, logical, stream

pytestmark = pytest.mark.gpu


def tokens(shape, dtype, seed, grow=True):
    """Normal rows whose sizes differ a lot from token to token (scales grow inside a page)."""
    r = np.random.default_rng(seed)
    x = r.normal(size=shape)
    if grow:
        x *= np.exp(1.5 * r.normal(size=(shape[0], 1, 1)))
    return torch.from_numpy(x).to(DT[dtype]).cuda()


class Model:
    """The definition's blocks of every sequence."""

    def __init__(self, lens, hkv, d, fmt):
        self.hkv, self.d, self.fmt = hkv, d, fmt
        self.blocks = [dict() for _ in lens]

    def write(self, b, pos, rows):
        """rows [m, Hkv, D] at positions pos ..., page by page as one call does."""
        m = len(rows)
        t = 0
        while t < m:
            lp, slot = divmod(pos + t, PAGE)
            step = min(PAGE - slot, m - t)
            for g in range(self.hkv):
                block = self.blocks[b].setdefault((lp, g), R.Block(self.d, self.fmt))
                block.write(slot, rows[t:t + step, g])
            t += step

    def values(self, b, n):
        out = np.zeros((n, self.hkv, self.d))
        for t in range(n):
            for g in range(self.hkv):
                out[t, g] = self.blocks[b][t // PAGE, g].values()[t % PAGE]
        return out


def counts(ms):
    return torch.tensor(np.concatenate([[0], np.cumsum(ms)]), dtype=torch.int32, device="cuda")


def write(L, d, paged, pool, ms, k, v, most=None, **kw):
    L.kv_write_q8(d, paged.table(), counts(ms), max(ms) if most is None else most, k, v, pool.cache, stream=stream(), **kw)


def read(L, d, paged, pool, ms, dtype, starts=None, most=None, fill=0.0):
    hkv, dim = pool.shape[1], pool.shape[3]
    out = [torch.full((max(sum(ms), 1), hkv, dim), fill, dtype=DT[dtype], device="cuda") for _ in range(2)]
    st = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
    L.kv_read_q8(d, paged.table(), counts(ms), max(ms) if most is None else most, st, pool.cache, *out, stream())
    return [host(x) for x in out]


SHAPES = [("bf16", "e4m3", 2, 128), ("bf16", "int8", 3, 64), ("f32", "e4m3", 1, 64), ("f32", "int8", 5, 128),
          ("bf16", "int8", 1, 128), ("f32", "e4m3", 4, 128)]


@pytest.mark.parametrize("dtype,fmt,hkv,dim", SHAPES)
def test_chunks_then_read_back(dtype, fmt, hkv, dim):
    # three chunks per sequence, starting and ending inside pages; an empty chunk; an empty sequence
    L = lib()
    chunks = [[1, 17, 40, 0, 33], [15, 0, 1, 0, 70], [30, 16, 5, 0, 2]]
    total = [sum(c[b] for c in chunks) for b in range(5)]
    paged = Paged([0] * 5, seed=1, room=max(total))
    pool = Pool8(paged.pages, hkv, dim, fmt, stale=0x7f)
    d = desc(hkv, hkv, dim, dtype, paged.pages)
    want = {w: Model(total, hkv, dim, fmt) for w in "kv"}
    done = [0] * 5
    for i, ms in enumerate(chunks):
        paged.set_lens([x + m for x, m in zip(done, ms)])
        k, v = tokens((sum(ms), hkv, dim), dtype, 10 + i), tokens((sum(ms), hkv, dim), dtype, 20 + i)
        write(L, d, paged, pool, ms, k, v, most=3 if i == 1 else None)      # the bound only sizes the launch
        row = 0
        for b, m in enumerate(ms):
            want["k"].write(b, done[b], host(k)[row:row + m])
            want["v"].write(b, done[b], host(v)[row:row + m])
            row += m
        done = list(paged.lens)
        got = read(L, d, paged, pool, done, dtype)
        row = 0
        for b, n in enumerate(done):
            assert np.array_equal(got[0][row:row + n], want["k"].values(b, n)), (i, b)
            assert np.array_equal(got[1][row:row + n], want["v"].values(b, n)), (i, b)
            row += n
    # slots behind the last token and pages of no sequence are as they were
    for b, n in enumerate(done):
        if n % PAGE:
            assert bool((pool.k[paged.phys(b, n // PAGE), :, n % PAGE:] == 0x7f).all())
    spare = sorted(set(range(paged.pages)) - set(paged.indices_h[:-1].tolist()))
    assert bool((pool.v[spare] == 0x7f).all()) and bool((pool.vs[spare] == 0).all())


@pytest.mark.parametrize("dtype,fmt,hkv,dim", SHAPES)
def test_append_token_by_token(dtype, fmt, hkv, dim):
    L = lib()
    paged = Paged([0, 0, 0], seed=2, room=40)
    pool = Pool8(paged.pages, hkv, dim, fmt, stale=0xff)
    d = desc(hkv, hkv, dim, dtype, paged.pages)
    model = {w: Model([0] * 3, hkv, dim, fmt) for w in "kv"}
    starts = [0, 5, 21]                        # the others join later: kv_len 0 is skipped
    for t in range(40):
        paged.set_lens([max(0, t + 1 - s) for s in starts])
        k, v = tokens((3, hkv, dim), dtype, 100 + t), tokens((3, hkv, dim), dtype, 200 + t)
        L.kv_append_q8(d, paged.table(), k, v, pool.cache, stream())
        for b, n in enumerate(paged.lens):
            if n:
                model["k"].write(b, n - 1, host(k)[b:b + 1])
                model["v"].write(b, n - 1, host(v)[b:b + 1])
    for b, n in enumerate(paged.lens):
        for w in "kv":
            got = logical(pool.numbers(w), paged, b).transpose(1, 0, 2)
            assert np.array_equal(got, model[w].values(b, n)), (b, w)


def test_append_layers_equals_single_appends():
    L = lib()
    hkv, dim, layers = 2, 64, 5
    paged = Paged([19, 1, 32], seed=3)
    d = desc(4, hkv, dim, "bf16", paged.pages)
    gen = torch.Generator(device="cuda").manual_seed(4)
    one = [Pool8(paged.pages, hkv, dim, "int8").fill(gen) for _ in range(layers)]
    all_ = [Pool8(paged.pages, hkv, dim, "int8") for _ in range(layers)]
    for a, b in zip(one, all_):
        for x, y in ((a.k, b.k), (a.v, b.v), (a.ks, b.ks), (a.vs, b.vs)):
            y.copy_(x)
    k, v = (torch.randn(layers, 3, hkv, dim, device="cuda").bfloat16() * 4 for _ in range(2))
    L.kv_append_layers_q8(d, paged.table(), k, v, [p.cache for p in all_], stream())
    for l in range(layers):
        L.kv_append_q8(d, paged.table(), k[l], v[l], one[l].cache, stream())
        for a, b in ((one[l].k, all_[l].k), (one[l].v, all_[l].v), (one[l].ks, all_[l].ks), (one[l].vs, all_[l].vs)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scales_at_their_borders(fmt, dtype):
    # one block per page: largest magnitudes at, just below and just above QMAX * 2^e; zeros; the smallest scale;
    # the largest finite values; subnormals
    L = lib()
    q = R.QMAX[fmt]
    info = torch.finfo(DT[dtype])
    tops = [q, q * (1 + info.eps), q * (1 - info.eps / 2), 1.0, 0.0, 2.0 ** -95, 2.0 ** -120, info.tiny / 4, info.max,
            q * 2.0 ** -100, 3.0e38]
    n = PAGE * len(tops)
    x = torch.randn(n, 1, 64, dtype=torch.float64).clamp(-3, 3) / 4
    for i, t in enumerate(tops):
        x[PAGE * i:PAGE * (i + 1)] *= t
        x[PAGE * i + 3, 0, 7] = t
    x = x.to(DT[dtype]).cuda()
    paged = Paged([n], seed=5)
    pool = Pool8(paged.pages, 1, 64, fmt)
    d = desc(1, 1, 64, dtype, paged.pages)
    write(L, d, paged, pool, [n], x, -x)
    m = Model([n], 1, 64, fmt)
    m.write(0, 0, host(x))
    k, v = read(L, d, paged, pool, [n], "f32" if dtype == "f32" else "bf16")
    # the type's largest values (above 2^127 * 1.9375) round to 2^128, which bf16 and fp32 hold as infinity
    with np.errstate(over="ignore"):
        ref = m.values(0, n).astype(np.float32).astype(np.float64)
    assert np.array_equal(k, ref) and np.array_equal(v, -ref)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_non_finite_values_mark_their_block_until_it_starts_anew(fmt, bad):
    L = lib()
    paged = Paged([40], seed=6)
    pool = Pool8(paged.pages, 2, 64, fmt)
    d = desc(2, 2, 64, "f32", paged.pages)
    x = torch.randn(40, 2, 64, device="cuda")
    x[20, 1, 3] = bad
    write(L, d, paged, pool, [40], x, x.abs())
    k, _ = read(L, d, paged, pool, [40], "f32")
    nan = np.isnan(k)
    assert nan[16:32, 1].all() and not nan[:16].any() and not nan[32:].any() and not nan[:, 0].any()
    # an appended finite token does not cure the block; writing its first slot does
    paged.set_lens([32])
    L.kv_append_q8(d, paged.table(), x[:1], x[:1], pool.cache, stream())
    assert np.isnan(read(L, d, paged, pool, [32], "f32")[0][16:32, 1]).all()
    paged.set_lens([17])
    L.kv_append_q8(d, paged.table(), x[:1], x[:1], pool.cache, stream())
    assert np.isfinite(read(L, d, paged, pool, [17], "f32")[0]).all()


def test_strided_rows():
    # k and v as slices of wider rows (a fused projection's output)
    L = lib()
    paged = Paged([50, 3], seed=7)
    d = desc(2, 2, 64, "bf16", paged.pages)
    wide = torch.randn(53, 3 * 2 * 64 + 8, device="cuda").bfloat16()
    k, v = wide[:, 128:256], wide[:, 256:384]
    a, b = Pool8(paged.pages, 2, 64, "e4m3"), Pool8(paged.pages, 2, 64, "e4m3")
    write(L, d, paged, a, [50, 3], k, v, row_stride=wide.stride(0))
    write(L, d, paged, b, [50, 3], k.contiguous(), v.contiguous())
    for x, y in ((a.k, b.k), (a.v, b.v), (a.ks, b.ks), (a.vs, b.vs)):
        assert torch.equal(x, y)


def test_read_back_of_ranges():
    # any first position; rows outside the context are left as they were
    L = lib()
    paged = Paged([100, 5, 0], seed=8)
    pool = Pool8(paged.pages, 3, 128, "int8").fill(torch.Generator(device="cuda").manual_seed(9))
    d = desc(3, 3, 128, "bf16", paged.pages)
    ms, starts = [30, 9, 4], [37, -2, 0]
    k, v = read(L, d, paged, pool, ms, "bf16", starts=starts, fill=7.0)
    for got, w in ((k, "k"), (v, "v")):
        num, row = pool.numbers(w), 0
        for b, (m, s) in enumerate(zip(ms, starts)):
            seq = logical(num, paged, b).transpose(1, 0, 2)
            for i in range(m):
                t = s + i
                want = seq[t] if 0 <= t < paged.lens[b] else np.full((3, 128), 7.0)
                assert np.array_equal(got[row + i], want), (b, i)
            row += m


def test_pages_outside_the_table_or_pool_are_skipped():
    # the kernels' own bounds checks; valid pages of the same call are written and read
    L = lib()
    paged = Paged([40, 16], seed=10)
    pool = Pool8(paged.pages, 1, 64, "int8")
    d = desc(1, 1, 64, "f32", paged.pages)
    x = torch.randn(56, 1, 64, device="cuda")
    broken = paged.indices.clone()
    broken[1] = paged.pages + 5                       # second page of sequence 0
    broken[paged.indptr_h[1]] = -3                    # the only page of sequence 1
    paged.indices = broken
    write(L, d, paged, pool, [40, 16], x, x)
    L.kv_append_q8(d, paged.table(), x[:2], x[:2], pool.cache, stream())
    k, _ = read(L, d, paged, pool, [40, 16], "f32", fill=5.0)
    assert np.all(k[16:32] == 5.0) and np.all(k[40:] == 5.0) and not np.any(k[:16] == 5.0)
    paged.kv_len.copy_(torch.tensor([4000, 16]))      # longer than its pages: the rows past them are left
    k, _ = read(L, d, paged, pool, [40, 16], "f32", starts=[30, 0], fill=5.0)
    assert np.all(k[18:40] == 5.0) and np.all(k[40:] == 5.0)


def test_offsets_past_32_bits():
    # a pool whose last pages lie behind 2^32 bytes
    L = lib()
    hkv, dim, pages = 64, 128, 32800                  # 131,072 bytes a page: 4.3e9 bytes a pool
    pool = Pool8(pages, hkv, dim, "int8")
    d = desc(hkv, hkv, dim, "bf16", pages)
    idx = torch.tensor([pages - 1, 32768, 3], dtype=torch.int32, device="cuda")
    ptr = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    n = torch.tensor([40], dtype=torch.int32, device="cuda")
    pt = L.DeltaPageTable(ptr.data_ptr(), idx.data_ptr(), n.data_ptr(), 1, 3)
    x = torch.randn(40, hkv, dim, device="cuda").bfloat16()
    L.kv_write_q8(d, pt, counts([40]), 40, x, -x, pool.cache, stream=stream())
    out = [torch.empty_like(x) for _ in range(2)]
    L.kv_read_q8(d, pt, counts([40]), 40, None, pool.cache, *out, stream())
    m = Model([40], hkv, dim, "int8")
    m.write(0, 0, host(x))
    ref = m.values(0, 40)
    assert np.array_equal(host(out[0]), ref) and np.array_equal(host(out[1]), -ref)
