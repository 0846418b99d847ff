"""GPU: outputs over the 8-bit cache are off by their own rounding and no more than 32-bit arithmetic explains,
also where blocks' scales lie far apart."""
import math

import numpy as np
import pytest
import torch

from oracle import operators as R
from tests.operator_helpers import (DT, HALF_STEP, PAGE, PAYLOAD, Pool8, assert_within, attention_tolerance, desc, flags, host, lib,
                                    stream, workspace)
from tests.test_gpu_attn_q8 import Case

pytestmark = pytest.mark.gpu

# A probability is the sum of two fp16 values: 22 bits and the signs, off by at most 2^-22 of itself.
P_PAIR = 2.0 ** -22


@pytest.mark.parametrize("fmt,G,hkv,d", [("e4m3", 5, 2, 128), ("int8", 4, 3, 64), ("int8", 7, 2, 128), ("e4m3", 2, 2, 64)])
@pytest.mark.parametrize("call", ["full", "delta", "sparse", "settled", "window"])
def test_bf16_outputs_round_once(call, fmt, G, hkv, d):
    # small queries: logits near 0, so that what the logits' own roundings may move is far below a bf16 step
    c = Case(fmt, "bf16", G, hkv, d, [3, 17, 40, 0, 1], seed=31, spread=0.0, qscale=0.05)
    L, st = c.L, stream()
    seen = lambda b, n: range(n)  # noqa: E731
    if call == "full":
        L.full_attn_q8(c.desc, c.pt, c.q, c.pool.cache, c.o, c.ws, c.bytes, st)
    elif call == "window":
        L.window_attn_q8(c.desc, c.pt, 12, 5, c.q, c.pool.cache, c.o, c.ws, c.bytes, st)
        seen = lambda b, n: R.visible(n, 12, 5)  # noqa: E731
    elif call == "delta":
        sp = L.DeltaSelectParams(1, 16, 16, L.DELTA_HEAD_SUM)
        cnt = torch.zeros(5, dtype=torch.int32, device="cuda")
        pages = torch.zeros(5, 4, dtype=torch.int32, device="cuda")
        L.select_attn_q8(c.desc, c.pt, sp, c.q, c.pool.cache, c.o, cnt, pages, 4, None, c.ws, c.bytes, st)
    else:
        cnt = torch.tensor([1, 1, 2, 0, 1], dtype=torch.int32, device="cuda")
        pages = torch.tensor([[0, 0], [1, 0], [0, 2], [0, 0], [0, 0]], dtype=torch.int32, device="cuda")
        fn = L.sparse_attn_q8 if call == "sparse" else L.sparse_attn_settled_q8
        torch.cuda.synchronize()
        fn(c.desc, c.pt, cnt, pages, 2, c.q, c.pool.cache, c.o, c.ws, c.bytes, st)
        at = [[0], [1], [0, 2], [], [0]]
        seen = lambda b, n: [t for j in at[b] for t in range(j * PAGE, min(n, (j + 1) * PAGE))]  # noqa: E731
    assert flags(c.ws) == 0
    got = host(c.o)
    for b, n in enumerate(c.lens):
        K, V = c.kv(b)
        at_b = list(seen(b, n))
        q = host(c.q)[b]
        ref = R.attention(q, K, V, at_b)
        assert_within(got[b], ref, attention_tolerance(q, K[:, at_b], V[:, at_b], ref, "bf16", P_PAIR, fmt=fmt), f"{call} b={b}")


# (log2 of the large block's V scale, its tokens' logit in nats): without weight in the output (-60), and with a
# probability of 2^-37.5 that its values make up for
APART = [(8, -60.0), (12, -60.0), (16, -60.0), (20, -60.0), (24, -60.0), (40, -26.0)]


@pytest.mark.parametrize("power,logit", APART)
@pytest.mark.parametrize("fmt,dtype", [("e4m3", "bf16"), ("int8", "bf16"), ("e4m3", "f32"), ("int8", "f32")])
def test_a_block_of_far_larger_values(fmt, dtype, power, logit):
    # 320 (sequence, KV head) units leave one CTA of 8 warps a unit, so that warp 0 streams every eighth page: one
    # token at logit 0, then a block with V 2^power times larger, 1,375 tokens at logit -8.5 (e4m3: -8) around it; the tokens of
    # the other warps' pages are at -60.  The first token's values nearly cancel the others' sum.
    L = lib()
    B, hkv, G, d, pages = 5, 64, 2, 64, 8 * 88
    gen = torch.Generator(device="cuda").manual_seed(power)
    pool = Pool8(pages, hkv, d, fmt)
    whole = lambda t: t.to(PAYLOAD[fmt]).view(torch.uint8)  # noqa: E731
    v = torch.randint(40, 101, pool.shape, generator=gen, device="cuda").float()
    v[0, :, 0] = -20.0
    pool.v.copy_(whole(v))
    logits = torch.full((pages, PAGE), -60.0, device="cuda")
    logits[::8] = -8.5
    logits[0, 0] = 0.0
    logits[2 * 8] = logit
    pool.k[..., 0] = whole(2 * logits)[:, None, :]              # q0 = 4: the logit is 4 k0 / sqrt(64)
    logits = pool.k[:, 0, :, 0].view(PAYLOAD[fmt]).double() / 2  # (-8 where e4m3 has no -17)
    pool.ks.fill_(1.0)
    pool.vs.fill_(1.0)
    pool.vs[2 * 8] = 2.0 ** power
    q = torch.randn(B, hkv * G, d, generator=gen, device="cuda")
    q[..., 0] = 4.0
    q = q.to(DT[dtype])
    dd = desc(hkv * G, hkv, d, dtype, pages)
    ptr = torch.arange(B + 1, dtype=torch.int32, device="cuda") * pages
    idx = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(B)
    n = torch.full((B,), pages * PAGE, dtype=torch.int32, device="cuda")
    pt = L.DeltaPageTable(ptr.data_ptr(), idx.data_ptr(), n.data_ptr(), B, pages)
    nb = L.workspace_size_q8(dd, B, pages)
    ws = workspace(nb)
    o = torch.empty_like(q)
    L.full_attn_q8(dd, pt, q, pool.cache, o, ws, nb, stream())
    assert flags(ws) == 0
    w = torch.softmax(logits.flatten(), 0).cpu().numpy()
    # A weight's roundings: the product 4 k0 is exact and the other dimensions add zeros, so a logit of at most 38 in
    # base 2 (those with any weight) is rounded at most four times; exp2 2^-22; the pair.  The second fp16 value
    # ends at 2^-25, or 2^-39 of the largest probability, and the largest block's V scale up to 2^6 of a block whose
    # scale is folded in: 2^-32 a token relative to it.
    top = 38.0 if power == 40 else 12.3
    rel = math.log(2) * 4 * 2.0 ** -24 * top + 2.0 ** -22 + P_PAIR + pages * PAGE * 2.0 ** -32
    for h in (0, 41):
        V = (pool.v[:, h].view(PAYLOAD[fmt]).double() * pool.vs[:, h].double()[:, None, None]).cpu().numpy()
        W = float((w.reshape(pages, PAGE) * np.abs(V).max((1, 2))[:, None]).sum())     # at least sum of w |v|
        ref = w @ V.reshape(-1, d)
        tol = (2 * rel + (pages // 8 + 32) * 2.0 ** -24) * W       # 88 pages a warp
        tol = tol * (1 + HALF_STEP[dtype]) + np.abs(ref) * HALF_STEP[dtype]
        for b in (0, B - 1):
            for x in (2 * h, 2 * h + 1):
                assert_within(host(o[b, x]), ref, tol, f"head {x} b={b}")
