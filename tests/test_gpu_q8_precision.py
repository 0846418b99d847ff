"""GPU: outputs over the 8-bit cache are off by their own rounding and no more than 32-bit arithmetic explains."""
import pytest
import torch

from oracle import operators as R
from tests.operator_helpers import PAGE, assert_within, attention_tolerance, flags, host, stream
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
