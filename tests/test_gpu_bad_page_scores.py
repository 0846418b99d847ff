"""GPU: a page outside the pool is flagged, skipped and scores 0 in a delta-layer, whatever the calls before left in
the workspace."""
import numpy as np
import pytest
import torch

from tests.operator_helpers import DT, PAGE, Paged, Pool8, desc, flags, host, lib, logical, stream, workspace
from tests.test_gpu_attn_q8 import probabilities

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("reduce", ["sum", "max"])
@pytest.mark.parametrize("cache,dtype", [("plain", "bf16"), ("plain", "f32"), ("e4m3", "bf16"), ("int8", "bf16"), ("int8", "f32")])
@pytest.mark.parametrize("lens,bad", [([700, 90], (0, 13)), ([90, 33], (1, 1)), ([5000], (0, 200)), ([333], (0, 20))])
def test_score_of_a_bad_page(cache, dtype, reduce, lens, bad):
    L = lib()
    hkv, G, d = 2, 3, 64
    paged = Paged(lens, seed=4)
    gen = torch.Generator(device="cuda").manual_seed(6)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(DT[dtype])  # noqa: E731
    if cache == "plain":
        k, v = (rand(paged.pages, hkv, PAGE, d) for _ in "kv")
        store, K = (k, v), host(k)
    else:
        pool = Pool8(paged.pages, hkv, d, cache).fill(gen)
        store, K = (pool.cache,), pool.numbers("k")
    dd = desc(hkv * G, hkv, d, dtype, paged.pages)
    mode = L.DELTA_HEAD_SUM if reduce == "sum" else L.DELTA_HEAD_MAX
    sp = L.DeltaSelectParams(4, 0, 0, mode)
    size = L.workspace_size_reduce if cache == "plain" else L.workspace_size_q8
    nb = size(dd, len(lens), paged.longest, mode)
    ws = workspace(nb)
    q = rand(len(lens), hkv * G, d)
    o = torch.empty_like(q)
    cnt = torch.zeros(len(lens), dtype=torch.int32, device="cuda")
    pages = torch.zeros(len(lens), 4, dtype=torch.int32, device="cuda")
    scores = torch.zeros(len(lens), paged.longest, device="cuda")
    fn = L.select_attn if cache == "plain" else L.select_attn_q8

    def call(x):
        fn(dd, paged.table(), sp, x, *store, o, cnt, pages, 4, scores, ws, nb, stream())
    b, j = bad
    # the bad page's own tokens had large logits in the call before (this page's first key as the query)
    big = q.clone()
    big[b] = (4 * torch.from_numpy(K[paged.phys(b, j), :, 0]).repeat_interleave(G, 0)).to(DT[dtype]).cuda()
    call(big)
    assert flags(ws) == 0 and int(cnt[b]) == min(4, -(-lens[b] // PAGE)) and j in pages[b].tolist()
    keep = paged.indices.clone()
    paged.indices[int(paged.indptr_h[b]) + j] = paged.pages
    call(q)
    assert flags(ws) == 1
    paged.indices.copy_(keep)
    got = scores.double().cpu().numpy()
    for i, n in enumerate(lens):
        N = -(-n // PAGE)
        at = [t for t in range(n) if i != b or t // PAGE != j]
        p = probabilities(host(q)[i], logical(K, paged, i)[:, at])
        w = p.sum(0) if reduce == "sum" else p.max(0)
        S = np.zeros(N)
        np.add.at(S, np.array(at) // PAGE, w)
        # logits of size A rounded d + 8 times, in the page's sum and in the normaliser; a bf16 query over int8 keys by
        # 2^-22 of its largest element; log2, exp2 and values up to 64 in base 2 (the plain bf16 cache: the same sums)
        A = np.abs(K).max() * np.abs(host(q)[i]).sum(1).max() / np.sqrt(d) * 1.4427
        rel = 2 * ((d + 8) * 2.0 ** -24 * A + 4 * 2.0 ** -22 + 64 * 2.0 ** -24) + 2 * 2.0 ** -22 * np.abs(K).max() * d * np.abs(host(q)[i]).max()
        assert np.all(np.abs(got[i, :N] - S) <= rel * S + hkv * 2.0 ** -55), i
        best = sorted(range(N), key=lambda x: (-got[i, x], x))[:4]
        assert sorted(best) == pages[i, : int(cnt[i])].tolist()
    assert got[b, j] == 0.0
