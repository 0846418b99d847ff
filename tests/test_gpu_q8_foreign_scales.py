"""GPU: tokens written into blocks whose scales are not the ones this library makes (any finite scale >= 0)."""
import math

import numpy as np
import pytest
import torch

from oracle import operators as R
from tests.operator_helpers import DT, PAGE, PAYLOAD, Paged, Pool8, desc, host, lib, stream
from tests.test_gpu_cache_q8 import counts

pytestmark = pytest.mark.gpu

SCALES = [0.7, 1.3, 1.0, 3.0 * 2.0 ** -110, 2.0 ** -120, 0.0, 2.0 ** 126 * 0.75, 2.0 ** 127]


@pytest.mark.parametrize("call", ["append", "write"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_tokens_written_behind_such_a_scale(fmt, dtype, call):
    L = lib()
    hkv, d, slot, m = 2, 64, 5, 1 if call == "append" else 3
    grow = (1.0, 30.0, 1000.0)             # the new tokens against what the block's scale can hold (about 0.1 to 100)
    todo = [(s, g) for s in SCALES for g in grow if s < 1e30 or g == 1.0]
    paged = Paged([slot + m] * len(todo), seed=3)
    gen = torch.Generator(device="cuda").manual_seed(5)
    pool = Pool8(paged.pages, hkv, d, fmt).fill(gen)
    old = torch.tensor([s for s, _ in todo], dtype=torch.float32, device="cuda")
    page = torch.tensor([paged.phys(b, 0) for b in range(len(todo))], device="cuda")
    pool.ks[page] = old[:, None]
    pool.vs[page] = old[:, None]
    before = {w: (p.view(PAYLOAD[fmt]).double().cpu().numpy(), s.double().cpu().numpy())
              for w, p, s in (("k", pool.k, pool.ks), ("v", pool.v, pool.vs))}
    size = torch.tensor([s * 0.3 if s > 1e30 else (s if s > 2.0 ** -100 else 1.0) * g * 2.0 for s, g in todo], device="cuda")
    k, v = ((torch.randn(len(todo), m, hkv, d, generator=gen, device="cuda").clamp(-3, 3) * size[:, None, None, None]).to(DT[dtype])
            for _ in "kv")
    dd = desc(hkv, hkv, d, dtype, paged.pages)
    if call == "append":
        L.kv_append_q8(dd, paged.table(), k, v, pool.cache, stream())
    else:
        L.kv_write_q8(dd, paged.table(), counts([m] * len(todo)), m, k, v, pool.cache, stream=stream())
    for w, x, payload, scale in (("k", k, pool.k, pool.ks), ("v", v, pool.v, pool.vs)):
        payload, scale = payload.view(PAYLOAD[fmt]).double().cpu().numpy(), scale.double().cpu().numpy()
        for b, (s, g) in enumerate(todo):
            p = paged.phys(b, 0)
            for h in range(hkv):
                s0 = before[w][1][p, h]
                fresh = host(x)[b, :, h]
                now = max(s0, R.block_scale(np.abs(fresh).max(), fmt))
                assert scale[p, h] == now, (s, g)
                got = payload[p, h, :slot + m] * now
                was = before[w][0][p, h, :slot] * s0
                if now == s0:
                    assert np.array_equal(got[:slot], was), (s, g)       # untouched
                want = np.concatenate([was, fresh])
                # half a step of the 8-bit type, and the quotient's own roundings: 1 / scale and the product, 2^-24 each
                # (a scale of 2^127: its inverse 2^-127 is exact)
                y = np.abs(want) / now
                step = np.ones_like(y) if fmt == "int8" else np.ldexp(1.0, np.maximum(np.frexp(np.maximum(y, 1e-30))[1] - 1, -6) - 3)
                assert np.all(np.abs(got - want) <= now * (0.5 * step * (1 + 2.0 ** -20) + y * 2.0 ** -22)), (s, g, w, h)
    # blocks of pages without new tokens are as they were
    spare = sorted(set(range(paged.pages)) - {paged.phys(b, 0) for b in range(len(todo))})
    for w, pp, ss in (("k", pool.k, pool.ks), ("v", pool.v, pool.vs)):
        assert np.array_equal(pp.view(PAYLOAD[fmt]).double().cpu().numpy()[spare], before[w][0][spare])
        assert np.array_equal(ss.double().cpu().numpy()[spare], before[w][1][spare])
    assert math.isfinite(float(pool.ks.max())) and PAGE == 16
