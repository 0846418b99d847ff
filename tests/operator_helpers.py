"""Inputs, device buffers and derived tolerances of the operator tests (rotary, 8-bit cache, window).

Tolerances count roundings.  A rounding to a type is off by at most finfo.eps / 2 relative to the value.
Attention: with w the weights, an output is sum_t w_t v_t; a relative error d_t of each weight (the same weights
normalise) moves it by at most 2 max|d_t| max|v|.  A weight's relative error is ln 2 times the absolute error of
its base-2 logit plus exp2's (2^-22) plus the rounding of p for the matrix product.  A logit is a sum of D
products: at most (D + 8) roundings of partial sums no larger than A = max_t sum_i |q_i k_ti| / sqrt(D) * log2 e.
bf16 queries over the int8 cache are 23-bit fixed point: an element is off by at most Q_PART of the head's largest,
which moves a logit by at most that times sum_i |k_ti| / sqrt(D) nats (e4m3: fp16, 2^-24 below 2^-14 of 2^14).
The sum over tokens runs over at most n / 16 + 32 fp32 additions of partial sums no larger than max|v|.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from oracle import operators as R

PAGE = 16
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
P_ROUND = {"bf16": 2.0 ** -11, "f32": 2.0 ** -22}      # p as one fp16 value, or as the sum of two
Q_PART = {"e4m3": 2.0 ** -39, "int8": 2.0 ** -22}      # half a step of the smallest unit
PAYLOAD = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def lib():
    import long_context_layer_b200 as L
    return L


def stream():
    return torch.cuda.current_stream().cuda_stream


def attention_tolerance(q, K, V, ref, dtype, p_round=None, fmt=None):
    """Element-wise bound of |kernel - fp64| for q [Hq, D], K and V [Hkv, n, D], ref [Hq, D]; fmt: the 8-bit
    cache's format."""
    if K.shape[1] == 0:
        return np.zeros_like(ref)
    Hq, D = q.shape
    G = Hq // K.shape[0]
    p_round = P_ROUND[dtype] if p_round is None else p_round
    tol = np.zeros_like(ref)
    for h in range(Hq):
        A = float((np.abs(K[h // G]) @ np.abs(q[h])).max()) / math.sqrt(D) * math.log2(math.e)
        rel = math.log(2) * (D + 8) * 2.0 ** -24 * A + 2.0 ** -22 + p_round
        if fmt is not None and dtype == "bf16":
            rel += Q_PART[fmt] * np.abs(q[h]).max() * np.abs(K[h // G]).sum(1).max() / math.sqrt(D)
        vmax = np.abs(V[h // G]).max()
        tol[h] = 2 * vmax * rel + (K.shape[1] / 16 + 32) * 2.0 ** -24 * vmax
    # the result itself, and its distance from the exact one, are rounded to the output type
    return tol * (1 + HALF_STEP[dtype]) + np.abs(ref) * HALF_STEP[dtype]


def assert_within(got, ref, tol, what=""):
    got, ref = np.asarray(got, dtype=np.float64), np.asarray(ref, dtype=np.float64)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, worst {np.abs(got - ref)[bad].max():.3e}, " \
                          f"allowed there {np.broadcast_to(tol, ref.shape)[bad].min():.3e}"


class Paged:
    """A page table over a shuffled pool with spare pages, for sequences of the given lengths."""

    def __init__(self, lens, seed=0, room=None, spare=3):
        r = np.random.default_rng(seed)
        n_pages = [-(-(n if room is None else room) // PAGE) for n in lens]
        self.pages = sum(n_pages) + spare
        perm = r.permutation(self.pages)[: sum(n_pages)]
        self.indptr_h = np.concatenate([[0], np.cumsum(n_pages)]).astype(np.int32)
        self.indices_h = np.concatenate([perm, [0]]).astype(np.int32)
        self.lens = list(lens)
        self.longest = max(1, max(n_pages))
        self.indptr = torch.from_numpy(self.indptr_h).cuda()
        self.indices = torch.from_numpy(self.indices_h).cuda()
        self.kv_len = torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    def set_lens(self, lens):
        self.lens = list(lens)
        self.kv_len.copy_(torch.tensor(self.lens, dtype=torch.int32))

    def table(self):
        return lib().DeltaPageTable(self.indptr.data_ptr(), self.indices.data_ptr(), self.kv_len.data_ptr(), len(self.lens),
                                    self.longest)

    def phys(self, b, lp):
        return int(self.indices_h[self.indptr_h[b] + lp])

    def rows(self, b, n=None):
        """(physical page, slot) of every token of sequence b."""
        t = np.arange(self.lens[b] if n is None else n)
        return self.indices_h[self.indptr_h[b] + t // PAGE], t % PAGE


class Pool8:
    """K and V pools of an 8-bit cache on the device, their DeltaQ8Cache and what they stand for."""

    def __init__(self, pages, hkv, d, fmt, payload=None, scale=None, stale=None):
        L = lib()
        self.fmt, self.shape = fmt, (pages, hkv, PAGE, d)
        self.k = torch.zeros(self.shape, dtype=torch.uint8, device="cuda")
        self.v = torch.zeros_like(self.k)
        if stale is not None:
            self.k.fill_(stale)
            self.v.fill_(stale)
        self.ks = torch.zeros((pages, hkv), device="cuda")
        self.vs = torch.zeros_like(self.ks)
        self.cache = L.DeltaQ8Cache(self.k.data_ptr(), self.v.data_ptr(), self.ks.data_ptr(), self.vs.data_ptr(),
                                    L.DELTA_E4M3 if fmt == "e4m3" else L.DELTA_INT8)

    def fill(self, gen, spread=0.0, std=1.0):
        """Quantised normal blocks, block sizes varying by 2^N(0, spread)."""
        for pool, scale in ((self.k, self.ks), (self.v, self.vs)):
            x = torch.randn(self.shape, generator=gen, device="cuda") * std
            x *= torch.exp2(spread * torch.randn(self.shape[:2], generator=gen, device="cuda"))[..., None, None]
            m, e = torch.frexp(x.abs().amax((2, 3)))
            top, shift = (0.875, 9) if self.fmt == "e4m3" else (0.9921875, 7)
            s = ((e - shift + (m > top).int() + 127).clamp_min(27) << 23).view(torch.float32)
            y = x / s[..., None, None]
            pool.copy_((y.to(torch.float8_e4m3fn) if self.fmt == "e4m3" else y.round().to(torch.int8)).view(torch.uint8))
            scale.copy_(s)
        return self

    def numbers(self, which):
        """What the pool stands for, fp64 [pages, hkv, 16, d]."""
        pool, scale = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        return (pool.view(PAYLOAD[self.fmt]).double() * scale.double()[..., None, None]).cpu().numpy()


def logical(numbers, paged, b, n=None):
    """[Hkv, n, D] of sequence b."""
    page, slot = paged.rows(b, n)
    return numbers[page, :, slot].transpose(1, 0, 2)


def desc(hq, hkv, d, dtype, pages):
    L = lib()
    return L.DeltaDesc(hq, hkv, d, PAGE, L.DELTA_BF16 if dtype == "bf16" else L.DELTA_F32, 0.0, pages)


def workspace(size):
    L = lib()
    ws = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
    L.workspace_init(ws, ws.numel(), stream())
    return ws


def flags(ws):
    return lib().read_device_error(ws, stream())[1]


def host(x):
    return x.double().cpu().numpy()


__all__ = [n for n in dir() if not n.startswith("_")]
