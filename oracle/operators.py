"""fp64 definitions of the operators around the cache: rotary positions, the 8-bit block cache and window
attention.  Plain numpy, written from the definitions in include/delta_attn.h."""
from __future__ import annotations

import math

import numpy as np

PAGE = 16
QMAX = {"e4m3": 448.0, "int8": 127.0}
SCALE_MIN = 2.0 ** -100


# ------------------------------------------------------------------ rotary positions
def rope_turns(rotary_dim, scaling="plain", base=10000.0, factor=1.0, original_len=0.0, low=0.0, high=1.0):
    """Turns per token of each pair."""
    out = []
    for j in range(rotary_dim // 2):
        f = base ** (-2.0 * j / rotary_dim)
        if scaling == "linear":
            f = f / factor
        elif scaling == "bands":
            r = original_len * f / (2 * math.pi)
            w = min(1.0, max(0.0, (r - low) / (high - low)))
            f = w * f + (1 - w) * f / factor
        out.append(f / (2 * math.pi))
    return np.array(out)


def rope(x, positions, turns, layout="half", magnitude=1.0):
    """x [rows, heads, D] rotated at positions [rows] (the first 2 * len(turns) dimensions)."""
    x = np.asarray(x, dtype=np.float64)
    out = x.copy()
    half = len(turns)
    for r, pos in enumerate(positions):
        for j, f in enumerate(turns):
            a, b = (j, j + half) if layout == "half" else (2 * j, 2 * j + 1)
            angle = 2 * math.pi * math.fmod(float(pos) * f, 1.0)
            c, s = magnitude * math.cos(angle), magnitude * math.sin(angle)
            out[r, :, a] = x[r, :, a] * c - x[r, :, b] * s
            out[r, :, b] = x[r, :, b] * c + x[r, :, a] * s
    return out


# ------------------------------------------------------------------ the 8-bit cache
def block_scale(amax, fmt):
    """The smallest power of two >= 2^-100 with amax <= QMAX * scale; NaN when amax is not finite."""
    if not math.isfinite(amax):
        return math.nan
    s = SCALE_MIN
    while amax > QMAX[fmt] * s:
        s *= 2.0
    return s


def round8(y, fmt):
    """The nearest 8-bit value, ties to even (y within the format's range)."""
    y = np.asarray(y, dtype=np.float64)
    if fmt == "int8":
        return np.rint(y)
    _, e = np.frexp(np.abs(y))                  # |y| = m * 2^e, 0.5 <= m < 1
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.rint(y / step) * step


class Block:
    """16 tokens x D of one (page, KV head): stored numbers (unscaled) and the scale."""

    def __init__(self, d, fmt, payload=None, scale=1.0):
        self.fmt = fmt
        self.payload = np.zeros((PAGE, d)) if payload is None else np.array(payload, dtype=np.float64)
        self.scale = scale

    def write(self, first, rows):
        """Tokens at slots first, first + 1, ...: the larger scale, older slots rounded again when it grew."""
        rows = np.asarray(rows, dtype=np.float64)
        need = block_scale(np.abs(rows).max() if np.isfinite(rows).all() else math.inf, self.fmt)
        if first > 0:
            now = math.nan if math.isnan(self.scale) or math.isnan(need) else max(self.scale, need)
            if not math.isnan(now) and now != self.scale:
                self.payload[:first] = round8(self.payload[:first] * (self.scale / now), self.fmt)
        else:
            now = need
        self.scale = now
        self.payload[first:first + len(rows)] = 0.0 if math.isnan(now) else round8(rows / now, self.fmt)

    def values(self):
        return self.payload * self.scale


# ------------------------------------------------------------------ attention
def visible(n, window, sink):
    """Tokens a window layer sees."""
    return [t for t in range(n) if t < sink or t >= n - window]


def attention(q, K, V, tokens=None, scale=None):
    """q [Hq, D], K, V [Hkv, n, D]: softmax over the given tokens (default all); 0 without any."""
    Hq, D = q.shape
    G = Hq // K.shape[0]
    idx = np.arange(K.shape[1]) if tokens is None else np.asarray(tokens, dtype=np.int64)
    out = np.zeros((Hq, D))
    if len(idx) == 0:
        return out
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    for h in range(Hq):
        s = K[h // G][idx] @ q[h] * scale
        p = np.exp(s - s.max())
        out[h] = (p / p.sum()) @ V[h // G][idx]
    return out
