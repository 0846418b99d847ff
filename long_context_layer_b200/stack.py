"""One DELTA decode step over a whole layer stack, through the C ABI.

Layer schedule (DELTA: Dynamic Layer-Aware Token Attention, ai.info summary,
"Methodology in Plain English"): layers before the first delta-layer run full
attention; a delta-layer runs full attention and refreshes the page selection;
every other layer runs sparse attention over the selection of the most recent
delta-layer of the same decode step.  The step starts by appending the current
token's k and v to every layer's paged pool in one launch (the cache is kept in full).

Beyond that schedule a stack may hold window layers (the first tokens and the last ones), keep its
cache in 8 bits with a scale per block (Q8Pools), and rotate q and the new k itself (Rotary).

The runner only sequences C-ABI calls on one CUDA stream; it can capture the
whole step in a CUDA graph so one replay launches every kernel of the step.
"""
from __future__ import annotations

import torch

from . import _native as N

FULL, DELTA, SPARSE, WINDOW = "full", "delta", "sparse", "window"
FORMATS = {"e4m3": N.DELTA_E4M3, "int8": N.DELTA_INT8}


def layer_kinds(num_layers: int, delta_layers) -> list:
    first = min(delta_layers)
    return [DELTA if l in delta_layers else (FULL if l < first else SPARSE) for l in range(num_layers)]


class Q8Pools:
    """One layer's cache in 8 bits: payloads k, v [num_phys_pages, Hkv, 16, D] uint8 and block scales
    k_scale, v_scale [num_phys_pages, Hkv] fp32 (format "e4m3" or "int8"); `c` is the descriptor the entry
    points take (kv_write_q8 fills it from a prompt, kv_read_q8 reads it back)."""

    def __init__(self, num_phys_pages: int, num_kv_heads: int, head_dim: int, format: str, device="cuda"):
        if format not in FORMATS:
            raise ValueError(f"format must be one of {sorted(FORMATS)}")
        self.format = format
        self.shape = (num_phys_pages, num_kv_heads, 16, head_dim)
        self.k = torch.zeros(self.shape, dtype=torch.uint8, device=device)
        self.v = torch.zeros_like(self.k)
        self.k_scale = torch.zeros(num_phys_pages, num_kv_heads, dtype=torch.float32, device=device)
        self.v_scale = torch.zeros_like(self.k_scale)
        self.c = N.DeltaQ8Cache(self.k.data_ptr(), self.v.data_ptr(), self.k_scale.data_ptr(), self.v_scale.data_ptr(),
                                FORMATS[format])


class Rotary:
    """Rotary positions of a stack: the device table of delta_rope with its layout and magnitude.

    scaling: "plain", "linear" (factor) or "bands" (factor, original_len, low_turns, high_turns), as
    delta_rope_table defines them; layout: "half" or "interleaved"."""

    def __init__(self, rotary_dim: int, base: float = 10000.0, layout: str = "half", scaling: str = "plain",
                 factor: float = 1.0, original_len: float = 0.0, low_turns: float = 0.0, high_turns: float = 0.0,
                 magnitude: float = 1.0, device="cuda"):
        layouts = {"half": N.DELTA_ROPE_HALF, "interleaved": N.DELTA_ROPE_INTERLEAVED}
        kinds = {"plain": N.DELTA_ROPE_PLAIN, "linear": N.DELTA_ROPE_LINEAR, "bands": N.DELTA_ROPE_BANDS}
        if layout not in layouts:
            raise ValueError(f"layout must be one of {sorted(layouts)}")
        if scaling not in kinds:
            raise ValueError(f"scaling must be one of {sorted(kinds)}")
        table = N.rope_table(N.DeltaRopeParams(rotary_dim, kinds[scaling], base, factor, original_len, low_turns, high_turns))
        self.turns = torch.tensor(table, dtype=torch.float64, device=device)
        self.rotary_dim, self.layout, self.magnitude = rotary_dim, layouts[layout], magnitude

    def plan(self, positions: torch.Tensor, offset: int = 0) -> N.DeltaRope:
        """delta_rope's plan for rows at positions[r % len] + offset (int32, on the device)."""
        return N.DeltaRope(self.turns.data_ptr(), self.rotary_dim, self.layout, self.magnitude, positions.data_ptr(),
                           positions.numel(), offset)


class DeltaStack:
    """Buffers and call sequence of one decode step.

    Tensors (all on one CUDA device):
      indptr [B+1], indices [nnz], kv_len [B]  int32 page table shared by all layers
      k_pools[l], v_pools[l]                   [num_phys_pages, Hkv, 16, D] per layer
      q [L, B, Hq, D], k_new / v_new [L, B, Hkv, D], out [L, B, Hq, D]

    cache "e4m3" or "int8": the cache is held in 8 bits; k_pools is then a list of Q8Pools and v_pools None.
    window_tokens, window_sinks: what the layers of kind "window" see.
    rotary: q and k_new arrive unrotated and are rotated to each sequence's newest position first (the inputs
    are left as they are).
    """

    def __init__(self, kinds, num_q_heads: int, num_kv_heads: int, head_dim: int, dtype: torch.dtype,
                 indptr: torch.Tensor, indices: torch.Tensor, kv_len: torch.Tensor, max_pages_per_seq: int,
                 num_phys_pages: int, budget_pages: int = 0, sink_tokens: int = 0, recency_tokens: int = 0,
                 sm_scale: float = 0.0, keep_scores: bool = False, reduce: int = N.DELTA_HEAD_SUM,
                 cache: str | None = None, window_tokens: int = 0, window_sinks: int = 0,
                 rotary: Rotary | None = None):
        self.kinds = list(kinds)
        unknown = set(self.kinds) - {FULL, DELTA, SPARSE, WINDOW}
        if unknown:
            raise ValueError(f"unknown layer kinds {sorted(unknown)}")
        if cache is not None and cache not in FORMATS:
            raise ValueError(f"cache must be None or one of {sorted(FORMATS)}")
        if WINDOW in self.kinds and (window_tokens < 0 or window_sinks < 0 or window_tokens + window_sinks == 0):
            raise ValueError("window layers need window_tokens and window_sinks >= 0, not both 0")
        self.cache, self.window = cache, (window_tokens, window_sinks)
        self.device = indptr.device
        self.batch = int(kv_len.numel())
        self.dtype = dtype
        dt = N.DELTA_BF16 if dtype == torch.bfloat16 else N.DELTA_F32
        if dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("dtype must be bfloat16 or float32")
        self.desc = N.DeltaDesc(num_q_heads, num_kv_heads, head_dim, 16, dt, sm_scale, num_phys_pages)
        self.indptr, self.indices, self.kv_len = indptr, indices, kv_len
        self.pt = N.DeltaPageTable(indptr.data_ptr(), indices.data_ptr(), kv_len.data_ptr(), self.batch,
                                   max_pages_per_seq)
        self.sp = N.DeltaSelectParams(budget_pages, sink_tokens, recency_tokens, reduce)
        self.max_pages = max_pages_per_seq
        size = N.workspace_size_reduce if cache is None else N.workspace_size_q8
        self.ws_bytes = size(self.desc, self.batch, max_pages_per_seq, reduce)
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
        N.workspace_init(self.workspace, self.ws_bytes, torch.cuda.current_stream(self.device).cuda_stream)
        self.sel_stride = max(N.sel_capacity(self.sp), 1)
        self.delta_layers = [l for l, k in enumerate(self.kinds) if k == DELTA]
        nd = max(len(self.delta_layers), 1)
        self.sel_cnt = torch.zeros(nd, self.batch, dtype=torch.int32, device=self.device)
        self.sel_pages = torch.zeros(nd, self.batch, self.sel_stride, dtype=torch.int32, device=self.device)
        self.page_scores = (torch.zeros(nd, self.batch, max_pages_per_seq, dtype=torch.float32, device=self.device)
                            if keep_scores else None)
        if any(k == SPARSE for k in self.kinds):
            first_sparse = self.kinds.index(SPARSE)
            if not any(k == DELTA for k in self.kinds[:first_sparse]):
                raise ValueError("a sparse layer needs an earlier delta-layer")
        self.graph = None
        self.rope = None
        if rotary is not None:
            self.rotary, self.rope = rotary, rotary.plan(kv_len, -1)
            L = len(self.kinds)
            self.q_rot = torch.empty(L, self.batch, num_q_heads, head_dim, dtype=dtype, device=self.device)
            self.k_rot = torch.empty(L, self.batch, num_kv_heads, head_dim, dtype=dtype, device=self.device)

    # ------------------------------------------------------------------ one step
    def launches_per_step(self, append: bool = True) -> int:
        # a delta-layer scoring with HEAD_SUM selects its pages inside its decode kernel; HEAD_MAX
        # adds a selection kernel
        per = {FULL: 1, DELTA: 1 if self.sp.reduce == N.DELTA_HEAD_SUM else 2, SPARSE: 1, WINDOW: 1}
        return sum(per[k] for k in self.kinds) + (1 if append else 0) + (1 if self.rope is not None else 0)

    def _rotate(self, q, k_new, a: int, b: int, st):
        """q and k_new (None: q alone) of layers [a, b), rotated when the stack has rotary positions
        (one launch)."""
        if self.rope is None:
            return q, k_new
        k, k_out = (None, None) if k_new is None else (k_new[a:b], self.k_rot[a:b])
        for x in (q[a:b], k):
            if x is not None and not x.is_contiguous():
                raise ValueError("q and k_new must be contiguous [layers, batch, heads, head_dim]")
        N.rope(self.desc, self.rope, (b - a) * self.batch, q[a:b], self.q_rot[a:b], k, k_out, stream=st)
        return self.q_rot, None if k_new is None else self.k_rot

    def _append(self, k_new, v_new, k_pools, v_pools, a: int, b: int, st):
        """The new token of layers [a, b) in one launch (layers do not read each other's pools)."""
        if self.cache is None:
            N.kv_append_layers(self.desc, self.pt, k_new[a:b], v_new[a:b], k_pools[a:b], v_pools[a:b], st)
        else:
            N.kv_append_layers_q8(self.desc, self.pt, k_new[a:b], v_new[a:b], [x.c for x in k_pools[a:b]], st)

    def _check_pools(self, pools):
        """Every layer's pools, before a step launches anything (the kernels read as many pages as desc names)."""
        if self.cache is None:
            return
        d = self.desc
        shape = (d.num_phys_pages, d.num_kv_heads, 16, d.head_dim)
        for x in pools:
            if not isinstance(x, Q8Pools) or x.format != self.cache or x.shape != shape:
                raise ValueError(f"a stack with a {self.cache} cache takes Q8Pools of its format and shape")

    def step(self, q, k_new, v_new, k_pools, v_pools, out, append: bool = True, stream: int | None = None):
        st = torch.cuda.current_stream(self.device).cuda_stream if stream is None else stream
        cur = -1
        self._check_pools(k_pools)
        q, k_new = self._rotate(q, k_new, 0, len(self.kinds), st)
        if append:
            self._append(k_new, v_new, k_pools, v_pools, 0, len(self.kinds), st)
        for l, kind in enumerate(self.kinds):
            # a sparse layer after a sparse or window layer uses the settled entry: the selection and
            # the appended tokens were final before the previous layer's kernel began its work (it
            # waited on the delta-layer that wrote the selection), so this layer may read them early
            self._layer(l, kind, cur, q, k_pools, v_pools, out, st, l > 0)
            if kind == DELTA:
                cur = self.delta_layers.index(l)

    # ------------------------------------------------------------------ host buffers
    def step_host(self, q_host, k_new_host, v_new_host, k_pools, v_pools, out_host, q_dev, k_new_dev, v_new_dev,
                  out_dev, append: bool = True, early_layers: int = 2, out_chunks: int = 8):
        """One decode step whose inputs and outputs live in (pinned) host memory.

        On a copy stream: the first `early_layers` layers' q and appended tokens, then every other
        layer's, which arrive while the first layers compute (the append runs as two launches, one
        per group of layers).  The outputs return to the host on another stream in about `out_chunks`
        groups of consecutive layers, each as soon as its last layer is done (the last layer on its
        own, so that only its output is copied after the final kernel).  The compute stream
        joins the copy streams at those few points only, so most consecutive kernels keep their
        programmatic-launch overlap.  *_dev are device staging buffers of the same shapes.
        Everything is enqueued on the current stream (graph-capturable); out_host is complete once
        that stream reaches the end of the step.
        """
        self._check_pools(k_pools)
        main = torch.cuda.current_stream(self.device)
        if not hasattr(self, "_up"):
            self._up = torch.cuda.Stream(self.device)
            self._down = torch.cuda.Stream(self.device)
        up, down = self._up, self._down
        L = len(self.kinds)
        early = max(1, min(early_layers, L))
        up.wait_stream(main)
        down.wait_stream(main)
        groups = [(0, early)] + ([(early, L)] if early < L else [])
        ready = []
        with torch.cuda.stream(up):
            for a, b in groups:
                q_dev[a:b].copy_(q_host[a:b], non_blocking=True)
                k_new_dev[a:b].copy_(k_new_host[a:b], non_blocking=True)
                v_new_dev[a:b].copy_(v_new_host[a:b], non_blocking=True)
                ev = torch.cuda.Event()
                ev.record(up)
                ready.append(ev)
        st = main.cuda_stream
        per = -(-max(L - 1, 1) // max(1, out_chunks))
        cur, c0 = -1, 0
        for gi, (a, b) in enumerate(groups):
            main.wait_event(ready[gi])
            q_use, k_use = self._rotate(q_dev, k_new_dev, a, b, st)
            if append:
                self._append(k_use, v_new_dev, k_pools, v_pools, a, b, st)
            for l in range(a, b):
                kind = self.kinds[l]
                # (the first layer of a group stands behind the group's append and rotation, not behind a layer)
                self._layer(l, kind, cur, q_use, k_pools, v_pools, out_dev, st,
                            l > a or (l > 0 and not append and self.rope is None))
                if kind == DELTA:
                    cur = self.delta_layers.index(l)
                if l + 1 - c0 == per or l >= L - 2:
                    done = torch.cuda.Event()
                    done.record(main)
                    down.wait_event(done)
                    with torch.cuda.stream(down):
                        out_host[c0:l + 1].copy_(out_dev[c0:l + 1], non_blocking=True)
                    c0 = l + 1
        main.wait_stream(up)
        main.wait_stream(down)

    def _layer(self, l, kind, cur, q, k_pools, v_pools, out, st, behind_layer):
        """behind_layer: the launch before this one on the stream is layer l - 1's."""
        d, pt, ws, wb = self.desc, self.pt, self.workspace, self.ws_bytes
        # what the entry points of this cache take in the place of the pools
        pools = (k_pools[l], v_pools[l]) if self.cache is None else (k_pools[l].c,)
        q8 = self.cache is not None
        if kind == FULL:
            (N.full_attn_q8 if q8 else N.full_attn)(d, pt, q[l], *pools, out[l], ws, wb, st)
        elif kind == WINDOW:
            (N.window_attn_q8 if q8 else N.window_attn)(d, pt, *self.window, q[l], *pools, out[l], ws, wb, st)
        elif kind == DELTA:
            c = self.delta_layers.index(l)
            scores = self.page_scores[c] if self.page_scores is not None else None
            self._select(q[l], pools, out[l], self.sel_cnt[c], self.sel_pages[c], scores, st)
        else:
            settled = behind_layer and self.kinds[l - 1] in (SPARSE, WINDOW)
            fn = ((N.sparse_attn_settled_q8 if q8 else N.sparse_attn_settled) if settled
                  else (N.sparse_attn_q8 if q8 else N.sparse_attn))
            fn(d, pt, self.sel_cnt[cur], self.sel_pages[cur], self.sel_stride, q[l], *pools, out[l], ws, wb, st)

    def _select(self, q, pools, out, sel_cnt, sel_pages, scores, st):
        fn = N.select_attn if self.cache is None else N.select_attn_q8
        fn(self.desc, self.pt, self.sp, q, *pools, out, sel_cnt, sel_pages, self.sel_stride, scores, self.workspace,
           self.ws_bytes, st)

    # ------------------------------------------------------------------ CUDA graph
    def capture(self, *args, **kw) -> torch.cuda.CUDAGraph:
        """Capture one step (same arguments as step) into a CUDA graph and return it."""
        s = torch.cuda.Stream(self.device)
        s.wait_stream(torch.cuda.current_stream(self.device))
        with torch.cuda.stream(s):
            self.step(*args, **kw)          # warm: sets per-device kernel attributes outside capture
        torch.cuda.current_stream(self.device).wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.step(*args, **kw)
        self.graph = g
        return g

    def selection(self, delta_index: int = -1) -> list:
        """Host copy of a delta-layer's selection: list (per sequence) of ascending logical pages."""
        cnt = self.sel_cnt[delta_index].cpu().tolist()
        pages = self.sel_pages[delta_index].cpu()
        return [pages[b, :cnt[b]].tolist() for b in range(self.batch)]

    # ------------------------------------------------------------------ calibration
    def calibration_shifts(self, q, k_pools, v_pools, out, stream: int | None = None) -> torch.Tensor:
        """Per-layer shift [L, B]: shift[l][b] = 1 - cos(page scores of layer l-1, of layer l).

        Every layer from 1 on runs as a delta-layer (full attention plus page scores) on the
        current cache; layers 0 and 1 get shift 0.  DELTA's calibration (ai.info summary,
        "Methodology in Plain English") averages such shifts over several steps and inputs
        and places the delta-layers where they are large.
        """
        st = torch.cuda.current_stream(self.device).cuda_stream if stream is None else stream
        L = len(self.kinds)
        self._check_pools(k_pools)
        q, _ = self._rotate(q, None, 0, L, st)
        scores = torch.zeros(L, self.batch, self.max_pages, dtype=torch.float32, device=self.device)
        shift = torch.zeros(L, self.batch, dtype=torch.float32, device=self.device)
        sel_cnt = torch.zeros(self.batch, dtype=torch.int32, device=self.device)
        sel_pages = torch.zeros(self.batch, self.sel_stride, dtype=torch.int32, device=self.device)
        for l in range(1, L):
            pools = (k_pools[l], v_pools[l]) if self.cache is None else (k_pools[l].c,)
            self._select(q[l], pools, out[l], sel_cnt, sel_pages, scores[l], st)
            if l >= 2:
                N.layer_shift(self.pt, scores[l - 1], scores[l], shift[l], st)
        return shift


def choose_delta_layers(shift, count: int, first: int = 2, min_gap: int = 2) -> list:
    """Delta-layer placement from per-layer shifts (shift[l]: between layers l-1 and l), computed by
    the library's host function delta_choose_layers (the rule is stated in include/delta_attn.h)."""
    return N.choose_layers(shift, count, first, min_gap)
