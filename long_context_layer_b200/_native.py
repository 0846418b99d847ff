"""Binding of include/delta_attn.h (argument marshalling only): ctypes, and for the calls of the smallest
layers the module _fastcall, which does the same with less time a call.

Every function takes device pointers as integers or torch CUDA tensors and passes
them unchanged to the C ABI; all computation happens in libdelta_attn.so.  Importing
this module fails loudly when the library has not been built.
"""
from __future__ import annotations

import ctypes
import operator
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdelta_attn.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m long_context_layer_b200.build` "
        "(there is no fallback implementation)")

lib = ctypes.CDLL(LIB_PATH)

try:
    from ._fastcall import bind as _bind
except ImportError:     # not built for this interpreter: the same calls through ctypes, with more time a call
    _bind = None

DELTA_OK, DELTA_ERR_INVALID_ARG, DELTA_ERR_UNSUPPORTED, DELTA_ERR_WORKSPACE, DELTA_ERR_CUDA, DELTA_ERR_BOUNDS = range(6)
DELTA_F32, DELTA_BF16 = 0, 1
DELTA_HEAD_SUM, DELTA_HEAD_MAX = 0, 1
DELTA_E4M3, DELTA_INT8 = 0, 1
DELTA_ROPE_HALF, DELTA_ROPE_INTERLEAVED = 0, 1
DELTA_ROPE_PLAIN, DELTA_ROPE_LINEAR, DELTA_ROPE_BANDS = 0, 1, 2

EXPORTED = [
    "delta_workspace_size", "delta_workspace_size_reduce", "delta_workspace_init", "delta_sel_capacity", "delta_kv_append",
    "delta_kv_append_layers",
    "delta_full_attn", "delta_full_attn_noalloc", "delta_select_attn", "delta_sparse_attn",
    "delta_sparse_attn_settled",
    "delta_layer_shift", "delta_choose_layers", "delta_read_device_error",
    "delta_status_string",
    "delta_window_attn", "delta_rope_table", "delta_rope",
    "delta_kv_append_q8", "delta_kv_append_layers_q8", "delta_kv_write_q8", "delta_kv_read_q8",
    "delta_workspace_size_q8", "delta_full_attn_q8", "delta_select_attn_q8", "delta_sparse_attn_q8",
    "delta_sparse_attn_settled_q8", "delta_window_attn_q8",
]


class DeltaDesc(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("sm_scale", ctypes.c_float),
                ("num_phys_pages", ctypes.c_int64)]


class DeltaPageTable(ctypes.Structure):
    _fields_ = [("page_indptr", ctypes.c_void_p), ("page_indices", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("batch", ctypes.c_int32),
                ("max_pages_per_seq", ctypes.c_int32)]


class DeltaSelectParams(ctypes.Structure):
    _fields_ = [("budget_pages", ctypes.c_int32), ("sink_tokens", ctypes.c_int32),
                ("recency_tokens", ctypes.c_int32), ("reduce", ctypes.c_int32)]


class DeltaRopeParams(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("scaling", ctypes.c_int32), ("base", ctypes.c_double),
                ("factor", ctypes.c_double), ("original_len", ctypes.c_double), ("low_turns", ctypes.c_double),
                ("high_turns", ctypes.c_double)]


class DeltaRope(ctypes.Structure):
    """delta_rope_plan"""
    _fields_ = [("turns", ctypes.c_void_p), ("rotary_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("magnitude", ctypes.c_float), ("positions", ctypes.c_void_p), ("num_positions", ctypes.c_int32),
                ("offset", ctypes.c_int32)]


class DeltaQ8Cache(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("format", ctypes.c_int32)]


_vp, _sz, _i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
_D, _PT, _SP = ctypes.POINTER(DeltaDesc), ctypes.POINTER(DeltaPageTable), ctypes.POINTER(DeltaSelectParams)

lib.delta_workspace_size.argtypes = [_D, _i32, _i32]
lib.delta_workspace_size.restype = _sz
lib.delta_workspace_size_reduce.argtypes = [_D, _i32, _i32, _i32]
lib.delta_workspace_size_reduce.restype = _sz
lib.delta_workspace_init.argtypes = [_vp, _sz, _vp]
lib.delta_workspace_init.restype = _i32
lib.delta_sel_capacity.argtypes = [_SP, _i32]
lib.delta_sel_capacity.restype = _i32
lib.delta_kv_append.argtypes = [_D, _PT, _vp, _vp, _vp, _vp, _vp]
lib.delta_kv_append.restype = _i32
_vpp = ctypes.POINTER(ctypes.c_void_p)
lib.delta_kv_append_layers.argtypes = [_D, _PT, _i32, _vpp, _vpp, _vpp, _vpp, _vp]
lib.delta_kv_append_layers.restype = _i32
lib.delta_full_attn.argtypes = [_D, _PT, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
lib.delta_full_attn.restype = _i32
lib.delta_full_attn_noalloc.argtypes = [_D, _PT, _vp, _vp, _vp, _vp, _vp]
lib.delta_full_attn_noalloc.restype = _i32
lib.delta_select_attn.argtypes = [_D, _PT, _SP, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _sz, _vp]
lib.delta_select_attn.restype = _i32
lib.delta_sparse_attn.argtypes = [_D, _PT, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
lib.delta_sparse_attn.restype = _i32
lib.delta_sparse_attn_settled.argtypes = [_D, _PT, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
lib.delta_sparse_attn_settled.restype = _i32
lib.delta_layer_shift.argtypes = [_PT, _vp, _vp, _vp, _vp]
lib.delta_layer_shift.restype = _i32
lib.delta_choose_layers.argtypes = [ctypes.POINTER(ctypes.c_float), _i32, _i32, _i32, _i32,
                                    ctypes.POINTER(_i32), ctypes.POINTER(_i32)]
lib.delta_choose_layers.restype = _i32
_i64, _Q8 = ctypes.c_int64, ctypes.POINTER(DeltaQ8Cache)
for _name, _args in {
    "delta_window_attn": [_D, _PT, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _sz, _vp],
    "delta_rope_table": [ctypes.POINTER(DeltaRopeParams), ctypes.POINTER(ctypes.c_double)],
    "delta_rope": [_D, ctypes.POINTER(DeltaRope), _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp],
    "delta_kv_append_q8": [_D, _PT, _vp, _vp, _Q8, _vp],
    "delta_kv_append_layers_q8": [_D, _PT, _i32, _vpp, _vpp, _Q8, _vp],
    "delta_kv_write_q8": [_D, _PT, _vp, _i32, _vp, _vp, _i64, _Q8, _vp],
    "delta_kv_read_q8": [_D, _PT, _vp, _i32, _vp, _Q8, _vp, _vp, _vp],
    "delta_full_attn_q8": [_D, _PT, _vp, _Q8, _vp, _vp, _sz, _vp],
    "delta_select_attn_q8": [_D, _PT, _SP, _vp, _Q8, _vp, _vp, _vp, _i32, _vp, _vp, _sz, _vp],
    "delta_sparse_attn_q8": [_D, _PT, _vp, _vp, _i32, _vp, _Q8, _vp, _vp, _sz, _vp],
    "delta_sparse_attn_settled_q8": [_D, _PT, _vp, _vp, _i32, _vp, _Q8, _vp, _vp, _sz, _vp],
    "delta_window_attn_q8": [_D, _PT, _i32, _i32, _vp, _Q8, _vp, _vp, _sz, _vp],
}.items():      # for callers of lib itself, and where _fastcall is not built
    getattr(lib, _name).argtypes = _args
    getattr(lib, _name).restype = _i32
lib.delta_workspace_size_q8.argtypes = [_D, _i32, _i32, _i32]
lib.delta_workspace_size_q8.restype = _sz
lib.delta_read_device_error.argtypes = [_vp, ctypes.POINTER(_i32), _vp]
lib.delta_read_device_error.restype = _i32
lib.delta_status_string.argtypes = [_i32]
lib.delta_status_string.restype = ctypes.c_char_p


class DeltaError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_string(status)} (status {status})")
        self.status = status


def ptr(x) -> int | None:
    """Device address of a torch tensor, an int, or None."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def status_string(status: int) -> str:
    return lib.delta_status_string(status).decode()


def _check(status: int, where: str) -> int:
    if status != DELTA_OK:
        raise DeltaError(status, where)
    return status


def workspace_size(desc: DeltaDesc, batch: int, max_pages_per_seq: int) -> int:
    return lib.delta_workspace_size(ctypes.byref(desc), batch, max_pages_per_seq)


def workspace_size_reduce(desc: DeltaDesc, batch: int, max_pages_per_seq: int, reduce: int) -> int:
    return lib.delta_workspace_size_reduce(ctypes.byref(desc), batch, max_pages_per_seq, reduce)


def workspace_init(workspace, nbytes: int, stream: int = 0) -> None:
    _check(lib.delta_workspace_init(ptr(workspace), nbytes, stream), "delta_workspace_init")


def sel_capacity(sp: DeltaSelectParams, page_size: int = 16) -> int:
    return lib.delta_sel_capacity(ctypes.byref(sp), page_size)


def kv_append(desc, pt, k_new, v_new, k_pool, v_pool, stream: int = 0, check: bool = True) -> int:
    s = lib.delta_kv_append(ctypes.byref(desc), ctypes.byref(pt), ptr(k_new), ptr(v_new), ptr(k_pool),
                            ptr(v_pool), stream)
    return _check(s, "delta_kv_append") if check else s


def _ptr_array(xs):
    return (ctypes.c_void_p * len(xs))(*[ptr(x) for x in xs])


def kv_append_layers(desc, pt, k_new, v_new, k_pools, v_pools, stream: int = 0, check: bool = True) -> int:
    """k_new, v_new, k_pools, v_pools: sequences (one entry per layer) of device tensors or pointers."""
    n = len(k_pools)
    s = lib.delta_kv_append_layers(ctypes.byref(desc), ctypes.byref(pt), n, _ptr_array([k_new[l] for l in range(n)]),
                                   _ptr_array([v_new[l] for l in range(n)]), _ptr_array(list(k_pools)),
                                   _ptr_array(list(v_pools)), stream)
    return _check(s, "delta_kv_append_layers") if check else s


def full_attn(desc, pt, q, k_pool, v_pool, o, workspace, ws_bytes: int, stream: int = 0, check: bool = True) -> int:
    s = lib.delta_full_attn(ctypes.byref(desc), ctypes.byref(pt), ptr(q), ptr(k_pool), ptr(v_pool), ptr(o),
                            ptr(workspace), ws_bytes, stream)
    return _check(s, "delta_full_attn") if check else s


def full_attn_noalloc(desc, pt, q, k_pool, v_pool, o, stream: int = 0, check: bool = True) -> int:
    """delta_full_attn with the library's own fixed scratch instead of a caller workspace."""
    s = lib.delta_full_attn_noalloc(ctypes.byref(desc), ctypes.byref(pt), ptr(q), ptr(k_pool), ptr(v_pool), ptr(o),
                                    stream)
    return _check(s, "delta_full_attn_noalloc") if check else s


def select_attn(desc, pt, sp, q, k_pool, v_pool, o, sel_cnt, sel_pages, sel_stride: int, page_scores,
                workspace, ws_bytes: int, stream: int = 0, check: bool = True) -> int:
    s = lib.delta_select_attn(ctypes.byref(desc), ctypes.byref(pt), ctypes.byref(sp), ptr(q), ptr(k_pool),
                              ptr(v_pool), ptr(o), ptr(sel_cnt), ptr(sel_pages), sel_stride, ptr(page_scores),
                              ptr(workspace), ws_bytes, stream)
    return _check(s, "delta_select_attn") if check else s


def sparse_attn(desc, pt, sel_cnt, sel_pages, sel_stride: int, q, k_pool, v_pool, o, workspace, ws_bytes: int,
                stream: int = 0, check: bool = True) -> int:
    s = lib.delta_sparse_attn(ctypes.byref(desc), ctypes.byref(pt), ptr(sel_cnt), ptr(sel_pages), sel_stride,
                              ptr(q), ptr(k_pool), ptr(v_pool), ptr(o), ptr(workspace), ws_bytes, stream)
    return _check(s, "delta_sparse_attn") if check else s


def sparse_attn_settled(desc, pt, sel_cnt, sel_pages, sel_stride: int, q, k_pool, v_pool, o, workspace,
                        ws_bytes: int, stream: int = 0, check: bool = True) -> int:
    s = lib.delta_sparse_attn_settled(ctypes.byref(desc), ctypes.byref(pt), ptr(sel_cnt), ptr(sel_pages), sel_stride,
                                      ptr(q), ptr(k_pool), ptr(v_pool), ptr(o), ptr(workspace), ws_bytes, stream)
    return _check(s, "delta_sparse_attn_settled") if check else s


def layer_shift(pt, scores_a, scores_b, shift_out, stream: int = 0, check: bool = True) -> int:
    s = lib.delta_layer_shift(ctypes.byref(pt), ptr(scores_a), ptr(scores_b), ptr(shift_out), stream)
    return _check(s, "delta_layer_shift") if check else s


def choose_layers(shift, count: int, first: int = 2, min_gap: int = 2) -> list:
    """delta_choose_layers on a host sequence of per-layer shifts; returns the ascending layer ids."""
    vals = [float(x) for x in shift]
    arr = (ctypes.c_float * len(vals))(*vals)
    out = (_i32 * max(count, 1))()
    n = _i32(0)
    _check(lib.delta_choose_layers(arr, len(vals), count, first, min_gap, out, ctypes.byref(n)),
           "delta_choose_layers")
    return [int(out[i]) for i in range(n.value)]


def read_device_error(workspace, stream: int = 0) -> tuple:
    flags = _i32(0)
    s = lib.delta_read_device_error(ptr(workspace), ctypes.byref(flags), stream)
    return s, flags.value


# ------------------------------------------------------------------ calls through _fastcall
# "p" takes None, an int or a tensor; "i" and "q" a 32- or 64-bit integer; a structure is passed as it is.
def _fast(name: str, *kinds):
    if _bind is None:
        return _through_ctypes(name, kinds)
    return _bind(name, ctypes.cast(getattr(lib, name), ctypes.c_void_p).value, kinds)


_RANGE = {"p": (0, 2 ** 64 - 1), "i": (-2 ** 31, 2 ** 31 - 1), "q": (-2 ** 63, 2 ** 63 - 1)}


def _through_ctypes(name: str, kinds):
    """What _fastcall's bind gives, with its conversions and refusals."""
    types = {"p": ctypes.c_void_p, "i": ctypes.c_int32, "q": ctypes.c_int64}
    fn = ctypes.CFUNCTYPE(ctypes.c_int32, *[types.get(k, ctypes.c_void_p) for k in kinds])((name, lib))

    def word(kind, x):
        if not isinstance(kind, str):
            if type(x) is not kind:
                raise TypeError(f"expected {kind.__name__}, got {type(x).__name__}")
            return ctypes.addressof(x)      # the caller holds x during the call
        x = ptr(x) if kind == "p" else operator.index(x)
        if x is not None and not _RANGE[kind][0] <= x <= _RANGE[kind][1]:
            raise OverflowError(f"{x} does not fit the argument")
        return x

    def call(*args):
        if len(args) != len(kinds):
            raise TypeError(f"{name} takes {len(kinds)} positional arguments")
        return fn(*[word(k, x) for k, x in zip(kinds, args)])
    return call


def _done(status: int, where: str, check: bool) -> int:
    if status != DELTA_OK and check:
        raise DeltaError(status, where)
    return status


_ATTN = (DeltaDesc, DeltaPageTable)
_OUT = ("p", "p", "q", "p")        # o, workspace, its bytes, stream
_window_attn = _fast("delta_window_attn", *_ATTN, "i", "i", "p", "p", "p", *_OUT)
_rope = _fast("delta_rope", DeltaDesc, DeltaRope, "q", "p", "q", "p", "q", "p", "q", "p", "q", "p")
_kv_append_q8 = _fast("delta_kv_append_q8", *_ATTN, "p", "p", DeltaQ8Cache, "p")
_kv_append_layers_q8 = _fast("delta_kv_append_layers_q8", *_ATTN, "i", "p", "p", "p", "p")
_kv_write_q8 = _fast("delta_kv_write_q8", *_ATTN, "p", "i", "p", "p", "q", DeltaQ8Cache, "p")
_kv_read_q8 = _fast("delta_kv_read_q8", *_ATTN, "p", "i", "p", DeltaQ8Cache, "p", "p", "p")
_full_attn_q8 = _fast("delta_full_attn_q8", *_ATTN, "p", DeltaQ8Cache, *_OUT)
_select_attn_q8 = _fast("delta_select_attn_q8", *_ATTN, DeltaSelectParams, "p", DeltaQ8Cache, "p", "p", "p", "i", "p",
                        "p", "q", "p")
_sparse_attn_q8 = _fast("delta_sparse_attn_q8", *_ATTN, "p", "p", "i", "p", DeltaQ8Cache, *_OUT)
_sparse_attn_settled_q8 = _fast("delta_sparse_attn_settled_q8", *_ATTN, "p", "p", "i", "p", DeltaQ8Cache, *_OUT)
_window_attn_q8 = _fast("delta_window_attn_q8", *_ATTN, "i", "i", "p", DeltaQ8Cache, *_OUT)


# ------------------------------------------------------------------ window layers
def window_attn(desc, pt, window_tokens: int, sink_tokens: int, q, k_pool, v_pool, o, workspace, ws_bytes: int,
                stream: int = 0, check: bool = True) -> int:
    return _done(_window_attn(desc, pt, window_tokens, sink_tokens, q, k_pool, v_pool, o, workspace, ws_bytes, stream),
                 "delta_window_attn", check)


# ------------------------------------------------------------------ rotary positions
def rope_table(params: DeltaRopeParams) -> list:
    """delta_rope_table: turns per token of each pair (host doubles; copy them to the device once)."""
    out = (ctypes.c_double * max(params.rotary_dim // 2, 1))()
    _check(lib.delta_rope_table(ctypes.byref(params), out), "delta_rope_table")
    return list(out)


def rope(desc, plan: DeltaRope, rows: int, q, q_out, k, k_out, q_stride: int = 0, q_out_stride: int = 0,
         k_stride: int = 0, k_out_stride: int = 0, stream: int = 0, check: bool = True) -> int:
    return _done(_rope(desc, plan, rows, q, q_stride, q_out, q_out_stride, k, k_stride, k_out, k_out_stride, stream),
                 "delta_rope", check)


# ------------------------------------------------------------------ the cache held in 8 bits
def workspace_size_q8(desc, batch: int, max_pages_per_seq: int, reduce: int = DELTA_HEAD_SUM) -> int:
    return lib.delta_workspace_size_q8(ctypes.byref(desc), batch, max_pages_per_seq, reduce)


def kv_append_q8(desc, pt, k_new, v_new, cache: DeltaQ8Cache, stream: int = 0, check: bool = True) -> int:
    return _done(_kv_append_q8(desc, pt, k_new, v_new, cache, stream), "delta_kv_append_q8", check)


def kv_append_layers_q8(desc, pt, k_new, v_new, caches, stream: int = 0, check: bool = True) -> int:
    """k_new, v_new: one tensor or pointer per layer; caches: one DeltaQ8Cache per layer."""
    n = len(caches)
    ks, vs = _ptr_array([k_new[l] for l in range(n)]), _ptr_array([v_new[l] for l in range(n)])
    cs = (DeltaQ8Cache * n)(*caches)
    return _done(_kv_append_layers_q8(desc, pt, n, ctypes.addressof(ks), ctypes.addressof(vs), ctypes.addressof(cs), stream),
                 "delta_kv_append_layers_q8", check)


def kv_write_q8(desc, pt, token_indptr, max_tokens: int, k, v, cache: DeltaQ8Cache, row_stride: int = 0,
                stream: int = 0, check: bool = True) -> int:
    return _done(_kv_write_q8(desc, pt, token_indptr, max_tokens, k, v, row_stride, cache, stream), "delta_kv_write_q8",
                 check)


def kv_read_q8(desc, pt, token_indptr, max_tokens: int, token_start, cache: DeltaQ8Cache, k_out, v_out,
               stream: int = 0, check: bool = True) -> int:
    return _done(_kv_read_q8(desc, pt, token_indptr, max_tokens, token_start, cache, k_out, v_out, stream),
                 "delta_kv_read_q8", check)


def full_attn_q8(desc, pt, q, cache: DeltaQ8Cache, o, workspace, ws_bytes: int, stream: int = 0,
                 check: bool = True) -> int:
    return _done(_full_attn_q8(desc, pt, q, cache, o, workspace, ws_bytes, stream), "delta_full_attn_q8", check)


def select_attn_q8(desc, pt, sp, q, cache: DeltaQ8Cache, o, sel_cnt, sel_pages, sel_stride: int, page_scores, workspace,
                   ws_bytes: int, stream: int = 0, check: bool = True) -> int:
    return _done(_select_attn_q8(desc, pt, sp, q, cache, o, sel_cnt, sel_pages, sel_stride, page_scores, workspace,
                                 ws_bytes, stream), "delta_select_attn_q8", check)


def sparse_attn_q8(desc, pt, sel_cnt, sel_pages, sel_stride: int, q, cache: DeltaQ8Cache, o, workspace, ws_bytes: int,
                   stream: int = 0, check: bool = True) -> int:
    return _done(_sparse_attn_q8(desc, pt, sel_cnt, sel_pages, sel_stride, q, cache, o, workspace, ws_bytes, stream),
                 "delta_sparse_attn_q8", check)


def sparse_attn_settled_q8(desc, pt, sel_cnt, sel_pages, sel_stride: int, q, cache: DeltaQ8Cache, o, workspace,
                           ws_bytes: int, stream: int = 0, check: bool = True) -> int:
    return _done(_sparse_attn_settled_q8(desc, pt, sel_cnt, sel_pages, sel_stride, q, cache, o, workspace, ws_bytes,
                                         stream), "delta_sparse_attn_settled_q8", check)


def window_attn_q8(desc, pt, window_tokens: int, sink_tokens: int, q, cache: DeltaQ8Cache, o, workspace, ws_bytes: int,
                   stream: int = 0, check: bool = True) -> int:
    return _done(_window_attn_q8(desc, pt, window_tokens, sink_tokens, q, cache, o, workspace, ws_bytes, stream),
                 "delta_window_attn_q8", check)
