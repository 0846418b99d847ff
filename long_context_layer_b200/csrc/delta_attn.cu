// DELTA decode attention stack for B200 (sm_100a): the full, delta and sparse layers over the bf16 / fp32
// cache, the appends and the calibration calls of include/delta_attn.h.  (Window layers: window_attn.cu; the
// 8-bit cache: cache_q8.cu and attn_q8.cu; rotary positions: rope.cu.)
//
// Method: "DELTA: Dynamic Layer-Aware Token Attention for Efficient Long-Context Reasoning",
// ai.info summary, section "Methodology in Plain English".  Initial layers run full attention,
// delta-layers run full attention and score 16-token KV pages, sparse layers attend only to
// the selected pages; the paged KV cache is kept in full.
//
// Kernels (all launched on the caller's stream with programmatic dependent launch, none
// synchronises the host):
//   kv_append_kernel,     the current token's k, v into its page slot: one (sequence, KV head)
//   kv_append_layers_     per CTA (and per layer), 16-byte vector copies.
//     kernel
//   decode_mma_kernel     bf16 split-KV online-softmax decode on the tensor cores (mma.sync,
//                         decode_mma.cuh).  Grid (split, KV head, sequence) in thread-block
//                         clusters; each warp streams whole pages (K and V of one KV head) into
//                         its own shared-memory ring with 2-D TMA tensor copies.  Delta-layers
//                         also write each (head, page)'s log2-sum-exp and each split's per-head
//                         state; sparse layers walk the selected page list.  Splits merge by
//                         pushing their partials into the owning CTA of the cluster (st.async
//                         on its mbarrier); several clusters of one unit meet in the workspace,
//                         merged by whichever CTA arrives last (an atomic ticket; no CTA waits).
//   decode_kernel         the fp32 counterpart on the CUDA cores (decode_simt.cuh), same merge.
//   score_select_kernel   one thread-block cluster per sequence (select.cuh): page score = sum
//                         over heads of 2^(lse_hp - c_h), c_h from the splits' states; the k-th
//                         largest candidate by a bucket histogram and an exact in-bucket rank
//                         (one CTA) or an MSB-first radix select (cluster); lower-index tie-break,
//                         union with sink and recency pages, ascending compaction.
//   layer_shift_kernel    1 - cos between two layers' page-score vectors (calibration metric).
//
// Logits are carried in base 2 (q is pre-scaled by sm_scale*log2(e)) so every exponential is
// one exp2.  No floating-point atomics are used: results are deterministic run to run.

#include "delta_attn.h"

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <mutex>

#include "common.cuh"
#include "host.cuh"
#include "launch_plain.cuh"
#include "select.cuh"

namespace delta {

delta_status launch_score_select(const AttnCall& a, const DecodeParams& prm) {
    const int Hq = a.d->num_q_heads;
    SelectParams sp2{};
    sp2.indptr = a.pt->page_indptr;
    sp2.indices = a.pt->page_indices;
    sp2.num_phys_pages = a.d->num_phys_pages;
    sp2.kv_len = a.pt->kv_len;
    sp2.page_lse = prm.page_lse;
    sp2.split_ml = prm.split_ml;
    sp2.num_splits = prm.num_splits;
    sp2.num_q_heads = Hq;
    sp2.max_pages = a.pt->max_pages_per_seq;
    sp2.budget_pages = a.sp->budget_pages;
    sp2.sink_tokens = a.sp->sink_tokens;
    sp2.recency_tokens = a.sp->recency_tokens;
    sp2.sel_cnt = a.sel_cnt_out;
    sp2.sel_pages = a.sel_pages_out;
    sp2.sel_stride = a.sel_stride_out;
    sp2.page_scores = a.page_scores;
    sp2.logits = prm.logits;
    sp2.err = prm.err;
    // one cluster of C CTAs per sequence; HEAD_MAX scores every token of every head (a warp per
    // page), so a CTA takes about one page per warp
    const int maxp = a.pt->max_pages_per_seq;
    int C = (maxp + kSelectThreads / 32 - 1) / (kSelectThreads / 32);
    C = C < 1 ? 1 : (C > 16 ? 16 : C);
    const int chunk = (maxp + C - 1) / C;
    const SelectSmem SL{chunk, C};
    // 32,768 pages over 16 CTAs are 2,048 pages each
    if (chunk > kMaxSelectChunk) return DELTA_ERR_UNSUPPORTED;
    const size_t smem_max = SelectSmem{kMaxSelectChunk, 16}.bytes();
    if (!configure_kernel(reinterpret_cast<const void*>(score_select_kernel), smem_max)) return DELTA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(C, a.pt->batch);
    cfg.blockDim = dim3(kSelectThreads);
    cfg.dynamicSmemBytes = SL.bytes();
    cfg.stream = static_cast<cudaStream_t>(a.stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, score_select_kernel, sp2, chunk) != cudaSuccess) return DELTA_ERR_CUDA;
    return launch_status();
}

// The attention entry points over the bf16 / fp32 pools.
delta_status run_attention(int mode, const delta_desc* d, const delta_page_table* pt, const delta_select_params* sp,
                           const int32_t* sel_cnt_in, const int32_t* sel_pages_in, int32_t sel_stride_in,
                           const void* q, const void* k_pool, const void* v_pool, void* o, int32_t* sel_cnt_out,
                           int32_t* sel_pages_out, int32_t sel_stride_out, float* page_scores, void* ws,
                           size_t ws_bytes, void* stream, bool settled = false, size_t lead = 0) {
    AttnCall a;
    a.mode = mode;
    a.d = d;
    a.pt = pt;
    a.sp = sp;
    a.sel_cnt_in = sel_cnt_in;
    a.sel_pages_in = sel_pages_in;
    a.sel_stride_in = sel_stride_in;
    a.settled = settled;
    a.q = q;
    a.o = o;
    a.sel_cnt_out = sel_cnt_out;
    a.sel_pages_out = sel_pages_out;
    a.sel_stride_out = sel_stride_out;
    a.page_scores = page_scores;
    a.ws = ws;
    a.ws_bytes = ws_bytes;
    a.lead = lead;
    a.stream = stream;
    return run_attention_on(PlainCache<false>{k_pool, v_pool}, a);
}

// ------------------------------------------------------------------ allocation-free variant
// Scratch of delta_full_attn_noalloc: a fixed array in the library's own device memory, so the
// call needs no workspace from the caller.  Every GPU that loads the library holds it until the
// process exits.
constexpr size_t kStaticScratchBytes = size_t(8) << 20;   // 8 MiB
static __device__ __align__(256) unsigned char g_noalloc_scratch[kStaticScratchBytes];

// Device address of the scratch array on the current device, looked up once per device.  In
// host code the array's name only stands for the symbol; the kernel must get this address.
unsigned char* noalloc_scratch() {
    static unsigned char* addr[64] = {nullptr};
    std::lock_guard<std::recursive_mutex> lock(cache_mutex());
    const int dev = current_device();
    if (dev < 0) return nullptr;
    if (addr[dev] == nullptr) {
        void* ptr = nullptr;
        if (cudaGetSymbolAddress(&ptr, g_noalloc_scratch) != cudaSuccess || ptr == nullptr) return nullptr;
        addr[dev] = static_cast<unsigned char*>(ptr);
    }
    return addr[dev];
}

}  // namespace delta

using namespace delta;

// ================================================================== C ABI
extern "C" {

size_t delta_workspace_size(const delta_desc* desc, int32_t batch, int32_t max_pages_per_seq) {
    if (check_desc(desc) != DELTA_OK || batch < 0 || max_pages_per_seq < 0) return 0;
    return ws_layout(desc, batch, max_pages_per_seq).total;
}

size_t delta_workspace_size_reduce(const delta_desc* desc, int32_t batch, int32_t max_pages_per_seq, int32_t reduce) {
    if (check_desc(desc) != DELTA_OK || batch < 0 || max_pages_per_seq < 0) return 0;
    if (reduce != DELTA_HEAD_SUM && reduce != DELTA_HEAD_MAX) return 0;
    return ws_layout(desc, batch, max_pages_per_seq, reduce == DELTA_HEAD_MAX).total;
}

delta_status delta_workspace_init(void* workspace, size_t ws_bytes, void* stream) {
    if (workspace == nullptr) return DELTA_ERR_INVALID_ARG;
    if (cudaMemsetAsync(workspace, 0, ws_bytes, static_cast<cudaStream_t>(stream)) != cudaSuccess) return DELTA_ERR_CUDA;
    return DELTA_OK;
}

int32_t delta_sel_capacity(const delta_select_params* sp, int32_t page_size) {
    if (sp == nullptr || page_size <= 0 || sp->budget_pages < 0 || sp->sink_tokens < 0 || sp->recency_tokens < 0)
        return -1;
    const int32_t sink = (sp->sink_tokens + page_size - 1) / page_size;
    const int32_t rec = sp->recency_tokens > 0 ? (sp->recency_tokens + page_size - 1) / page_size + 1 : 0;
    return sp->budget_pages + sink + rec;
}

delta_status delta_kv_append(const delta_desc* desc, const delta_page_table* pt, const void* k_new,
                             const void* v_new, void* k_pool, void* v_pool, void* stream) {
    delta_status s = check_desc(desc);
    if (s != DELTA_OK) return s;
    s = check_pt(pt);
    if (s != DELTA_OK) return s;
    if (pt->batch == 0) return DELTA_OK;
    if (k_new == nullptr || v_new == nullptr || k_pool == nullptr || v_pool == nullptr) return DELTA_ERR_INVALID_ARG;
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_pool) || !aligned16(v_pool)) return DELTA_ERR_INVALID_ARG;
    // kv_append has no workspace to flag errors in: an out-of-range page is skipped, and the
    // attention call that follows on the same page table flags it.
    const int row_vecs = desc->head_dim * elem_bytes(desc->dtype) / 16;
    return launch_pdl(kv_append_kernel, dim3(pt->batch, desc->num_kv_heads), dim3(32), 0,
                      static_cast<cudaStream_t>(stream), static_cast<const uint4*>(k_new),
                      static_cast<const uint4*>(v_new), static_cast<uint4*>(k_pool), static_cast<uint4*>(v_pool),
                      pt->page_indptr, pt->page_indices, pt->kv_len, desc->num_kv_heads, row_vecs,
                      desc->num_phys_pages);
}

delta_status delta_kv_append_layers(const delta_desc* desc, const delta_page_table* pt, int32_t num_layers,
                                    const void* const* k_new, const void* const* v_new, void* const* k_pools,
                                    void* const* v_pools, void* stream) {
    delta_status s = check_desc(desc);
    if (s != DELTA_OK) return s;
    s = check_pt(pt);
    if (s != DELTA_OK) return s;
    if (num_layers < 0 || num_layers > kMaxAppendLayers) return num_layers < 0 ? DELTA_ERR_INVALID_ARG : DELTA_ERR_UNSUPPORTED;
    if (pt->batch == 0 || num_layers == 0) return DELTA_OK;
    if (k_new == nullptr || v_new == nullptr || k_pools == nullptr || v_pools == nullptr) return DELTA_ERR_INVALID_ARG;
    AppendLayers a = {};
    for (int l = 0; l < num_layers; ++l) {
        if (k_new[l] == nullptr || v_new[l] == nullptr || k_pools[l] == nullptr || v_pools[l] == nullptr)
            return DELTA_ERR_INVALID_ARG;
        if (!aligned16(k_new[l]) || !aligned16(v_new[l]) || !aligned16(k_pools[l]) || !aligned16(v_pools[l]))
            return DELTA_ERR_INVALID_ARG;
        a.k_new[l] = static_cast<const uint4*>(k_new[l]);
        a.v_new[l] = static_cast<const uint4*>(v_new[l]);
        a.k_pool[l] = static_cast<uint4*>(k_pools[l]);
        a.v_pool[l] = static_cast<uint4*>(v_pools[l]);
    }
    const int row_vecs = desc->head_dim * elem_bytes(desc->dtype) / 16;
    return launch_pdl(kv_append_layers_kernel, dim3(pt->batch, desc->num_kv_heads, num_layers), dim3(32), 0,
                      static_cast<cudaStream_t>(stream), a, pt->page_indptr, pt->page_indices, pt->kv_len,
                      desc->num_kv_heads, row_vecs, desc->num_phys_pages);
}

delta_status delta_full_attn(const delta_desc* desc, const delta_page_table* pt, const void* q, const void* k_pool,
                             const void* v_pool, void* o, void* workspace, size_t ws_bytes, void* stream) {
    return run_attention(kModeFull, desc, pt, nullptr, nullptr, nullptr, 0, q, k_pool, v_pool, o, nullptr, nullptr, 0,
                         nullptr, workspace, ws_bytes, stream);
}

delta_status delta_full_attn_noalloc(const delta_desc* desc, const delta_page_table* pt, const void* q,
                                     const void* k_pool, const void* v_pool, void* o, void* stream) {
    delta_status s = check_desc(desc);
    if (s != DELTA_OK) return s;
    s = check_pt(pt);
    if (s != DELTA_OK) return s;
    if (pt->batch == 0) return DELTA_OK;
    const WsLayout L = ws_layout(desc, pt->batch, pt->max_pages_per_seq);
    if (L.counters + L.scratch > kStaticScratchBytes) return DELTA_ERR_UNSUPPORTED;   // shape needs more scratch than the array holds
    unsigned char* ws = noalloc_scratch();
    if (ws == nullptr) return DELTA_ERR_CUDA;
    // the error word and the split-arrival tickets must start at zero; a full layer has no score accumulators, and the
    // rest is overwritten
    if (cudaMemsetAsync(ws, 0, L.counters, static_cast<cudaStream_t>(stream)) != cudaSuccess) return DELTA_ERR_CUDA;
    return run_attention(kModeFull, desc, pt, nullptr, nullptr, nullptr, 0, q, k_pool, v_pool, o, nullptr, nullptr, 0,
                         nullptr, ws, kStaticScratchBytes, stream, false, L.counters);
}

delta_status delta_select_attn(const delta_desc* desc, const delta_page_table* pt, const delta_select_params* sp,
                               const void* q, const void* k_pool, const void* v_pool, void* o, int32_t* sel_cnt,
                               int32_t* sel_pages, int32_t sel_stride, float* page_scores, void* workspace,
                               size_t ws_bytes, void* stream) {
    return run_attention(kModeDelta, desc, pt, sp, nullptr, nullptr, 0, q, k_pool, v_pool, o, sel_cnt, sel_pages,
                         sel_stride, page_scores, workspace, ws_bytes, stream);
}

delta_status delta_sparse_attn(const delta_desc* desc, const delta_page_table* pt, const int32_t* sel_cnt,
                               const int32_t* sel_pages, int32_t sel_stride, const void* q, const void* k_pool,
                               const void* v_pool, void* o, void* workspace, size_t ws_bytes, void* stream) {
    return run_attention(kModeSparse, desc, pt, nullptr, sel_cnt, sel_pages, sel_stride, q, k_pool, v_pool, o, nullptr,
                         nullptr, 0, nullptr, workspace, ws_bytes, stream);
}

delta_status delta_sparse_attn_settled(const delta_desc* desc, const delta_page_table* pt, const int32_t* sel_cnt,
                                       const int32_t* sel_pages, int32_t sel_stride, const void* q,
                                       const void* k_pool, const void* v_pool, void* o, void* workspace,
                                       size_t ws_bytes, void* stream) {
    return run_attention(kModeSparse, desc, pt, nullptr, sel_cnt, sel_pages, sel_stride, q, k_pool, v_pool, o, nullptr,
                         nullptr, 0, nullptr, workspace, ws_bytes, stream, true);
}

delta_status delta_layer_shift(const delta_page_table* pt, const float* scores_a, const float* scores_b,
                               float* shift_out, void* stream) {
    delta_status s = check_pt(pt);
    if (s != DELTA_OK) return s;
    if (pt->batch == 0) return DELTA_OK;
    if (scores_a == nullptr || scores_b == nullptr || shift_out == nullptr) return DELTA_ERR_INVALID_ARG;
    return launch_pdl(layer_shift_kernel, dim3(pt->batch), dim3(kShiftThreads), 0, static_cast<cudaStream_t>(stream),
                      scores_a, scores_b, pt->page_indptr, pt->kv_len, pt->max_pages_per_seq, shift_out);
}

delta_status delta_choose_layers(const float* shift, int32_t num_layers, int32_t count, int32_t first,
                                 int32_t min_gap, int32_t* out_layers, int32_t* out_count) {
    if (shift == nullptr || out_layers == nullptr || out_count == nullptr) return DELTA_ERR_INVALID_ARG;
    if (num_layers <= 0 || num_layers > 4096 || first < 0 || first >= num_layers || min_gap < 0)
        return DELTA_ERR_INVALID_ARG;
    for (int32_t l = 0; l < num_layers; ++l)
        if (!(shift[l] == shift[l])) return DELTA_ERR_INVALID_ARG;   // NaN has no order
    int32_t n = 0;
    out_layers[n++] = first;
    // candidates after `first` by decreasing shift, equal shifts lower layer first; a candidate is
    // kept when at least min_gap layers away from every kept layer
    bool used[4096] = {false};
    while (n < count) {
        int32_t best = -1;
        for (int32_t l = first + 1; l < num_layers; ++l) {
            if (used[l]) continue;
            if (best < 0 || shift[l] > shift[best]) best = l;
        }
        if (best < 0) break;
        used[best] = true;
        bool far = true;
        for (int32_t i = 0; i < n; ++i) {
            const int32_t d = best > out_layers[i] ? best - out_layers[i] : out_layers[i] - best;
            if (d < min_gap) far = false;
        }
        if (far) out_layers[n++] = best;
    }
    for (int32_t i = 1; i < n; ++i)   // ascending
        for (int32_t j = i; j > 0 && out_layers[j - 1] > out_layers[j]; --j) {
            const int32_t t = out_layers[j];
            out_layers[j] = out_layers[j - 1];
            out_layers[j - 1] = t;
        }
    *out_count = n;
    return DELTA_OK;
}

delta_status delta_read_device_error(void* workspace, int32_t* flags_out, void* stream) {
    if (workspace == nullptr) return DELTA_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int32_t h = 0;
    if (cudaMemcpyAsync(&h, workspace, sizeof(int32_t), cudaMemcpyDeviceToHost, st) != cudaSuccess) return DELTA_ERR_CUDA;
    if (cudaMemsetAsync(workspace, 0, sizeof(int32_t), st) != cudaSuccess) return DELTA_ERR_CUDA;
    if (cudaStreamSynchronize(st) != cudaSuccess) return DELTA_ERR_CUDA;
    if (flags_out != nullptr) *flags_out = h;
    return h ? DELTA_ERR_BOUNDS : DELTA_OK;
}

const char* delta_status_string(delta_status s) {
    switch (s) {
        case DELTA_OK: return "ok";
        case DELTA_ERR_INVALID_ARG: return "invalid argument";
        case DELTA_ERR_UNSUPPORTED: return "unsupported shape or mode";
        case DELTA_ERR_WORKSPACE: return "workspace missing, misaligned or too small";
        case DELTA_ERR_CUDA: return "CUDA launch or runtime error";
        case DELTA_ERR_BOUNDS: return "device-side bounds check failed";
        default: return "unknown status";
    }
}

}  // extern "C"
