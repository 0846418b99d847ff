// Host side shared by every translation unit of the library: argument checks, per-device caches, split
// plans over a kernel family, launches with programmatic dependent launch, and the driver of the
// attention entry points.
#pragma once

#include "delta_attn.h"

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <mutex>

#include "common.cuh"

namespace delta {

// A workspace is two areas: the counters and accumulators that every launch leaves at zero, from its start, and scratch,
// from workspace_lead(its bytes) on.  The lead depends on the workspace's size alone, so calls of any shapes that share
// one never put scratch where another's counters are.
struct WsLayout {
    size_t err, tickets, seq_tickets, counters, score_acc, zeros;            // from the start; bytes of the counters, of all
    size_t part_ml, part_o, page_lse, split_ml, keys, logits, scratch;       // from the lead; bytes of the area
    size_t total;                                                            // the smallest workspace that holds both
};

// (A 32nd: a page has 8 bytes of accumulators, and 4 (heads + 1) of scratch, 68 a head more for HEAD_MAX.)
constexpr size_t kLeadPart = 32;
inline size_t workspace_lead(size_t ws_bytes) { return ws_bytes / kLeadPart & ~size_t(255); }

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

inline int elem_bytes(int dtype) { return dtype == DELTA_BF16 ? 2 : 4; }

inline int current_device() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return -1;
    return dev;
}

// Guards the per-device caches below (SM count, kernel attributes, cluster occupancy, the tensor-map
// encoder and the scratch array's address): first calls from several host threads may race.
inline std::recursive_mutex& cache_mutex() {
    static std::recursive_mutex mu;
    return mu;
}

inline int device_sm_count() {
    static int cache[64] = {0};
    std::lock_guard<std::recursive_mutex> lock(cache_mutex());
    const int dev = current_device();
    if (dev < 0) return 148;
    if (cache[dev] == 0) {
        int sms = 0;
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) sms = 148;
        cache[dev] = sms;
    }
    return cache[dev];
}

// S: the most splits a plan can have (room for as many cluster partials: fit_plan never exceeds a plan's).
// with_logits: room for per-token logits of every query head (delta-layers scoring with HEAD_MAX)
inline WsLayout ws_layout_splits(const delta_desc* d, int batch, int max_pages, int S, bool with_logits) {
    WsLayout w{};
    const size_t rows = size_t(batch) * d->num_q_heads;
    const size_t pages = size_t(batch) * size_t(max_pages);
    size_t off = 0;
    auto area = [&](size_t bytes) {
        const size_t at = off;
        off += align256(bytes);
        return at;
    };
    w.err = area(64);
    w.tickets = area(size_t(batch) * d->num_kv_heads * sizeof(int));
    w.seq_tickets = area(size_t(batch) * sizeof(int));
    w.counters = off;
    // (4 KB from the tickets: the atomics on both are in flight together, and close by a 1 x 8k delta-layer takes 12.8
    // instead of 12.5 us)
    off = (off + 4095) & ~size_t(4095);
    w.score_acc = area(pages * sizeof(unsigned long long));
    w.zeros = off;
    off = 0;
    w.part_ml = area(rows * S * sizeof(float2));
    w.part_o = area(rows * S * d->head_dim * sizeof(float));
    w.page_lse = area(rows * size_t(max_pages) * sizeof(float));
    w.split_ml = area(rows * S * sizeof(float2));
    w.keys = area(pages * sizeof(uint32_t));
    const size_t logits = align256(rows * size_t(max_pages) * kPage * sizeof(float));
    // Without the logits the total leaves room for what they move the lead by, so that they add their own bytes only.
    const size_t for_zeros = kLeadPart * w.zeros;
    const size_t room = off + logits / kLeadPart;
    const size_t for_scratch = align256(room + room / (kLeadPart - 1) + 1);
    w.total = (for_zeros > for_scratch ? for_zeros : for_scratch) + (with_logits ? logits : 0);
    w.logits = area(with_logits ? logits : 0);
    w.scratch = off;
    return w;
}

inline delta_status check_desc(const delta_desc* d) {
    if (d == nullptr) return DELTA_ERR_INVALID_ARG;
    if (d->num_q_heads <= 0 || d->num_kv_heads <= 0 || d->head_dim <= 0 || d->page_size <= 0 ||
        d->num_phys_pages < 0)
        return DELTA_ERR_INVALID_ARG;
    if (d->num_q_heads % d->num_kv_heads != 0) return DELTA_ERR_INVALID_ARG;
    if (d->dtype != DELTA_F32 && d->dtype != DELTA_BF16) return DELTA_ERR_INVALID_ARG;
    if (!(d->sm_scale >= 0.f) || isinf(d->sm_scale)) return DELTA_ERR_INVALID_ARG;
    if (d->page_size != kPage) return DELTA_ERR_UNSUPPORTED;
    if (d->head_dim != 64 && d->head_dim != 128) return DELTA_ERR_UNSUPPORTED;
    if (d->num_q_heads / d->num_kv_heads > kMaxGroup) return DELTA_ERR_UNSUPPORTED;
    if (d->num_kv_heads > 64) return DELTA_ERR_UNSUPPORTED;
    // rows of the pool viewed as a [pages * Hkv * 16, D] matrix must fit a 32-bit TMA coordinate
    if (d->num_phys_pages * d->num_kv_heads * kPage > int64_t(INT32_MAX)) return DELTA_ERR_UNSUPPORTED;
    return DELTA_OK;
}

inline delta_status check_pt(const delta_page_table* pt) {
    if (pt == nullptr || pt->batch < 0) return DELTA_ERR_INVALID_ARG;
    if (pt->batch == 0) return DELTA_OK;
    if (pt->page_indptr == nullptr || pt->page_indices == nullptr || pt->kv_len == nullptr) return DELTA_ERR_INVALID_ARG;
    if (pt->max_pages_per_seq <= 0) return DELTA_ERR_INVALID_ARG;
    if (pt->batch > 65535) return DELTA_ERR_UNSUPPORTED;
    return DELTA_OK;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline delta_status launch_status() { return cudaPeekAtLastError() == cudaSuccess ? DELTA_OK : DELTA_ERR_CUDA; }

// ---- tensor maps (driver entry point resolved through the runtime; no libcuda link needed)
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    std::lock_guard<std::recursive_mutex> lock(cache_mutex());
    if (fn == nullptr) {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    }
    return fn;
}

// Split plan: about one full wave of CTAs over the GPU, at least one page per warp.  Up to 16
// splits form one thread-block cluster; more are grouped into clusters whose partials meet in the
// workspace.
struct SplitPlan {
    int cluster, clusters;
    int variant;   // kVarNarrow: 4-warp CTAs, 3 stages, two per SM; kVarWide: one 8-warp CTA per SM;
                   // kVarShort: 6-warp CTAs, 2 stages, two per SM (tensor-core kernel)
    int splits() const { return cluster * clusters; }
};

enum : int { kVarNarrow = 0, kVarWide = 1, kVarShort = 2 };   // tensor-core kernel variants

#ifndef DELTA_PAGES_PER_CLUSTER
#define DELTA_PAGES_PER_CLUSTER 256  // pages each cluster must get before a unit uses several
#endif
#ifndef DELTA_ONE_CLUSTER_PAGES
#define DELTA_ONE_CLUSTER_PAGES 512  // up to this many pages per unit, one cluster
#endif


// One-time per-device attributes of a decode kernel (shared-memory limit, cluster sizes > 8).
inline bool configure_kernel(const void* func, size_t smem) {
    constexpr int kSlots = 256;
    static const void* done_fn[64][kSlots];
    std::lock_guard<std::recursive_mutex> lock(cache_mutex());
    const int dev = current_device();
    if (dev < 0) return false;
    int i = 0;
    for (; i < kSlots && done_fn[dev][i] != nullptr; ++i)
        if (done_fn[dev][i] == func) return true;
    if (cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) != cudaSuccess ||
        cudaFuncSetAttribute(func, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return false;
    if (i < kSlots) done_fn[dev][i] = func;
    return true;
}

// Clusters of `cluster` CTAs of this kernel that can be resident at once (cached per device).
inline int max_active_clusters(const void* func, size_t smem, int cluster, int threads) {
    constexpr int kSlots = 512;
    struct Entry { const void* fn; int cluster; int n; };
    static Entry cache[64][kSlots];
    std::lock_guard<std::recursive_mutex> lock(cache_mutex());
    const int dev = current_device();
    if (dev < 0) return 1;
    int i = 0;
    for (; i < kSlots && cache[dev][i].fn != nullptr; ++i)
        if (cache[dev][i].fn == func && cache[dev][i].cluster == cluster) return cache[dev][i].n;
    if (!configure_kernel(func, smem)) return 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cluster, 1, 1);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, func, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = 1;
    }
    if (i < kSlots) cache[dev][i] = {func, cluster, n};
    return n;
}

// Fit a split plan to the clusters that can be resident at once.  Among cluster sizes C <= the
// plan's, pick the (C, clusters) pair with the most CTAs (C * clusters <= the plan's splits) whose
// units * clusters all fit in one wave; ties go to the larger cluster (fewer cross-cluster
// partials).  Long sequences thus keep ~one wave of CTAs even where large clusters do not pack
// into the GPCs.
// one_cluster_per_unit: delta-layers that select their pages at the end of the decode keep every
// (sequence, KV head) unit in one cluster, so each CTA gets the unit's per-head normalisers from the
// cluster merge (a unit spread over several clusters needs a second arrival stage).
// spare: clusters that must stay free.  A plan that takes every place can end in two waves behind a kernel that is
// still draining: 56 units of 16k tokens in clusters of 5 on 8-bit layers, 56 instead of 44 us (full) and 75 instead of
// 53 (delta-layer) against the next smaller clusters.
// kernel_of(variant, &smem, &threads): the kernel of that variant, its dynamic shared memory and threads.
template <typename KernelOf>
SplitPlan fit_plan_now(SplitPlan pl, const KernelOf& kernel_of, int units, int items, bool one_cluster_per_unit,
                       int spare) {
    const int s = pl.splits();
    // Clusters meet through the workspace only when each gets at least 256 pages (and the unit has
    // more than 512): below that the cross-cluster merge costs more than the extra CTAs gain.
    // Up to 512 pages per (sequence, KV head) one cluster is faster (measured on the 8k stack).
    constexpr int per_cluster = DELTA_PAGES_PER_CLUSTER, one_cluster = DELTA_ONE_CLUSTER_PAGES;
    const int max_clusters =
        (one_cluster_per_unit || items <= one_cluster || items / per_cluster < 1) ? 1 : items / per_cluster;
    SplitPlan best = pl;
    int best_ctas = -1;
    for (int c = pl.cluster; c >= 1; --c) {
        SplitPlan cand = pl;
        cand.cluster = c;
        cand.clusters = s / c < max_clusters ? s / c : max_clusters;
        if (cand.clusters < 1) continue;
        size_t smem = 0;
        int threads = 0;
        const void* fn = kernel_of(cand.variant, &smem, &threads);
        if (fn == nullptr) return pl;
        const int maxc = max_active_clusters(fn, smem, c, threads) - spare;
        if (int64_t(units) * cand.clusters > maxc) {
            cand.clusters = maxc / units;
            if (cand.clusters < 1) continue;
        }
        const int ctas = c * cand.clusters;
        if (ctas > best_ctas) {
            best = cand;
            best_ctas = ctas;
        }
    }
    if (best_ctas < 0) {   // more units than resident clusters even at size 1: several waves
        best.cluster = 1;
        best.clusters = 1;
        best.variant = kVarNarrow;
    }
    return best;
}

// fit_plan_now, remembered: a plan depends on the kernel and the sizes alone, and finding it asks for the cluster
// occupancy up to 16 times.
struct KnownPlan {
    const void* fn;
    int dev, cluster, clusters, units, items, one, spare;
    SplitPlan plan;
};
template <typename KernelOf>
SplitPlan fit_plan(SplitPlan pl, const KernelOf& kernel_of, int units, int items, bool one_cluster_per_unit = false,
                   int spare = 0) {
    constexpr int kSlots = 256;
    static KnownPlan known[kSlots];
    static int count = 0;
    size_t smem = 0;
    int threads = 0;
    const int dev = current_device();
    const KnownPlan key = {kernel_of(pl.variant, &smem, &threads), dev, pl.cluster, pl.clusters, units, items,
                           one_cluster_per_unit ? 1 : 0, spare, pl};
    std::lock_guard<std::recursive_mutex> lock(cache_mutex());
    for (int i = count - 1; i >= 0; --i) {
        const KnownPlan& k = known[i];
        if (k.fn == key.fn && k.dev == key.dev && k.units == key.units && k.items == key.items && k.one == key.one &&
            k.cluster == key.cluster && k.clusters == key.clusters && k.spare == key.spare)
            return k.plan;
    }
    const SplitPlan plan = fit_plan_now(pl, kernel_of, units, items, one_cluster_per_unit, spare);
    if (dev >= 0 && count < kSlots) {
        known[count] = key;
        known[count++].plan = plan;
    }
    return plan;
}

// Launch with programmatic dependent launch: the kernel may be scheduled while the previous
// kernel of the stream drains; it waits for it in pdl_wait() before touching global memory.
template <typename K, typename... Args>
inline delta_status launch_pdl(K kern, dim3 grid, dim3 block, size_t smem, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) return DELTA_ERR_CUDA;
    return launch_status();
}

// Launch a decode kernel as clusters of `cluster` CTAs along the split dimension.
template <typename K, typename... Args>
inline delta_status launch_clustered(K kern, size_t smem, int threads, const DecodeParams& prm, int cluster, int batch,
                              int Hkv, cudaStream_t st, Args... args) {
    if (!configure_kernel(reinterpret_cast<const void*>(kern), smem)) return DELTA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(prm.num_splits, Hkv, batch);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kern, prm, args...) != cudaSuccess) return DELTA_ERR_CUDA;
    return launch_status();
}

inline delta_status check_q8_cache(const delta_q8_cache* c) {
    if (c == nullptr || c->k_pool == nullptr || c->v_pool == nullptr || c->k_scale == nullptr || c->v_scale == nullptr)
        return DELTA_ERR_INVALID_ARG;
    if (c->format != DELTA_E4M3 && c->format != DELTA_INT8) return DELTA_ERR_INVALID_ARG;
    if (!aligned16(c->k_pool) || !aligned16(c->v_pool)) return DELTA_ERR_INVALID_ARG;
    if (((reinterpret_cast<uintptr_t>(c->k_scale) | reinterpret_cast<uintptr_t>(c->v_scale)) & 3u) != 0)
        return DELTA_ERR_INVALID_ARG;
    return DELTA_OK;
}

// Arguments of one attention call (the selection outputs and sp only for delta-layers, the selection
// inputs only for sparse layers, window and sink only for window layers).
struct AttnCall {
    int mode = kModeFull;
    const delta_desc* d = nullptr;
    const delta_page_table* pt = nullptr;
    const delta_select_params* sp = nullptr;
    const int32_t* sel_cnt_in = nullptr;
    const int32_t* sel_pages_in = nullptr;
    int32_t sel_stride_in = 0;
    bool settled = false;
    int32_t window = 0, sink = 0;
    const void* q = nullptr;
    void* o = nullptr;
    int32_t* sel_cnt_out = nullptr;
    int32_t* sel_pages_out = nullptr;
    int32_t sel_stride_out = 0;
    float* page_scores = nullptr;
    void* ws = nullptr;
    size_t ws_bytes = 0;
    size_t lead = 0;             // of a workspace that one shape alone uses (0: workspace_lead)
    void* stream = nullptr;
};

// The HEAD_MAX selection kernel of a delta-layer (select.cuh), launched behind its decode kernel.
delta_status launch_score_select(const AttnCall& a, const DecodeParams& prm);

// Driver of the attention entry points over one cache storage.  Backend:
//   delta_status check(d)                          its own arguments (pool pointers, alignment)
//   WsLayout layout(d, batch, max_pages, logits)   workspace
//   SplitPlan plan(d, batch, items, fused)         a plan that fits the GPU (fused: in-kernel selection)
//   void fill(prm)                                 pool pointers and the like
//   delta_status launch(d, prm, plan, batch, stream)
template <typename Backend>
delta_status run_attention_on(const Backend& be, const AttnCall& a) {
    const delta_desc* d = a.d;
    const delta_page_table* pt = a.pt;
    const delta_select_params* sp = a.sp;
    delta_status s = check_desc(d);
    if (s != DELTA_OK) return s;
    s = check_pt(pt);
    if (s != DELTA_OK) return s;
    if (a.mode == kModeDelta) {
        if (sp == nullptr) return DELTA_ERR_INVALID_ARG;
        if (sp->budget_pages < 0 || sp->sink_tokens < 0 || sp->recency_tokens < 0) return DELTA_ERR_INVALID_ARG;
        if (sp->reduce != DELTA_HEAD_SUM && sp->reduce != DELTA_HEAD_MAX) return DELTA_ERR_INVALID_ARG;
        if (d->num_q_heads > kMaxQHeadsSelect) return DELTA_ERR_UNSUPPORTED;
    }
    if (a.mode == kModeWindow && (a.window < 0 || a.sink < 0)) return DELTA_ERR_INVALID_ARG;
    if (pt->batch == 0) return DELTA_OK;
    if (a.q == nullptr || a.o == nullptr) return DELTA_ERR_INVALID_ARG;
    s = be.check(d);
    if (s != DELTA_OK) return s;
    if (!aligned16(a.q) || !aligned16(a.o)) return DELTA_ERR_INVALID_ARG;
    if (a.mode == kModeDelta) {
        if (a.sel_cnt_out == nullptr || a.sel_pages_out == nullptr) return DELTA_ERR_INVALID_ARG;
        if (a.sel_stride_out < delta_sel_capacity(sp, d->page_size)) return DELTA_ERR_INVALID_ARG;
        if (pt->max_pages_per_seq > kMaxSelectPages) return DELTA_ERR_UNSUPPORTED;
    }
    if (a.mode == kModeSparse) {
        if (a.sel_cnt_in == nullptr || a.sel_pages_in == nullptr || a.sel_stride_in <= 0) return DELTA_ERR_INVALID_ARG;
    }
    if (a.ws == nullptr || (reinterpret_cast<uintptr_t>(a.ws) & 255u) != 0) return DELTA_ERR_WORKSPACE;
    const bool head_max = a.mode == kModeDelta && sp->reduce == DELTA_HEAD_MAX;
    const WsLayout L = be.layout(d, pt->batch, pt->max_pages_per_seq, head_max);
    if (a.lead == 0 && a.ws_bytes < L.total) return DELTA_ERR_WORKSPACE;

    const int D = d->head_dim, Hq = d->num_q_heads, Hkv = d->num_kv_heads;
    int items = pt->max_pages_per_seq;
    if (a.mode == kModeSparse && a.sel_stride_in < items) items = a.sel_stride_in;
    if (a.mode == kModeWindow) {   // the sinks' pages, and the window's plus one when it starts inside a page
        const int64_t most = (int64_t(a.sink) + kPage - 1) / kPage + (a.window > 0 ? (int64_t(a.window) + kPage - 1) / kPage + 1 : 0);
        if (most < items) items = int(most < 1 ? 1 : most);
    }
    const bool fused = a.mode == kModeDelta && !head_max;
    const SplitPlan plan = be.plan(d, pt->batch, items, fused);
    // the in-kernel selection forms each unit's normalisers from its one cluster's merge
    if (fused && plan.clusters != 1) return DELTA_ERR_UNSUPPORTED;
    const int S = plan.splits();
    unsigned char* base = static_cast<unsigned char*>(a.ws);
    unsigned char* scratch = base + (a.lead != 0 ? a.lead : workspace_lead(a.ws_bytes));

    DecodeParams prm{};
    prm.q = a.q;
    be.fill(prm);
    prm.indptr = pt->page_indptr;
    prm.indices = pt->page_indices;
    prm.kv_len = pt->kv_len;
    prm.sel_cnt = a.sel_cnt_in;
    prm.sel_pages = a.sel_pages_in;
    prm.sel_stride = a.sel_stride_in;
    prm.num_q_heads = Hq;
    prm.num_kv_heads = Hkv;
    prm.items_per_split = (items + S - 1) / S;
    prm.num_splits = S;
    prm.max_pages = pt->max_pages_per_seq;
    prm.num_phys_pages = d->num_phys_pages;
    const float scale = d->sm_scale > 0.f ? d->sm_scale : 1.0f / sqrtf(float(D));
    prm.qscale = scale * 1.4426950408889634f;
    prm.mode = a.mode;
    prm.part_ml = reinterpret_cast<float2*>(scratch + L.part_ml);
    prm.part_o = reinterpret_cast<float*>(scratch + L.part_o);
    prm.page_lse = reinterpret_cast<float*>(scratch + L.page_lse);
    prm.split_ml = a.mode == kModeDelta ? reinterpret_cast<float2*>(scratch + L.split_ml) : nullptr;
    prm.err = reinterpret_cast<int*>(base + L.err);
    prm.o = a.o;
    prm.num_clusters = plan.clusters;
    prm.logits = head_max ? reinterpret_cast<float*>(scratch + L.logits) : nullptr;
    prm.tickets = reinterpret_cast<int*>(base + L.tickets);
    prm.settled = (a.mode == kModeSparse && a.settled) ? 1 : 0;
    prm.window = a.window;
    prm.sink = a.sink;
    // delta-layers scoring with HEAD_SUM select their pages at the end of the decode kernel
    prm.fuse_select = fused ? 1 : 0;
    if (prm.fuse_select) {
        prm.budget_pages = sp->budget_pages;
        prm.sink_tokens = sp->sink_tokens;
        prm.recency_tokens = sp->recency_tokens;
        prm.sel_cnt_out = a.sel_cnt_out;
        prm.sel_pages_out = a.sel_pages_out;
        prm.sel_stride_out = a.sel_stride_out;
        prm.page_scores = a.page_scores;
        prm.score_acc = reinterpret_cast<unsigned long long*>(base + L.score_acc);
        prm.keys = reinterpret_cast<uint32_t*>(scratch + L.keys);
        prm.seq_tickets = reinterpret_cast<int*>(base + L.seq_tickets);
    }
    s = be.launch(d, prm, plan, pt->batch, static_cast<cudaStream_t>(a.stream));
    if (s != DELTA_OK || !head_max) return s;
    return launch_score_select(a, prm);
}

}  // namespace delta
