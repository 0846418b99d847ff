// Split plans, kernel variants and launches of the decode kernels over the bf16 / fp32 pools (included by
// one translation unit per kernel family: WIN false, full, delta and sparse layers; WIN true, window
// layers).
#pragma once

#include "decode_mma.cuh"
#include "decode_simt.cuh"
#include "host.cuh"

namespace delta {

constexpr int kMmaStages = 3;      // tensor-core kernel: stages per warp (8 KB each for D = 128), 2 CTAs/SM
constexpr int kMmaWideWarps = 8;   // when a cluster per unit fits one CTA per SM: 8-warp CTAs
constexpr int kMmaShortWarps = 6;  // short page lists: 6 warps with 2 stages each (same shared memory)
constexpr int kMmaShortStages = 2;
constexpr int variant_threads(int v) { return 32 * (v == kVarWide ? kMmaWideWarps : v == kVarShort ? kMmaShortWarps : kWarps); }

// Stages of the CUDA-core kernel (fp32): about 24 KB of pages in flight per warp.
constexpr int simt_stages(int ebytes, int D) {
    return (24 * 1024) / (2 * kPage * D * ebytes) < 2   ? 2
           : (24 * 1024) / (2 * kPage * D * ebytes) > 4 ? 4
                                                        : (24 * 1024) / (2 * kPage * D * ebytes);
}

// Dynamic shared memory of the decode kernel that serves (dtype, D).
inline size_t decode_smem_bytes(int dtype, int D) {
    if (dtype == DELTA_BF16)
        return D == 128 ? MmaSmem<128, kMmaStages>::kBytes : MmaSmem<64, kMmaStages>::kBytes;
    return D == 128 ? DecodeSmem<float, 128, simt_stages(4, 128)>::kBytes : DecodeSmem<float, 64, simt_stages(4, 64)>::kBytes;
}

inline int ctas_per_sm(int dtype, int D) {
    const size_t per_sm = 233472;  // shared memory per SM on B200
    int c = int(per_sm / (decode_smem_bytes(dtype, D) + 1024));
    return c < 1 ? 1 : (c > 8 ? 8 : c);
}

// Split-plan constants (compile-time; a sweep rebuilds the library with -D overrides).
#ifndef DELTA_CTAS_PER_SM
#define DELTA_CTAS_PER_SM 0          // 0: as many CTAs per SM as shared memory allows
#endif
#ifndef DELTA_MAX_SPLITS
#define DELTA_MAX_SPLITS 0           // 0: no cap beyond kMaxSplits
#endif
#ifndef DELTA_MAX_WIDE_SPLITS
#define DELTA_MAX_WIDE_SPLITS 0      // 0: no extra cap on 8-warp plans
#endif
#ifndef DELTA_MAX_NARROW_SPLITS
#define DELTA_MAX_NARROW_SPLITS 0    // 0: no extra cap on 4- and 6-warp plans
#endif
#ifndef DELTA_WIDE
#define DELTA_WIDE 1                 // 0: never use 8-warp CTAs
#endif

inline int split_target_per_sm(int dtype, int D) {
    return DELTA_CTAS_PER_SM > 0 ? DELTA_CTAS_PER_SM : ctas_per_sm(dtype, D);
}

// About one wave of CTAs, at least one page per warp.  The splits of one (sequence, KV head) form
// clusters of at most 16 CTAs that merge through distributed shared memory; only long page lists
// (fit_plan) make several clusters meet in the workspace.
// The plan of one variant.
inline SplitPlan plan_variant(int dtype, int D, int batch, int Hkv, int items, int variant) {
    if (items <= 0) return {1, 1, kVarNarrow};
    const bool wide = variant == kVarWide;
    const int sms = device_sm_count();
    const int units = batch * Hkv;
    const int warps = variant_threads(variant) / 32;
    const int slots = wide ? sms : sms * split_target_per_sm(dtype, D);
    int s = slots / (units > 0 ? units : 1);
    // at least one page per warp; 4- and 6-warp tensor-core CTAs take at least 2 * warps - 1
    // (two pages for all warps but one): of the plans that give no warp more than one two-page
    // loop iteration, that one measured fastest on the 8k sparse layers (81 pages)
    const int per_cta = (!wide && dtype == DELTA_BF16) ? 2 * warps - 1 : warps;
    const int cap = (items + per_cta - 1) / per_cta;
    if (s > cap) s = cap;
    if (s > kMaxSplits) s = kMaxSplits;
    if (DELTA_MAX_SPLITS > 0 && s > DELTA_MAX_SPLITS) s = DELTA_MAX_SPLITS;
    if (wide && DELTA_MAX_WIDE_SPLITS > 0 && s > DELTA_MAX_WIDE_SPLITS) s = DELTA_MAX_WIDE_SPLITS;
    if (!wide && DELTA_MAX_NARROW_SPLITS > 0 && s > DELTA_MAX_NARROW_SPLITS) s = DELTA_MAX_NARROW_SPLITS;
    if (s < 1) s = 1;
    SplitPlan pl;
    pl.cluster = s < 16 ? s : 16;
    pl.clusters = s / pl.cluster;
    pl.variant = variant;
    return pl;
}

// delta_fused: a delta-layer that scores and selects its pages inside the decode (HEAD_SUM).
inline SplitPlan plan_splits(int dtype, int D, int batch, int Hkv, int items, bool delta_fused = false) {
    // One 8-warp CTA per SM, each warp streaming half the pages of a 4-warp CTA's warp (the per-warp
    // chain of dependent MMAs, exponentials and shuffles, not the memory system, bounds such layers):
    //  - few (sequence, KV head) units, so that a full cluster per unit fits one CTA per SM, and at
    //    least two pages per warp of such a cluster (short lists of such batches, sparse layers, keep
    //    smaller CTAs, two per SM, so the next layer's CTAs find room beside them and start early);
    //  - mid-size batches, where a 16-CTA cluster per unit would not fit but every unit still gets
    //    at least four SMs, for every layer kind (measured: the 8-sequence 16k-32k stack's step
    //    640 -> 551 us and the 4-sequence 64k stack's 1296 -> 1239 us, every layer kind faster,
    //    against 4- and 6-warp CTAs two per SM).
    const int64_t units = int64_t(batch) * Hkv;
    const int sms = device_sm_count();
    const bool few_units = units * 16 <= sms && items >= 16 * kMmaWideWarps * 2;
    const bool mid_units = units * 16 > sms && units * 4 <= sms;
    const bool wide = DELTA_WIDE && dtype == DELTA_BF16 && (few_units || mid_units);
    if (wide) return plan_variant(dtype, D, batch, Hkv, items, kVarWide);
    // 6 warps with 2 stages each (the same shared memory and pages in flight as 4 warps x 3 stages,
    // spread over more warps) for three kinds of list:
    //  - lists that 4-warp CTAs would cover with at most two pages per warp (a sparse layer of a
    //    small batch), so more warps share the few pages;
    //  - short lists (sparse layers, at most kShortListPages) that still give a 4-warp CTA at least
    //    kShortLongCta pages (a sparse layer of a large batch): each warp streams fewer pages, so the
    //    slowest warp, which ends the layer, finishes sooner (measured: 29.0 instead of 30.1 us per
    //    sparse layer of the 16-sequence 16k stack with 81 pages per CTA; slower at 32 pages per CTA
    //    on the 4-sequence 64k stack, 17.2 instead of 16.0 us);
    //  - delta-layers of large batches (at most two splits per unit, at least 64 pages per CTA): the
    //    page terms add work to every page, which more warps share (measured: 167 instead of 171 us
    //    per delta-layer of the 16-sequence 16k stack; at nine splits per unit, the 64k stack's, the
    //    6-warp plan ran slower, 204 instead of 178 us).
    //  Other long lists (full layers) keep 3 stages per warp.
    constexpr int kShortListPages = 512, kShortLongCta = 48;
    const SplitPlan narrow = plan_variant(dtype, D, batch, Hkv, items, kVarNarrow);
    const int per_cta = (items + narrow.splits() - 1) / narrow.splits();
    const bool short_list = per_cta <= 2 * kWarps || (items <= kShortListPages && per_cta >= kShortLongCta);
    const bool delta_large_batch = delta_fused && narrow.splits() <= 2 && per_cta >= 64;
    if (dtype == DELTA_BF16 && (short_list || delta_large_batch))
        return plan_variant(dtype, D, batch, Hkv, items, kVarShort);
    return narrow;
}

// Most splits any launch on page lists of at most max_pages can get (workspace bound): both
// variants' split counts grow with the page count.
inline int max_splits_for(int dtype, int D, int batch, int Hkv, int max_pages) {
    // (a short-list plan never has more splits than the 4-warp plan of the same list)
    const int a = plan_variant(dtype, D, batch, Hkv, max_pages, kVarNarrow).splits();
    const int b = plan_variant(dtype, D, batch, Hkv, max_pages, kVarWide).splits();
    return a > b ? a : b;
}

inline WsLayout ws_layout(const delta_desc* d, int batch, int max_pages, bool with_logits = false) {
    const int S = max_splits_for(d->dtype, d->head_dim, batch, d->num_kv_heads, max_pages);
    return ws_layout_splits(d, batch, max_pages, S, with_logits);
}

// A bf16 pool [pages][Hkv][16][D] seen as a [pages*Hkv*16, D] matrix, 16-row x 64-column boxes,
// 128-byte swizzle (what the ldmatrix addressing of the tensor-core kernel assumes).
inline bool make_pool_map(CUtensorMap* map, const void* pool, const delta_desc* d) {
    EncodeTiledFn enc = encode_fn();
    if (enc == nullptr) return false;
    const cuuint64_t dims[2] = {cuuint64_t(d->head_dim), cuuint64_t(d->num_phys_pages) * d->num_kv_heads * kPage};
    const cuuint64_t strides[1] = {cuuint64_t(d->head_dim) * 2};
    const cuuint32_t box[2] = {64, kPage};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(pool), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ---- kernel selection and cluster occupancy
template <int D, int G, bool WIN>
const void* mma_ptr(int variant, size_t* smem) {
    if (variant == kVarWide) {
        *smem = MmaSmem<D, kMmaStages, kMmaWideWarps>::kBytes;
        return reinterpret_cast<const void*>(decode_mma_kernel<D, G, kMmaStages, kMmaWideWarps, WIN>);
    }
    if (variant == kVarShort) {
        *smem = MmaSmem<D, kMmaShortStages, kMmaShortWarps>::kBytes;
        return reinterpret_cast<const void*>(decode_mma_kernel<D, G, kMmaShortStages, kMmaShortWarps, WIN>);
    }
    *smem = MmaSmem<D, kMmaStages>::kBytes;
    return reinterpret_cast<const void*>(decode_mma_kernel<D, G, kMmaStages, kWarps, WIN>);
}
template <int D, int G, bool WIN>
const void* simt_ptr(size_t* smem) {
    constexpr int STAGES = simt_stages(4, D);
    *smem = DecodeSmem<float, D, STAGES>::kBytes;
    return reinterpret_cast<const void*>(decode_kernel<float, D, G, STAGES, WIN>);
}
#define DELTA_G_PTR(G, CALL)  \
    switch (G) {               \
        case 1: return CALL(1); \
        case 2: return CALL(2); \
        case 3: return CALL(3); \
        case 4: return CALL(4); \
        case 5: return CALL(5); \
        case 6: return CALL(6); \
        case 7: return CALL(7); \
        case 8: return CALL(8); \
        default: return nullptr; \
    }
template <bool WIN>
const void* decode_ptr(int dtype, int D, int G, int variant, size_t* smem) {
    if (dtype == DELTA_BF16) {
        if (D == 128) {
#define CALL(g) mma_ptr<128, g, WIN>(variant, smem)
            DELTA_G_PTR(G, CALL)
#undef CALL
        }
#define CALL(g) mma_ptr<64, g, WIN>(variant, smem)
        DELTA_G_PTR(G, CALL)
#undef CALL
    }
    if (D == 128) {
#define CALL(g) simt_ptr<128, g, WIN>(smem)
        DELTA_G_PTR(G, CALL)
#undef CALL
    }
#define CALL(g) simt_ptr<64, g, WIN>(smem)
    DELTA_G_PTR(G, CALL)
#undef CALL
}

template <typename T, int D, int G, bool WIN>
delta_status launch_simt_g(const DecodeParams& prm, int cluster, int batch, int Hkv, cudaStream_t st) {
    constexpr int STAGES = simt_stages(int(sizeof(T)), D);
    return launch_clustered(decode_kernel<T, D, G, STAGES, WIN>, DecodeSmem<T, D, STAGES>::kBytes, kThreads, prm, cluster,
                            batch, Hkv, st);
}

template <int D, int G, bool WIN>
delta_status launch_mma_g(const DecodeParams& prm, const CUtensorMap& mk, const CUtensorMap& mv, int cluster,
                          int variant, int batch, int Hkv, cudaStream_t st) {
    if (variant == kVarWide)
        return launch_clustered(decode_mma_kernel<D, G, kMmaStages, kMmaWideWarps, WIN>,
                                MmaSmem<D, kMmaStages, kMmaWideWarps>::kBytes, kMmaWideWarps * 32, prm, cluster, batch,
                                Hkv, st, mk, mv);
    if (variant == kVarShort)
        return launch_clustered(decode_mma_kernel<D, G, kMmaShortStages, kMmaShortWarps, WIN>,
                                MmaSmem<D, kMmaShortStages, kMmaShortWarps>::kBytes, kMmaShortWarps * 32, prm, cluster,
                                batch, Hkv, st, mk, mv);
    return launch_clustered(decode_mma_kernel<D, G, kMmaStages, kWarps, WIN>, MmaSmem<D, kMmaStages>::kBytes, kThreads, prm,
                            cluster, batch, Hkv, st, mk, mv);
}

#define DELTA_G_SWITCH(G, CALL) \
    switch (G) {                  \
        case 1: return CALL(1);   \
        case 2: return CALL(2);   \
        case 3: return CALL(3);   \
        case 4: return CALL(4);   \
        case 5: return CALL(5);   \
        case 6: return CALL(6);   \
        case 7: return CALL(7);   \
        case 8: return CALL(8);   \
        default: return DELTA_ERR_UNSUPPORTED; \
    }

template <bool WIN>
delta_status launch_decode(const delta_desc* d, const DecodeParams& prm, int cluster, int variant, int batch,
                           cudaStream_t st) {
    const int Hkv = d->num_kv_heads, G = d->num_q_heads / Hkv;
    if (d->dtype == DELTA_BF16) {
        CUtensorMap mk, mv;
        if (!make_pool_map(&mk, prm.k_pool, d) || !make_pool_map(&mv, prm.v_pool, d)) return DELTA_ERR_CUDA;
        if (d->head_dim == 128) {
#define CALL(g) launch_mma_g<128, g, WIN>(prm, mk, mv, cluster, variant, batch, Hkv, st)
            DELTA_G_SWITCH(G, CALL)
#undef CALL
        } else {
#define CALL(g) launch_mma_g<64, g, WIN>(prm, mk, mv, cluster, variant, batch, Hkv, st)
            DELTA_G_SWITCH(G, CALL)
#undef CALL
        }
    }
    if (d->head_dim == 128) {
#define CALL(g) launch_simt_g<float, 128, g, WIN>(prm, cluster, batch, Hkv, st)
        DELTA_G_SWITCH(G, CALL)
#undef CALL
    }
#define CALL(g) launch_simt_g<float, 64, g, WIN>(prm, cluster, batch, Hkv, st)
    DELTA_G_SWITCH(G, CALL)
#undef CALL
}

// The bf16 / fp32 pools (WIN: the window kernels over them).
template <bool WIN>
struct PlainCache {
    const void* k_pool;
    const void* v_pool;
    delta_status check(const delta_desc*) const {
        if (k_pool == nullptr || v_pool == nullptr || !aligned16(k_pool) || !aligned16(v_pool)) return DELTA_ERR_INVALID_ARG;
        return DELTA_OK;
    }
    WsLayout layout(const delta_desc* d, int batch, int max_pages, bool logits) const {
        return ws_layout(d, batch, max_pages, logits);
    }
    SplitPlan plan(const delta_desc* d, int batch, int items, bool fused) const {
        const int dtype = d->dtype, D = d->head_dim, Hkv = d->num_kv_heads, G = d->num_q_heads / Hkv;
        auto kernel_of = [&](int variant, size_t* smem, int* threads) {
            *threads = dtype == DELTA_BF16 ? variant_threads(variant) : kThreads;
            return decode_ptr<WIN>(dtype, D, G, variant, smem);
        };
        return fit_plan(plan_splits(dtype, D, batch, Hkv, items, fused), kernel_of, batch * Hkv, items, fused,
                        WIN ? 1 : 0);
    }
    void fill(DecodeParams& prm) const {
        prm.k_pool = k_pool;
        prm.v_pool = v_pool;
    }
    delta_status launch(const delta_desc* d, const DecodeParams& prm, const SplitPlan& plan, int batch,
                        cudaStream_t st) const {
        return launch_decode<WIN>(d, prm, plan.cluster, plan.variant, batch, st);
    }
};

}  // namespace delta
