// Entry points of attention over the 8-bit cache: split plans, tensor maps and the shared driver.
#include "attn_q8.cuh"
#include "q8.cuh"

namespace delta {

// A pool of blocks seen as a [pages * Hkv * 16, D] byte matrix, one block a box, swizzled over its rows' width
// (what the ldmatrix addressing of the kernel assumes).
bool make_block_map(CUtensorMap* map, const void* pool, const delta_desc* d) {
    EncodeTiledFn enc = encode_fn();
    if (enc == nullptr) return false;
    const cuuint64_t dims[2] = {cuuint64_t(d->head_dim), cuuint64_t(d->num_phys_pages) * d->num_kv_heads * kPage};
    const cuuint64_t strides[1] = {cuuint64_t(d->head_dim)};
    const cuuint32_t box[2] = {cuuint32_t(d->head_dim), kPage};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(pool), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE,
               d->head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// About one wave of CTAs, at least a page per warp.
SplitPlan plan_q8_variant(int D, int batch, int Hkv, int items, int variant) {
    if (items <= 0) return {1, 1, kVarNarrow};
    const bool wide = variant == kVarWide;
    const int warps = q8_warps(D, wide);
    const int slots = device_sm_count() * (wide ? 1 : 2);
    int s = int(slots / (int64_t(batch) * Hkv));     // (the size function takes any batch)
    const int per_cta = wide ? warps : 2 * warps - 1;
    s = min(s, (items + per_cta - 1) / per_cta);
    s = max(1, min(s, kMaxSplits));
    SplitPlan pl;
    pl.cluster = s < 16 ? s : 16;
    pl.clusters = s / pl.cluster;
    pl.variant = variant;
    return pl;
}

// One wide CTA an SM where plan_splits has one for the bf16 cache, by the same rules: a full cluster for each of a
// few units with long lists (one sequence: 8k full layer 7.2 instead of 7.6 us, 32k 14.5 instead of 18), and
// mid-size batches (4 x 64k 86 instead of 87 us, its delta-layer 99 instead of 119); else two narrow ones.
SplitPlan plan_q8(int dtype, int D, int batch, int Hkv, int items) {
    const int64_t units = int64_t(batch) * Hkv;
    const int sms = device_sm_count();
    const bool few_units = units * 16 <= sms && items >= 16 * q8_warps(D, true) * 2;
    const bool mid_units = units * 16 > sms && units * 4 <= sms;
    return plan_q8_variant(D, batch, Hkv, items, dtype == DELTA_BF16 && (few_units || mid_units) ? kVarWide : kVarNarrow);
}

WsLayout q8_layout(const delta_desc* d, int batch, int max_pages, bool logits) {
    const int a = plan_q8_variant(d->head_dim, batch, d->num_kv_heads, max_pages, kVarNarrow).splits();
    const int b = plan_q8_variant(d->head_dim, batch, d->num_kv_heads, max_pages, kVarWide).splits();
    return ws_layout_splits(d, batch, max_pages, a > b ? a : b, logits);
}

struct Q8Cache {
    const delta_q8_cache* c;
    delta_status check(const delta_desc*) const { return check_q8_cache(c); }
    WsLayout layout(const delta_desc* d, int batch, int max_pages, bool logits) const {
        return q8_layout(d, batch, max_pages, logits);
    }
    SplitPlan plan(const delta_desc* d, int batch, int items, bool fused) const {
        const int dtype = d->dtype, D = d->head_dim, Hkv = d->num_kv_heads, G = d->num_q_heads / Hkv;
        const int format = c->format;
        auto kernel_of = [&](int variant, size_t* smem, int* threads) {
            const Q8Kernel k = format == DELTA_E4M3 ? q8_kernel<kE4M3>(dtype, D, G, variant)
                                                    : q8_kernel<kInt8>(dtype, D, G, variant);
            *smem = k.smem;
            *threads = k.threads;
            return k.fn;
        };
        return fit_plan(plan_q8(dtype, D, batch, Hkv, items), kernel_of, batch * Hkv, items, fused, 1);
    }
    void fill(DecodeParams& prm) const {
        prm.k_pool = c->k_pool;
        prm.v_pool = c->v_pool;
        prm.k_scale = c->k_scale;
        prm.v_scale = c->v_scale;
    }
    delta_status launch(const delta_desc* d, const DecodeParams& prm, const SplitPlan& plan, int batch,
                        cudaStream_t st) const {
        CUtensorMap mk, mv;
        if (!make_block_map(&mk, c->k_pool, d) || !make_block_map(&mv, c->v_pool, d)) return DELTA_ERR_CUDA;
        return c->format == DELTA_E4M3 ? q8_launch<kE4M3>(d, prm, mk, mv, plan, batch, st)
                                       : q8_launch<kInt8>(d, prm, mk, mv, plan, batch, st);
    }
};

AttnCall q8_call(int mode, const delta_desc* d, const delta_page_table* pt, const void* q, void* o, void* ws,
                 size_t ws_bytes, void* stream) {
    AttnCall a;
    a.mode = mode;
    a.d = d;
    a.pt = pt;
    a.q = q;
    a.o = o;
    a.ws = ws;
    a.ws_bytes = ws_bytes;
    a.stream = stream;
    return a;
}

}  // namespace delta

using namespace delta;

extern "C" {

size_t delta_workspace_size_q8(const delta_desc* desc, int32_t batch, int32_t max_pages_per_seq, int32_t reduce) {
    if (check_desc(desc) != DELTA_OK || batch < 0 || max_pages_per_seq < 0) return 0;
    if (reduce != DELTA_HEAD_SUM && reduce != DELTA_HEAD_MAX) return 0;
    return q8_layout(desc, batch < 1 ? 1 : batch, max_pages_per_seq, reduce == DELTA_HEAD_MAX).total;
}

delta_status delta_full_attn_q8(const delta_desc* desc, const delta_page_table* pt, const void* q,
                                const delta_q8_cache* cache, void* o, void* workspace, size_t ws_bytes, void* stream) {
    return run_attention_on(Q8Cache{cache}, q8_call(kModeFull, desc, pt, q, o, workspace, ws_bytes, stream));
}

delta_status delta_select_attn_q8(const delta_desc* desc, const delta_page_table* pt, const delta_select_params* sp,
                                  const void* q, const delta_q8_cache* cache, void* o, int32_t* sel_cnt,
                                  int32_t* sel_pages, int32_t sel_stride, float* page_scores, void* workspace,
                                  size_t ws_bytes, void* stream) {
    AttnCall a = q8_call(kModeDelta, desc, pt, q, o, workspace, ws_bytes, stream);
    a.sp = sp;
    a.sel_cnt_out = sel_cnt;
    a.sel_pages_out = sel_pages;
    a.sel_stride_out = sel_stride;
    a.page_scores = page_scores;
    return run_attention_on(Q8Cache{cache}, a);
}

static delta_status sparse_q8(const delta_desc* desc, const delta_page_table* pt, const int32_t* sel_cnt,
                              const int32_t* sel_pages, int32_t sel_stride, const void* q, const delta_q8_cache* cache,
                              void* o, void* workspace, size_t ws_bytes, void* stream, bool settled) {
    AttnCall a = q8_call(kModeSparse, desc, pt, q, o, workspace, ws_bytes, stream);
    a.sel_cnt_in = sel_cnt;
    a.sel_pages_in = sel_pages;
    a.sel_stride_in = sel_stride;
    a.settled = settled;
    return run_attention_on(Q8Cache{cache}, a);
}

delta_status delta_sparse_attn_q8(const delta_desc* desc, const delta_page_table* pt, const int32_t* sel_cnt,
                                  const int32_t* sel_pages, int32_t sel_stride, const void* q,
                                  const delta_q8_cache* cache, void* o, void* workspace, size_t ws_bytes,
                                  void* stream) {
    return sparse_q8(desc, pt, sel_cnt, sel_pages, sel_stride, q, cache, o, workspace, ws_bytes, stream, false);
}

delta_status delta_sparse_attn_settled_q8(const delta_desc* desc, const delta_page_table* pt, const int32_t* sel_cnt,
                                          const int32_t* sel_pages, int32_t sel_stride, const void* q,
                                          const delta_q8_cache* cache, void* o, void* workspace, size_t ws_bytes,
                                          void* stream) {
    return sparse_q8(desc, pt, sel_cnt, sel_pages, sel_stride, q, cache, o, workspace, ws_bytes, stream, true);
}

delta_status delta_window_attn_q8(const delta_desc* desc, const delta_page_table* pt, int32_t window_tokens,
                                  int32_t sink_tokens, const void* q, const delta_q8_cache* cache, void* o,
                                  void* workspace, size_t ws_bytes, void* stream) {
    AttnCall a = q8_call(kModeWindow, desc, pt, q, o, workspace, ws_bytes, stream);
    a.window = window_tokens;
    a.sink = sink_tokens;
    return run_attention_on(Q8Cache{cache}, a);
}

}  // extern "C"
