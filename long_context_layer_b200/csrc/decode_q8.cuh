// Split-KV decode attention over the 8-bit cache on the tensor cores (included by the q8 attention
// translation units).
//
// Grid, clusters, page rings and the merge are those of the bf16 kernel (decode_mma.cuh); what differs is
// what 8-bit blocks with one scale each allow and ask for.  Per page (16 tokens x D bytes of K and of V):
//   S^T[16 x 8] = K8[16 x D] . Q^T[D x 8]   mma.m16n8k16 in fp16: an e4m3 or int8 value is exact in fp16, and
//        one ldmatrix row of 16 bytes holds 16 dimensions, so a 4-byte register holds two 2-value fragments
//        of one token: dimensions 4 t4 + {0, 1} and 4 t4 + {2, 3} of the chunk.  The product sums over
//        dimensions, so their order is free as long as Q's fragments follow it.
//   s = S * (Q's factor per head) * (K's block scale): powers of two and the softmax scale, in fp32.
//        Q is scaled per head by a power of two so that its largest element is in [2^14, 2^15): a bf16 value
//        keeps all its bits in fp16 down to 2^-28 of the largest.  fp32 queries are a sum of two fp16 values
//        (22 bits and the sign), which costs a second MMA.
//   online softmax as in decode_mma.cuh, with p = 2^(s - m + 14) so that fp16 holds small probabilities
//        (to 2^-39 of the largest; the offset cancels in o = acc / l), l summed from the rounded p that
//        weigh V (fp32: p too is a sum of two fp16 values).
//   O^T[D x 8] += (V's block scale) * V8^T[D x 16] . P^T[16 x 8]   ldmatrix.trans moves 2-byte units, that is
//        two dimensions of one token; a byte permute separates them, and the accumulator's rows g4 and g4 + 8
//        are dimensions 2 g4 and 2 g4 + 1 of the 16-dimension tile.
// Block scales stay out of the fp16 operands (their range is 2^-100..2^122): K's multiplies the logits and V's
// the page's product before it joins the fp32 accumulator.
#pragma once

#include "decode_mma.cuh"
#include "q8.cuh"

namespace delta {

// Shared-memory plan: WARPS rings of STAGES pages (K block, V block).
template <int D, int STAGES, int WARPS>
struct Q8Smem {
    static constexpr uint32_t kBlock = kPage * D;             // one K or V block
    static constexpr uint32_t kPage2 = 2 * kBlock;
    static constexpr size_t kStages = size_t(WARPS) * STAGES * kPage2;
    static_assert(size_t(STAGES) * kPage2 >= (size_t(kMaxGroup) * (D + 4) + 4 * kMaxGroup) * sizeof(float), "merge record");
    static constexpr size_t kBars = size_t(WARPS) * STAGES * sizeof(uint64_t);
    static constexpr size_t kRecv = size_t(recv_floats<D>()) * sizeof(float);
    static constexpr size_t kBytes = 1024 /* alignment slack */ + kStages + kBars + kRecv;
};

__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack_f16(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

// Bytes (i, j) of four payload bytes as two fp16 values.  e4m3: sign, 4 exponent bits and 3 mantissa bits
// moved to fp16's places, which is the value times 2^-8 (subnormals too; kFold puts 2^8 back).  int8: the
// byte with its sign bit flipped is value + 128, as fp16's 1024 + u, minus 1152.
template <int FMT>
struct Half8 {
    static constexpr float kFold = FMT == kE4M3 ? 256.f : 1.f;
    static __device__ __forceinline__ uint32_t ready(uint32_t x) { return FMT == kE4M3 ? x : x ^ 0x80808080u; }
    template <int I, int J>
    static __device__ __forceinline__ uint32_t pair(uint32_t x) {
        if constexpr (FMT == kE4M3) {
            const uint32_t y = __byte_perm(x, 0u, 0x0404 | (I << 4) | (J << 12));    // bytes into the high halves
            return (y & 0x80008000u) | ((y >> 1) & 0x3f803f80u);
        } else {
            const uint32_t y = __byte_perm(x, 0x64646464u, 0x4040 | I | (J << 8));
            __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&y), __half2half2(__ushort_as_half(0x6480)));
            return *reinterpret_cast<const uint32_t*>(&h);
        }
    }
};

// Pages of a warp with their block scales, a lane holding one page of each of two chunks of 32.
struct Q8Pages {
    int lp_a, ph_a, lp_b, ph_b, cur;
    float ks_a, vs_a, ks_b, vs_b;
};

template <int W>
__device__ __forceinline__ void q8_lookup(const DecodeParams& p, const SeqExtent& ex, int b, int i0, int warp, int nk,
                                          int kbase, int lane, int& lp, int& ph) {
    const int k = kbase + lane;
    lp = -1;
    ph = -1;
    if (k >= nk) return;
    const int i = i0 + warp + k * W;
    lp = p.mode == kModeSparse ? __ldcg(p.sel_pages + size_t(b) * p.sel_stride + i) : p.mode == kModeWindow ? window_page(ex, i) : i;
    if (lp < 0 || lp >= ex.N) {
        atomicOr(p.err, kErrSel);
        lp = -1;
        return;
    }
    const int64_t x = p.indices[ex.pbeg + lp];
    if (x < 0 || x >= p.num_phys_pages) {
        atomicOr(p.err, kErrPage);
        return;
    }
    ph = int(x);
}
// skip: the page whose scale the previous kernel may still write (-1: none).
__device__ __forceinline__ void q8_scales(const DecodeParams& p, int g, int lp, int ph, int skip, float& ks, float& vs) {
    ks = vs = 0.f;
    if (ph < 0 || lp == skip) return;
    const size_t i = size_t(ph) * p.num_kv_heads + g;
    ks = __ldcg(p.k_scale + i);
    vs = __ldcg(p.v_scale + i);
}

// T: dtype of q and o.  FMT: payload format.
template <typename T, int FMT, int D, int G, int STAGES, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, WARPS <= 8 ? 2 : 1) decode_q8_kernel(const DecodeParams p,
                                                                  const __grid_constant__ CUtensorMap tmap_k,
                                                                  const __grid_constant__ CUtensorMap tmap_v) {
    using S = Q8Smem<D, STAGES, WARPS>;
    using H = Half8<FMT>;
    constexpr bool kTwo = sizeof(T) == 4;      // fp32 queries and outputs: fp16 pairs
    constexpr int KS = D / 16;                 // k-steps of the QK product = M-tiles of the PV product
    constexpr int CH = D / 32;                 // ldmatrix.x4 of a block
    constexpr float kShift = 14.f, kUnshift = 6.103515625e-05f;    // 2^14, 2^-14
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem =
        smem_raw + ((1024 - (static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw)) & 1023)) & 1023);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kStages);
    float* recv = reinterpret_cast<float*>(smem + S::kStages + S::kBars);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g4 = lane >> 2, t4 = lane & 3;
    const int b = blockIdx.z, g = blockIdx.y, split = blockIdx.x;
    const int Hq = p.num_q_heads;
    const int h0 = g * G;

    uint64_t* wbar = bars + warp * STAGES;
    unsigned char* wst = smem + size_t(warp) * STAGES * S::kPage2;
    if (lane == 0) {
#pragma unroll
        for (int s = 0; s < STAGES; ++s) mbar_init(&wbar[s], 1);
        fence_mbar_init();
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_k)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_v)) : "memory");
    }
    __syncwarp();
    merge_prologue(recv);
    SeqExtent ex = seq_extent(p, b);
    int i0 = 0, nk = 0;
    Q8Pages pages;
    const uint64_t policy = evict_first_policy();
    // The newest token's page and its scales may still be written by the previous kernel until the wait
    // (settled inputs: not).
    const int newest = p.settled ? -1 : ex.N - 1;
    auto setup = [&](int skip) {
        if (p.mode == kModeWindow) seq_window(p, ex);
        else seq_count(p, b, ex);
        i0 = split * p.items_per_split;
        const int i1 = min(i0 + p.items_per_split, ex.count);
        nk = (i1 - i0 > warp) ? (i1 - i0 - warp + WARPS - 1) / WARPS : 0;   // pages of this warp
        pages.cur = 0;
        q8_lookup<WARPS>(p, ex, b, i0, warp, nk, 0, lane, pages.lp_a, pages.ph_a);
        q8_lookup<WARPS>(p, ex, b, i0, warp, nk, 32, lane, pages.lp_b, pages.ph_b);
        q8_scales(p, g, pages.lp_a, pages.ph_a, skip, pages.ks_a, pages.vs_a);
        q8_scales(p, g, pages.lp_b, pages.ph_b, skip, pages.ks_b, pages.vs_b);
    };
    // all lanes call, at the top of iteration k
    auto advance = [&](int k) {
        if (k > 0 && (k & 31) == 0) {
            pages.cur = k >> 5;
            pages.lp_a = pages.lp_b;
            pages.ph_a = pages.ph_b;
            pages.ks_a = pages.ks_b;
            pages.vs_a = pages.vs_b;
            q8_lookup<WARPS>(p, ex, b, i0, warp, nk, (pages.cur + 1) * 32, lane, pages.lp_b, pages.ph_b);
            q8_scales(p, g, pages.lp_b, pages.ph_b, -1, pages.ks_b, pages.vs_b);
        }
    };
    auto page_at = [&](int k, int& lp, int& ph) {
        const bool a = (k >> 5) == pages.cur;
        lp = __shfl_sync(0xffffffffu, a ? pages.lp_a : pages.lp_b, k & 31);
        ph = __shfl_sync(0xffffffffu, a ? pages.ph_a : pages.ph_b, k & 31);
    };
    auto scales_at = [&](int k, float& ks, float& vs) {
        const bool a = (k >> 5) == pages.cur;
        ks = __shfl_sync(0xffffffffu, a ? pages.ks_a : pages.ks_b, k & 31);
        vs = __shfl_sync(0xffffffffu, a ? pages.vs_a : pages.vs_b, k & 31);
    };
    // all lanes call; lane 0 issues the copies of page k into stage k % STAGES
    auto issue = [&](int k) {
        int lp, ph;
        page_at(k, lp, ph);
        if (lane != 0) return;
        const int s = k % STAGES;
        if (ph < 0) {
            mbar_arrive(&wbar[s]);   // completes the phase with no data; the page is skipped
            return;
        }
        unsigned char* dst = wst + size_t(s) * S::kPage2;
        const int y = (ph * p.num_kv_heads + g) * kPage;
        mbar_expect_tx(&wbar[s], S::kPage2);
        tma_load_2d(dst, &tmap_k, 0, y, &wbar[s], policy);
        tma_load_2d(dst + S::kBlock, &tmap_v, 0, y, &wbar[s], policy);
    };

    if (threadIdx.x == 0)
        prefetch_l2(reinterpret_cast<const T*>(p.q) + (size_t(b) * Hq + h0) * D, G * D * sizeof(T));
    // Before the wait: every page but the newest (all of a settled selection); the first sparse layer behind
    // a delta-layer waits, its page list is that layer's output.
    const bool known = p.mode != kModeSparse || p.settled;
    uint32_t early = 0;       // bit k: page k's copies were issued before the wait
    if (known) {
        setup(newest);
        for (int k = 0; k < min(STAGES, nk); ++k) {
            int lp, ph;
            page_at(k, lp, ph);
            if (ph >= 0 && lp != newest) {
                issue(k);
                early |= 1u << k;
            }
        }
    }
    pdl_wait();
    pdl_trigger();
    if (!known) setup(-1);
    for (int k = 0; k < min(STAGES, nk); ++k)
        if (!((early >> k) & 1u)) issue(k);
    if (known && newest >= 0) {   // the newest page's scales, if this lane holds it
        if (pages.lp_a == newest) q8_scales(p, g, pages.lp_a, pages.ph_a, -1, pages.ks_a, pages.vs_a);
        if (pages.lp_b == newest) q8_scales(p, g, pages.lp_b, pages.ph_b, -1, pages.ks_b, pages.vs_b);
    }

    // ---- Q^T fragments of head g4: dimensions 16 kk + 4 t4 + {0, 1} and {2, 3}
    uint32_t qb[KS][2], ql[kTwo ? KS : 1][2];
    float qf0, qf1;           // factors of this lane's logits (heads 2 t4, 2 t4 + 1)
    {
        float q[KS][4];
        const T* qp = reinterpret_cast<const T*>(p.q) + (size_t(b) * Hq + h0 + g4) * D + 4 * t4;
        uint32_t amax = 0;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
            if (g4 < G) load_row<T, 4>(qp + kk * 16, q[kk]);
            else q[kk][0] = q[kk][1] = q[kk][2] = q[kk][3] = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) amax = max(amax, __float_as_uint(q[kk][j]) & 0x7fffffffu);
        }
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // 2^x <= |q|max < 2^(x + 1), x at least -100; a head with a non-finite query gives NaN logits
        const int x = max(int(amax >> 23) - 127, -100);
        const bool fine = amax < 0x7f800000u;
        const float up = fine ? __uint_as_float(uint32_t(14 - x + 127) << 23) : 0.f;
        const float factor = fine ? p.qscale * H::kFold * __uint_as_float(uint32_t(x - 14 + 127) << 23) : __uint_as_float(0x7fc00000u);
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
#pragma unroll
            for (int j = 0; j < 4; ++j) q[kk][j] = fine ? q[kk][j] * up : 0.f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                qb[kk][j] = pack_f16(q[kk][2 * j], q[kk][2 * j + 1]);
                if constexpr (kTwo) {
                    const float2 r = unpack_f16(qb[kk][j]);
                    ql[kk][j] = pack_f16(q[kk][2 * j] - r.x, q[kk][2 * j + 1] - r.y);
                }
            }
        }
        qf0 = __shfl_sync(0xffffffffu, factor, 8 * t4);
        qf1 = __shfl_sync(0xffffffffu, factor, 8 * t4 + 4);
    }

    float m_run[2] = {-INFINITY, -INFINITY};   // heads 2*t4, 2*t4+1
    float l_run[2] = {0.f, 0.f};               // this lane's tokens only; summed over the lanes at the end
    float dl_run[2] = {0.f, 0.f};              // delta-layers: the same over the unrounded terms
    float acc[KS][4];
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) acc[mt][0] = acc[mt][1] = acc[mt][2] = acc[mt][3] = 0.f;

    // ldmatrix roles of this lane: matrix lj = (rows 8 (lj & 1) .. + 7, 16-byte chunk 2 c + (lj >> 1))
    const int row = (lane & 7) + (((lane >> 3) & 1) << 3);
    const int sub = lane >> 4;
    const int swz = D == 128 ? (row & 7) : ((row >> 1) & 3);     // TMA swizzle: 128-byte or 64-byte rows
    const uint32_t row_off = uint32_t(row) * D;
    bool failed = false;
    int consumed = 0;

    // base-2 logits of the page in stage s: tokens g4, g4 + 8, heads 2 t4, 2 t4 + 1
    auto qk_page = [&](int s, int lp, float ks, float (&sc)[4]) {
        const uint32_t base = smem_addr(wst + size_t(s) * S::kPage2) + row_off;
        float c0[4] = {0.f, 0.f, 0.f, 0.f}, c1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            uint32_t r0, r1, r2, r3;
            ldmatrix_x4(base + (((2 * c + sub) ^ swz) << 4), r0, r1, r2, r3);
            r0 = H::ready(r0);
            r1 = H::ready(r1);
            r2 = H::ready(r2);
            r3 = H::ready(r3);
            const uint32_t a0 = H::template pair<0, 1>(r0), a1 = H::template pair<0, 1>(r1);
            const uint32_t a2 = H::template pair<2, 3>(r0), a3 = H::template pair<2, 3>(r1);
            const uint32_t b0 = H::template pair<0, 1>(r2), b1 = H::template pair<0, 1>(r3);
            const uint32_t b2 = H::template pair<2, 3>(r2), b3 = H::template pair<2, 3>(r3);
            mma_f16_16816(c0, a0, a1, a2, a3, qb[2 * c][0], qb[2 * c][1]);
            mma_f16_16816(c1, b0, b1, b2, b3, qb[2 * c + 1][0], qb[2 * c + 1][1]);
            if constexpr (kTwo) {
                mma_f16_16816(c0, a0, a1, a2, a3, ql[2 * c][0], ql[2 * c][1]);
                mma_f16_16816(c1, b0, b1, b2, b3, ql[2 * c + 1][0], ql[2 * c + 1][1]);
            }
        }
        const int t = lp * kPage + g4;
        bool ok0 = t < ex.n, ok1 = t + 8 < ex.n;
        if (p.mode == kModeWindow) {
            ok0 = ok0 && (t < p.sink || t >= ex.from);
            ok1 = ok1 && (t + 8 < p.sink || t + 8 >= ex.from);
        }
        sc[0] = ok0 ? (c0[0] + c1[0]) * qf0 * ks : -INFINITY;
        sc[1] = ok0 ? (c0[1] + c1[1]) * qf1 * ks : -INFINITY;
        sc[2] = ok1 ? (c0[2] + c1[2]) * qf0 * ks : -INFINITY;
        sc[3] = ok1 ? (c0[3] + c1[3]) * qf1 * ks : -INFINITY;
    };
    // delta-layers: a page's log2-sum-exp per head from the terms 2^(s - m + 14), as in decode_mma.cuh
    auto page_partials = [&](const float (&pa)[4], const float (&pb)[4], float mn0, float mn1, float al0, float al1,
                             bool vA, bool vB, int lpA, int lpB) {
        float ea0 = pa[0] + pa[2], ea1 = pa[1] + pa[3], eb0 = pb[0] + pb[2], eb1 = pb[1] + pb[3];
        dl_run[0] = dl_run[0] * al0 + (ea0 + eb0);
        dl_run[1] = dl_run[1] * al1 + (ea1 + eb1);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            ea0 += __shfl_xor_sync(0xffffffffu, ea0, o);
            ea1 += __shfl_xor_sync(0xffffffffu, ea1, o);
            eb0 += __shfl_xor_sync(0xffffffffu, eb0, o);
            eb1 += __shfl_xor_sync(0xffffffffu, eb1, o);
        }
        const int hA = 2 * t4, hB = 2 * t4 + 1;
        if (g4 == 0) {
            float* out = p.page_lse + (size_t(b) * Hq + h0) * p.max_pages;
            const float u0 = mn0 - kShift, u1 = mn1 - kShift;
            if (vA && hA < G) out[size_t(hA) * p.max_pages + lpA] = u0 + log2_approx(ea0);
            if (vA && hB < G) out[size_t(hB) * p.max_pages + lpA] = u1 + log2_approx(ea1);
            if (vB && hA < G) out[size_t(hA) * p.max_pages + lpB] = u0 + log2_approx(eb0);
            if (vB && hB < G) out[size_t(hB) * p.max_pages + lpB] = u1 + log2_approx(eb1);
        }
    };
    auto store_logits = [&](const float (&sc)[4], int lp) {      // HEAD_MAX scoring
        float* lg = p.logits + (size_t(b) * Hq + h0) * (size_t(p.max_pages) * kPage) + size_t(lp) * kPage;
        const size_t hs = size_t(p.max_pages) * kPage;
        if (2 * t4 < G) { lg[2 * t4 * hs + g4] = sc[0]; lg[2 * t4 * hs + g4 + 8] = sc[2]; }
        if (2 * t4 + 1 < G) { lg[(2 * t4 + 1) * hs + g4] = sc[1]; lg[(2 * t4 + 1) * hs + g4 + 8] = sc[3]; }
    };
    // Tile pair c (dimensions 32 c .. 32 c + 31) of V^T . P^T of the page in stage s, added to d0 and d1.  Hidden
    // tokens weigh exactly 0 and any payload byte is a finite fp16 value, so stale slots need no clearing.
    auto pv_tile = [&](int s, int c, const uint32_t (&pt)[kTwo ? 4 : 2], float (&d0)[4], float (&d1)[4]) {
        const uint32_t base = smem_addr(wst + size_t(s) * S::kPage2) + S::kBlock + row_off;
        uint32_t r0, r1, r2, r3;
        ldmatrix_x4_trans(base + (((2 * c + sub) ^ swz) << 4), r0, r1, r2, r3);
        r0 = H::ready(r0);
        r1 = H::ready(r1);
        r2 = H::ready(r2);
        r3 = H::ready(r3);
        const uint32_t a0 = H::template pair<0, 2>(r0), a1 = H::template pair<1, 3>(r0);
        const uint32_t a2 = H::template pair<0, 2>(r1), a3 = H::template pair<1, 3>(r1);
        const uint32_t b0 = H::template pair<0, 2>(r2), b1 = H::template pair<1, 3>(r2);
        const uint32_t b2 = H::template pair<0, 2>(r3), b3 = H::template pair<1, 3>(r3);
        mma_f16_16816(d0, a0, a1, a2, a3, pt[0], pt[1]);
        mma_f16_16816(d1, b0, b1, b2, b3, pt[0], pt[1]);
        if constexpr (kTwo) {
            mma_f16_16816(d0, a0, a1, a2, a3, pt[2], pt[3]);
            mma_f16_16816(d1, b0, b1, b2, b3, pt[2], pt[3]);
        }
    };
    // the rounded probabilities of a page as P^T fragments; adds them to this lane's sums
    auto round_p = [&](const float (&e)[4], uint32_t (&pt)[kTwo ? 4 : 2], float& s0, float& s1) {
        const uint32_t x0 = pack_f16(e[0], e[1]), x1 = pack_f16(e[2], e[3]);
        const float2 r0 = unpack_f16(x0), r1 = unpack_f16(x1);
        s0 += r0.x + r1.x;
        s1 += r0.y + r1.y;
        pt[0] = movmatrix_trans(x0);
        pt[1] = movmatrix_trans(x1);
        if constexpr (kTwo) {
            const uint32_t y0 = pack_f16(e[0] - r0.x, e[1] - r0.y), y1 = pack_f16(e[2] - r1.x, e[3] - r1.y);
            const float2 u0 = unpack_f16(y0), u1 = unpack_f16(y1);
            s0 += u0.x + u1.x;
            s1 += u0.y + u1.y;
            pt[2] = movmatrix_trans(y0);
            pt[3] = movmatrix_trans(y1);
        }
    };

    for (int k = 0; k < nk; k += 2) {
        advance(k);
        const bool two = k + 1 < nk;
        const int sA = k % STAGES, sB = (k + 1) % STAGES;
        if (!mbar_wait(&wbar[sA], (k / STAGES) & 1) || (two && !mbar_wait(&wbar[sB], ((k + 1) / STAGES) & 1))) {
            if (lane == 0) atomicOr(p.err, kErrTimeout);
            failed = true;
            break;
        }
        consumed = k + (two ? 2 : 1);
        int lpA, phA, lpB = -1, phB = -1;
        float ksA, vsA, ksB = 0.f, vsB = 0.f;
        page_at(k, lpA, phA);
        scales_at(k, ksA, vsA);
        if (two) {
            page_at(k + 1, lpB, phB);
            scales_at(k + 1, ksB, vsB);
        }
        const bool vA = phA >= 0, vB = phB >= 0;
        float scA[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        float scB[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (vA) qk_page(sA, lpA, ksA, scA);
        if (vB) qk_page(sB, lpB, ksB, scB);
        if (vA || vB) {
            if (p.logits != nullptr) {
                if (vA) store_logits(scA, lpA);
                if (vB) store_logits(scB, lpB);
            }
            float mx0 = fmaxf(fmaxf(scA[0], scA[2]), fmaxf(scB[0], scB[2]));
            float mx1 = fmaxf(fmaxf(scA[1], scA[3]), fmaxf(scB[1], scB[3]));
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
                mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
            }
            // the lowest finite value when every logit is NaN (fmaxf drops them): the sums then are NaN
            const float mn0 = fmaxf(fmaxf(m_run[0], mx0), -3.402823466e38f);
            const float mn1 = fmaxf(fmaxf(m_run[1], mx1), -3.402823466e38f);
            const float al0 = exp2_approx(m_run[0] - mn0), al1 = exp2_approx(m_run[1] - mn1);
            const float u0 = kShift - mn0, u1 = kShift - mn1;
            const float pa[4] = {exp2_approx(scA[0] + u0), exp2_approx(scA[1] + u1), exp2_approx(scA[2] + u0),
                                 exp2_approx(scA[3] + u1)};
            const float pb[4] = {exp2_approx(scB[0] + u0), exp2_approx(scB[1] + u1), exp2_approx(scB[2] + u0),
                                 exp2_approx(scB[3] + u1)};
            if (p.mode == kModeDelta) page_partials(pa, pb, mn0, mn1, al0, al1, vA, vB, lpA, lpB);
            uint32_t ptA[kTwo ? 4 : 2], ptB[kTwo ? 4 : 2];
            float s0 = 0.f, s1 = 0.f;
            round_p(pa, ptA, s0, s1);
            round_p(pb, ptB, s0, s1);
            l_run[0] = l_run[0] * al0 + s0;
            l_run[1] = l_run[1] * al1 + s1;
            m_run[0] = mn0;
            m_run[1] = mn1;
            // The two pages' products share one accumulator when their V scales are equal (mostly: powers of
            // two of similar blocks), else each is scaled by its own.
            const float wA = vsA * (H::kFold * kUnshift), wB = vsB * (H::kFold * kUnshift);
            const bool joint = vA && vB && vsA == vsB;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                float d0[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f};
                float(&a0)[4] = acc[2 * c];
                float(&a1)[4] = acc[2 * c + 1];
                if (vA) pv_tile(sA, c, ptA, d0, d1);
                if (joint) pv_tile(sB, c, ptB, d0, d1);
                const float w = vA ? wA : 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float al = (j & 1) ? al1 : al0;
                    a0[j] = fmaf(d0[j], w, a0[j] * al);
                    a1[j] = fmaf(d1[j], w, a1[j] * al);
                }
                if (vB && !joint) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) d0[j] = d1[j] = 0.f;
                    pv_tile(sB, c, ptB, d0, d1);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        a0[j] = fmaf(d0[j], wB, a0[j]);
                        a1[j] = fmaf(d1[j], wB, a1[j]);
                    }
                }
            }
        }
        __syncwarp();
        if (k + STAGES < nk) issue(k + STAGES);
        if (two && k + 1 + STAGES < nk) issue(k + 1 + STAGES);
    }
    if (failed) {
        // drain this warp's copies still in flight (bounded) before shared memory is released
        for (int k = consumed + 1; k < min(consumed + STAGES, nk); ++k) mbar_wait(&wbar[k % STAGES], (k / STAGES) & 1);
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            l_run[j] += __shfl_xor_sync(0xffffffffu, l_run[j], o);
            dl_run[j] += __shfl_xor_sync(0xffffffffu, dl_run[j], o);
        }
    }

    // ---- this warp's state into its own stage area, then the merge of the CTA's warps and of the splits
    __syncwarp();
    constexpr int kRow = D + 4;
    float* po = reinterpret_cast<float*>(wst);           // [8][D + 4] outputs
    float* pml = po + kMaxGroup * kRow;                   // [8][2] (max, sum)
    float* pdl = pml + kMaxGroup * 2;                     // [8][2] delta-layers: over the unrounded terms
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) {
        const int d = mt * 16 + 2 * g4;
        *reinterpret_cast<float2*>(po + (2 * t4) * kRow + d) = make_float2(acc[mt][0], acc[mt][2]);
        *reinterpret_cast<float2*>(po + (2 * t4 + 1) * kRow + d) = make_float2(acc[mt][1], acc[mt][3]);
    }
    if (g4 == 0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            pml[(2 * t4 + j) * 2] = m_run[j];
            pml[(2 * t4 + j) * 2 + 1] = l_run[j] * kUnshift;
            pdl[(2 * t4 + j) * 2] = m_run[j];
            pdl[(2 * t4 + j) * 2 + 1] = dl_run[j] * kUnshift;
        }
    }
    __syncthreads();
    constexpr int kPart = STAGES * int(S::kPage2) / 4;    // floats between two warps' records
    const float* mo0 = reinterpret_cast<const float*>(smem);
    float pre[2][G];   // delta-layers: this CTA's page terms, loaded before the merge
    if (p.fuse_select) select_preload<WARPS * 32, G>(p, b, g, ex.N, pre);
    merge_epilogue<T, D, G, WARPS, WARPS * 32, kRow>(
        p, smem, mo0, mo0 + kMaxGroup * kRow, recv, b, g, kPart, kPart,
        (p.mode == kModeDelta) ? mo0 + kMaxGroup * kRow + kMaxGroup * 2 : nullptr);
    if (p.fuse_select) select_tail<WARPS * 32, G, D>(p, smem, S::kStages, recv, b, g, ex.n, ex.N, pre);
}

}  // namespace delta
