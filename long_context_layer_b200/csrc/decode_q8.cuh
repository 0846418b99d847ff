// Split-KV decode attention over the 8-bit cache on the tensor cores (included by the q8 attention
// translation units).
//
// Grid, clusters, page rings and the merge are those of the bf16 kernel (decode_mma.cuh); what differs is
// what 8-bit blocks with one scale each allow and ask for.  Per page (16 tokens x D bytes of K and of V):
//   S^T[16 x 8] = K8[16 x D] . Q^T[D x 8]
//        e4m3: mma.m16n8k16 in fp16, in which an e4m3 value is exact.  Q is scaled per head by a power of two so
//        that its largest element is in [2^14, 2^15): a bf16 keeps its bits down to 2^-28 of the largest.  A
//        4-byte register of an ldmatrix row holds two 2-value fragments of one token, dimensions 4 t4 + {0, 1}
//        and 4 t4 + {2, 3} of a 16-byte chunk; the product sums over dimensions, so their order is free as long
//        as Q's fragments follow it.  (The 8-bit mma.m16n8k32 over e4m3 operands is executed as two fp16
//        products with conversions of both operands, a tenth slower for the delta-layer of 16 x 16k.)
//        int8: the payload is an operand of mma.m16n8k32 over bytes, and a query is 23-bit fixed point, its high
//        bytes (signed), middle and low bytes (unsigned) on three integer accumulators: exact down to 2^-14 of
//        the head's largest element, the others to 2^-22 of it.  No conversion of K (4 x 64k 86 us,
//        in fp16 91; 16 x 16k 84 and 90).  Two bytes would do for even queries and save 2 to 6 % where lists are short, but leave
//        2^-15 of the largest element, which queries with an outlying dimension would show.
//        fp32 queries: the fp16 form with a query as the sum of two values (22 bits and the sign).
//   s = S * (Q's factor per head) * (K's block scale): powers of two and the softmax scale, in fp32.
//   online softmax as in decode_mma.cuh, with p = 2^(s - m + 14) so that fp16 holds small probabilities
//        (to 2^-38 of the largest; the offset cancels in o = acc / l).  For the product p is the sum of two fp16
//        values (22 bits and the signs), so that an output is off by its own rounding and what fp32 sums explain.
//        l sums the fp32 terms, which are also the page terms of a delta-layer.
//   O^T[D x 8] += V8^T[D x 16] . (V's block scale / unit * P^T)[16 x 8]   ldmatrix.trans moves 2-byte units, that is
//        two dimensions of one token; a byte permute separates them, and the accumulator's rows g4 and g4 + 8
//        are dimensions 2 g4 and 2 g4 + 1 of the 16-dimension tile.
// Block scales range over 2^-100..2^122: K's multiplies the logits; V's joins P relative to the accumulators' unit,
// the largest scale so far.  (Scaling the product instead costs 64 multiply-adds a pair of pages, and about a third of
// the pages of caches with ordinary spread differ from the unit.)
#pragma once

#include "decode_mma.cuh"
#include "q8.cuh"

#include <type_traits>

namespace delta {

// Shared-memory plan: WARPS rings of STAGES pages (K block, V block).
template <int D, int STAGES, int WARPS>
struct Q8Smem {
    static constexpr uint32_t kBlock = kPage * D;             // one K or V block
    static constexpr uint32_t kPage2 = 2 * kBlock;
    static constexpr size_t kStages = size_t(WARPS) * STAGES * kPage2;
    static_assert(size_t(STAGES) * kPage2 >= (size_t(kMaxGroup) * (D + 4) + 4 * kMaxGroup) * sizeof(float), "merge record");
    static constexpr size_t kBars = size_t(WARPS) * STAGES * sizeof(uint64_t);
    static_assert(kBars % 16 == 0, "the merge's receive area starts on 16 bytes");
    static constexpr size_t kRecv = size_t(recv_floats<D>()) * sizeof(float);
    static constexpr size_t kBytes = 1024 /* alignment slack */ + kStages + kBars + kRecv;
};

// (Not volatile: the products depend on their registers alone, so independent chains interleave.)
__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_s8s8_16832(int (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_s8u8_16832(int (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.u8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack_f16(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

// Four payload bytes as fp16 pairs: near() gives bytes (0, 1) and (2, 3), apart() (0, 2) and (1, 3).
// e4m3: the conversion instruction (after a byte permute for the pairs that are apart).  int8: a byte with its
// sign bit flipped is value + 128; as the low byte of 0x6400 it is fp16's 1024 + (value + 128), minus 1152.
template <int FMT>
struct Half8;
template <>
struct Half8<kE4M3> {
    static __device__ __forceinline__ uint32_t cvt(uint32_t two) {
        uint32_t h;
        asm("{ .reg .b16 l, u; mov.b32 {l, u}, %1; cvt.rn.f16x2.e4m3x2 %0, l; }" : "=r"(h) : "r"(two));
        return h;
    }
    static __device__ __forceinline__ uint32_t cvt_high(uint32_t two) {
        uint32_t h;
        asm("{ .reg .b16 l, u; mov.b32 {l, u}, %1; cvt.rn.f16x2.e4m3x2 %0, u; }" : "=r"(h) : "r"(two));
        return h;
    }
    static __device__ __forceinline__ void near(uint32_t x, uint32_t& lo, uint32_t& hi) {
        lo = cvt(x);
        hi = cvt_high(x);
    }
    static __device__ __forceinline__ void apart(uint32_t x, uint32_t& even, uint32_t& odd) {
        near(__byte_perm(x, 0u, 0x3120), even, odd);
    }
};
template <>
struct Half8<kInt8> {
    static __device__ __forceinline__ uint32_t less(uint32_t y) {
        const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&y), __half2half2(__ushort_as_half(0x6480)));
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ void near(uint32_t x, uint32_t& lo, uint32_t& hi) {
        x ^= 0x80808080u;
        lo = less(__byte_perm(x, 0x64646464u, 0x4140));
        hi = less(__byte_perm(x, 0x64646464u, 0x4342));
    }
    static __device__ __forceinline__ void apart(uint32_t x, uint32_t& even, uint32_t& odd) {
        x ^= 0x80808080u;
        even = less(__byte_perm(x, 0x64646464u, 0x4240));
        odd = less(__byte_perm(x, 0x64646464u, 0x4341));
    }
};

// Pages of a warp with their block scales, a lane holding one page of each of two chunks of 32 (a: the chunk
// of the page in hand).  A page to be skipped has lp = ph = -1.
struct Q8Pages {
    int lp_a, ph_a, lp_b, ph_b, cur;
    float ks_a, vs_a, ks_b, vs_b;
};

// QUIET: a speculative lookup before the wait, which raises no flags.
template <int W, bool QUIET = false>
__device__ __forceinline__ void q8_lookup(const DecodeParams& p, const SeqExtent& ex, int b, int i0, int warp, int nk,
                                          int kbase, int lane, int& lp, int& ph) {
    const int k = kbase + lane;
    lp = -1;
    ph = -1;
    if (k >= nk) return;
    const int i = i0 + warp + k * W;
    lp = p.mode == kModeSparse ? __ldcg(p.sel_pages + size_t(b) * p.sel_stride + i) : p.mode == kModeWindow ? window_page(ex, i) : i;
    if (lp < 0 || lp >= ex.N) {
        if (!QUIET) atomicOr(p.err, kErrSel);
        lp = -1;
        return;
    }
    const int64_t x = p.indices[ex.pbeg + lp];
    if (x < 0 || x >= p.num_phys_pages) {
        if (!QUIET) atomicOr(p.err, kErrPage);
        lp = -1;
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
    constexpr bool kTwo = sizeof(T) == 4;      // fp32 queries: fp16 pairs
    constexpr bool kHalf = kTwo || FMT == kE4M3;    // QK in fp16, else in 8-bit integers
    constexpr int KS = D / 16;                 // k-steps of the QK product = M-tiles of the PV product
    constexpr int CH = D / 32;                 // ldmatrix.x4 of a block
    constexpr bool kTwin = G <= 4;             // columns 4..7 of the products are the heads 0..3 once more
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
    auto phys_at = [&](int k) {
        return __shfl_sync(0xffffffffu, (k >> 5) == pages.cur ? pages.ph_a : pages.ph_b, k & 31);
    };
    // lane 0: the copies of a page into stage s
    auto copy_page = [&](int ph, int s) {
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
    // all lanes call
    auto issue = [&](int k, int s) {
        const int ph = phys_at(k);
        if (lane == 0) copy_page(ph, s);
    };

    if (threadIdx.x == 0)
        prefetch_l2(reinterpret_cast<const T*>(p.q) + (size_t(b) * Hq + h0) * D, G * D * sizeof(T));
    // Before the wait: every page but the newest (all of a settled selection).  The first sparse layer behind a
    // delta-layer guesses that the selection is already the new one (mostly the last step's still holds) and
    // checks it after the wait.
    const bool known = p.mode != kModeSparse || p.settled;
    uint32_t early = 0;       // bit k: page k's copies were issued before the wait
    uint32_t parity = 0;      // of the phases of the pages in hand
    if (known) {
        setup(newest);
    } else {
        ex.count = min(max(__ldcg(p.sel_cnt + b), 0), min(p.sel_stride, p.items_per_split * p.num_splits));
        i0 = split * p.items_per_split;
        const int i1 = min(i0 + p.items_per_split, ex.count);
        nk = (i1 - i0 > warp) ? (i1 - i0 - warp + WARPS - 1) / WARPS : 0;
        pages.cur = 0;
        q8_lookup<WARPS, true>(p, ex, b, i0, warp, nk, 0, lane, pages.lp_a, pages.ph_a);
        q8_scales(p, g, pages.lp_a, pages.ph_a, newest, pages.ks_a, pages.vs_a);
        pages.lp_b = pages.ph_b = -1;
    }
    for (int k = 0; k < min(STAGES, nk); ++k) {
        const int lp = __shfl_sync(0xffffffffu, pages.lp_a, k);
        if (lp >= 0 && lp != newest) {
            issue(k, k);
            early |= 1u << k;
        }
    }
    pdl_wait();
    pdl_trigger();
    if (!known) {
        // the selection's entries at the guessed places, loaded together with its count
        const int guess_nk = nk;
        const int lp = lane < nk ? __ldcg(p.sel_pages + size_t(b) * p.sel_stride + i0 + warp + lane * WARPS) : -1;
        seq_count(p, b, ex);
        const int i1 = min(i0 + p.items_per_split, ex.count);
        nk = (i1 - i0 > warp) ? (i1 - i0 - warp + WARPS - 1) / WARPS : 0;
        if (nk == guess_nk && __all_sync(0xffffffffu, lane >= nk || (lp == pages.lp_a && lp >= 0))) {
            q8_lookup<WARPS>(p, ex, b, i0, warp, nk, 32, lane, pages.lp_b, pages.ph_b);
            q8_scales(p, g, pages.lp_b, pages.ph_b, -1, pages.ks_b, pages.vs_b);
        } else {
            // spend the first phase of every stage: wait for the guessed copies (bounded), pass the others
            for (int k = 0; k < STAGES; ++k) {
                if ((early >> k) & 1u) {
                    if (!mbar_wait(&wbar[k], 0) && lane == 0) atomicOr(p.err, kErrTimeout);
                } else {
                    if (lane == 0) mbar_arrive(&wbar[k]);
                }
            }
            __syncwarp();
            early = 0;
            parity = 1;
            setup(-1);
        }
    }
    for (int k = 0; k < min(STAGES, nk); ++k)
        if (!((early >> k) & 1u)) issue(k, k);
    if (newest >= 0) {   // the newest page's scales, if this lane holds it
        if (pages.lp_a == newest) q8_scales(p, g, pages.lp_a, pages.ph_a, -1, pages.ks_a, pages.vs_a);
        if (pages.lp_b == newest) q8_scales(p, g, pages.lp_b, pages.ph_b, -1, pages.ks_b, pages.vs_b);
    }

    // ---- Q^T fragments of head g4 (kTwin: g4 & 3): dimensions 16 kk + 4 t4 + {0, 1, 2, 3} are this lane's
    constexpr int kTop = kHalf ? 14 : 21;    // the largest element is scaled into [2^kTop, 2^(kTop + 1))
    constexpr bool kThree = !kHalf;          // 24-bit fixed point in three bytes: qa, qc, qx
    uint32_t qa[KS], qc[KS], qx[kTwo || kThree ? KS : 1], qy[kTwo ? KS : 1];
    float qf0, qf1;           // factors of this lane's logits (heads 2 t4, 2 t4 + 1)
    {
        // bf16: two registers of two; fp32: four
        uint32_t raw[KS][kTwo ? 4 : 2];
        const int hq = kTwin ? g4 & 3 : g4;
        const T* qp = reinterpret_cast<const T*>(p.q) + (size_t(b) * Hq + h0 + hq) * D + 4 * t4;
        uint32_t amax = 0;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
            if constexpr (kTwo) {
                const uint4 w = hq < G ? *reinterpret_cast<const uint4*>(qp + kk * 16) : make_uint4(0, 0, 0, 0);
                raw[kk][0] = w.x;
                raw[kk][1] = w.y;
                raw[kk][2] = w.z;
                raw[kk][3] = w.w;
            } else {
                const uint2 w = hq < G ? *reinterpret_cast<const uint2*>(qp + kk * 16) : make_uint2(0, 0);
                raw[kk][0] = w.x;
                raw[kk][1] = w.y;
            }
        }
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
            if constexpr (kTwo) amax = Raw16<float>::more(amax, make_uint4(raw[kk][0], raw[kk][1], raw[kk][2], raw[kk][3]));
            else amax = __vimax3_u16x2(amax, raw[kk][0] & 0x7fff7fffu, raw[kk][1] & 0x7fff7fffu);
        }
        if constexpr (!kTwo) amax = Raw16<__nv_bfloat16>::top(amax);
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // 2^x <= |q|max < 2^(x + 1), x at least -100; a head with a non-finite query gives NaN logits
        const int x = max(int(amax >> 23) - 127, -100);
        const bool fine = amax < 0x7f800000u;
        const float up = fine ? __uint_as_float(uint32_t(kTop - x + 127) << 23) : 0.f;
        const float factor = fine ? p.qscale * __uint_as_float(uint32_t(x - kTop + 127) << 23) : __uint_as_float(0x7fc00000u);
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
            float q[4];
            if constexpr (kTwo) {
#pragma unroll
                for (int j = 0; j < 4; ++j) q[j] = __uint_as_float(raw[kk][j]);
            } else {
                unpack_bf16x2(raw[kk][0], q[0], q[1]);
                unpack_bf16x2(raw[kk][1], q[2], q[3]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) q[j] = fine ? q[j] * up : 0.f;
            if constexpr (kHalf) {
                qa[kk] = pack_f16(q[0], q[1]);
                qc[kk] = pack_f16(q[2], q[3]);
                if constexpr (kTwo) {
                    const float2 ra = unpack_f16(qa[kk]), rc = unpack_f16(qc[kk]);
                    qx[kk] = pack_f16(q[0] - ra.x, q[1] - ra.y);
                    qy[kk] = pack_f16(q[2] - rc.x, q[3] - rc.y);
                }
            } else {
                // the nearest integer, within +-2^22, from the bits of q + 1.5 * 2^23
                uint32_t i[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) i[j] = __float_as_uint(q[j] + 12582912.f) - 0x4b400000u;
                qa[kk] = __byte_perm(__byte_perm(i[0], i[1], 0x0062), __byte_perm(i[2], i[3], 0x0062), 0x5410);
                qc[kk] = __byte_perm(__byte_perm(i[0], i[1], 0x0051), __byte_perm(i[2], i[3], 0x0051), 0x5410);
                qx[kk] = __byte_perm(__byte_perm(i[0], i[1], 0x0040), __byte_perm(i[2], i[3], 0x0040), 0x5410);
            }
        }
        qf0 = __shfl_sync(0xffffffffu, factor, 8 * t4);
        qf1 = __shfl_sync(0xffffffffu, factor, 8 * t4 + 4);
    }

    // reference of the base-2 logits of heads 2 t4, 2 t4 + 1 (within 1 below their maximum or above it)
    float m_run[2] = {-3.402823466e38f, -3.402823466e38f};
    float l_run[2] = {0.f, 0.f};               // this lane's tokens only; summed over the lanes at the end
    float acc[KS][4];
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) acc[mt][0] = acc[mt][1] = acc[mt][2] = acc[mt][3] = 0.f;
    // unit of acc: the largest V scale so far, at first of the warp's first 32 pages (from 2^-126; NaN if one is)
    float vref = __uint_as_float(max(0x00800000u, __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(pages.vs_a)))));
    float vinv = 1.f / vref;

    // ldmatrix roles of this lane: matrix lj = (rows 8 (lj & 1) .. + 7, 16-byte chunk 2 c + (lj >> 1))
    const int row = (lane & 7) + (((lane >> 3) & 1) << 3);
    const int sub = lane >> 4;
    const int swz = D == 128 ? (row & 7) : ((row >> 1) & 3);     // TMA swizzle: 128-byte or 64-byte rows
    bool failed = false;
    int consumed = 0;

    uint32_t off[CH];         // this lane's ldmatrix offsets in a block
#pragma unroll
    for (int c = 0; c < CH; ++c) off[c] = uint32_t(row) * D + (((2 * c + sub) ^ swz) << 4);
    const uint32_t st0 = smem_addr(wst);

    // K . Q^T of 32 dimensions of the page in stage s.  c0 and c1: of the chunk's two halves (fp16); or c0, c1, c2:
    // the products with Q's bytes, high to low.
    using Sum = std::conditional_t<kHalf, float, int>;
    auto qk_chunk = [&](int s, int c, Sum (&c0)[4], Sum (&c1)[4], Sum (&c2)[4]) {
        uint32_t r[4];
        ldmatrix_x4(st0 + uint32_t(s) * S::kPage2 + off[c], r[0], r[1], r[2], r[3]);
        if constexpr (kHalf) {
            uint32_t a0, a1, a2, a3;
            H::near(r[0], a0, a2);
            H::near(r[1], a1, a3);
            mma_f16_16816(c0, a0, a1, a2, a3, qa[2 * c], qc[2 * c]);
            if constexpr (kTwo) mma_f16_16816(c0, a0, a1, a2, a3, qx[2 * c], qy[2 * c]);
            H::near(r[2], a0, a2);
            H::near(r[3], a1, a3);
            mma_f16_16816(c1, a0, a1, a2, a3, qa[2 * c + 1], qc[2 * c + 1]);
            if constexpr (kTwo) mma_f16_16816(c1, a0, a1, a2, a3, qx[2 * c + 1], qy[2 * c + 1]);
        } else {
            mma_s8s8_16832(c0, r, qa[2 * c], qa[2 * c + 1]);
            mma_s8u8_16832(c1, r, qc[2 * c], qc[2 * c + 1]);
            mma_s8u8_16832(c2, r, qx[2 * c], qx[2 * c + 1]);
        }
    };
    auto sum_of = [](Sum x, Sum y, Sum z) {
        if constexpr (std::is_same_v<Sum, int>) return fmaf(float(x), 65536.f, float(y * 256 + z));   // below 2^31 each
        else return x + y;
    };
    // base-2 logits of a page: tokens g4, g4 + 8, heads 2 t4, 2 t4 + 1
    auto logits_of = [&](const Sum (&c0)[4], const Sum (&c1)[4], const Sum (&c2)[4], float ks, int lp, int s, float (&sc)[4]) {
        const float f0 = qf0 * ks, f1 = qf1 * ks;
        sc[0] = sum_of(c0[0], c1[0], c2[0]) * f0;
        sc[1] = sum_of(c0[1], c1[1], c2[1]) * f1;
        sc[2] = sum_of(c0[2], c1[2], c2[2]) * f0;
        sc[3] = sum_of(c0[3], c1[3], c2[3]) * f1;
        const int t0 = lp * kPage;
        const bool whole = t0 + kPage <= ex.n && (p.mode != kModeWindow || t0 + kPage <= p.sink || t0 >= ex.from);
        if (!whole) {      // the last page, and pages at the edge of the sinks or the window
            const int t = t0 + g4;
            bool ok0 = t < ex.n, ok1 = t + 8 < ex.n;
            if (p.mode == kModeWindow) {
                ok0 = ok0 && (t < p.sink || t >= ex.from);
                ok1 = ok1 && (t + 8 < p.sink || t + 8 >= ex.from);
            }
            if (!ok0) sc[0] = sc[1] = -INFINITY;
            if (!ok1) sc[2] = sc[3] = -INFINITY;
            // slots past the end and hidden tokens may hold e4m3's NaN: their V rows become zeros
            int lo = 0, hi = 0;
            if (p.mode == kModeWindow) window_gap(p, ex, lp, lo, hi);
            uint4* vz = reinterpret_cast<uint4*>(wst + size_t(s) * S::kPage2 + S::kBlock);
            for (int i = lane; i < kPage * (D / 16); i += 32) {
                const int r = i / (D / 16);
                if (t0 + r >= ex.n || (r >= lo && r < hi)) vz[i] = make_uint4(0, 0, 0, 0);
            }
            __syncwarp();
            if (lane == 0) fence_proxy_async_smem();    // ahead of the copy that reuses the stage
        }
    };
    // Delta-layers: a page's log2-sum-exp per head from the terms 2^(s - m + 14), summed over the g4 lanes.  The four
    // sums of a lane (pages A and B, heads 2 t4 and 2 t4 + 1) are scattered as they are reduced, so each lane
    // ends with one of them: page B where lane & 16, head 2 t4 + 1 where lane & 8.
    const bool pick_b = lane & 16, pick_1 = lane & 8;
    const int lse_head = 2 * t4 + (pick_1 ? 1 : 0);
    float* lse_row = p.page_lse + (size_t(b) * Hq + h0 + (lse_head < G ? lse_head : 0)) * p.max_pages;
    auto page_partials = [&](const float (&pa)[4], const float (&pb)[4], float mn0, float mn1, int lpA, int lpB) {
        const float ea0 = pa[0] + pa[2], ea1 = pa[1] + pa[3], eb0 = pb[0] + pb[2], eb1 = pb[1] + pb[3];
        float e0 = pick_b ? eb0 : ea0, e1 = pick_b ? eb1 : ea1;
        e0 += __shfl_xor_sync(0xffffffffu, pick_b ? ea0 : eb0, 16);
        e1 += __shfl_xor_sync(0xffffffffu, pick_b ? ea1 : eb1, 16);
        float e = pick_1 ? e1 : e0;
        e += __shfl_xor_sync(0xffffffffu, pick_1 ? e0 : e1, 8);
        e += __shfl_xor_sync(0xffffffffu, e, 4);
        const int lp = pick_b ? lpB : lpA;
        if ((lane & 4) == 0 && lp >= 0 && lse_head < G) lse_row[lp] = (pick_1 ? mn1 : mn0) - kShift + log2_approx(e);
    };
    auto store_logits = [&](const float (&sc)[4], int lp) {      // HEAD_MAX scoring
        float* lg = p.logits + (size_t(b) * Hq + h0) * (size_t(p.max_pages) * kPage) + size_t(lp) * kPage;
        const size_t hs = size_t(p.max_pages) * kPage;
        if (2 * t4 < G) { lg[2 * t4 * hs + g4] = sc[0]; lg[2 * t4 * hs + g4 + 8] = sc[2]; }
        if (2 * t4 + 1 < G) { lg[(2 * t4 + 1) * hs + g4] = sc[1]; lg[(2 * t4 + 1) * hs + g4 + 8] = sc[3]; }
    };
    // Tile pair c (dimensions 32 c .. 32 c + 31) of V^T . P^T of the page in stage s, added to d0 and d1.
    using Probs = uint32_t[kTwin ? 2 : 4];
    auto pv_tile = [&](int s, int c, const Probs& pt, float (&d0)[4], float (&d1)[4]) {
        uint32_t r0, r1, r2, r3, a0, a1, a2, a3;
        ldmatrix_x4_trans(st0 + uint32_t(s) * S::kPage2 + S::kBlock + off[c], r0, r1, r2, r3);
        H::apart(r0, a0, a1);
        H::apart(r1, a2, a3);
        mma_f16_16816(d0, a0, a1, a2, a3, pt[0], pt[1]);
        if constexpr (!kTwin) mma_f16_16816(d0, a0, a1, a2, a3, pt[2], pt[3]);
        H::apart(r2, a0, a1);
        H::apart(r3, a2, a3);
        mma_f16_16816(d1, a0, a1, a2, a3, pt[0], pt[1]);
        if constexpr (!kTwin) mma_f16_16816(d1, a0, a1, a2, a3, pt[2], pt[3]);
    };
    // The probabilities of a page, weighted, as P^T fragments: the fp16 value and what it leaves, rounded again.  Up to
    // four heads leave half of the eight columns free: the heads' twins in columns 4..7 carry the second values
    // through the same products (joined at the end); more heads take a second product.  w0, w1: of heads 2 t4, 2 t4 + 1.
    auto round_p = [&](const float (&e)[4], float w0, float w1, Probs& pt) {
        const float x[4] = {e[0] * w0, e[1] * w1, e[2] * w0, e[3] * w1};
        const uint32_t x0 = pack_f16(x[0], x[1]), x1 = pack_f16(x[2], x[3]);
        const float2 r0 = unpack_f16(x0), r1 = unpack_f16(x1);
        const uint32_t y0 = pack_f16(x[0] - r0.x, x[1] - r0.y), y1 = pack_f16(x[2] - r1.x, x[3] - r1.y);
        if constexpr (kTwin) {
            pt[0] = movmatrix_trans(t4 < 2 ? x0 : y0);
            pt[1] = movmatrix_trans(t4 < 2 ? x1 : y1);
        } else {
            pt[0] = movmatrix_trans(x0);
            pt[1] = movmatrix_trans(x1);
            pt[2] = movmatrix_trans(y0);
            pt[3] = movmatrix_trans(y1);
        }
    };
    // A page whose V scale does not go with the accumulators' unit (the largest scale so far): a larger one, which
    // becomes the unit, or one below 2^-6 of it (or NaN).  Its product is scaled in fp32, and the probabilities of each
    // head by the power of two that brings the page's largest to [2^14, 2^15): they keep 22 bits down to 2^-16 of it,
    // however small the page's weight is next to the reference (large values may make up for it).
    auto pv_rescaled = [&](int s, const float (&e)[4], float vs) {
        if (!(fabsf(vs) <= vref)) {
            const float r = vref / fabsf(vs);
            vref = fabsf(vs);
            vinv = 1.f / vref;
#pragma unroll
            for (int mt = 0; mt < KS; ++mt)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[mt][j] *= r;
        }
        float top[2] = {fmaxf(e[0], e[2]), fmaxf(e[1], e[3])}, up[2], down[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], o));
            const uint32_t x = max((__float_as_uint(top[j]) >> 23) & 0xffu, 27u);     // 2^(x - 127) <= top, from 2^-100
            up[j] = __uint_as_float((127u + 14u + 127u - x) << 23);
            down[j] = vs / vref * __uint_as_float((x - 14u) << 23);
        }
        Probs pt;
        round_p(e, up[0], up[1], pt);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float d0[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f};
            pv_tile(s, c, pt, d0, d1);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[2 * c][j] = fmaf(d0[j], down[j & 1], acc[2 * c][j]);
                acc[2 * c + 1][j] = fmaf(d1[j], down[j & 1], acc[2 * c + 1][j]);
            }
        }
    };

    const uint32_t parity0 = parity;
    int sA = 0;               // stage of page k: k % STAGES
    for (int k = 0; k < nk; k += 2) {
        advance(k);
        const bool two = k + 1 < nk;
        const int sB = sA + 1 == STAGES ? 0 : sA + 1;
        const uint32_t parity_b = sB == 0 ? parity ^ 1u : parity;
        if (!mbar_wait(&wbar[sA], parity) || (two && !mbar_wait(&wbar[sB], parity_b))) {
            if (lane == 0) atomicOr(p.err, kErrTimeout);
            failed = true;
            break;
        }
        consumed = k + (two ? 2 : 1);
        const int src = k & 31;      // k is even: both pages are in chunk a
        const int lpA = __shfl_sync(0xffffffffu, pages.lp_a, src);
        const float ksA = __shfl_sync(0xffffffffu, pages.ks_a, src), vsA = __shfl_sync(0xffffffffu, pages.vs_a, src);
        const int lpB = two ? __shfl_sync(0xffffffffu, pages.lp_a, src + 1) : -1;
        const float ksB = __shfl_sync(0xffffffffu, pages.ks_a, src + 1), vsB = __shfl_sync(0xffffffffu, pages.vs_a, src + 1);
        const bool vA = lpA >= 0, vB = lpB >= 0;
        if (vA || vB) {
            // a page that is skipped, or missing behind the last, is stood in for by the other with weights of 0
            const int pA = vA ? sA : sB, pB = vB ? sB : sA;
            const float kA = vA ? ksA : ksB, kB = vB ? ksB : ksA, wA = vA ? vsA : vsB, wB = vB ? vsB : vsA;
            float scA[4], scB[4];
            {
                Sum a0[4] = {0, 0, 0, 0}, a1[4] = {0, 0, 0, 0}, a2[4] = {0, 0, 0, 0};
                Sum b0[4] = {0, 0, 0, 0}, b1[4] = {0, 0, 0, 0}, b2[4] = {0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    qk_chunk(pA, c, a0, a1, a2);
                    qk_chunk(pB, c, b0, b1, b2);
                }
                logits_of(a0, a1, a2, kA, vA ? lpA : lpB, pA, scA);
                logits_of(b0, b1, b2, kB, vB ? lpB : lpA, pB, scB);
            }
            if (!vA) scA[0] = scA[1] = scA[2] = scA[3] = -INFINITY;
            if (!vB) scB[0] = scB[1] = scB[2] = scB[3] = -INFINITY;
            if (p.logits != nullptr) {
                if (vA) store_logits(scA, lpA);
                if (vB) store_logits(scB, lpB);
            }
            float mx0 = fmaxf(fmaxf(scA[0], scA[2]), fmaxf(scB[0], scB[2]));
            float mx1 = fmaxf(fmaxf(scA[1], scA[3]), fmaxf(scB[1], scB[3]));
            // The reference m need not be the maximum, only so near it that 2^(s - m + 14) fits fp16 (below 2^16):
            // it moves when a logit passes it by more than 1, rarely after a few pages.  (NaN logits never do;
            // their sums are NaN.)
            if (__any_sync(0xffffffffu, mx0 > m_run[0] + 1.f || mx1 > m_run[1] + 1.f)) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
                    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
                }
                const float m0 = fmaxf(m_run[0], mx0), m1 = fmaxf(m_run[1], mx1);
                const float al0 = exp2_approx(m_run[0] - m0), al1 = exp2_approx(m_run[1] - m1);
                m_run[0] = m0;
                m_run[1] = m1;
                l_run[0] *= al0;
                l_run[1] *= al1;
#pragma unroll
                for (int mt = 0; mt < KS; ++mt) {
                    acc[mt][0] *= al0;
                    acc[mt][1] *= al1;
                    acc[mt][2] *= al0;
                    acc[mt][3] *= al1;
                }
            }
            const float mn0 = m_run[0], mn1 = m_run[1];
            const float u0 = kShift - mn0, u1 = kShift - mn1;
            const float pa[4] = {exp2_approx(scA[0] + u0), exp2_approx(scA[1] + u1), exp2_approx(scA[2] + u0),
                                 exp2_approx(scA[3] + u1)};
            const float pb[4] = {exp2_approx(scB[0] + u0), exp2_approx(scB[1] + u1), exp2_approx(scB[2] + u0),
                                 exp2_approx(scB[3] + u1)};
            l_run[0] += (pa[0] + pa[2]) + (pb[0] + pb[2]);
            l_run[1] += (pa[1] + pa[3]) + (pb[1] + pb[3]);
            if (p.mode == kModeDelta) page_partials(pa, pb, mn0, mn1, lpA, lpB);
            // A page's V scale in the accumulators' unit goes into its probabilities: a power of two of at least 2^-6, so p keeps
            // 22 bits down to 2^-10 of the largest, and what is lost below (2^-33 of the largest, in the page's own V
            // scale) adds up to an fp32 rounding over some thousand tokens a warp.
            constexpr float kFold = 0.015625f;
            const float rA = wA * vinv, rB = wB * vinv;
            if (rA <= 1.f && rA >= kFold && rB <= 1.f && rB >= kFold) {
                Probs ptA, ptB;
                round_p(pa, rA, rA, ptA);
                round_p(pb, rB, rB, ptB);
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    pv_tile(pA, c, ptA, acc[2 * c], acc[2 * c + 1]);
                    pv_tile(pB, c, ptB, acc[2 * c], acc[2 * c + 1]);
                }
            } else {
                pv_rescaled(pA, pa, wA);
                pv_rescaled(pB, pb, wB);
            }
        }
        __syncwarp();
        if (k + STAGES < nk) {
            const int ph0 = phys_at(k + STAGES), ph1 = phys_at(k + STAGES + 1);
            if (lane == 0) {
                copy_page(ph0, sA);
                if (k + STAGES + 1 < nk) copy_page(ph1, sB);
            }
        }
        sA = sB + 1 == STAGES ? 0 : sB + 1;
        parity = sA == 0 ? parity_b ^ 1u : parity_b;
    }
    if (failed) {
        // drain this warp's copies still in flight (bounded) before shared memory is released
        for (int k = consumed + 1; k < min(consumed + STAGES, nk); ++k)
            mbar_wait(&wbar[k % STAGES], parity0 ^ ((k / STAGES) & 1));
    }
    const float unit = vref * kUnshift;      // of the accumulators
    if constexpr (kTwin) {
#pragma unroll
        for (int mt = 0; mt < KS; ++mt)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[mt][j] += __shfl_xor_sync(0xffffffffu, acc[mt][j], 2);
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            l_run[j] += __shfl_xor_sync(0xffffffffu, l_run[j], o);
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if (l_run[j] == 0.f) m_run[j] = -INFINITY;   // no token (a token at the reference weighs 2^13 or more)

    // ---- this warp's state into its own stage area, then the merge of the CTA's warps and of the splits
    __syncwarp();
    constexpr int kRow = D + 4;
    float* po = reinterpret_cast<float*>(wst);           // [8][D + 4] outputs
    float* pml = po + kMaxGroup * kRow;                   // [8][2] (max, sum)
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) {
        const int d = mt * 16 + 2 * g4;
        *reinterpret_cast<float2*>(po + (2 * t4) * kRow + d) = make_float2(acc[mt][0] * unit, acc[mt][2] * unit);
        *reinterpret_cast<float2*>(po + (2 * t4 + 1) * kRow + d) = make_float2(acc[mt][1] * unit, acc[mt][3] * unit);
    }
    if (g4 == 0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            pml[(2 * t4 + j) * 2] = m_run[j];
            pml[(2 * t4 + j) * 2 + 1] = l_run[j] * kUnshift;
        }
    }
    __syncthreads();
    constexpr int kPart = STAGES * int(S::kPage2) / 4;    // floats between two warps' records
    const float* mo0 = reinterpret_cast<const float*>(smem);
    float pre[2][G];   // delta-layers: this CTA's page terms, loaded before the merge
    if (p.fuse_select) select_preload<WARPS * 32, G>(p, b, g, ex.N, pre);
    merge_epilogue<T, D, G, WARPS, WARPS * 32, kRow>(
        p, smem, mo0, mo0 + kMaxGroup * kRow, recv, b, g, kPart, kPart);
    if (p.fuse_select) select_tail<WARPS * 32, G, D>(p, smem, S::kStages, recv, b, g, ex.n, ex.N, pre);
}

}  // namespace delta
