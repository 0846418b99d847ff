// Kernel variants and launches of the 8-bit decode kernel for one payload format (included by one
// translation unit per format), and what the entry points see of them.
#pragma once

#include "host.cuh"

namespace delta {

// Narrow CTAs, two an SM (kVarNarrow), or, bf16 queries, one CTA of twice the warps an SM (kVarWide).  A warp's ring
// holds 4 pages: while a pair of pages is worked on, the next pair is on its way.  head_dim 128: 6 warps, 96 KB a
// CTA (8 warps with 3 pages: 16 x 16k full layer 97 instead of 84 us, sparse 22 instead of 19).  head_dim 64: the
// pages are half as large for nearly the same work, so 8 warps (16 x 16k full layer 58 us; 6 warps with 8 pages
// 66, 10 warps 76).
constexpr int q8_warps(int D, bool wide) { return (D == 128 ? 6 : 8) * (wide ? 2 : 1); }
constexpr int kQ8Stages = 4;

struct Q8Kernel {
    const void* fn;
    size_t smem;
    int threads;
};
template <int FMT>
Q8Kernel q8_kernel(int dtype, int D, int G, int variant);
template <int FMT>
delta_status q8_launch(const delta_desc* d, const DecodeParams& prm, const CUtensorMap& mk, const CUtensorMap& mv,
                       const SplitPlan& plan, int batch, cudaStream_t st);

}  // namespace delta
