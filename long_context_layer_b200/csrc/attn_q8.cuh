// Kernel variants and launches of the 8-bit decode kernel for one payload format (included by one
// translation unit per format), and what the entry points see of them.
#pragma once

#include "host.cuh"

namespace delta {

// 6-warp CTAs, two an SM (kVarNarrow), or, bf16 queries, one 12-warp CTA an SM (kVarWide); a warp's ring holds
// 16 KB of pages (two pairs of pages of head_dim 128).
constexpr int kQ8Warps = 6, kQ8WideWarps = 12;
constexpr int q8_stages(int D) { return 512 / D; }

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
