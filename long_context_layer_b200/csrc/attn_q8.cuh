// Kernel variants and launches of the 8-bit decode kernel for one payload format (included by one
// translation unit per format), and what the entry points see of them.
#pragma once

#include "host.cuh"

namespace delta {

// bf16 queries: 8-warp CTAs, two an SM (kVarNarrow), or one 16-warp CTA an SM (kVarWide); the same pages in
// flight.  fp32 queries carry every fragment twice and keep to 8 warps.
#ifndef Q8_WIDE
#define Q8_WIDE 3
#endif
#ifndef Q8_STAGES
#define Q8_STAGES 3
#endif
constexpr int kQ8Warps = 8, kQ8WideWarps = 16, kQ8Stages = Q8_STAGES;

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
