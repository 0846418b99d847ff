// Instantiations of the 8-bit decode kernel for the payload format DELTA_Q8_FMT.
#include "attn_q8.cuh"
#include "decode_q8.cuh"

namespace delta {

namespace {

template <typename T, int D, int G, int WARPS>
Q8Kernel entry() {
    return {reinterpret_cast<const void*>(decode_q8_kernel<T, DELTA_Q8_FMT, D, G, kQ8Stages, WARPS>),
            Q8Smem<D, kQ8Stages, WARPS>::kBytes, WARPS * 32};
}
template <int D, int G>
Q8Kernel by_variant(int dtype, int variant) {
    if (dtype == DELTA_F32) return entry<float, D, G, q8_warps(D, false)>();
    return variant == kVarWide ? entry<__nv_bfloat16, D, G, q8_warps(D, true)>()
                               : entry<__nv_bfloat16, D, G, q8_warps(D, false)>();
}
template <int D>
Q8Kernel by_group(int dtype, int G, int variant) {
    switch (G) {
        case 1: return by_variant<D, 1>(dtype, variant);
        case 2: return by_variant<D, 2>(dtype, variant);
        case 3: return by_variant<D, 3>(dtype, variant);
        case 4: return by_variant<D, 4>(dtype, variant);
        case 5: return by_variant<D, 5>(dtype, variant);
        case 6: return by_variant<D, 6>(dtype, variant);
        case 7: return by_variant<D, 7>(dtype, variant);
        case 8: return by_variant<D, 8>(dtype, variant);
        default: return {nullptr, 0, 0};
    }
}

}  // namespace

template <>
Q8Kernel q8_kernel<DELTA_Q8_FMT>(int dtype, int D, int G, int variant) {
    return D == 128 ? by_group<128>(dtype, G, variant) : by_group<64>(dtype, G, variant);
}

template <>
delta_status q8_launch<DELTA_Q8_FMT>(const delta_desc* d, const DecodeParams& prm, const CUtensorMap& mk,
                                     const CUtensorMap& mv, const SplitPlan& plan, int batch, cudaStream_t st) {
    const int Hkv = d->num_kv_heads;
    const Q8Kernel k = q8_kernel<DELTA_Q8_FMT>(d->dtype, d->head_dim, d->num_q_heads / Hkv, plan.variant);
    if (k.fn == nullptr) return DELTA_ERR_UNSUPPORTED;
    using Fn = void (*)(const DecodeParams, const CUtensorMap, const CUtensorMap);
    return launch_clustered(reinterpret_cast<Fn>(const_cast<void*>(k.fn)), k.smem, k.threads, prm, plan.cluster, batch,
                            Hkv, st, mk, mv);
}

}  // namespace delta
