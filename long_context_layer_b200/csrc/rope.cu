// Rotary positions of q and k.
//
// Pair j of a head turns by the angle 2 pi * position * turns[j].  Far positions make the product large, so
// it is formed in double precision and reduced to a fraction of a turn before it is rounded to float; what
// is left is at most half a turn, whose sine and cosine are accurate to a few float ulps at any position.
//
// Bound: HBM, one read and one write of the rows.  A warp takes a row (or a share of its heads, when there are few
// rows): it forms the row's sines and cosines once, each lane keeps those of the 16 bytes of a head that it
// turns, and then streams heads, four groups in flight.  In the half layout a value's partner lies
// rotary_dim/2 dimensions away, in another lane's 16 bytes (at any offset: widths need not divide): the group
// passes through shared memory, which also makes in-place safe, a group being read whole before it is written.

#include "host.cuh"
#include "q8.cuh"

namespace delta {

// Four groups of heads (512 bytes each) in flight a warp, four blocks an SM (64 registers).  16,384 rows of 32 + 8
// heads of 128 in bf16 (336 MB moved): adjacent pairs 58 us, 5.8 TB/s, at any width; halves 65 us (5.1 TB/s), 76 us
// where the partner's offset is no multiple of 16 bytes; fp32 108 and 112 us (6.2 TB/s).  Two groups 73 us (halves),
// three blocks an SM 70 us; partners by shuffles instead of shared memory 66 and 80 us.
constexpr int kRopeWarps = 8;
constexpr int kRopeBatch = 4;

struct RopeParams {
    const double* turns;
    const int32_t* positions;
    int32_t num_positions, offset, rotary_dim;
    float magnitude;
    int64_t rows;
    int32_t split;                // warps a row is shared by: 1, 2, 4 or 8
    const void* x[2];             // q, k
    void* y[2];
    int64_t xs[2], ys[2];         // row strides in elements
    int32_t heads[2];
};

__device__ __forceinline__ uint32_t rope_bf16x2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint4 pack16(const float (&x)[8]) {
    uint4 w;
    w.x = rope_bf16x2(x[0], x[1]);
    w.y = rope_bf16x2(x[2], x[3]);
    w.z = rope_bf16x2(x[4], x[5]);
    w.w = rope_bf16x2(x[6], x[7]);
    return w;
}
__device__ __forceinline__ uint4 pack16(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}

template <typename T, int D, bool HALF>
__global__ void __launch_bounds__(kRopeWarps * 32, 4) rope_kernel(const RopeParams p) {
    constexpr int V = Raw16<T>::N, U = D / V, HP = 32 / U;   // values a lane, lanes a head, heads a group
    constexpr int TV = HALF ? V : V / 2;                     // sines and cosines a lane
    __shared__ float2 table[kRopeWarps][D / 2];
    __shared__ uint4 swap[HALF ? kRopeWarps : 1][kRopeBatch][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t at = int64_t(blockIdx.x) * kRopeWarps + warp;
    const int64_t row = at / p.split;
    const int part = int(at - row * p.split);
    const int rd = p.rotary_dim, pairs = rd / 2;
    // the table of turns is set up once by the caller; positions may be another kernel's output
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (row >= p.rows) return;
    {
        const int64_t pos = int64_t(p.positions[row < p.num_positions ? row : row % p.num_positions]) + p.offset;
        for (int j = lane; j < pairs; j += 32) {
            const double t = double(pos) * p.turns[j];
            float s, c;
            sincospif(2.0f * float(t - rint(t)), &s, &c);
            table[warp][j] = make_float2(c * p.magnitude, s * p.magnitude);
        }
        __syncwarp();
    }
    const int sub = lane / U, u = lane % U, d0 = u * V;      // the lane's head in a group and its dimensions
    const bool turned = d0 < rd;                             // (some of them)
    float cs[TV], sn[TV];
#pragma unroll
    for (int i = 0; i < TV; ++i) {
        const int d = HALF ? d0 + i : d0 + 2 * i;
        const bool first = d < pairs;
        const int j = HALF ? (first ? d : d - pairs) : d / 2;
        // a value that passes through is x * 1 + 0 * -0: itself, its sign of zero too
        const float2 t = d < rd ? table[warp][j] : make_float2(1.f, -0.f);
        cs[i] = t.x;
        sn[i] = HALF && d < rd && first ? -t.y : t.y;
    }
    const bool whole = HALF && pairs % V == 0;      // a lane's partners are one other lane's values
    const int lane2 = sub * U + (!turned ? u : (d0 < pairs ? d0 + pairs : d0 - pairs) / V);
    const int groups_q = p.x[0] == nullptr ? 0 : (p.heads[0] + HP - 1) / HP;
    const int groups = groups_q + (p.x[1] == nullptr ? 0 : (p.heads[1] + HP - 1) / HP);
    const bool pass_q = p.x[0] != p.y[0], pass_k = p.x[1] != p.y[1];     // out of place: the rest is copied
    for (int g0 = part; g0 < groups; g0 += p.split * kRopeBatch) {
        uint4 raw[kRopeBatch];
        uint32_t live = 0;
#pragma unroll
        for (int k = 0; k < kRopeBatch; ++k) {
            const int g = g0 + k * p.split;
            const bool is_k = g >= groups_q;
            const int head = (is_k ? g - groups_q : g) * HP + sub;
            raw[k] = make_uint4(0, 0, 0, 0);
            if (g < groups && head < (is_k ? p.heads[1] : p.heads[0]) && (turned || (is_k ? pass_k : pass_q))) {
                const T* x = static_cast<const T*>(is_k ? p.x[1] : p.x[0]) + row * (is_k ? p.xs[1] : p.xs[0]);
                raw[k] = __ldcs(reinterpret_cast<const uint4*>(x + head * D + d0));
                live |= 1u << k;
            }
        }
        if constexpr (HALF) {
#pragma unroll
            for (int k = 0; k < kRopeBatch; ++k) swap[warp][k][lane] = raw[k];
            __syncwarp();
        }
#pragma unroll
        for (int k = 0; k < kRopeBatch; ++k) {
            if (!((live >> k) & 1u)) continue;
            uint4 out = raw[k];
            if (turned) {
                float x[V], r[V];
                Raw16<T>::get(out, x);
                if constexpr (HALF) {
                    float other[V];
                    if (whole) {
                        Raw16<T>::get(swap[warp][k][lane2], other);
                    } else {
                        const T* head = reinterpret_cast<const T*>(&swap[warp][k][sub * U]);
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            const int d = d0 + i;
                            other[i] = d < rd ? Elem<T>::to_f(head[d < pairs ? d + pairs : d - pairs]) : 0.f;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < V; ++i) r[i] = fmaf(x[i], cs[i], other[i] * sn[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < V; i += 2) {
                        const bool in = d0 + i < rd;
                        r[i] = in ? x[i] * cs[i / 2] - x[i + 1] * sn[i / 2] : x[i];
                        r[i + 1] = in ? x[i + 1] * cs[i / 2] + x[i] * sn[i / 2] : x[i + 1];
                    }
                }
                out = pack16(r);
            }
            const int g = g0 + k * p.split;
            const bool is_k = g >= groups_q;
            const int head = (is_k ? g - groups_q : g) * HP + sub;
            T* y = static_cast<T*>(is_k ? p.y[1] : p.y[0]) + row * (is_k ? p.ys[1] : p.ys[0]);
            __stcs(reinterpret_cast<uint4*>(y + head * D + d0), out);
        }
        if constexpr (HALF) __syncwarp();      // the next groups overwrite the swapped ones
    }
}

template <typename T, int D>
delta_status launch_rope(RopeParams p, bool half, cudaStream_t st) {
    p.split = 1;
    while (p.split < 8 && p.rows * p.split * 2 <= int64_t(device_sm_count()) * 32) p.split *= 2;
    const int64_t blocks = (p.rows * p.split + kRopeWarps - 1) / kRopeWarps;
    if (blocks > INT32_MAX) return DELTA_ERR_UNSUPPORTED;
    const dim3 grid{unsigned(blocks)}, block{kRopeWarps * 32};
    return half ? launch_pdl(rope_kernel<T, D, true>, grid, block, 0, st, p)
                : launch_pdl(rope_kernel<T, D, false>, grid, block, 0, st, p);
}

}  // namespace delta

using namespace delta;

extern "C" {

delta_status delta_rope_table(const delta_rope_params* params, double* turns_out) {
    if (params == nullptr || turns_out == nullptr) return DELTA_ERR_INVALID_ARG;
    const delta_rope_params& a = *params;
    if (a.rotary_dim < 2 || a.rotary_dim % 2 != 0 || a.rotary_dim > 4096) return DELTA_ERR_INVALID_ARG;
    if (!(a.base > 1.0) || isinf(a.base)) return DELTA_ERR_INVALID_ARG;
    if (a.scaling != DELTA_ROPE_PLAIN && a.scaling != DELTA_ROPE_LINEAR && a.scaling != DELTA_ROPE_BANDS)
        return DELTA_ERR_INVALID_ARG;
    if (a.scaling != DELTA_ROPE_PLAIN && (!(a.factor >= 1.0) || isinf(a.factor))) return DELTA_ERR_INVALID_ARG;
    if (a.scaling == DELTA_ROPE_BANDS &&
        (!(a.original_len > 0.0) || isinf(a.original_len) || !(a.low_turns >= 0.0) || !(a.high_turns > a.low_turns) ||
         isinf(a.high_turns)))
        return DELTA_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925;
    for (int32_t j = 0; j < a.rotary_dim / 2; ++j) {
        const double f = pow(a.base, -2.0 * j / a.rotary_dim) / two_pi;
        double t = f;
        if (a.scaling == DELTA_ROPE_LINEAR) t = f / a.factor;
        if (a.scaling == DELTA_ROPE_BANDS) {
            double w = (f * a.original_len - a.low_turns) / (a.high_turns - a.low_turns);
            w = w < 0.0 ? 0.0 : (w > 1.0 ? 1.0 : w);
            t = w * f + (1.0 - w) * f / a.factor;
        }
        turns_out[j] = t;
    }
    return DELTA_OK;
}

delta_status delta_rope(const delta_desc* desc, const delta_rope_plan* rope, int64_t rows, const void* q,
                        int64_t q_stride, void* q_out, int64_t q_out_stride, const void* k, int64_t k_stride,
                        void* k_out, int64_t k_out_stride, void* stream) {
    delta_status s = check_desc(desc);
    if (s != DELTA_OK) return s;
    if (rope == nullptr || rows < 0) return DELTA_ERR_INVALID_ARG;
    if (rope->rotary_dim < 2 || rope->rotary_dim % 2 != 0 || rope->rotary_dim > desc->head_dim) return DELTA_ERR_INVALID_ARG;
    if (rope->layout != DELTA_ROPE_HALF && rope->layout != DELTA_ROPE_INTERLEAVED) return DELTA_ERR_INVALID_ARG;
    if (!isfinite(rope->magnitude)) return DELTA_ERR_INVALID_ARG;
    if ((q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_out == nullptr)) return DELTA_ERR_INVALID_ARG;
    RopeParams p{};
    const int V = 16 / elem_bytes(desc->dtype);
    p.heads[0] = desc->num_q_heads;
    p.heads[1] = desc->num_kv_heads;
    p.x[0] = q;
    p.x[1] = k;
    p.y[0] = q_out;
    p.y[1] = k_out;
    const int64_t xs[2] = {q_stride, k_stride}, ys[2] = {q_out_stride, k_out_stride};
    for (int i = 0; i < 2; ++i) {
        const int64_t row = int64_t(p.heads[i]) * desc->head_dim;
        p.xs[i] = xs[i] == 0 ? row : xs[i];
        p.ys[i] = ys[i] == 0 ? row : ys[i];
        if (p.x[i] == nullptr) continue;
        if (p.xs[i] < row || p.ys[i] < row || p.xs[i] % V != 0 || p.ys[i] % V != 0) return DELTA_ERR_INVALID_ARG;
        if (!aligned16(p.x[i]) || !aligned16(p.y[i])) return DELTA_ERR_INVALID_ARG;
        if (p.x[i] == p.y[i] && p.xs[i] != p.ys[i]) return DELTA_ERR_INVALID_ARG;
    }
    if (rows == 0 || (q == nullptr && k == nullptr)) return DELTA_OK;
    if (rope->turns == nullptr || rope->positions == nullptr || rope->num_positions < 1) return DELTA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(rope->turns) & 7u) != 0) return DELTA_ERR_INVALID_ARG;
    p.turns = rope->turns;
    p.positions = rope->positions;
    p.num_positions = rope->num_positions;
    p.offset = rope->offset;
    p.rotary_dim = rope->rotary_dim;
    p.magnitude = rope->magnitude;
    p.rows = rows;
    const bool half = rope->layout == DELTA_ROPE_HALF;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (desc->dtype == DELTA_BF16)
        return desc->head_dim == 128 ? launch_rope<__nv_bfloat16, 128>(p, half, st) : launch_rope<__nv_bfloat16, 64>(p, half, st);
    return desc->head_dim == 128 ? launch_rope<float, 128>(p, half, st) : launch_rope<float, 64>(p, half, st);
}

}  // extern "C"
