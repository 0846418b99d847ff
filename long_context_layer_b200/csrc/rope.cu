// Rotary positions of q and k.
//
// Pair j of a head turns by the angle 2 pi * position * turns[j].  Far positions make the product large, so
// it is formed in double precision and reduced to a fraction of a turn before it is rounded to float; what
// is left is at most half a turn, whose sine and cosine are accurate to a few float ulps at any position.
//
// Bound: HBM, one read and one write of the rows (arithmetic: 3 flops a value and one sine and cosine per
// (row, pair), shared by all heads of the row through shared memory).

#include "host.cuh"

namespace delta {

constexpr int kRopeThreads = 256;
constexpr int kRopeRows = 4;      // rows a block takes when there are many

struct RopeParams {
    const double* turns;
    const int32_t* positions;
    int32_t num_positions, offset, rotary_dim, head_dim;
    float magnitude;
    int64_t rows;
    const void* x[2];             // q, k
    void* y[2];
    int64_t xs[2], ys[2];         // row strides in elements
    int32_t heads[2];
};

template <typename T, int V>
struct __align__(sizeof(T) * V) RopeVec {
    T v[V];
};

// One row's (cos, sin) * magnitude of every pair, then its heads: a work item is the V pairs that a vector
// (or, HALF, two vectors rotary_dim/2 apart) holds, or V values that pass through.  V = 1: odd sizes.
template <typename T, bool HALF, int V>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p, int rows_per_block) {
    __shared__ float2 cs[kRopeRows][64];
    const int pairs = p.rotary_dim / 2;
    const int64_t r0 = int64_t(blockIdx.x) * rows_per_block;
    const int nr = int(min(int64_t(rows_per_block), p.rows - r0));
    // the table is set up once by the caller; positions may be another kernel's output
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int i = threadIdx.x; i < nr * pairs; i += kRopeThreads) {
        const int r = i / pairs, j = i - r * pairs;
        const int64_t pos = int64_t(p.positions[(r0 + r) % p.num_positions]) + p.offset;
        const double t = double(pos) * p.turns[j];
        float s, c;
        sincospif(2.0f * float(t - rint(t)), &s, &c);
        cs[r][j] = make_float2(c * p.magnitude, s * p.magnitude);
    }
    __syncthreads();
    // items of a head: rotated, then (unless in place) copied ones
    const int rot = HALF ? pairs / V : (V == 1 ? pairs : p.rotary_dim / V);
    const int rest = (p.head_dim - p.rotary_dim) / V;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        if (p.x[which] == nullptr) continue;
        const bool same = p.x[which] == p.y[which];
        const int items = rot + (same ? 0 : rest);
        const int per_row = p.heads[which] * items;
        for (int i = threadIdx.x; i < nr * per_row; i += kRopeThreads) {
            const int r = i / per_row;
            const int in_row = i - r * per_row;
            const int h = in_row / items, u = in_row - h * items;
            const T* x = static_cast<const T*>(p.x[which]) + (r0 + r) * p.xs[which] + int64_t(h) * p.head_dim;
            T* y = static_cast<T*>(p.y[which]) + (r0 + r) * p.ys[which] + int64_t(h) * p.head_dim;
            using Vec = RopeVec<T, V>;
            if (u >= rot) {
                const int d = p.rotary_dim + (u - rot) * V;
                *reinterpret_cast<Vec*>(y + d) = *reinterpret_cast<const Vec*>(x + d);
            } else if constexpr (HALF) {
                const int j = u * V;
                Vec a = *reinterpret_cast<const Vec*>(x + j);
                Vec b = *reinterpret_cast<const Vec*>(x + pairs + j);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float2 t = cs[r][j + k];
                    const float fa = Elem<T>::to_f(a.v[k]), fb = Elem<T>::to_f(b.v[k]);
                    a.v[k] = Elem<T>::from_f(fa * t.x - fb * t.y);
                    b.v[k] = Elem<T>::from_f(fb * t.x + fa * t.y);
                }
                *reinterpret_cast<Vec*>(y + j) = a;
                *reinterpret_cast<Vec*>(y + pairs + j) = b;
            } else if constexpr (V == 1) {
                const float2 t = cs[r][u];
                const float fa = Elem<T>::to_f(x[2 * u]), fb = Elem<T>::to_f(x[2 * u + 1]);
                y[2 * u] = Elem<T>::from_f(fa * t.x - fb * t.y);
                y[2 * u + 1] = Elem<T>::from_f(fb * t.x + fa * t.y);
            } else {
                Vec a = *reinterpret_cast<const Vec*>(x + u * V);
#pragma unroll
                for (int k = 0; k < V; k += 2) {
                    const float2 t = cs[r][(u * V + k) / 2];
                    const float fa = Elem<T>::to_f(a.v[k]), fb = Elem<T>::to_f(a.v[k + 1]);
                    a.v[k] = Elem<T>::from_f(fa * t.x - fb * t.y);
                    a.v[k + 1] = Elem<T>::from_f(fb * t.x + fa * t.y);
                }
                *reinterpret_cast<Vec*>(y + u * V) = a;
            }
        }
    }
}

template <typename T>
delta_status launch_rope(const RopeParams& p, bool half, cudaStream_t st) {
    constexpr int V = 16 / int(sizeof(T));
    const int rd = p.rotary_dim;
    const bool wide = half ? (rd / 2) % V == 0 : rd % V == 0;   // every vector whole (head_dim is a multiple of V)
    const int rows = p.rows >= int64_t(device_sm_count()) * 8 * kRopeRows ? kRopeRows : 1;
    const int64_t blocks = (p.rows + rows - 1) / rows;
    if (blocks > INT32_MAX) return DELTA_ERR_UNSUPPORTED;
    const dim3 grid{unsigned(blocks)}, block{kRopeThreads};
    if (half)
        return wide ? launch_pdl(rope_kernel<T, true, V>, grid, block, 0, st, p, rows)
                    : launch_pdl(rope_kernel<T, true, 1>, grid, block, 0, st, p, rows);
    return wide ? launch_pdl(rope_kernel<T, false, V>, grid, block, 0, st, p, rows)
                : launch_pdl(rope_kernel<T, false, 1>, grid, block, 0, st, p, rows);
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
    p.head_dim = desc->head_dim;
    p.magnitude = rope->magnitude;
    p.rows = rows;
    const bool half = rope->layout == DELTA_ROPE_HALF;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return desc->dtype == DELTA_BF16 ? launch_rope<__nv_bfloat16>(p, half, st) : launch_rope<float>(p, half, st);
}

}  // extern "C"
