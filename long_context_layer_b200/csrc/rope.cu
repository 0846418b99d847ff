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
// Rows a block takes when there are many, and vectors a thread has in flight: 8 and 4 rotate 32,768 rows of 32 +
// 8 heads of 128 (671 MB moved) in 105 us, 6.4 TB/s; 4 rows 131 us, 2 vectors 127 us, both without the
// streaming loads and stores, which gave 124 -> 105 us.
constexpr int kRopeRows = 8;
constexpr int kRopeBatch = 4;

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
    uint32_t magic[2];            // ceil(2^32 / heads): i / heads = i * magic >> 32 for i * heads < 2^32
};

template <typename T, int V>
struct __align__(sizeof(T) * V) RopeVec {
    T v[V];
};

// Rows are read once and written once: evict-first in the caches.
template <typename Vec>
__device__ __forceinline__ Vec rope_load(const void* p) {
    if constexpr (sizeof(Vec) == 16) {
        const uint4 w = __ldcs(static_cast<const uint4*>(p));
        return *reinterpret_cast<const Vec*>(&w);
    } else {
        return *static_cast<const Vec*>(p);
    }
}
template <typename Vec>
__device__ __forceinline__ void rope_store(void* p, const Vec& v) {
    if constexpr (sizeof(Vec) == 16) __stcs(static_cast<uint4*>(p), *reinterpret_cast<const uint4*>(&v));
    else *static_cast<Vec*>(p) = v;
}

// A head's work items: `rot` vectors of pairs (V pairs in two vectors rotary_dim/2 apart, HALF; V / 2 adjacent
// pairs; one pair where V is 1: odd widths), then, unless in place, vectors that pass through.  A thread keeps
// one item u and walks over the (row, head) list, kRopeBatch of them in flight.
template <typename T, bool HALF, int V>
__device__ __forceinline__ void rope_rows(const RopeParams& p, const float2 (*cs)[64], const T* x, T* y, int64_t xs,
                                          int64_t ys, int heads, uint32_t magic, int64_t r0, int nr) {
    using Vec = RopeVec<T, V>;
    const int pairs = p.rotary_dim / 2;
    const int rot = HALF ? pairs / V : (V == 1 ? pairs : p.rotary_dim / V);
    const int items = rot + (x == y ? 0 : (p.head_dim - p.rotary_dim) / V);
    if (items == 0) return;
    const int slots = kRopeThreads / items, n = nr * heads;      // items <= head_dim <= 128
    const int slot = threadIdx.x / items, u = threadIdx.x - slot * items;
    if (slot >= slots) return;
    const bool pass = u >= rot;
    // offsets of the item's one or two vectors
    const int d0 = pass ? p.rotary_dim + (u - rot) * V : HALF || V > 1 ? u * V : 2 * u;
    const int d1 = HALF ? d0 + pairs : d0 + 1;
    constexpr bool kSecond = HALF || V == 1;
    for (int i0 = slot; i0 < n; i0 += kRopeBatch * slots) {
        Vec a[kRopeBatch], b[kSecond ? kRopeBatch : 1];
        int row[kRopeBatch], head[kRopeBatch];
#pragma unroll
        for (int k = 0; k < kRopeBatch; ++k) {
            const int i = i0 + k * slots;
            row[k] = heads == 1 ? i : int(__umulhi(uint32_t(i), magic));
            head[k] = i - row[k] * heads;
            if (i >= n) continue;
            const T* src = x + (r0 + row[k]) * xs + head[k] * p.head_dim;
            a[k] = rope_load<Vec>(src + d0);
            if constexpr (kSecond) {
                if (!pass) b[k] = rope_load<Vec>(src + d1);
            }
        }
#pragma unroll
        for (int k = 0; k < kRopeBatch; ++k) {
            if (i0 + k * slots >= n) continue;
            T* dst = y + (r0 + row[k]) * ys + head[k] * p.head_dim;
            if (!pass) {
                const float2* t = cs[row[k]] + (HALF || V == 1 ? u * V : u * V / 2);
                if constexpr (kSecond) {
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float fa = Elem<T>::to_f(a[k].v[j]), fb = Elem<T>::to_f(b[k].v[j]);
                        a[k].v[j] = Elem<T>::from_f(fa * t[j].x - fb * t[j].y);
                        b[k].v[j] = Elem<T>::from_f(fb * t[j].x + fa * t[j].y);
                    }
                    rope_store(dst + d1, b[k]);
                } else {
#pragma unroll
                    for (int j = 0; j < V; j += 2) {
                        const float fa = Elem<T>::to_f(a[k].v[j]), fb = Elem<T>::to_f(a[k].v[j + 1]);
                        a[k].v[j] = Elem<T>::from_f(fa * t[j / 2].x - fb * t[j / 2].y);
                        a[k].v[j + 1] = Elem<T>::from_f(fb * t[j / 2].x + fa * t[j / 2].y);
                    }
                }
            }
            rope_store(dst + d0, a[k]);
        }
    }
}

// One block: the (cos, sin) * magnitude of its rows' pairs, then the rows' heads.
template <typename T, bool HALF, int V>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p, int rows_per_block) {
    __shared__ __align__(16) float2 cs[kRopeRows][64];
    const int pairs = p.rotary_dim / 2;
    const int64_t r0 = int64_t(blockIdx.x) * rows_per_block;
    const int nr = int(min(int64_t(rows_per_block), p.rows - r0));
    // the table is set up once by the caller; positions may be another kernel's output
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int i = threadIdx.x; i < nr * pairs; i += kRopeThreads) {
        const int r = i / pairs, j = i - r * pairs;
        const int64_t row = r0 + r;
        const int32_t at = row < p.num_positions ? int32_t(row) : int32_t(row % p.num_positions);
        const int64_t pos = int64_t(p.positions[at]) + p.offset;
        const double t = double(pos) * p.turns[j];
        float s, c;
        sincospif(2.0f * float(t - rint(t)), &s, &c);
        cs[r][j] = make_float2(c * p.magnitude, s * p.magnitude);
    }
    __syncthreads();
    if (p.x[0] != nullptr)
        rope_rows<T, HALF, V>(p, cs, static_cast<const T*>(p.x[0]), static_cast<T*>(p.y[0]), p.xs[0], p.ys[0], p.heads[0],
                              p.magic[0], r0, nr);
    if (p.x[1] != nullptr)
        rope_rows<T, HALF, V>(p, cs, static_cast<const T*>(p.x[1]), static_cast<T*>(p.y[1]), p.xs[1], p.ys[1], p.heads[1],
                              p.magic[1], r0, nr);
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
        p.magic[i] = uint32_t((0x100000000ull + p.heads[i] - 1) / p.heads[i]);
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
