// Writing the 8-bit cache (the tokens of a decode step, or a prompt) and reading it back.
//
// One warp owns one block (page, KV head, K or V), so a block's scale, its older values and its new ones are
// one warp's business: no atomics, no second pass.  The new values are loaded once into registers (16
// bytes a lane and row group), their largest magnitude is one warp reduction, and the payload is written
// once.  Bound: HBM for prompts (bf16: 2 bytes read and 1 written a value); for a decode step, latency.

#include "host.cuh"
#include "q8.cuh"

namespace delta {

// Bulk calls run one-warp blocks: a block of more waits for its slowest warp.  The write of 4 x 16k tokens of 8
// heads takes 65 us (6.2 TB/s; 69 with 2 or 4 warps a block), the read back 71 us (5.7 TB/s; 74).  A warp of a long
// write takes 4 consecutive pages, whose table entries it looks up at once (with two warps a block 69 us, two
// pages a warp 72).  The largest magnitude is taken from the raw bits, two halfwords at a time: 79 -> 69 us.
constexpr int kMaxColumns = 16384;   // grid columns; more pages are strided over
constexpr int kWarpsPerSm = 64;      // warps an SM gets before a warp takes more than one page
constexpr int kMaxChunk = 4;

// The lanes of a warp over rows of D elements of T, 16 bytes a lane.
template <typename T, int D, int ROWS>
struct Rows {
    static constexpr int V = Raw16<T>::N;               // elements of a 16-byte load
    static constexpr int LPR = D / V;                   // lanes a row takes
    static constexpr int RPI = 32 / LPR;                // rows of one pass over the lanes
    static constexpr int ITERS = (ROWS + RPI - 1) / RPI;
};

// Rows [f0, f1) of a block from src (row f0 first, `stride` elements apart); zeros elsewhere.
template <typename T, int D, int ROWS>
__device__ __forceinline__ void load_rows(const T* src, int64_t stride, int f0, int f1, int lane,
                                          uint4 (&raw)[Rows<T, D, ROWS>::ITERS]) {
    using R = Rows<T, D, ROWS>;
    const int r = lane / R::LPR, c = (lane % R::LPR) * R::V;
#pragma unroll
    for (int i = 0; i < R::ITERS; ++i) {
        const int row = f0 + i * R::RPI + r;
        raw[i] = make_uint4(0, 0, 0, 0);
        if (row < f1) raw[i] = *reinterpret_cast<const uint4*>(src + int64_t(row - f0) * stride + c);
    }
}

// Writes those rows into a block and rounds its older rows [0, f0) again when the scale grows.
template <typename T, int D, int FMT, int ROWS>
__device__ __forceinline__ void store_block(const uint4 (&raw)[Rows<T, D, ROWS>::ITERS], int f0, int f1, uint8_t* block,
                                            float* scale, int lane) {
    using R = Rows<T, D, ROWS>;
    constexpr int V = R::V;
    const int r = lane / R::LPR, c = (lane % R::LPR) * V;
    const uint32_t before = f0 > 0 ? __float_as_uint(__ldcg(scale)) & 0x7fffffffu : 0u;
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < R::ITERS; ++i) amax = Raw16<T>::more(amax, raw[i]);
    amax = __reduce_max_sync(0xffffffffu, Raw16<T>::top(amax));
    const uint32_t now = max(before, block_scale_bits<FMT>(amax));
    const bool fine = scale_finite(now);
    const float inv = fine ? scale_inverse(now) : 0.f;
    if (f0 > 0 && now != before && fine) {
        const float ratio = __uint_as_float(before) * inv;      // <= 1/2 and a power of two (a block written elsewhere: < 1)
        for (int i = lane; i < f0 * D / 16; i += 32) {
            uint4* p = reinterpret_cast<uint4*>(block) + i;
            uint4 w = __ldcg(p);
            uint32_t* u = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 lo = unpack8x2<FMT>(u[k]), hi = unpack8x2<FMT>(u[k] >> 16);
                u[k] = pack8x4<FMT>(lo.x * ratio, lo.y * ratio, hi.x * ratio, hi.y * ratio);
            }
            *p = w;
        }
    }
#pragma unroll
    for (int i = 0; i < R::ITERS; ++i) {
        const int row = f0 + i * R::RPI + r;
        if (row >= f1) continue;
        float x[V];
        Raw16<T>::get(raw[i], x);
        uint32_t out[V / 4];
#pragma unroll
        for (int k = 0; k < V; k += 4)
            out[k / 4] = fine ? pack8x4<FMT>(x[k] * inv, x[k + 1] * inv, x[k + 2] * inv, x[k + 3] * inv) : 0u;
        uint8_t* dst = block + row * D + c;
        if constexpr (V == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
        else *reinterpret_cast<uint32_t*>(dst) = out[0];
    }
    if (lane == 0) *scale = __uint_as_float(now);
}

struct Q8Pools {
    uint8_t* pool[2];    // K, V
    float* scale[2];
};
struct AppendQ8Layers {
    const void* k_new[64];
    const void* v_new[64];
    Q8Pools cache[64];
};
static_assert(sizeof(AppendQ8Layers) < 4000, "kernel parameters");

// One appended token of every (sequence, KV head, layer): warp 0 its K, warp 1 its V.
template <typename T, int D, int FMT>
__global__ void __launch_bounds__(64) append_q8_kernel(const __grid_constant__ AppendQ8Layers a,
                                                       const int32_t* __restrict__ indptr,
                                                       const int32_t* __restrict__ indices,
                                                       const int32_t* __restrict__ kv_len, int64_t num_phys_pages) {
    const int b = blockIdx.x, g = blockIdx.y, l = blockIdx.z, Hkv = gridDim.y;
    const int kv = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the page table and kv_len are inputs of the whole step: looked up before the wait
    const int n = kv_len[b];
    const int lp = n > 0 ? (n - 1) / kPage : 0, slot = n > 0 ? (n - 1) % kPage : 0;
    const int pbeg = indptr[b], npg = indptr[b + 1] - pbeg;
    int64_t phys = -1;
    if (n > 0 && lp < npg) phys = indices[pbeg + lp];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (phys < 0 || phys >= num_phys_pages) return;   // flagged by the attention call that follows
    const T* src = static_cast<const T*>(kv ? a.v_new[l] : a.k_new[l]) + (size_t(b) * Hkv + g) * D;
    const size_t block = size_t(phys) * Hkv + g;
    uint4 raw[1];
    load_rows<T, D, 1>(src, 0, slot, slot + 1, lane, raw);
    store_block<T, D, FMT, 1>(raw, slot, slot + 1, (kv ? a.cache[l].pool[1] : a.cache[l].pool[0]) + block * kPage * D,
                              (kv ? a.cache[l].scale[1] : a.cache[l].scale[0]) + block, lane);
}

struct BulkQ8 {
    const int32_t* indptr;
    const int32_t* indices;
    const int32_t* kv_len;
    const int32_t* tokens;      // [B + 1] rows of each sequence
    const int32_t* start;       // [B] first position (read back), or null: the last tokens
    int64_t num_phys_pages;
    int64_t stride;             // elements between rows of in[] / out[]
    const void* in[2];          // k, v rows (write)
    void* out[2];               // k, v rows (read back)
    Q8Pools cache;
    int32_t Hkv;
    int32_t chunk;              // consecutive pages a warp takes, 1..32
};

// The positions [lo, hi) of sequence b that a bulk call covers, and the row of position 0 (may be negative).
__device__ __forceinline__ void bulk_range(const BulkQ8& p, int b, int64_t& lo, int64_t& hi, int64_t& row0) {
    const int64_t n = max(p.kv_len[b], 0), t0 = p.tokens[b], m = max(int64_t(p.tokens[b + 1]) - t0, int64_t(0));
    const int64_t first = p.start != nullptr ? int64_t(p.start[b]) : n - m;
    lo = max(first, int64_t(0));
    hi = min(first + m, n);
    row0 = t0 - first;
}

// Physical pages of the warp's chunk of logical pages lp0 .. lp0 + cnt - 1, one a lane; -1 where the table or the
// pool has none (the attention calls flag those).
__device__ __forceinline__ int chunk_pages(const BulkQ8& p, int b, int lp0, int cnt, int lane) {
    if (lane >= cnt) return -1;
    const int pbeg = p.indptr[b], npg = p.indptr[b + 1] - pbeg;
    if (lp0 + lane >= npg) return -1;
    const int64_t phys = p.indices[pbeg + lp0 + lane];
    return phys < 0 || phys >= p.num_phys_pages ? -1 : int(phys);
}

// Grid (chunks of pages, sequences, (K or V, KV head) items), a warp each.
template <typename T, int D, int FMT>
__global__ void __launch_bounds__(32) write_q8_kernel(const BulkQ8 p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int ITERS = Rows<T, D, kPage>::ITERS;
    const int b = blockIdx.y, lane = threadIdx.x, item = blockIdx.z;
    int64_t lo, hi, row0;
    bulk_range(p, b, lo, hi, row0);
    if (lo < hi) {
        const int kv = item >= p.Hkv ? 1 : 0, g = item - kv * p.Hkv;
        const T* in = static_cast<const T*>(kv ? p.in[1] : p.in[0]) + int64_t(g) * D;
        uint8_t* pool = (kv ? p.cache.pool[1] : p.cache.pool[0]);
        float* scale = (kv ? p.cache.scale[1] : p.cache.scale[0]);
        const int first = int(lo / kPage), last = int((hi - 1) / kPage);
        for (int64_t at = first + int64_t(blockIdx.x) * p.chunk; at <= last; at += int64_t(gridDim.x) * p.chunk) {
            const int lp0 = int(at), cnt = min(p.chunk, last - lp0 + 1);
            auto range = [&](int lp, int& f0, int& f1) {
                f0 = int(max(lo - int64_t(lp) * kPage, int64_t(0)));
                f1 = int(min(hi - int64_t(lp) * kPage, int64_t(kPage)));
            };
            auto load = [&](int lp, uint4 (&raw)[ITERS]) {
                int f0, f1;
                range(lp, f0, f1);
                load_rows<T, D, kPage>(in + (row0 + int64_t(lp) * kPage + f0) * p.stride, p.stride, f0, f1, lane, raw);
            };
            uint4 raw[ITERS];
            load(lp0, raw);
            const int pages = chunk_pages(p, b, lp0, cnt, lane);
            for (int i = 0; i < cnt; ++i) {
                const int phys = __shfl_sync(0xffffffffu, pages, i);
                if (phys >= 0) {
                    int f0, f1;
                    range(lp0 + i, f0, f1);
                    const size_t block = size_t(phys) * p.Hkv + g;
                    store_block<T, D, FMT, kPage>(raw, f0, f1, pool + block * kPage * D, scale + block, lane);
                }
                if (i + 1 < cnt) load(lp0 + i + 1, raw);
            }
        }
    }
    // The next kernel may load pages (through the asynchronous proxy) before it waits for this grid;
    // it is not started before every block is done, and these fences put the warp's writes ahead of
    // that (one lane's, behind the warp barrier).
    __syncwarp();
    if (lane == 0) {
        __threadfence();
        asm volatile("fence.proxy.async.global;" ::: "memory");
    }
}

// The same grid, a page at a time: the payload is 16 bytes a lane and pass.
template <typename T, int D, int FMT>
__global__ void __launch_bounds__(32) read_q8_kernel(const BulkQ8 p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int b = blockIdx.y, lane = threadIdx.x, item = blockIdx.z;
    int64_t lo, hi, row0;
    bulk_range(p, b, lo, hi, row0);
    if (lo >= hi) return;
    constexpr int LPR = D / 16, RPI = 32 / LPR, ITERS = kPage / RPI;
    const int kv = item >= p.Hkv ? 1 : 0, g = item - kv * p.Hkv;
    const int r = lane / LPR, c = (lane % LPR) * 16;
    const uint8_t* pool = (kv ? p.cache.pool[1] : p.cache.pool[0]);
    const float* scale = (kv ? p.cache.scale[1] : p.cache.scale[0]);
    T* out = static_cast<T*>(kv ? p.out[1] : p.out[0]) + int64_t(g) * D + c;
    const int pbeg = p.indptr[b], npg = p.indptr[b + 1] - pbeg;
    const int first = int(lo / kPage), last = min(int((hi - 1) / kPage), npg - 1);
    for (int64_t lp = first + int64_t(blockIdx.x); lp <= last; lp += gridDim.x) {
        const int64_t phys = p.indices[pbeg + lp];
        if (phys < 0 || phys >= p.num_phys_pages) continue;     // flagged by the attention calls
        const size_t block = size_t(phys) * p.Hkv + g;
        uint4 w[ITERS];
#pragma unroll
        for (int i = 0; i < ITERS; ++i)
            w[i] = *reinterpret_cast<const uint4*>(pool + block * kPage * D + (i * RPI + r) * D + c);
        const float s = scale[block];
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const int64_t pos = lp * kPage + i * RPI + r;
            if (pos < lo || pos >= hi) continue;
            T* dst = out + (row0 + pos) * p.stride;
            const uint32_t* u = reinterpret_cast<const uint32_t*>(&w[i]);
            float x[16];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 a = unpack8x2<FMT>(u[j]), d = unpack8x2<FMT>(u[j] >> 16);
                x[4 * j] = a.x * s;
                x[4 * j + 1] = a.y * s;
                x[4 * j + 2] = d.x * s;
                x[4 * j + 3] = d.y * s;
            }
            if constexpr (sizeof(T) == 2) {
                uint4 o[2];
                uint32_t* q = reinterpret_cast<uint32_t*>(o);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
                    q[j] = *reinterpret_cast<const uint32_t*>(&h);
                }
                reinterpret_cast<uint4*>(dst)[0] = o[0];
                reinterpret_cast<uint4*>(dst)[1] = o[1];
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    reinterpret_cast<float4*>(dst)[j] = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
            }
        }
    }
}

// One of the eight (dtype, head_dim, format) instantiations of a kernel template: f<T, D, FMT>().
template <typename F>
delta_status for_types(const delta_desc* d, int format, const F& f) {
    auto by_format = [&](auto t, auto dim) {
        using T = decltype(t);
        constexpr int D = decltype(dim)::value;
        return format == kE4M3 ? f.template operator()<T, D, kE4M3>() : f.template operator()<T, D, kInt8>();
    };
    auto by_dim = [&](auto t) {
        return d->head_dim == 128 ? by_format(t, std::integral_constant<int, 128>{})
                                  : by_format(t, std::integral_constant<int, 64>{});
    };
    return d->dtype == DELTA_BF16 ? by_dim(__nv_bfloat16{}) : by_dim(float{});
}

struct LaunchAppend {
    const AppendQ8Layers& a;
    const delta_page_table* pt;
    const delta_desc* d;
    int layers;
    cudaStream_t st;
    template <typename T, int D, int FMT>
    delta_status operator()() const {
        return launch_pdl(append_q8_kernel<T, D, FMT>, dim3(pt->batch, d->num_kv_heads, layers), dim3(64), 0, st, a,
                          pt->page_indptr, pt->page_indices, pt->kv_len, d->num_phys_pages);
    }
};
struct LaunchBulk {
    const BulkQ8& p;
    dim3 grid;
    bool write;
    cudaStream_t st;
    template <typename T, int D, int FMT>
    delta_status operator()() const {
        return write ? launch_pdl(write_q8_kernel<T, D, FMT>, grid, dim3(32), 0, st, p)
                     : launch_pdl(read_q8_kernel<T, D, FMT>, grid, dim3(32), 0, st, p);
    }
};

delta_status append_layers(const delta_desc* desc, const delta_page_table* pt, int32_t num_layers,
                           const void* const* k_new, const void* const* v_new, const delta_q8_cache* caches,
                           void* stream) {
    delta_status s = check_desc(desc);
    if (s != DELTA_OK) return s;
    s = check_pt(pt);
    if (s != DELTA_OK) return s;
    if (num_layers < 0) return DELTA_ERR_INVALID_ARG;
    if (num_layers > 64) return DELTA_ERR_UNSUPPORTED;
    if (pt->batch == 0 || num_layers == 0) return DELTA_OK;
    if (k_new == nullptr || v_new == nullptr || caches == nullptr) return DELTA_ERR_INVALID_ARG;
    AppendQ8Layers a{};
    for (int l = 0; l < num_layers; ++l) {
        s = check_q8_cache(&caches[l]);
        if (s != DELTA_OK) return s;
        if (caches[l].format != caches[0].format) return DELTA_ERR_INVALID_ARG;
        if (k_new[l] == nullptr || v_new[l] == nullptr || !aligned16(k_new[l]) || !aligned16(v_new[l]))
            return DELTA_ERR_INVALID_ARG;
        a.k_new[l] = k_new[l];
        a.v_new[l] = v_new[l];
        a.cache[l] = {{static_cast<uint8_t*>(caches[l].k_pool), static_cast<uint8_t*>(caches[l].v_pool)},
                      {caches[l].k_scale, caches[l].v_scale}};
    }
    return for_types(desc, caches[0].format, LaunchAppend{a, pt, desc, num_layers, static_cast<cudaStream_t>(stream)});
}

delta_status bulk(const delta_desc* desc, const delta_page_table* pt, const int32_t* tokens, int32_t max_tokens,
                  const int32_t* start, const void* const (&in)[2], void* const (&out)[2], bool write,
                  int64_t row_stride, const delta_q8_cache* cache, void* stream) {
    delta_status s = check_desc(desc);
    if (s != DELTA_OK) return s;
    s = check_pt(pt);
    if (s != DELTA_OK) return s;
    if (max_tokens < 0) return DELTA_ERR_INVALID_ARG;
    const int64_t row = int64_t(desc->num_kv_heads) * desc->head_dim;
    if (row_stride == 0) row_stride = row;
    if (row_stride < row || row_stride * elem_bytes(desc->dtype) % 16 != 0) return DELTA_ERR_INVALID_ARG;
    if (pt->batch == 0 || max_tokens == 0) return DELTA_OK;
    s = check_q8_cache(cache);
    if (s != DELTA_OK) return s;
    if (tokens == nullptr) return DELTA_ERR_INVALID_ARG;
    BulkQ8 p{};
    for (int i = 0; i < 2; ++i) {
        const void* x = write ? in[i] : out[i];
        if (x == nullptr || !aligned16(x)) return DELTA_ERR_INVALID_ARG;
        p.in[i] = in[i];
        p.out[i] = out[i];
    }
    p.indptr = pt->page_indptr;
    p.indices = pt->page_indices;
    p.kv_len = pt->kv_len;
    p.tokens = tokens;
    p.start = start;
    p.num_phys_pages = desc->num_phys_pages;
    p.stride = row_stride;
    p.cache = {{static_cast<uint8_t*>(cache->k_pool), static_cast<uint8_t*>(cache->v_pool)},
               {cache->k_scale, cache->v_scale}};
    p.Hkv = desc->num_kv_heads;
    // max_tokens tokens overlap at most one page more than they fill
    const int64_t pages = (int64_t(max_tokens) + kPage - 1) / kPage + 1;
    const int items = 2 * desc->num_kv_heads;
    const int64_t warps = pages * pt->batch * items / (int64_t(device_sm_count()) * kWarpsPerSm);
    p.chunk = !write || warps < 1 ? 1 : warps > kMaxChunk ? kMaxChunk : int(warps);
    const int64_t columns = (pages + p.chunk - 1) / p.chunk;
    const dim3 grid(unsigned(columns < kMaxColumns ? columns : kMaxColumns), pt->batch, items);
    return for_types(desc, cache->format, LaunchBulk{p, grid, write, static_cast<cudaStream_t>(stream)});
}

}  // namespace delta

using namespace delta;

extern "C" {

delta_status delta_kv_append_layers_q8(const delta_desc* desc, const delta_page_table* pt, int32_t num_layers,
                                       const void* const* k_new, const void* const* v_new,
                                       const delta_q8_cache* caches, void* stream) {
    return append_layers(desc, pt, num_layers, k_new, v_new, caches, stream);
}

delta_status delta_kv_append_q8(const delta_desc* desc, const delta_page_table* pt, const void* k_new,
                                const void* v_new, const delta_q8_cache* cache, void* stream) {
    return append_layers(desc, pt, 1, &k_new, &v_new, cache, stream);
}

delta_status delta_kv_write_q8(const delta_desc* desc, const delta_page_table* pt, const int32_t* token_indptr,
                               int32_t max_tokens, const void* k, const void* v, int64_t row_stride,
                               const delta_q8_cache* cache, void* stream) {
    return bulk(desc, pt, token_indptr, max_tokens, nullptr, {k, v}, {nullptr, nullptr}, true, row_stride, cache, stream);
}

delta_status delta_kv_read_q8(const delta_desc* desc, const delta_page_table* pt, const int32_t* token_indptr,
                              int32_t max_tokens, const int32_t* token_start, const delta_q8_cache* cache, void* k_out,
                              void* v_out, void* stream) {
    return bulk(desc, pt, token_indptr, max_tokens, token_start, {nullptr, nullptr}, {k_out, v_out}, false, 0, cache,
                stream);
}

}  // extern "C"
