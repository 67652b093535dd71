// Learned embeddings: the lookup with a scale and its gradient.
//
//   forward   out[i, :] = s * T[id_i, :]
//   backward  grad[v, :] = s * sum over i with id_i = v, i ascending, of g[i, :]
//
// Both are bound by memory: the forward reads each row and writes it; the
// backward reads every row of g once and writes each distinct ID's row once.
//
// The backward sorts the positions by ID (stable LSD radix sort, 8 bits a
// pass, so equal IDs keep ascending positions), then cuts the sorted list
// into chunks of equal length, whatever the IDs' frequencies: a warp sums the
// rows of its chunk run by run.  A run that lies inside a chunk is written
// at once; the pieces of a run that crosses chunk borders are left in the
// workspace and joined in chunk order by k_embed_join.  So one hot ID costs no
// more than many cold ones, and every sum has one order: no float atomics.
#include <cuda_bf16.h>
#include <string.h>

#include "sg_internal.cuh"

SGI_ERROR_WORD(embed)

using namespace sgi;

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 8;
constexpr int kSortItems = 16;                    // keys a thread of the sort
constexpr int kSortTile = kThreads * kSortItems;  // 4096 keys a block
constexpr int kDigits = 256;
constexpr int kScanThreads = 1024;
constexpr int kChunk = 32;  // sorted positions a warp sums

size_t a256(size_t x) { return (x + 255) & ~(size_t)255; }

__device__ __forceinline__ int64_t count_of(const int32_t* d_n, int64_t n_cap) {
    if (!d_n) return n_cap;
    const int64_t n = *d_n;
    return n < 0 ? 0 : (n < n_cap ? n : n_cap);
}

// ------------------------------------------------- VEC elements at a time
template <int VEC>
__device__ __forceinline__ void load_vec(const float* p, float (&v)[VEC]) {
    if constexpr (VEC % 4 == 0) {
#pragma unroll
        for (int q = 0; q < VEC / 4; ++q) {
            const float4 t = __ldg(reinterpret_cast<const float4*>(p) + q);
            v[4 * q] = t.x, v[4 * q + 1] = t.y, v[4 * q + 2] = t.z, v[4 * q + 3] = t.w;
        }
    } else {
#pragma unroll
        for (int q = 0; q < VEC; ++q) v[q] = __ldg(p + q);
    }
}
__device__ __forceinline__ void unpack2(uint32_t u, float& lo, float& hi) {
    lo = __uint_as_float(u << 16);
    hi = __uint_as_float(u & 0xFFFF0000u);
}
template <int VEC>
__device__ __forceinline__ void load_vec(const __nv_bfloat16* p, float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        const uint4 t = __ldg(reinterpret_cast<const uint4*>(p));
        unpack2(t.x, v[0], v[1]);
        unpack2(t.y, v[2], v[3]);
        unpack2(t.z, v[4], v[5]);
        unpack2(t.w, v[6], v[7]);
    } else if constexpr (VEC == 4) {
        const uint2 t = __ldg(reinterpret_cast<const uint2*>(p));
        unpack2(t.x, v[0], v[1]);
        unpack2(t.y, v[2], v[3]);
    } else {
#pragma unroll
        for (int q = 0; q < VEC; ++q) v[q] = __bfloat162float(p[q]);
    }
}
template <int VEC>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[VEC]) {
    if constexpr (VEC % 4 == 0) {
#pragma unroll
        for (int q = 0; q < VEC / 4; ++q)
            reinterpret_cast<float4*>(p)[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
    } else {
#pragma unroll
        for (int q = 0; q < VEC; ++q) p[q] = v[q];
    }
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&t);
}
template <int VEC>
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        *reinterpret_cast<uint4*>(p) =
            make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
    } else if constexpr (VEC == 4) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
    } else {
#pragma unroll
        for (int q = 0; q < VEC; ++q) p[q] = __float2bfloat16_rn(v[q]);
    }
}

// ---------------------------------------------------------------- forward
// Flat over (row, unit of VEC elements), consecutive threads on consecutive
// units, kUnroll loads in flight a thread; (i, c) advance by the grid stride
// without a division (stride = step_rows * units + step_rem).
template <typename TI, typename TO, int VEC>
__global__ void __launch_bounds__(kThreads) k_embed_fwd(const TI* __restrict__ table, int64_t n_rows, int64_t ld_table,
                                                        const int32_t* __restrict__ ids, int64_t n_cap,
                                                        const int32_t* __restrict__ d_n, float scale, int32_t units,
                                                        int64_t step_rows, int32_t step_rem, TO* __restrict__ out,
                                                        int64_t ld_out) {
    pdl_start();
    const int64_t total = count_of(d_n, n_cap) * units;
    const int64_t stride = (int64_t)gridDim.x * kThreads;
    int64_t t = blockIdx.x * (int64_t)kThreads + threadIdx.x;
    int64_t i = t / units;
    int32_t c = (int32_t)(t - i * units);
    while (t < total) {
        float v[kUnroll][VEC];
        int64_t dst[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            dst[u] = -1;
            if (t < total) {
                const int32_t g = __ldg(ids + i);
                dst[u] = i * ld_out + (int64_t)c * VEC;
                if (g < 0 || (int64_t)g >= n_rows) {
                    if (c == 0 && g != -1) dev_err(ERR_INDEX);
#pragma unroll
                    for (int q = 0; q < VEC; ++q) v[u][q] = 0.f;
                } else {
                    load_vec<VEC>(table + (int64_t)g * ld_table + (int64_t)c * VEC, v[u]);
                }
            }
            t += stride;
            i += step_rows;
            c += step_rem;
            if (c >= units) {
                c -= units;
                ++i;
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (dst[u] < 0) continue;
#pragma unroll
            for (int q = 0; q < VEC; ++q) v[u][q] *= scale;
            store_vec<VEC>(out + dst[u], v[u]);
        }
    }
}

// ------------------------------------------------------------------- sort
// Key of position i: its ID, or n_rows (sorted last) for one that takes no part.
__device__ __forceinline__ uint32_t key_of(const int32_t* __restrict__ ids, int64_t i, int64_t n_rows) {
    const int32_t g = ids[i];
    if (g < 0 || (int64_t)g >= n_rows) {
        if (g != -1) dev_err(ERR_INDEX);
        return (uint32_t)n_rows;
    }
    return (uint32_t)g;
}

// Digit histogram of block b's tile, digit-major: hist[digit * nb + b].  The
// first pass reads the IDs (keys NULL).
__global__ void __launch_bounds__(kThreads) k_sort_hist(const uint32_t* __restrict__ keys,
                                                        const int32_t* __restrict__ ids, int64_t n_rows, int64_t n_cap,
                                                        const int32_t* __restrict__ d_n, int shift, int mask,
                                                        uint32_t* __restrict__ hist, int64_t nb) {
    pdl_start();
    __shared__ uint32_t h[kDigits];
    h[threadIdx.x] = 0;
    __syncthreads();
    const int64_t n = count_of(d_n, n_cap), i0 = (int64_t)blockIdx.x * kSortTile;
    for (int r = 0; r < kSortItems; ++r) {
        const int64_t i = i0 + r * kThreads + threadIdx.x;
        if (i < n) atomicAdd(&h[((keys ? keys[i] : key_of(ids, i, n_rows)) >> shift) & mask], 1u);
    }
    __syncthreads();
    hist[(int64_t)threadIdx.x * nb + blockIdx.x] = h[threadIdx.x];
}

// Exclusive scan of m entries in place, one block.
__global__ void __launch_bounds__(kScanThreads) k_sort_scan(uint32_t* __restrict__ a, int64_t m) {
    pdl_start();
    __shared__ uint32_t sh[kScanThreads / 32 + 1];
    uint32_t base = 0;
    for (int64_t i0 = 0; i0 < m; i0 += kScanThreads) {
        const int64_t i = i0 + threadIdx.x;
        const uint32_t x = i < m ? a[i] : 0;
        uint32_t total;
        const uint32_t e = block_excl_scan<kScanThreads, uint32_t>(x, sh, total);
        if (i < m) a[i] = base + e;
        base += total;
    }
}

// Stable scatter of block b's tile (in rounds of kThreads items): a warp ranks
// its lanes by digit, the warps' counts become offsets.
__global__ void __launch_bounds__(kThreads) k_sort_scatter(const uint32_t* __restrict__ keys_in,
                                                           const int32_t* __restrict__ vals_in,
                                                           const int32_t* __restrict__ ids, int64_t n_rows,
                                                           int64_t n_cap, const int32_t* __restrict__ d_n, int shift,
                                                           int mask, const uint32_t* __restrict__ offs, int64_t nb,
                                                           uint32_t* __restrict__ keys_out,
                                                           int32_t* __restrict__ vals_out) {
    pdl_start();
    __shared__ uint32_t run[kDigits];
    __shared__ uint32_t wcnt[kThreads / 32][kDigits];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    run[threadIdx.x] = offs[(int64_t)threadIdx.x * nb + blockIdx.x];
    const int64_t n = count_of(d_n, n_cap), i0 = (int64_t)blockIdx.x * kSortTile;
    for (int r = 0; r < kSortItems; ++r) {
        if (i0 + r * kThreads >= n) break;  // the same in every thread
        const int64_t i = i0 + r * kThreads + threadIdx.x;
        const bool valid = i < n;
        uint32_t key = 0;
        int32_t val = 0;
        if (valid) {
            val = keys_in ? vals_in[i] : (int32_t)i;
            key = keys_in ? keys_in[i] : key_of(ids, i, n_rows);
        }
        const uint32_t d = valid ? (key >> shift) & mask : 0x100u + (uint32_t)lane;  // invalid lanes match none
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) wcnt[w][threadIdx.x] = 0;
        __syncthreads();
        const unsigned peers = __match_any_sync(0xFFFFFFFFu, d);
        const uint32_t rank = __popc(peers & lanemask_lt());
        if (valid && rank == 0) wcnt[warp][d] = __popc(peers);
        __syncthreads();
        {
            uint32_t acc = run[threadIdx.x];
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) {
                const uint32_t c = wcnt[w][threadIdx.x];
                wcnt[w][threadIdx.x] = acc;
                acc += c;
            }
            run[threadIdx.x] = acc;
        }
        __syncthreads();
        if (valid) {
            const uint32_t pos = wcnt[warp][d] + rank;
            keys_out[pos] = key;
            vals_out[pos] = val;
        }
        __syncthreads();
    }
}

// ------------------------------------------------------- runs of equal IDs
// Run starts of each chunk of the sorted list (IDs that take part only).
__global__ void __launch_bounds__(kThreads) k_run_count(const uint32_t* __restrict__ keys, int64_t n_rows,
                                                        int64_t n_cap, const int32_t* __restrict__ d_n,
                                                        int32_t* __restrict__ starts, int64_t chunks) {
    pdl_start();
    const int64_t n = count_of(d_n, n_cap);
    const int64_t c = blockIdx.x * (int64_t)(kThreads / 32) + (threadIdx.x >> 5);
    if (c >= chunks) return;
    const int64_t p = c * kChunk + (threadIdx.x & 31);
    const bool start = p < n && keys[p] < (uint32_t)n_rows && (p == 0 || keys[p - 1] != keys[p]);
    const unsigned b = __ballot_sync(0xFFFFFFFFu, start);
    if ((threadIdx.x & 31) == 0) starts[c] = __popc(b);
}

// starts -> exclusive prefix; the total is the number of distinct IDs.
__global__ void __launch_bounds__(kScanThreads) k_run_base(int32_t* __restrict__ starts, int64_t chunks,
                                                           int32_t* __restrict__ n_out) {
    pdl_start();
    __shared__ int32_t sh[kScanThreads / 32 + 1];
    int32_t base = 0;
    for (int64_t i0 = 0; i0 < chunks; i0 += kScanThreads) {
        const int64_t i = i0 + threadIdx.x;
        int32_t total;
        const int32_t e = block_excl_scan<kScanThreads, int32_t>(i < chunks ? starts[i] : 0, sh, total);
        if (i < chunks) starts[i] = base + e;
        base += total;
    }
    if (threadIdx.x == 0) *n_out = base;
}

template <typename TO>
struct SumArgs {
    const uint32_t* keys;   // sorted
    const int32_t* vals;    // positions
    const int32_t* d_n;
    int64_t n_cap, n_rows;
    int64_t ld_g;
    int32_t dim, units, col_blocks, lanes;  // lanes: of a warp, for one chunk's rows
    int32_t mode;
    float scale;
    const int32_t* starts;  // SG_GRAD_ROWS: distinct IDs before each chunk
    int32_t* rows;
    TO* grad;
    int64_t ld_grad;
    float* head;  // [chunks][dim] sums of runs that began in an earlier chunk
    float* tail;  // [chunks][dim] sums of runs that go on in the next chunk
};

// Row of the gradient for the run of `key` (the j-th run).
template <typename TO, int VEC>
__device__ __forceinline__ void put_row(const SumArgs<TO>& a, uint32_t key, int32_t j, int32_t col,
                                        const float (&acc)[VEC]) {
    const int64_t row = a.mode == SG_GRAD_ROWS ? (int64_t)j : (int64_t)key;
    if (a.mode == SG_GRAD_ROWS && col == 0) a.rows[j] = (int32_t)key;
    TO* p = a.grad + row * a.ld_grad + col;
    float v[VEC];
#pragma unroll
    for (int q = 0; q < VEC; ++q) v[q] = acc[q] * a.scale;
    if (a.mode == SG_GRAD_ADD) {
        float o[VEC];
        if constexpr (sizeof(TO) == 4) {
#pragma unroll
            for (int q = 0; q < VEC; ++q) o[q] = p[q];
        } else {
#pragma unroll
            for (int q = 0; q < VEC; ++q) o[q] = __bfloat162float(p[q]);
        }
#pragma unroll
        for (int q = 0; q < VEC; ++q) v[q] += o[q];
    }
    store_vec<VEC>(p, v);
}

// Lanes of a warp in groups of a.lanes; each group sums one chunk's rows over
// 32 / lanes... units of VEC columns (column block cb), run by run.
template <typename TI, typename TO, int VEC>
__global__ void __launch_bounds__(kThreads) k_embed_sum(const TI* __restrict__ g, SumArgs<TO> a) {
    pdl_start();
    const int64_t n = count_of(a.d_n, a.n_cap);
    const int64_t group = (blockIdx.x * (int64_t)kThreads + threadIdx.x) / a.lanes;
    const int32_t lane = (int32_t)(threadIdx.x % (unsigned)a.lanes);
    const int64_t c = group / a.col_blocks;
    const int32_t unit = (int32_t)(group - c * a.col_blocks) * a.lanes + lane;
    const int64_t p0 = c * kChunk;
    if (p0 >= n || unit >= a.units) return;
    const int32_t col = unit * VEC;
    const int64_t p1 = p0 + kChunk < n ? p0 + kChunk : n;
    const uint32_t none = (uint32_t)a.n_rows;
    uint32_t key = a.keys[p0];
    if (key == none) return;
    bool head = p0 > 0 && a.keys[p0 - 1] == key;
    int32_t j = a.mode == SG_GRAD_ROWS ? a.starts[c] - (head ? 1 : 0) : 0;
    float acc[VEC];
#pragma unroll
    for (int q = 0; q < VEC; ++q) acc[q] = 0.f;
    bool last = false;
    for (int64_t p = p0; p < p1 && !last; p += kUnroll) {
        uint32_t k[kUnroll];
        float v[kUnroll][VEC];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            k[u] = p + u < p1 ? a.keys[p + u] : none;
            if (k[u] != none) load_vec<VEC>(g + (int64_t)a.vals[p + u] * a.ld_g + col, v[u]);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (last) continue;
            if (p + u >= p1 || k[u] == none) {
                last = true;
                continue;
            }
            if (k[u] != key) {
                if (head) store_vec<VEC>(a.head + c * a.dim + col, acc);
                else put_row<TO, VEC>(a, key, j, col, acc);
                head = false;
                ++j;
                key = k[u];
#pragma unroll
                for (int q = 0; q < VEC; ++q) acc[q] = 0.f;
            }
#pragma unroll
            for (int q = 0; q < VEC; ++q) acc[q] += v[u][q];
        }
    }
    if (head) store_vec<VEC>(a.head + c * a.dim + col, acc);
    else if (p1 < n && a.keys[p1] == key) store_vec<VEC>(a.tail + c * a.dim + col, acc);
    else put_row<TO, VEC>(a, key, j, col, acc);
}

// Joins the runs that cross chunks: chunk c owns the run that begins in it
// and goes on; the sum is tail[c] + head[c + 1] + ..., in this order.
template <typename TO, int VEC>
__global__ void __launch_bounds__(kThreads) k_embed_join(SumArgs<TO> a) {
    pdl_start();
    const int64_t n = count_of(a.d_n, a.n_cap);
    const int64_t group = (blockIdx.x * (int64_t)kThreads + threadIdx.x) / a.lanes;
    const int32_t lane = (int32_t)(threadIdx.x % (unsigned)a.lanes);
    const int64_t c = group / a.col_blocks;
    const int32_t unit = (int32_t)(group - c * a.col_blocks) * a.lanes + lane;
    const int64_t p0 = c * kChunk, p1 = p0 + kChunk;
    if (p1 >= n || unit >= a.units) return;  // nothing after this chunk
    const uint32_t key = a.keys[p1 - 1];
    if (key == (uint32_t)a.n_rows || a.keys[p1] != key) return;
    if (p0 > 0 && a.keys[p0] == key && a.keys[p0 - 1] == key) return;  // the run began earlier
    const int32_t col = unit * VEC;
    float acc[VEC];
    load_vec<VEC>(a.tail + c * a.dim + col, acc);
    for (int64_t d = c + 1; d * kChunk < n && a.keys[d * kChunk] == key; ++d) {
        float v[VEC];
        load_vec<VEC>(a.head + d * a.dim + col, v);
#pragma unroll
        for (int q = 0; q < VEC; ++q) acc[q] += v[q];
    }
    put_row<TO, VEC>(a, key, a.mode == SG_GRAD_ROWS ? a.starts[c + 1] - 1 : 0, col, acc);
}

// ------------------------------------------------------------------- host
bool dtype_ok(int32_t d) { return d == SG_F32 || d == SG_BF16; }
int elem(int32_t d) { return d == SG_F32 ? 4 : 2; }

// Widest unit (8, 4 or 1 elements) that both sides allow: bf16 input moves 8
// elements (16 bytes) at a time, fp32 input 4; every row has to start on the
// unit's boundary and hold a whole number of units.
int vec_for(const void* in, int32_t dtype_in, int64_t ld_in, const void* out, int32_t dtype_out, int64_t ld_out,
            int32_t dim) {
    for (int v = dtype_in == SG_BF16 ? 8 : 4; v >= 4; v /= 2) {
        const int ai = v * elem(dtype_in) < 16 ? v * elem(dtype_in) : 16;
        const int ao = v * elem(dtype_out) < 16 ? v * elem(dtype_out) : 16;
        if (dim % v == 0 && (uintptr_t)in % ai == 0 && (ld_in * elem(dtype_in)) % ai == 0 && (uintptr_t)out % ao == 0 &&
            (ld_out * elem(dtype_out)) % ao == 0)
            return v;
    }
    return 1;
}

template <typename TI, typename TO, int VEC>
sg_status launch_fwd(const void* table, int64_t n_rows, int32_t dim, int64_t ld_table, const int32_t* ids,
                     int64_t n_cap, const int32_t* d_n, float scale, void* out, int64_t ld_out, cudaStream_t s) {
    const int32_t units = dim / VEC;
    int64_t blocks = cdiv(cdiv(n_cap * units, kThreads), kUnroll);
    if (blocks > (int64_t)num_sms() * 8) blocks = (int64_t)num_sms() * 8;
    if (blocks < 1) blocks = 1;
    const int64_t stride = blocks * kThreads;
    SG_CUDA(launch_pdl(k_embed_fwd<TI, TO, VEC>, dim3((unsigned)blocks), dim3(kThreads), 0, s, (const TI*)table, n_rows,
                       ld_table, ids, n_cap, d_n, scale, units, stride / units, (int32_t)(stride % units), (TO*)out,
                       ld_out));
    return SG_OK;
}

template <typename TI, typename TO>
sg_status run_fwd(int vec, const void* table, int64_t n_rows, int32_t dim, int64_t ld_table, const int32_t* ids,
                  int64_t n_cap, const int32_t* d_n, float scale, void* out, int64_t ld_out, cudaStream_t s) {
    if constexpr (sizeof(TI) == 2)
        if (vec == 8) return launch_fwd<TI, TO, 8>(table, n_rows, dim, ld_table, ids, n_cap, d_n, scale, out, ld_out, s);
    if (vec == 4) return launch_fwd<TI, TO, 4>(table, n_rows, dim, ld_table, ids, n_cap, d_n, scale, out, ld_out, s);
    return launch_fwd<TI, TO, 1>(table, n_rows, dim, ld_table, ids, n_cap, d_n, scale, out, ld_out, s);
}

struct BwdLayout {
    int64_t nb, chunks;
    size_t keys0, keys1, vals0, vals1, hist, starts, head, tail, total;
};

BwdLayout bwd_layout(int64_t n_cap, int32_t dim) {
    BwdLayout L;
    L.nb = cdiv(n_cap, kSortTile);
    L.chunks = cdiv(n_cap, kChunk);
    size_t o = 0;
    const auto put = [&o](size_t bytes) {
        const size_t at = o;
        o += a256(bytes);
        return at;
    };
    L.keys0 = put((size_t)n_cap * 4);
    L.keys1 = put((size_t)n_cap * 4);
    L.vals0 = put((size_t)n_cap * 4);
    L.vals1 = put((size_t)n_cap * 4);
    L.hist = put((size_t)kDigits * L.nb * 4);
    L.starts = put((size_t)(L.chunks + 1) * 4);
    L.head = put((size_t)L.chunks * dim * 4);
    L.tail = put((size_t)L.chunks * dim * 4);
    L.total = o;
    return L;
}

template <typename TI, typename TO, int VEC>
sg_status launch_sum(const void* g, SumArgs<TO> a, cudaStream_t s) {
    a.units = a.dim / VEC;
    a.lanes = 1;
    while (a.lanes < 32 && a.lanes < a.units) a.lanes *= 2;
    a.col_blocks = (int32_t)cdiv(a.units, a.lanes);
    const int64_t threads = cdiv(a.n_cap, kChunk) * a.col_blocks * a.lanes;
    const int64_t blocks = cdiv(threads, kThreads);
    if (blocks > 2147483647LL) return fail(SG_ERR_INVALID_ARG, "sg_embed_bwd: n_cap x dim too large");
    SG_CUDA(launch_pdl(k_embed_sum<TI, TO, VEC>, dim3((unsigned)blocks), dim3(kThreads), 0, s, (const TI*)g, a));
    SG_CUDA(launch_pdl(k_embed_join<TO, VEC>, dim3((unsigned)blocks), dim3(kThreads), 0, s, a));
    return SG_OK;
}

template <typename TI, typename TO>
sg_status run_sum(int vec, const void* g, SumArgs<TO> a, cudaStream_t s) {
    if constexpr (sizeof(TI) == 2)
        if (vec == 8) return launch_sum<TI, TO, 8>(g, a, s);
    if (vec == 4) return launch_sum<TI, TO, 4>(g, a, s);
    return launch_sum<TI, TO, 1>(g, a, s);
}

template <typename TO>
sg_status run_bwd(const int32_t* ids, int64_t n_cap, const int32_t* d_n, int64_t n_rows, const void* g, int32_t dtype_g,
                  int32_t dim, int64_t ld_g, float scale, int32_t mode, int32_t* rows, int32_t* n_out, TO* grad,
                  int32_t dtype_grad, int64_t ld_grad, char* ws, cudaStream_t s) {
    const BwdLayout L = bwd_layout(n_cap, dim);
    uint32_t* keys[2] = {(uint32_t*)(ws + L.keys0), (uint32_t*)(ws + L.keys1)};
    int32_t* vals[2] = {(int32_t*)(ws + L.vals0), (int32_t*)(ws + L.vals1)};
    uint32_t* hist = (uint32_t*)(ws + L.hist);
    int bits = 1;
    while (bits < 32 && (n_rows >> bits) != 0) ++bits;  // keys 0 .. n_rows
    const int passes = (bits + 7) / 8, per = (bits + passes - 1) / passes;
    int cur = 0;
    for (int p = 0; p < passes; ++p) {
        const uint32_t* ki = p ? keys[cur] : nullptr;
        const int32_t* vi = p ? vals[cur] : nullptr;
        const int shift = p * per, mask = (1 << per) - 1;
        SG_CUDA(launch_pdl(k_sort_hist, dim3((unsigned)L.nb), dim3(kThreads), 0, s, ki, ids, n_rows, n_cap, d_n, shift,
                           mask, hist, L.nb));
        SG_CUDA(launch_pdl(k_sort_scan, dim3(1), dim3(kScanThreads), 0, s, hist, (int64_t)kDigits * L.nb));
        SG_CUDA(launch_pdl(k_sort_scatter, dim3((unsigned)L.nb), dim3(kThreads), 0, s, ki, vi, ids, n_rows, n_cap, d_n,
                           shift, mask, (const uint32_t*)hist, L.nb, keys[cur ^ 1], vals[cur ^ 1]));
        cur ^= 1;
    }
    int32_t* starts = (int32_t*)(ws + L.starts);
    if (mode == SG_GRAD_ROWS) {
        SG_CUDA(launch_pdl(k_run_count, dim3((unsigned)cdiv(L.chunks + 1, kThreads / 32)), dim3(kThreads), 0, s,
                           (const uint32_t*)keys[cur], n_rows, n_cap, d_n, starts, L.chunks + 1));
        SG_CUDA(launch_pdl(k_run_base, dim3(1), dim3(kScanThreads), 0, s, starts, L.chunks + 1, n_out));
    } else if (mode == SG_GRAD_DENSE) {
        SG_CUDA(cudaMemset2DAsync(grad, (size_t)ld_grad * sizeof(TO), 0, (size_t)dim * sizeof(TO), (size_t)n_rows, s));
    }
    SumArgs<TO> a;
    memset(&a, 0, sizeof(a));
    a.keys = keys[cur];
    a.vals = vals[cur];
    a.d_n = d_n;
    a.n_cap = n_cap;
    a.n_rows = n_rows;
    a.ld_g = ld_g;
    a.dim = dim;
    a.mode = mode;
    a.scale = scale;
    a.starts = starts;
    a.rows = rows;
    a.grad = grad;
    a.ld_grad = ld_grad;
    a.head = (float*)(ws + L.head);
    a.tail = (float*)(ws + L.tail);
    const int vec = vec_for(g, dtype_g, ld_g, grad, dtype_grad, ld_grad, dim);
    return dtype_g == SG_F32 ? run_sum<float, TO>(vec, g, a, s) : run_sum<__nv_bfloat16, TO>(vec, g, a, s);
}

}  // namespace

extern "C" sg_status sg_embed_fwd(const void* d_table, int32_t dtype_table, int64_t n_rows, int32_t dim,
                                  int64_t ld_table, const int32_t* d_ids, int64_t n_cap, const int32_t* d_n,
                                  float scale, void* d_out, int32_t dtype_out, int64_t ld_out, sg_stream_t stream) {
    if (!dtype_ok(dtype_table) || !dtype_ok(dtype_out)) return fail(SG_ERR_UNSUPPORTED, "sg_embed_fwd: dtype");
    if (n_rows < 0 || n_rows > 2147483647LL || n_cap < 0 || n_cap > 2147483647LL || dim <= 0)
        return fail(SG_ERR_INVALID_ARG, "sg_embed_fwd: bad sizes");
    if (ld_table < dim || ld_out < dim) return fail(SG_ERR_INVALID_ARG, "sg_embed_fwd: a row stride is below dim");
    if (n_cap == 0) return SG_OK;
    if ((!d_table && n_rows > 0) || !d_ids || !d_out) return fail(SG_ERR_INVALID_ARG, "sg_embed_fwd: NULL array");
    if ((uintptr_t)d_table % elem(dtype_table) || (uintptr_t)d_out % elem(dtype_out) || (uintptr_t)d_ids % 4)
        return fail(SG_ERR_INVALID_ARG, "sg_embed_fwd: an array is not aligned to its elements");
    cudaStream_t s = (cudaStream_t)stream;
    const int vec = vec_for(d_table, dtype_table, ld_table, d_out, dtype_out, ld_out, dim);
    using B = __nv_bfloat16;
    const bool ti = dtype_table == SG_F32, to = dtype_out == SG_F32;
    if (ti && to) return run_fwd<float, float>(vec, d_table, n_rows, dim, ld_table, d_ids, n_cap, d_n, scale, d_out, ld_out, s);
    if (ti) return run_fwd<float, B>(vec, d_table, n_rows, dim, ld_table, d_ids, n_cap, d_n, scale, d_out, ld_out, s);
    if (to) return run_fwd<B, float>(vec, d_table, n_rows, dim, ld_table, d_ids, n_cap, d_n, scale, d_out, ld_out, s);
    return run_fwd<B, B>(vec, d_table, n_rows, dim, ld_table, d_ids, n_cap, d_n, scale, d_out, ld_out, s);
}

extern "C" size_t sg_embed_bwd_workspace(int64_t n_cap, int64_t n_rows, int32_t dim, int32_t mode) {
    if (n_cap <= 0 || n_cap > 2147483647LL || n_rows <= 0 || n_rows > 2147483647LL || dim <= 0 || mode < SG_GRAD_ROWS ||
        mode > SG_GRAD_ADD)
        return 0;
    return bwd_layout(n_cap, dim).total;
}

extern "C" sg_status sg_embed_bwd(const int32_t* d_ids, int64_t n_cap, const int32_t* d_n, int64_t n_rows,
                                  const void* d_g, int32_t dtype_g, int32_t dim, int64_t ld_g, float scale,
                                  int32_t mode, int32_t* d_rows, int32_t* d_n_rows, void* d_grad, int32_t dtype_grad,
                                  int64_t ld_grad, void* d_workspace, size_t workspace_bytes, sg_stream_t stream) {
    if (!dtype_ok(dtype_g) || !dtype_ok(dtype_grad)) return fail(SG_ERR_UNSUPPORTED, "sg_embed_bwd: dtype");
    if (mode < SG_GRAD_ROWS || mode > SG_GRAD_ADD) return fail(SG_ERR_INVALID_ARG, "sg_embed_bwd: mode");
    if (n_cap < 0 || n_cap > 2147483647LL || n_rows <= 0 || n_rows > 2147483647LL || dim <= 0)
        return fail(SG_ERR_INVALID_ARG, "sg_embed_bwd: bad sizes");
    if (ld_g < dim || ld_grad < dim) return fail(SG_ERR_INVALID_ARG, "sg_embed_bwd: a row stride is below dim");
    if (mode == SG_GRAD_ROWS && (!d_rows || !d_n_rows))
        return fail(SG_ERR_INVALID_ARG, "sg_embed_bwd: SG_GRAD_ROWS needs d_rows and d_n_rows");
    if (mode != SG_GRAD_ROWS && (d_rows || d_n_rows))
        return fail(SG_ERR_INVALID_ARG, "sg_embed_bwd: d_rows and d_n_rows belong to SG_GRAD_ROWS");
    if (!d_grad) return fail(SG_ERR_INVALID_ARG, "sg_embed_bwd: NULL array");
    if ((uintptr_t)d_g % elem(dtype_g) || (uintptr_t)d_grad % elem(dtype_grad) || (uintptr_t)d_ids % 4)
        return fail(SG_ERR_INVALID_ARG, "sg_embed_bwd: an array is not aligned to its elements");
    cudaStream_t s = (cudaStream_t)stream;
    if (n_cap == 0) {  // nothing to add
        if (mode == SG_GRAD_ROWS) SG_CUDA(cudaMemsetAsync(d_n_rows, 0, sizeof(int32_t), s));
        if (mode == SG_GRAD_DENSE)
            SG_CUDA(cudaMemset2DAsync(d_grad, (size_t)ld_grad * elem(dtype_grad), 0, (size_t)dim * elem(dtype_grad),
                                      (size_t)n_rows, s));
        return SG_OK;
    }
    if (!d_ids || !d_g || !d_workspace) return fail(SG_ERR_INVALID_ARG, "sg_embed_bwd: NULL array");
    if ((uintptr_t)d_workspace % 256) return fail(SG_ERR_INVALID_ARG, "sg_embed_bwd: workspace must be 256-byte aligned");
    const size_t need = bwd_layout(n_cap, dim).total;
    if (workspace_bytes < need) return fail(SG_ERR_INVALID_ARG, "sg_embed_bwd: workspace needs %zu bytes", need);
    if (dtype_grad == SG_F32)
        return run_bwd<float>(d_ids, n_cap, d_n, n_rows, d_g, dtype_g, dim, ld_g, scale, mode, d_rows, d_n_rows,
                              (float*)d_grad, dtype_grad, ld_grad, (char*)d_workspace, s);
    return run_bwd<__nv_bfloat16>(d_ids, n_cap, d_n, n_rows, d_g, dtype_g, dim, ld_g, scale, mode, d_rows, d_n_rows,
                                  (__nv_bfloat16*)d_grad, dtype_grad, ld_grad, (char*)d_workspace, s);
}
