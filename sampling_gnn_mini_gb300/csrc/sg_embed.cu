// Learned embeddings: the lookup with a scale and its gradient.
//
//   forward   out[i, :] = s * T[id_i, :]
//   backward  grad[v, :] = s * sum over i with id_i = v, i ascending, of g[i, :]
//
// Both are bound by memory: the forward reads each row and writes it; the
// backward reads every row of g once and writes each distinct ID's row once.
//
// The backward sorts (ID, position) pairs by ID (stable radix sort, up to 8 bits
// a pass, so equal IDs keep ascending positions), then cuts the sorted list
// into chunks of equal length, whatever the IDs' frequencies: a group of lanes
// that covers a row's columns sums the rows of its chunk, run by run.  A run
// that lies inside a chunk is written at once; the pieces of a run that
// crosses chunks meet in shared memory, in chunk order, and those of a run
// that crosses blocks are left in the workspace and joined in block order by
// k_embed_join.  So one hot ID costs no more than many cold ones, and every
// sum has one order: no float atomics.
//
// The sort: up to kSmallSort positions in one block's shared memory
// (k_sort_small); up to kClusterSort by one cluster, where the device takes it
// (k_sort_cluster); else one histogram launch for all passes, then one launch a
// pass, whose tiles learn their digits' offsets from the tiles before them
// (decoupled look-back, one thread a digit).
#include <cuda_bf16.h>
#include <string.h>

#include "sg_internal.cuh"
#include "sg_tc.cuh"

SGI_ERROR_WORD(embed)

using namespace sgi;

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 8;
constexpr int kDigits = 256;
constexpr int kMaxPasses = 4;
constexpr int kCopies = 8;            // of the digit counts, which blocks add to in turn
constexpr int kSortThreads = 512;     // of a pass
constexpr int kSmallThreads = 1024;
constexpr int kSmallSort = 3 * kSmallThreads;  // positions sorted by one block (us for the dense / compact gradient of 64
                                               // columns, one block: 1,000 positions 11.0 / 11.5, 3,000 14.1 / 14.9, 4,000
                                               // 16.7 / 17.7, 5,000 17.4 / 18.5; a cluster of 8: 14.6 / 16.7, 14.9 / 17.4,
                                               // 15.4 / 17.4, 15.4 / 17.7)
constexpr int kSortCtas = 16;                  // blocks of a cluster that sorts more; 8 where they hold the list (6,000
                                               // positions 15.4 / 18.0, by 16 blocks 16.4 / 19.2)
constexpr int kClusterSort = kSortCtas * 2 * kSmallThreads;
constexpr int kRunTile = kThreads * 16;   // sorted positions a block of k_runs looks at
constexpr int kFewBlocks = 76;           // half the SMs: below this many blocks chunks are 8 positions, not 32
constexpr uint32_t kNoKey = 0xFFFFFFFFu;  // beside the list's ends

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
// VEC elements as they were loaded (16 bytes at most), unpacked when used.
template <typename T, int VEC>
struct Raw {
    uint32_t w[(VEC * sizeof(T) + 3) / 4];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (VEC * sizeof(T) == 16) {
            const uint4 t = __ldg(reinterpret_cast<const uint4*>(p));
            w[0] = t.x, w[1] = t.y, w[2] = t.z, w[3] = t.w;
        } else if constexpr (VEC * sizeof(T) == 8) {
            const uint2 t = __ldg(reinterpret_cast<const uint2*>(p));
            w[0] = t.x, w[1] = t.y;
        } else if constexpr (sizeof(T) == 4) {
            w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
        } else {
            w[0] = (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(p)) << 16;
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (uint32_t& x : w) x = 0;
    }
    __device__ __forceinline__ float operator[](int q) const {
        if constexpr (sizeof(T) == 4 || VEC == 1) return __uint_as_float(w[q]);
        else return __uint_as_float(q & 1 ? w[q / 2] & 0xFFFF0000u : w[q / 2] << 16);
    }
};

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
// A block takes kThreads * kUnroll consecutive units of VEC elements, flat over
// the rows: consecutive threads on consecutive units, kUnroll loads in flight a
// thread, no loop.  Measured on 600,001 x 128 fp32 rows of a 10 GB table: 91 us
// (6.7 TB/s, the rate of a copy); with a grid of 8 blocks an SM that loops, 112.
// (i, c), row and unit, advance by kThreads without a division:
// kThreads = step_rows * units + step_rem.
template <typename TI, typename TO, int VEC>
__global__ void __launch_bounds__(kThreads) k_embed_fwd(const TI* __restrict__ table, int64_t n_rows, int64_t ld_table,
                                                        const int32_t* __restrict__ ids, int64_t n_cap,
                                                        const int32_t* __restrict__ d_n, float scale, int32_t units,
                                                        int32_t step_rows, int32_t step_rem, TO* __restrict__ out,
                                                        int64_t ld_out) {
    pdl_start();
    const int32_t n = (int32_t)count_of(d_n, n_cap);
    const int64_t t0 = (int64_t)blockIdx.x * (kThreads * kUnroll);
    int32_t i0 = (int32_t)(t0 / units), c0 = (int32_t)(t0 - (int64_t)i0 * units) + (int32_t)threadIdx.x;
    i0 += c0 / units;
    c0 %= units;
    int32_t id[kUnroll];
    {
        int32_t i = i0, c = c0;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            id[u] = i < n ? __ldg(ids + i) : -1;
            i += step_rows;
            c += step_rem;
            if (c >= units) c -= units, ++i;
        }
    }
    Raw<TI, VEC> v[kUnroll];
    {
        int32_t i = i0, c = c0;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            v[u].zero();
            if (id[u] >= 0 && id[u] < n_rows) v[u].load(table + (int64_t)id[u] * ld_table + (int64_t)c * VEC);
            else if (c == 0 && id[u] != -1) dev_err(ERR_INDEX);
            i += step_rows;
            c += step_rem;
            if (c >= units) c -= units, ++i;
        }
    }
    int32_t i = i0, c = c0;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if (i < n) {
            float x[VEC];
#pragma unroll
            for (int q = 0; q < VEC; ++q) x[q] = v[u][q] * scale;
            store_vec<VEC>(out + (int64_t)i * ld_out + (int64_t)c * VEC, x);
        }
        i += step_rows;
        c += step_rem;
        if (c >= units) c -= units, ++i;
    }
}

// ------------------------------------------------------------------- sort
// Key of an ID: itself, or n_rows (sorted last) for one that takes no part.
// (Taken from loaded IDs, so that a thread's loads are all issued before the
// first is looked at.)
__device__ __forceinline__ uint32_t key_of(int32_t g, int64_t n_rows) {
    if (g < 0 || (int64_t)g >= n_rows) {
        if (g != -1) dev_err(ERR_INDEX);
        return (uint32_t)n_rows;
    }
    return (uint32_t)g;
}

// How the keys' bits are dealt to passes of `per` bits.
struct Digits {
    int32_t passes, per;
};

// Device state of the multi-block sort; cleared before every use.
struct SortState {
    uint32_t hist[kCopies][kMaxPasses][kDigits];
    uint32_t ticket[kMaxPasses + 1];  // tiles handed out (the last: of k_runs)
};

// The lanes of `valid` whose digit (below 256) is this lane's: one ballot a
// bit.  (match_any takes a turn for each distinct digit of the warp: measured
// 1,235 cycles for 16 items of few digits and 6,000 of many.)
__device__ __forceinline__ unsigned digit_peers(int32_t d, unsigned valid) {
    unsigned peers = valid;
#pragma unroll
    for (int b = 0; b < 8; ++b) {
        const bool bit = (d >> b) & 1;
        const unsigned with = __ballot_sync(0xFFFFFFFFu, bit);
        peers &= bit ? with : ~with;
    }
    return peers;
}

// Clears the sort's state.  (A kernel, so that the next one's launch overlaps it;
// with cudaMemsetAsync in its place the gradient of 65,536 positions of 1024 bf16
// columns takes 69.5 us, not 66.7.)
__global__ void __launch_bounds__(kThreads) k_sort_clear(uint4* __restrict__ p, int64_t words) {
    pdl_start();
    const int64_t i0 = blockIdx.x * (int64_t)(kThreads * 4) + threadIdx.x;
#pragma unroll
    for (int u = 0; u < 4; ++u)
        if (i0 + u * kThreads < words) p[i0 + u * kThreads] = make_uint4(0, 0, 0, 0);
}

// Digit counts of all passes, in kCopies copies (800,003 positions: 6 us; with one
// copy, whose counters 304 blocks add to in turn, 19).
__global__ void __launch_bounds__(kThreads) k_sort_hist(const int32_t* __restrict__ ids, int64_t n_rows, int64_t n_cap,
                                                        const int32_t* __restrict__ d_n, Digits dg,
                                                        SortState* __restrict__ st) {
    pdl_start();
    __shared__ uint32_t h[kMaxPasses][kDigits];
    for (int p = 0; p < dg.passes; ++p) h[p][threadIdx.x] = 0;
    __syncthreads();
    const int64_t n = count_of(d_n, n_cap), stride = (int64_t)gridDim.x * kThreads;
    const uint32_t mask = (1u << dg.per) - 1;
    for (int64_t i0 = blockIdx.x * (int64_t)kThreads; i0 < n; i0 += 8 * stride) {
        int32_t g[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int64_t i = i0 + u * stride + threadIdx.x;
            g[u] = i < n ? __ldg(ids + i) : -2;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (i0 + u * stride + threadIdx.x >= n) continue;
            const uint32_t k = key_of(g[u], n_rows);
            for (int p = 0; p < dg.passes; ++p) atomicAdd(&h[p][(k >> (p * dg.per)) & mask], 1u);
        }
    }
    __syncthreads();
    for (int p = 0; p < dg.passes; ++p)
        if (h[p][threadIdx.x]) atomicAdd(&st->hist[blockIdx.x % kCopies][p][threadIdx.x], h[p][threadIdx.x]);
}

// Ranks a warp's items (item i of lane l before item i of lane l + 1 and
// before item i + 1) within their digits: on return rank[i] counts the warp's
// earlier items of the same digit and cnt[digit] all of them.  Items that are
// not valid have digit -1.
template <int ITEMS, typename C>
__device__ __forceinline__ void warp_rank(const int32_t (&d)[ITEMS], C* cnt, uint32_t (&rank)[ITEMS]) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) rank[i] = digit_peers(d[i], __ballot_sync(0xFFFFFFFFu, d[i] >= 0));
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const unsigned peers = rank[i];
        const uint32_t before = __popc(peers & lanemask_lt());
        const uint32_t old = d[i] >= 0 ? cnt[d[i]] : 0;  // all lanes of a digit read the same count
        __syncwarp();
        if (d[i] >= 0 && before == 0) cnt[d[i]] = (C)(old + __popc(peers));
        __syncwarp();
        rank[i] = old + before;
    }
}

__device__ __forceinline__ uint32_t ld_relaxed(const uint32_t* p) {
    uint32_t v;
    asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void st_relaxed(uint32_t* p, uint32_t v) {
    asm volatile("st.relaxed.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// One pass: a stable scatter of (key, position) pairs by the pass's digit.
// Thread t looks back for digit t: status[tile][digit] = flag | count, flag 1
// the tile's own count, 2 the count up to and including the tile.  Tiles are
// handed out in order, so every tile looked at is running or done.  A pass of
// 800,003 positions (131 tiles): 13 us, latencies: 1,000 cycles for the loads, 5,000 for
// the ranks, 4,000 for the look-back.
template <int ITEMS>
__global__ void __launch_bounds__(kSortThreads, 1) k_sort_pass(const int32_t* __restrict__ ids, const uint2* __restrict__ in,
                                                        int64_t n_rows, int64_t n_cap, const int32_t* __restrict__ d_n,
                                                        int pass, int per, SortState* __restrict__ st,
                                                        uint32_t* __restrict__ status, uint2* __restrict__ out) {
    pdl_start();
    constexpr int kWarps = kSortThreads / 32, kTile = kSortThreads * ITEMS;
    __shared__ uint32_t cnt[kWarps][kDigits];
    __shared__ uint32_t sh[kWarps + 1];
    __shared__ uint32_t tile_sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool digit = threadIdx.x < kDigits;  // threads that look after a digit
    if (threadIdx.x == 0) tile_sh = atomicAdd(&st->ticket[pass], 1u);
    for (int i = threadIdx.x; i < kWarps * kDigits; i += kSortThreads) (&cnt[0][0])[i] = 0;
    __syncthreads();
    const uint32_t tile = tile_sh;
    const int64_t n = count_of(d_n, n_cap), i0 = (int64_t)tile * kTile + warp * 32 * ITEMS + lane;
    if ((int64_t)tile * kTile >= n) return;  // no later tile has items either
    uint32_t count = 0;
    if (digit)
#pragma unroll
        for (int c = 0; c < kCopies; ++c) count += st->hist[c][pass][threadIdx.x];
    uint2 kv[ITEMS];
    int32_t d[ITEMS];
    uint32_t rank[ITEMS];
    if (in) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
            kv[i] = i0 + i * 32 < n ? in[i0 + i * 32] : make_uint2(0, 0);
    } else {
        int32_t g[ITEMS];
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) g[i] = i0 + i * 32 < n ? __ldg(ids + i0 + i * 32) : -1;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) kv[i] = make_uint2(key_of(g[i], n_rows), (uint32_t)(i0 + i * 32));
    }
    uint32_t total;
    const uint32_t base = block_excl_scan<kSortThreads, uint32_t>(count, sh, total);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
        d[i] = i0 + i * 32 < n ? (int32_t)((kv[i].x >> (pass * per)) & ((1u << per) - 1)) : -1;
    warp_rank<ITEMS>(d, cnt[warp], rank);
    __syncthreads();
    if (digit) {
        uint32_t mine = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mine += cnt[w][threadIdx.x];
        uint32_t* word = status + (int64_t)tile * kDigits + threadIdx.x;
        uint32_t before = 0;
        if (tile == 0) {
            st_relaxed(word, (2u << 30) | mine);
        } else {
            st_relaxed(word, (1u << 30) | mine);
            // kBack tiles' words at a time: most tiles of one wave are still at
            // flag 1, so a walk one by one would cost a memory latency a tile
            constexpr int kBack = 16;
            int64_t t = (int64_t)tile - 1;  // next tile to add
            bool done = false;
            int spins = 0;
            while (!done && spins < kLookbackSpins) {
                uint32_t v[kBack];
#pragma unroll
                for (int u = 0; u < kBack; ++u) v[u] = t - u >= 0 ? ld_relaxed(word - (tile - t + u) * kDigits) : 2u << 30;
#pragma unroll
                for (int u = 0; u < kBack; ++u) {
                    if (done || (v[u] >> 30) == 0) {  // not there yet: ask again from here
                        ++spins;
                        break;
                    }
                    before += v[u] & 0x3FFFFFFFu;
                    done = (v[u] >> 30) == 2;
                    --t;
                }
            }
            const bool late = !done;
            if (late) dev_err(ERR_TIMEOUT);
            st_relaxed(word, (2u << 30) | (before + mine));
        }
        uint32_t run = base + before;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const uint32_t c = cnt[w][threadIdx.x];
            cnt[w][threadIdx.x] = run;
            run += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
        if (d[i] >= 0) {
            const uint32_t to = cnt[warp][d[i]] + rank[i];
            if (to < (uint32_t)n) out[to] = kv[i];  // always, unless a look-back gave up
        }
}

// starts[p / span] = distinct IDs before sorted position p, for every p that
// is a multiple of span (a power of two of at least 32) up to the end of the
// list; the number of distinct IDs follows at the end.  800,003 positions: 12 us,
// most of it the look-back's chain.
__global__ void __launch_bounds__(kThreads) k_runs(const uint2* __restrict__ kv, int64_t n_rows, int64_t n_cap,
                                                   const int32_t* __restrict__ d_n, int32_t span,
                                                   SortState* __restrict__ st, unsigned long long* __restrict__ status,
                                                   int32_t* __restrict__ starts, int32_t* __restrict__ n_out) {
    pdl_start();
    __shared__ int32_t sh[kThreads / 32 + 1];
    __shared__ int32_t tile_sh, before_sh;
    if (threadIdx.x == 0) tile_sh = (int32_t)atomicAdd(&st->ticket[kMaxPasses], 1u);
    __syncthreads();
    const int32_t tile = tile_sh;
    const int warp = (int)(threadIdx.x >> 5), lane = (int)lane_id();
    const int64_t n = count_of(d_n, n_cap), p0 = (int64_t)tile * kRunTile + warp * 512;  // a warp's 16 x 32 positions
    if ((int64_t)tile * kRunTile >= n) {
        if (tile == 0 && threadIdx.x == 0) *n_out = 0;
        return;
    }
    uint32_t k[16];
#pragma unroll
    for (int q = 0; q < 16; ++q) {
        const int64_t p = p0 + q * 32 + lane;
        k[q] = p < n ? kv[p].x : kNoKey;
    }
    uint32_t last = p0 > 0 && p0 - 1 < n ? kv[p0 - 1].x : kNoKey;
    int32_t before[16], mine = 0;  // run starts of the warp before round q
#pragma unroll
    for (int q = 0; q < 16; ++q) {
        const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, k[q], 1), prev = lane ? up : last;
        before[q] = mine;
        mine += __popc(__ballot_sync(0xFFFFFFFFu, k[q] < (uint32_t)n_rows && k[q] != prev));
        last = __shfl_sync(0xFFFFFFFFu, k[q], 31);
    }
    int32_t total;
    const int32_t e = block_excl_scan<kThreads, int32_t>(lane == 0 ? mine : 0, sh, total);  // lane 0: the warps before
    if (threadIdx.x < 32) {
        bool late = false;
        const int32_t x = chain_lookback(status, tile, 0, total, &late);
        if (late && threadIdx.x == 0) dev_err(ERR_TIMEOUT);
        if (threadIdx.x == 0) before_sh = x;
    }
    __syncthreads();
    if (lane == 0) {
#pragma unroll
        for (int q = 0; q < 16; ++q) {
            const int64_t p = p0 + q * 32;
            if (p < n && p % span == 0) starts[p / span] = before_sh + e + before[q];
        }
    }
    if (threadIdx.x == 0 && (int64_t)(tile + 1) * kRunTile >= n) {
        starts[(n + span - 1) / span] = before_sh + total;
        *n_out = before_sh + total;
    }
}

// All of it for a short list, in one block: up to 3 items a thread, passes in shared
// memory.
template <int ITEMS>
__global__ void __launch_bounds__(kSmallThreads) k_sort_small(const int32_t* __restrict__ ids, int64_t n_rows,
                                                              int32_t n_cap, const int32_t* __restrict__ d_n, Digits dg,
                                                              int32_t span, uint2* __restrict__ out,
                                                              int32_t* __restrict__ starts, int32_t* __restrict__ n_out) {
    pdl_start();
    constexpr int kItems = ITEMS, kWarps = kSmallThreads / 32, kParts = kSmallThreads / kDigits, kPer = kWarps / kParts;
    extern __shared__ __align__(16) uint8_t dsm[];
    uint32_t* key = reinterpret_cast<uint32_t*>(dsm);                            // [kSmallSort]
    uint16_t* pos = reinterpret_cast<uint16_t*>(key + kSmallSort);               // [kSmallSort]
    uint16_t(*cnt)[kDigits] = reinterpret_cast<uint16_t(*)[kDigits]>(pos + kSmallSort);  // [kWarps][kDigits]
    __shared__ uint32_t sh[kWarps + 1];
    __shared__ uint32_t psum[kParts][kDigits];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int digit = threadIdx.x % kDigits, q4 = threadIdx.x / kDigits;  // a digit, and kPer of the warps
    const int32_t n = (int32_t)count_of(d_n, n_cap);
    uint32_t k[kItems], v[kItems], rank[kItems], total;
    int32_t d[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        v[i] = (uint32_t)(warp * 32 * kItems + i * 32 + lane);
        d[i] = (int32_t)v[i] < n ? __ldg(ids + v[i]) : -1;
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) k[i] = (int32_t)v[i] < n ? key_of(d[i], n_rows) : kNoKey;
    for (int p = 0; p < dg.passes; ++p) {
        uint32_t* zero = reinterpret_cast<uint32_t*>(&cnt[warp][0]);
#pragma unroll
        for (int i = 0; i < kDigits / 64; ++i) zero[lane + 32 * i] = 0;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kItems; ++i)
            d[i] = k[i] != kNoKey ? (int32_t)((k[i] >> (p * dg.per)) & ((1u << dg.per) - 1)) : -1;
        warp_rank<kItems>(d, cnt[warp], rank);
        __syncthreads();
        uint32_t mine = 0;
#pragma unroll
        for (int w = 0; w < kPer; ++w) mine += cnt[q4 * kPer + w][digit];
        psum[q4][digit] = mine;
        __syncthreads();
        uint32_t all = 0, before = 0;
#pragma unroll
        for (int p4 = 0; p4 < kParts; ++p4) {
            all += psum[p4][digit];
            before += p4 < q4 ? psum[p4][digit] : 0;
        }
        const uint32_t e = block_excl_scan<kSmallThreads, uint32_t>(q4 == 0 ? all : 0, sh, total);
        if (q4 == 0) psum[0][digit] = e;  // (its own total has been read: the scan has barriers)
        __syncthreads();
        uint32_t run = psum[0][digit] + before;
#pragma unroll
        for (int w = 0; w < kPer; ++w) {
            const uint32_t c = cnt[q4 * kPer + w][digit];
            cnt[q4 * kPer + w][digit] = (uint16_t)run;
            run += c;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kItems; ++i)
            if (d[i] >= 0) {
                const uint32_t to = cnt[warp][d[i]] + rank[i];
                key[to] = k[i];
                pos[to] = (uint16_t)v[i];
            }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int32_t q = warp * 32 * kItems + i * 32 + lane;
            k[i] = q < n ? key[q] : kNoKey;
            v[i] = q < n ? pos[q] : 0;
        }
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const int32_t q = warp * 32 * kItems + i * 32 + lane;
        if (q < n) out[q] = make_uint2(k[i], v[i]);
    }
    if (!n_out) return;
    constexpr int kRun = 4;  // run starts, 4 positions a thread
    static_assert(kRun * kSmallThreads >= kSmallSort);
    const int32_t p0 = (int32_t)threadIdx.x * kRun;
    uint32_t prev = p0 > 0 && p0 - 1 < n ? key[p0 - 1] : kNoKey, mine = 0;
    for (int q = 0; q < kRun; ++q) {
        const uint32_t x = p0 + q < n ? key[p0 + q] : kNoKey;
        mine += x < (uint32_t)n_rows && x != prev;
        prev = x;
    }
    const uint32_t e = block_excl_scan<kSmallThreads, uint32_t>(mine, sh, total);
    if (p0 < n && p0 % span == 0) starts[p0 / span] = (int32_t)e;
    if (threadIdx.x == 0) {
        starts[(n + span - 1) / span] = (int32_t)total;
        *n_out = (int32_t)total;
    }
}
constexpr int kSmallSmem = kSmallSort * 6 + (kSmallThreads / 32) * kDigits * 2;

// A list of up to kClusterSort positions, in one launch: a cluster of CTAS
// blocks, block r holding positions [r, r + 1) ITEMS 1024 in every pass's
// order.  The blocks exchange their digit counts in shared memory and the
// pairs through memory (L2), written to their places and read back after a
// cluster barrier.  Measured, us for the whole gradient, this / a launch a
// pass: 20,000 positions of 1024 bf16 columns 48 / 52, of 64 fp32 columns
// 24 / 27; 40,000 of 256 fp32 columns 51 / 49.  (With the pairs sent straight
// into the other blocks' shared memory, 8 bytes at a time: 53 for the first.)
template <int ITEMS, int CTAS>
__global__ void __launch_bounds__(kSmallThreads) k_sort_cluster(const int32_t* __restrict__ ids, int64_t n_rows,
                                                                int32_t n_cap, const int32_t* __restrict__ d_n, Digits dg,
                                                                int32_t span, uint2* kv0, uint2* kv1,
                                                                int32_t* __restrict__ starts, int32_t* __restrict__ n_out) {
    pdl_start();
    constexpr int kWarps = kSmallThreads / 32, kParts = kSmallThreads / kDigits, kPer = kWarps / kParts;
    __shared__ __align__(16) uint16_t cnt[kWarps][kDigits];
    __shared__ uint32_t theirs[CTAS][kDigits];
    __shared__ uint32_t sh[kWarps + 1];
    __shared__ uint32_t psum[kParts][kDigits], base[kDigits];
    __shared__ uint32_t runs[CTAS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int digit = threadIdx.x % kDigits, q4 = threadIdx.x / kDigits;  // a digit, and kPer of the warps
    const uint32_t rank = cluster_rank();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");
    const int32_t n = (int32_t)count_of(d_n, n_cap);
    const int32_t first = (int32_t)rank * ITEMS * kSmallThreads + warp * 32 * ITEMS + lane;
    uint2 x[ITEMS];
    uint32_t rk[ITEMS], total;
    int32_t d[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) d[i] = first + i * 32 < n ? __ldg(ids + first + i * 32) : -1;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
        x[i] = make_uint2(first + i * 32 < n ? key_of(d[i], n_rows) : kNoKey, (uint32_t)(first + i * 32));
    for (int p = 0; p < dg.passes; ++p) {
        uint2* to_kv = p & 1 ? kv1 : kv0;
        uint32_t* zero = reinterpret_cast<uint32_t*>(&cnt[warp][0]);
#pragma unroll
        for (int i = 0; i < kDigits / 64; ++i) zero[lane + 32 * i] = 0;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
            d[i] = x[i].x != kNoKey ? (int32_t)((x[i].x >> (p * dg.per)) & ((1u << dg.per) - 1)) : -1;
        warp_rank<ITEMS>(d, cnt[warp], rk);
        __syncthreads();
        uint32_t part = 0;
#pragma unroll
        for (int w = 0; w < kPer; ++w) part += cnt[q4 * kPer + w][digit];
        psum[q4][digit] = part;
        __syncthreads();
        uint32_t all = 0, run = 0, lower = 0;  // this block's; of the warps before; of the blocks before
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
            all += psum[k][digit];
            run += k < q4 ? psum[k][digit] : 0;
        }
        // every block runs: its shared memory may be written
        if (p == 0) asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");
#pragma unroll
        for (int c = 0; c < CTAS / kParts; ++c)
            asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(
                             map_rank(smem_addr(&theirs[rank][digit]), (uint32_t)(c * kParts + q4))),
                         "r"(all)
                         : "memory");
        cluster_sync();
        all = 0;
#pragma unroll
        for (uint32_t c = 0; c < CTAS; ++c) {
            all += theirs[c][digit];
            lower += c < rank ? theirs[c][digit] : 0;
        }
        const uint32_t e = block_excl_scan<kSmallThreads, uint32_t>(q4 == 0 ? all : 0, sh, total);
        if (q4 == 0) base[digit] = e + lower;
#pragma unroll
        for (int w = 0; w < kPer; ++w) {
            const uint32_t c = cnt[q4 * kPer + w][digit];
            cnt[q4 * kPer + w][digit] = (uint16_t)run;
            run += c;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
            if (d[i] >= 0) to_kv[base[d[i]] + cnt[warp][d[i]] + rk[i]] = x[i];
        if (p + 1 == dg.passes && !n_out) return;
        cluster_sync();
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)  // (past L1, which may hold what an earlier pass read here)
            x[i] = first + i * 32 < n ? __ldcg(to_kv + first + i * 32) : make_uint2(kNoKey, 0);
    }
    // run starts: round i of a warp is 32 positions in a row
    uint32_t last = first - lane > 0 && first - lane - 1 < n ? __ldcg(((dg.passes & 1 ? kv0 : kv1) + first - lane - 1)).x : kNoKey;
    int32_t before[ITEMS], mine = 0;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, x[i].x, 1), prev = lane ? up : last;
        before[i] = mine;
        mine += __popc(__ballot_sync(0xFFFFFFFFu, x[i].x < (uint32_t)n_rows && x[i].x != prev));
        last = __shfl_sync(0xFFFFFFFFu, x[i].x, 31);
    }
    int32_t e = (int32_t)block_excl_scan<kSmallThreads, uint32_t>(lane == 0 ? (uint32_t)mine : 0, sh, total);
    if (threadIdx.x < CTAS)
        asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(map_rank(smem_addr(runs + rank), threadIdx.x)), "r"(total)
                     : "memory");
    cluster_sync();
    uint32_t sum = 0;
#pragma unroll
    for (uint32_t c = 0; c < CTAS; ++c) {
        e += c < rank ? (int32_t)runs[c] : 0;
        sum += runs[c];
    }
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
            if (first + i * 32 < n && (first + i * 32) % span == 0) starts[(first + i * 32) / span] = e + before[i];
    }
    if (rank == 0 && threadIdx.x == 0) {
        starts[(n + span - 1) / span] = (int32_t)sum;
        *n_out = (int32_t)sum;
    }
}

// ------------------------------------------------------- runs of equal IDs
template <typename TO>
struct SumArgs {
    const uint2* kv;  // sorted (ID, position)
    const int32_t* d_n;
    int64_t n_cap, n_rows;
    int64_t ld_g;
    int32_t dim, units, col_blocks, lanes;  // units of VEC columns; lanes that cover a column block
    int32_t mode;
    float scale;
    const int32_t* starts;  // SG_GRAD_ROWS: distinct IDs before each tile
    int32_t* rows;
    TO* grad;
    int64_t ld_grad;
    float* head;          // [tiles][dim] sums of runs that began in an earlier tile
    float* tail;          // [tiles][dim] sums of runs that go on in the next tile
    int32_t zero_blocks;  // SG_GRAD_DENSE: blocks that fill the rows without an ID
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

// Zero rows for the IDs that do not occur: a warp looks kZeroRows IDs up in the
// sorted list, a lane each, first among kSamples keys that the block has taken
// at equal distances into shared memory (a search in memory alone costs a
// latency a step: 16 for 65,536 positions, instead of 5).
constexpr int kSamples = 2048;
constexpr int kZeroRows = 8;  // few, so that the rows of a wide table spread evenly over the SMs
template <typename TO, int VEC>
__device__ __forceinline__ void zero_rows(const SumArgs<TO>& a, int64_t n, int32_t block, uint32_t* sample) {
    const int lane = (int)lane_id();
    const int64_t every = n > kSamples ? cdiv(n, kSamples) : 1;
    const int32_t samples = n > 0 ? (int32_t)cdiv(n, every) : 0;
#pragma unroll
    for (int u = 0; u < kSamples / kThreads; ++u) {
        const int32_t i = u * kThreads + (int32_t)threadIdx.x;
        if (i < samples) sample[i] = __ldg(&a.kv[i * every].x);
    }
    __syncthreads();
    const int64_t r0 = ((int64_t)block * (kThreads / 32) + (threadIdx.x >> 5)) * kZeroRows;
    if (r0 >= a.n_rows) return;
    const uint32_t id = (uint32_t)(r0 + lane % kZeroRows);
    int32_t s0 = 0, s1 = samples;  // first sample that is not below id
    while (s0 < s1) {
        const int32_t mid = (s0 + s1) >> 1;
        if (sample[mid] < id) s0 = mid + 1;
        else s1 = mid;
    }
    int64_t lo = s0 > 0 ? (s0 - 1) * every + 1 : 0, hi = s0 < samples ? s0 * every : n;
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (__ldg(&a.kv[mid].x) < id) lo = mid + 1;
        else hi = mid;
    }
    const bool absent = (int64_t)id < a.n_rows && (lo >= n || __ldg(&a.kv[lo].x) != id);
    const float none[VEC] = {};
    for (unsigned todo = __ballot_sync(0xFFFFFFFFu, absent && lane < kZeroRows); todo; todo &= todo - 1) {
        TO* p = a.grad + (r0 + __ffs(todo) - 1) * a.ld_grad;
        for (int32_t u = lane; u < a.units; u += 32) store_vec<VEC>(p + (int64_t)u * VEC, none);
    }
}

// A block takes a tile of the sorted list and a column block of a.lanes units;
// a group of a.lanes lanes takes a chunk of CH positions of it.  Memory bounds it:
// 800,003 positions of 256 fp32 columns 167 us (6.7 TB/s), 65,536 of 1024 bf16
// columns with the zero rows of a 50,001-row gradient 40 us (5.4 TB/s: short, and
// its runs are uneven).
template <typename TI, typename TO, int VEC, int CH>
__global__ void __launch_bounds__(kThreads) k_embed_sum(const TI* __restrict__ g, SumArgs<TO> a) {
    pdl_start();
    constexpr int kMaxTile = CH == 32 ? 1024 : 2048;  // 32-long chunks go with 8 lanes or more
    __shared__ uint2 kv[kMaxTile + 2];                // the tile's pairs, and one on either side
    __shared__ __align__(16) float part[kThreads * VEC];  // the chunks' heads
    __shared__ int32_t first[kThreads];
    __shared__ int32_t sh[kThreads / 32 + 1];
    const int64_t n = count_of(a.d_n, a.n_cap);
    int32_t block = (int32_t)blockIdx.x;
    if (a.zero_blocks) {
        // zero blocks are spread evenly over the grid: their look-ups are latency, the sums bandwidth
        const int32_t z = (int32_t)(((int64_t)block * a.zero_blocks) / gridDim.x);
        if ((int32_t)(((int64_t)(block + 1) * a.zero_blocks) / gridDim.x) != z) {
            zero_rows<TO, VEC>(a, n, z, reinterpret_cast<uint32_t*>(kv));
            return;
        }
        block -= z;
    }
    const int32_t tile = block / a.col_blocks, cb = block - tile * a.col_blocks;
    const int32_t chunks = kThreads / a.lanes, span = chunks * CH;
    const int64_t p0 = (int64_t)tile * span;
    if (p0 >= n) return;
    for (int32_t i = threadIdx.x; i < span + 2; i += kThreads) {
        const int64_t p = p0 - 1 + i;
        kv[i] = p >= 0 && p < n ? a.kv[p] : make_uint2(kNoKey, 0);
    }
    __syncthreads();
    const int32_t chunk = (int32_t)threadIdx.x / a.lanes, lane = (int32_t)threadIdx.x - chunk * a.lanes;
    const int32_t unit = cb * a.lanes + lane, col = unit * VEC;
    const bool active = unit < a.units;
    const uint2* c = kv + 1 + chunk * CH;  // the chunk; c[-1], c[CH] are its neighbours
    const uint32_t none = (uint32_t)a.n_rows;
    int32_t j = 0;
    if (a.mode == SG_GRAD_ROWS) {  // distinct IDs before the chunk
        int32_t starts = 0;
        if (lane == 0)
            for (int i = 0; i < CH; ++i) starts += c[i].x < none && c[i].x != c[i - 1].x;
        int32_t total;
        const int32_t e = block_excl_scan<kThreads, int32_t>(starts, sh, total);
        if (lane == 0) first[chunk] = a.starts[tile] + e;
        __syncthreads();
        j = first[chunk];
    }
    float acc[VEC];
#pragma unroll
    for (int q = 0; q < VEC; ++q) acc[q] = 0.f;
    uint32_t key = c[0].x;
    const bool any = key < none && active;
    const bool enters = any && c[-1].x == key;  // the first run began before this chunk
    bool head = enters;
    if (head) --j;
    float* my_head = &part[threadIdx.x * VEC];
    if (any) {
#pragma unroll 1
        for (int b = 0; b < CH; b += kUnroll) {
            if (c[b].x >= none) break;
            Raw<TI, VEC> v[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (c[b + u].x < none) v[u].load(g + (int64_t)(int32_t)c[b + u].y * a.ld_g + col);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const uint32_t k = c[b + u].x;
                if (k >= none) continue;
                if (k != key) {
                    if (head) store_vec<VEC>(my_head, acc);
                    else put_row<TO, VEC>(a, key, j, col, acc);
                    head = false;
                    ++j;
                    key = k;
#pragma unroll
                    for (int q = 0; q < VEC; ++q) acc[q] = 0.f;
                }
#pragma unroll
                for (int q = 0; q < VEC; ++q) acc[q] += v[u][q];
            }
        }
        if (head) store_vec<VEC>(my_head, acc);
    }
    const bool goes_on = any && !head && c[CH].x == key;  // the last run began here and goes on
    if (any && !head && !goes_on) put_row<TO, VEC>(a, key, j, col, acc);
    __syncthreads();
    // joins within the tile: the chunk a run begins in adds the heads of the
    // chunks it enters; chunk 0 does so for the run that enters the tile
    const auto add_heads = [&](uint32_t id) {
        int32_t d = chunk + 1;
        for (; d < chunks && kv[1 + d * CH].x == id; ++d) {
            const float* h = &part[(d * a.lanes + lane) * VEC];
#pragma unroll
            for (int q = 0; q < VEC; ++q) acc[q] += h[q];
        }
        return d;
    };
    if (goes_on) {
        const int32_t d = add_heads(key);
        if (d == chunks && kv[1 + span].x == key) store_vec<VEC>(a.tail + (int64_t)tile * a.dim + col, acc);
        else put_row<TO, VEC>(a, key, j, col, acc);
    }
    if (enters && chunk == 0) {
#pragma unroll
        for (int q = 0; q < VEC; ++q) acc[q] = my_head[q];
        add_heads(c[0].x);
        store_vec<VEC>(a.head + (int64_t)tile * a.dim + col, acc);
    }
}

// Joins the runs that cross tiles: the tile a run begins in adds, in order,
// its tail and the heads of the tiles the run enters.  A warp looks at one
// tile and column block and joins a short run itself; a run of more than
// kUnroll heads is split over the block's warps, whose sums are then added in
// order (800,003 positions of a power-law list: 13 us; a warp alone, 692, for a run of
// 1,075 heads).
template <typename TO, int VEC>
__global__ void __launch_bounds__(kThreads) k_embed_join(SumArgs<TO> a, int32_t span, int64_t items) {
    pdl_start();
    constexpr int kWarps = kThreads / 32;
    __shared__ __align__(16) float part[kWarps][32 * VEC];
    __shared__ int32_t heads[kWarps];  // of the run that begins in the warp's tile
    const int64_t n = count_of(a.d_n, a.n_cap);
    const int warp = (int)(threadIdx.x >> 5), lane = (int)lane_id();
    const int64_t item0 = (int64_t)blockIdx.x * kWarps;
    // the key whose run begins in tile t and goes on, or kNoKey
    const auto owned = [&](int64_t t) {
        const int64_t p0 = t * span, p1 = p0 + span;
        if (p1 >= n) return kNoKey;
        const uint32_t k0 = p0 > 0 ? a.kv[p0 - 1].x : kNoKey, k1 = a.kv[p0].x, k2 = a.kv[p1 - 1].x, k3 = a.kv[p1].x;
        if (k2 >= (uint32_t)a.n_rows || k3 != k2 || (k1 == k2 && k0 == k2)) return kNoKey;
        return k2;
    };
    const auto add = [&](float (&acc)[VEC], int64_t t0, int64_t t1, int32_t col) {
        for (int64_t t = t0; t < t1; t += kUnroll) {
            float v[kUnroll][VEC];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (t + u < t1) load_vec<VEC>(a.head + (t + u) * a.dim + col, v[u]);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (t + u < t1)
#pragma unroll
                    for (int q = 0; q < VEC; ++q) acc[q] += v[u][q];
        }
    };
    {
        const int64_t item = item0 + warp, tile = item / a.col_blocks;
        const uint32_t key = item < items ? owned(tile) : kNoKey;
        int32_t count = 0;
        if (key != kNoKey) {  // the same in the whole warp
            // last tile the run enters: 32 probes at a time
            int64_t lo = tile + 1, hi = (n - 1) / span;  // tile lo is entered, tiles past hi do not exist
            while (lo < hi) {
                const int64_t step = (hi - lo + 31) / 32, t = lo + (lane + 1) * step;
                const bool in = t <= hi && a.kv[t * span].x == key;
                const int hits = __popc(__ballot_sync(0xFFFFFFFFu, in));  // a prefix of the lanes
                lo += hits * step;
                if (hits < 32) hi = lo + step - 1 < hi ? lo + step - 1 : hi;
            }
            count = (int32_t)(lo - tile);
            const int32_t unit = (int32_t)(item - tile * a.col_blocks) * a.lanes + lane, col = unit * VEC;
            if (count <= kUnroll && lane < a.lanes && unit < a.units) {
                float acc[VEC];
                load_vec<VEC>(a.tail + tile * a.dim + col, acc);
                add(acc, tile + 1, tile + 1 + count, col);
                put_row<TO, VEC>(a, key, a.mode == SG_GRAD_ROWS ? a.starts[tile + 1] - 1 : 0, col, acc);
            }
        }
        if (lane == 0) heads[warp] = count;
    }
    __syncthreads();
#pragma unroll 1
    for (int w = 0; w < kWarps; ++w) {
        const int32_t count = heads[w];
        if (count <= kUnroll) continue;
        const int64_t item = item0 + w, tile = item / a.col_blocks;
        const int32_t unit = (int32_t)(item - tile * a.col_blocks) * a.lanes + lane, col = unit * VEC;
        const bool active = lane < a.lanes && unit < a.units;
        const int64_t per = (count + kWarps - 1) / kWarps, t0 = min((int64_t)count, warp * per), t1 = min((int64_t)count, t0 + per);
        float acc[VEC];
#pragma unroll
        for (int q = 0; q < VEC; ++q) acc[q] = 0.f;
        if (active) {
            if (warp == 0) load_vec<VEC>(a.tail + tile * a.dim + col, acc);
            add(acc, tile + 1 + t0, tile + 1 + t1, col);
            store_vec<VEC>(&part[warp][lane * VEC], acc);
        }
        __syncthreads();
        if (warp == 0 && active) {
            for (int i = 1; i < kWarps; ++i)
#pragma unroll
                for (int q = 0; q < VEC; ++q) acc[q] += part[i][lane * VEC + q];
            const uint32_t key = a.kv[(tile + 1) * span].x;
            put_row<TO, VEC>(a, key, a.mode == SG_GRAD_ROWS ? a.starts[tile + 1] - 1 : 0, col, acc);
        }
        __syncthreads();
    }
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
    const int64_t blocks = cdiv(n_cap * units, kThreads * kUnroll);
    if (blocks > 2147483647LL) return fail(SG_ERR_INVALID_ARG, "sg_embed_fwd: n_cap x dim too large");
    SG_CUDA(launch_pdl(k_embed_fwd<TI, TO, VEC>, dim3((unsigned)blocks), dim3(kThreads), 0, s, (const TI*)table, n_rows,
                       ld_table, ids, n_cap, d_n, scale, units, (int32_t)(kThreads / units), (int32_t)(kThreads % units),
                       (TO*)out, ld_out));
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

// How the sum is cut for units of vec columns.  A chunk is 32 positions, or 8
// (one batch of loads) when that leaves too few blocks.  Measured, us for the
// whole gradient, 8 / 32: 256 fp32 columns, 4,999 positions (40 blocks of 32)
// 28 / 31, 20,000 (158 blocks) 43 / 42; 1024 bf16 columns, 4,999 positions (80
// blocks) 49 / 40, 65,536 (1,024 blocks) 85 / 75.
struct Cut {
    int32_t units, lanes, col_blocks, span;  // span: positions of a tile
    int64_t most;                            // tiles of a list of up to n_cap positions
};
Cut cut_for(int64_t n_cap, int32_t dim, int vec) {
    Cut c;
    c.units = dim / vec;
    c.lanes = 1;
    while (c.lanes < 32 && c.lanes < c.units) c.lanes *= 2;
    c.col_blocks = (int32_t)cdiv(c.units, c.lanes);
    const int32_t chunks = kThreads / c.lanes;
    const bool wide = c.lanes >= 8 && cdiv(n_cap, chunks * 32) * c.col_blocks >= kFewBlocks;
    c.span = chunks * (wide ? 32 : 8);
    c.most = cdiv(n_cap, c.span);
    if (wide) {  // the longest list of short chunks, which may have more tiles
        const int64_t few = (int64_t)((kFewBlocks - 1) / c.col_blocks) * 4;
        if (few > c.most) c.most = few;
    }
    return c;
}

struct BwdLayout {
    int64_t tiles;       // bound on the sum's tiles, of this list and of every shorter one
    int64_t sort_tiles;  // bound on a pass's tiles
    size_t kv0, kv1, state, status, run_status, starts, head, tail, total;  // state .. status: cleared for a sort
};

BwdLayout bwd_layout(int64_t n_cap, int32_t dim) {
    BwdLayout L;
    L.tiles = 0;
    for (int vec = 1; vec <= 8; vec *= 2)  // the strides and addresses decide between units of 1, 4 and 8
        if (vec != 2 && dim % vec == 0) {
            const int64_t t = cut_for(n_cap, dim, vec).most;
            if (t > L.tiles) L.tiles = t;
        }
    L.sort_tiles = n_cap <= kSmallSort ? 0 : cdiv(n_cap, kSortThreads * 4);
    size_t o = 0;
    const auto put = [&o](size_t bytes) {
        const size_t at = o;
        o += a256(bytes);
        return at;
    };
    L.kv0 = put((size_t)n_cap * 8);
    L.kv1 = put((size_t)n_cap * 8);
    L.state = put(sizeof(SortState));
    L.run_status = put((size_t)cdiv(n_cap, kRunTile) * 8);
    L.status = put((size_t)L.sort_tiles * kDigits * kMaxPasses * 4);
    L.starts = put((size_t)(L.tiles + 2) * 4);
    L.head = put((size_t)L.tiles * dim * 4);
    L.tail = put((size_t)L.tiles * dim * 4);
    L.total = o;
    return L;
}

template <typename TI, typename TO, int VEC>
sg_status launch_sum(const void* g, SumArgs<TO> a, int32_t span, cudaStream_t s) {
    const int64_t tiles = cdiv(a.n_cap, span), blocks = tiles * a.col_blocks;
    const int64_t zero = a.mode == SG_GRAD_DENSE ? cdiv(a.n_rows, kThreads / 32 * kZeroRows) : 0;
    if (blocks + zero > 2147483647LL) return fail(SG_ERR_INVALID_ARG, "sg_embed_bwd: n_cap x dim too large");
    a.zero_blocks = (int32_t)zero;
    if (span * a.lanes == kThreads * 32)
        SG_CUDA(launch_pdl(k_embed_sum<TI, TO, VEC, 32>, dim3((unsigned)(blocks + zero)), dim3(kThreads), 0, s,
                           (const TI*)g, a));
    else
        SG_CUDA(launch_pdl(k_embed_sum<TI, TO, VEC, 8>, dim3((unsigned)(blocks + zero)), dim3(kThreads), 0, s,
                           (const TI*)g, a));
    if (tiles > 1)
        SG_CUDA(launch_pdl(k_embed_join<TO, VEC>, dim3((unsigned)cdiv(blocks, kThreads / 32)), dim3(kThreads), 0, s, a,
                           span, blocks));
    return SG_OK;
}

template <typename TI, typename TO>
sg_status run_sum(int vec, const void* g, const SumArgs<TO>& a, int32_t span, cudaStream_t s) {
    if constexpr (sizeof(TI) == 2)
        if (vec == 8) return launch_sum<TI, TO, 8>(g, a, span, s);
    if (vec == 4) return launch_sum<TI, TO, 4>(g, a, span, s);
    return launch_sum<TI, TO, 1>(g, a, span, s);
}

// A launch of the sort by one cluster of CTAS blocks; at: its two attributes.
template <int CTAS>
cudaLaunchConfig_t cluster_config(cudaLaunchAttribute (&at)[2], cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CTAS);
    cfg.blockDim = dim3(kSmallThreads);
    cfg.stream = s;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = CTAS;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cfg;
}

// Whether the current device takes such a cluster (looked up once for each
// device): a part of a device may have fewer SMs side by side than it needs.
template <int ITEMS, int CTAS>
bool cluster_fits() {
    static OncePerDevice set;
    static std::atomic<uint64_t> yes{0};  // by device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        return false;
    }
    set(dev, [&] {
        cudaLaunchAttribute at[2];
        cudaLaunchConfig_t cfg = cluster_config<CTAS>(at, nullptr);
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaFuncSetAttribute(k_sort_cluster<ITEMS, CTAS>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
            cudaOccupancyMaxActiveClusters(&n, k_sort_cluster<ITEMS, CTAS>, &cfg) == cudaSuccess && n > 0)
            yes.fetch_or((uint64_t)1 << dev);
        else
            cudaGetLastError();
        return 0;
    });
    return (yes.load() >> dev) & 1;
}

// Sorts by one cluster of CTAS blocks; *taken: whether the device takes it.
template <int ITEMS, int CTAS>
cudaError_t sort_by_cluster(const int32_t* ids, int64_t n_rows, int64_t n_cap, const int32_t* d_n, Digits dg, int32_t span,
                            uint2* const (&kv)[2], int32_t* starts, int32_t* n_out, cudaStream_t s, bool* taken) {
    *taken = cluster_fits<ITEMS, CTAS>();
    if (!*taken) return cudaSuccess;
    cudaLaunchAttribute at[2];
    const cudaLaunchConfig_t cfg = cluster_config<CTAS>(at, s);
    return cudaLaunchKernelEx(&cfg, k_sort_cluster<ITEMS, CTAS>, ids, n_rows, (int32_t)n_cap, d_n, dg, span, kv[0], kv[1], starts,
                              n_out);
}

// Sorted pairs in *sorted; with rows, the distinct IDs before each tile of
// `span` positions in starts.
sg_status run_sort(const int32_t* ids, int64_t n_cap, const int32_t* d_n, int64_t n_rows, bool rows, int32_t span,
                   int32_t* n_out, const BwdLayout& L, char* ws, uint2** sorted, cudaStream_t s) {
    uint2* kv[2] = {(uint2*)(ws + L.kv0), (uint2*)(ws + L.kv1)};
    SortState* st = (SortState*)(ws + L.state);
    int32_t* starts = (int32_t*)(ws + L.starts);
    int bits = 1;
    while (bits < 32 && (n_rows >> bits) != 0) ++bits;  // keys 0 .. n_rows
    Digits dg;
    dg.passes = (bits + 7) / 8;
    dg.per = (bits + dg.passes - 1) / dg.passes;
    *sorted = kv[0];
    if (n_cap <= kSmallSort) {
        const int32_t items = (int32_t)cdiv(n_cap, kSmallThreads);  // a thread
        const auto go = [&](auto kernel) {
            return launch_pdl(kernel, dim3(1), dim3(kSmallThreads), kSmallSmem, s, ids, n_rows, (int32_t)n_cap, d_n, dg,
                              span, kv[0], starts, rows ? n_out : nullptr);
        };
        static OncePerDevice set1, set3;
        SG_CUDA(allow_smem(set1, k_sort_small<1>, kSmallSmem));
        SG_CUDA(allow_smem(set3, k_sort_small<3>, kSmallSmem));
        SG_CUDA(items <= 1 ? go(k_sort_small<1>) : go(k_sort_small<3>));
        return SG_OK;
    }
    if (n_cap <= kClusterSort) {
        int32_t* const distinct = rows ? n_out : nullptr;
        const auto sort = n_cap <= kClusterSort / 4   ? sort_by_cluster<1, kSortCtas / 2>
                          : n_cap <= kClusterSort / 2 ? sort_by_cluster<1, kSortCtas>
                                                      : sort_by_cluster<2, kSortCtas>;
        bool taken = false;
        SG_CUDA(sort(ids, n_rows, n_cap, d_n, dg, span, kv, starts, distinct, s, &taken));
        *sorted = kv[(dg.passes & 1) ^ 1];
        if (taken) return SG_OK;
    }
    // the fewest items a thread (4, 8 or 12) with which every tile has an SM of
    // its own: two tiles on an SM take twice as long as one, and every later
    // tile waits for them (us for the whole gradient of 256 columns, 4 / 8 / 12:
    // 100,000 positions 65 / 70 / -, 620,000 191 / 189 / 193, 800,003 242 / 245 / 238)
    const int64_t wave = (int64_t)num_sms() * kSortThreads;
    const int items = n_cap <= 4 * wave ? 4 : n_cap <= 8 * wave ? 8 : 12;
    const int64_t tiles = cdiv(n_cap, kSortThreads * items);
    const int64_t words = (int64_t)(L.status - L.state) / 16 + dg.passes * tiles * (kDigits / 4);  // of 16 bytes
    SG_CUDA(launch_pdl(k_sort_clear, dim3((unsigned)cdiv(words, kThreads * 4)), dim3(kThreads), 0, s,
                       (uint4*)(ws + L.state), words));
    const int64_t hb = cdiv(n_cap, kThreads * 8) < num_sms() * 2 ? cdiv(n_cap, kThreads * 8) : num_sms() * 2;
    SG_CUDA(launch_pdl(k_sort_hist, dim3((unsigned)hb), dim3(kThreads), 0, s, ids, n_rows, n_cap, d_n, dg, st));
    for (int p = 0; p < dg.passes; ++p) {
        uint32_t* status = (uint32_t*)(ws + L.status) + p * tiles * kDigits;
        const uint2* in = p ? kv[(p & 1) ^ 1] : nullptr;
        uint2* out = kv[p & 1];
        const auto kernel = items == 4 ? k_sort_pass<4> : items == 8 ? k_sort_pass<8> : k_sort_pass<12>;
        SG_CUDA(launch_pdl(kernel, dim3((unsigned)tiles), dim3(kSortThreads), 0, s, ids, in, n_rows, n_cap, d_n, p,
                           (int)dg.per, st, status, out));
        *sorted = out;
    }
    if (rows)
        SG_CUDA(launch_pdl(k_runs, dim3((unsigned)cdiv(n_cap, kRunTile)), dim3(kThreads), 0, s, (const uint2*)*sorted,
                           n_rows, n_cap, d_n, span, st, (unsigned long long*)(ws + L.run_status), starts, n_out));
    return SG_OK;
}

template <typename TO>
sg_status run_bwd(const int32_t* ids, int64_t n_cap, const int32_t* d_n, int64_t n_rows, const void* g, int32_t dtype_g,
                  int32_t dim, int64_t ld_g, float scale, int32_t mode, int32_t* rows, int32_t* n_out, TO* grad,
                  int32_t dtype_grad, int64_t ld_grad, char* ws, cudaStream_t s) {
    const BwdLayout L = bwd_layout(n_cap, dim);
    const int vec = vec_for(g, dtype_g, ld_g, grad, dtype_grad, ld_grad, dim);
    SumArgs<TO> a;
    memset(&a, 0, sizeof(a));
    const Cut cut = cut_for(n_cap, dim, vec);
    a.units = cut.units;
    a.lanes = cut.lanes;
    a.col_blocks = cut.col_blocks;
    const int32_t span = cut.span;
    uint2* sorted = nullptr;
    const sg_status st = run_sort(ids, n_cap, d_n, n_rows, mode == SG_GRAD_ROWS, span, n_out, L, ws, &sorted, s);
    if (st != SG_OK) return st;
    a.kv = sorted;
    a.d_n = d_n;
    a.n_cap = n_cap;
    a.n_rows = n_rows;
    a.ld_g = ld_g;
    a.dim = dim;
    a.mode = mode;
    a.scale = scale;
    a.starts = (const int32_t*)(ws + L.starts);
    a.rows = rows;
    a.grad = grad;
    a.ld_grad = ld_grad;
    a.head = (float*)(ws + L.head);
    a.tail = (float*)(ws + L.tail);
    return dtype_g == SG_F32 ? run_sum<float, TO>(vec, g, a, span, s) : run_sum<__nv_bfloat16, TO>(vec, g, a, span, s);
}

}  // namespace

extern "C" sg_status sg_embed_fwd(const void* d_table, int32_t dtype_table, int64_t n_rows, int32_t dim,
                                  int64_t ld_table, const int32_t* d_ids, int64_t n_cap, const int32_t* d_n,
                                  float scale, void* d_out, int32_t dtype_out, int64_t ld_out, sg_stream_t stream) {
    if (!dtype_ok(dtype_table) || !dtype_ok(dtype_out)) return fail(SG_ERR_UNSUPPORTED, "sg_embed_fwd: dtype");
    if (n_rows < 0 || n_rows > 2147483647LL || n_cap < 0 || n_cap >= (1LL << 30) || dim <= 0)
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
    if (n_cap <= 0 || n_cap >= (1LL << 30) || n_rows <= 0 || n_rows > 2147483647LL || dim <= 0 || mode < SG_GRAD_ROWS ||
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
    if (n_cap < 0 || n_cap >= (1LL << 30) || n_rows <= 0 || n_rows > 2147483647LL || dim <= 0)
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
