// Orthogonalised updates (the Muon optimiser's step) by Newton-Schulz products:
//   X = U / (||U||_F + eps), on the smaller side (transposed when rows > cols)
//   steps times:  A = X X^T;  B = a I + b A + c A A;  X <- B X
// with U the matrix itself (sg_orthogonalise) or the momentum update of
// sg_muon_step, and the weights updated from the result.
//
// Here m = min(rows, cols), n = max(rows, cols); X is held as m rows of n.
//
// Number format.  The iteration multiplies small singular values by up to
// a = 3.44 a step (485 in five), and an operand's rounding error with them, so
// one 16-bit operand a product (off by up to 2^-8 in bf16, 2^-11 in fp16) would leave
// errors of a percent and more.  Every operand is held as two fp16 terms,
// hi + lo, of 256 times its value: the iterates are bounded (singular values
// up to about 1.2), so 256 x stays inside fp16's range, and the pair carries 22
// bits while lo is above fp16's subnormals (entries from 2^-11, 5e-4); below, x is off by
// up to 2^-33 (half of lo's last step).  A first iterate's entry is about 1 / sqrt(m n):
// 5e-4 for 1024 x 4096, 4e-5 at the largest sizes (18 bits).  A product is three tensor-core
// products, hi hi + hi lo + lo hi, with fp32 accumulation in tensor memory.
// Folding a I into B makes X <- B X one product with nothing to add.
// The tensor core cuts a sum's low bits at every accumulation, always towards
// zero.  So the two cross products, 2^-11 as large, have an accumulator of their
// own, and hi hi is taken out of tensor memory every 4 or 8 accumulations and
// summed in registers.  Relative error and time, 1024 x 4096: 1.9e-5 with all
// accumulations in one place; 6.7e-6 and 263 us with 16 or 32 in one; 3.4e-6, 266
// with 8 or 16; 1.9e-6, 276 with 4 or 8 (fp32 products: 3.8e-6; the pairs
// themselves, in exact arithmetic: 5e-7).  512 x 2048: 6.5, 5.6 and 3.1e-6 (fp32 3.4e-6).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <string.h>

#include "sg_internal.cuh"
#include "sg_tc.cuh"

SGI_ERROR_WORD(muon)

using namespace sgi;

namespace {

constexpr int kThreads = 256;
constexpr int kNormParts = 256;  // partial sums of squares of a matrix, at most
constexpr float kScale = 256.f;  // of every fp16 pair
constexpr int kTile = 128;       // rows of an output tile (and columns of a symmetric one)
constexpr int kBK = 64;          // K elements of a stage: one 128-byte swizzle row
constexpr int kOperand = kTile * kBK * 2;  // bytes of one operand tile: 16 KB
// A product's block: kSumWarps warps sum and write the tile, one more feeds the
// copies, one the tensor core.
constexpr int kSumWarps = kThreads / 32;
constexpr int kProductThreads = kThreads + 64;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// A matrix held as two fp16 planes of `ld` columns (a multiple of 8).
struct Planes {
    __half* hi;
    __half* lo;
};

// What enters: a matrix of type T (mom_out NULL), or gradient and momentum.
template <typename T>
struct Source {
    const T* g;
    int64_t ld;
    const float* mom;
    float* mom_out;
    float mu;
    int32_t nesterov;
    int32_t vec;  // 1: g, 2: the momentum may be read 16 bytes at a time
};

// Two values as packed hi and lo.  (x - hi is exact, in one instruction that
// takes hi as fp16; with the sums in pairs of fp32 values the passes over tensor
// memory are a third shorter in instructions: 128 x 200 49.3 -> 47.6 us.)
__device__ __forceinline__ void split2(f2 x, uint32_t& hi, uint32_t& lo) {
    asm("{\n"
        ".reg .b16 h0, h1, m;\n"
        ".reg .f32 a, b, r0, r1;\n"
        "mov.b64 {a, b}, %2;\n"
        "cvt.rn.f16x2.f32 %0, b, a;\n"
        "mov.b32 {h0, h1}, %0;\n"
        "mov.b16 m, 0xBC00;\n"  // -1
        "fma.rn.f32.f16 r0, h0, m, a;\n"
        "fma.rn.f32.f16 r1, h1, m, b;\n"
        "cvt.rn.f16x2.f32 %1, r1, r0;\n"
        "}\n"
        : "=&r"(hi), "=r"(lo)
        : "l"(x));
}
__device__ __forceinline__ void split8(const f2 (&v)[4], uint4& hi, uint4& lo) {
    split2(v[0], hi.x, lo.x);
    split2(v[1], hi.y, lo.y);
    split2(v[2], hi.z, lo.z);
    split2(v[3], hi.w, lo.w);
}
__device__ __forceinline__ void split8(const float (&v)[8], uint4& hi, uint4& lo) {
    const f2 p[4] = {pair(v[0], v[1]), pair(v[2], v[3]), pair(v[4], v[5]), pair(v[6], v[7])};
    split8(p, hi, lo);
}

// ------------------------------------------------------------ norm and split
// Elements t .. t + 3 of a row, as far as there are that many (0 past the end).
template <typename T>
__device__ __forceinline__ void load4(const T* p, int32_t valid, bool vec, float (&v)[4]) {
    if (vec && valid >= 4) {
        if constexpr (sizeof(T) == 4) {
            const float4 a = *reinterpret_cast<const float4*>(p);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        } else {
            const uint2 a = *reinterpret_cast<const uint2*>(p);
            v[0] = __uint_as_float(a.x << 16), v[1] = __uint_as_float(a.x & 0xFFFF0000u);
            v[2] = __uint_as_float(a.y << 16), v[3] = __uint_as_float(a.y & 0xFFFF0000u);
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = k < valid ? to_f(p[k]) : 0.f;
}

// New momentum, and partial sums of the squares of U: a warp takes rows in
// turn, 4 x 4 elements a lane at a time.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_ns_norm(Source<T> src, int32_t rows, int32_t cols,
                                                      double* __restrict__ part) {
    pdl_next();
    pdl_start();
    __shared__ double sh[kThreads / 32];
    const int64_t q = blockIdx.y;
    const int warp = (int)(threadIdx.x >> 5), lane = (int)(threadIdx.x & 31);
    const int32_t pieces = (cols + 511) / 512;  // of a row
    const int64_t items = (int64_t)rows * pieces;
    float sum = 0.f;
    for (int64_t it = blockIdx.x * (int64_t)(kThreads / 32) + warp; it < items; it += (int64_t)gridDim.x * (kThreads / 32)) {
        const int32_t r = (int32_t)(it / pieces), c0 = (int32_t)(it - (int64_t)r * pieces) * 512 + lane * 4;
        const T* g = src.g + (q * rows + r) * src.ld + c0;
        float u[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) load4(g + k * 128, cols - c0 - k * 128, (src.vec & 1) != 0, u[k]);
        if (src.mom_out) {
            const int64_t at = (q * rows + r) * cols + c0;
            float m[4][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) load4(src.mom + at + k * 128, cols - c0 - k * 128, (src.vec & 2) != 0, m[k]);
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    m[k][e] = src.mu * m[k][e] + u[k][e];
                    if (c0 + k * 128 + e < cols) src.mom_out[at + k * 128 + e] = m[k][e];
                    u[k][e] = src.nesterov ? u[k][e] + src.mu * m[k][e] : m[k][e];
                }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum += u[k][e] * u[k][e];
    }
    double s = warp_sum((double)sum);
    if (lane == 0) sh[warp] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kThreads / 32; ++w) s += sh[w];
        part[q * gridDim.x + blockIdx.x] = s;
    }
}

// X = U / (||U|| + eps) as planes, transposed when rows > cols; a block takes
// 64 rows x 32 columns of U (tall) or 32 x 64, and writes 8 elements a thread.
constexpr int kSplitN = 64, kSplitM = 32;  // of X
template <typename T>
__global__ void __launch_bounds__(kThreads) k_ns_split(Source<T> src, int32_t rows, int32_t cols,
                                                       const double* __restrict__ part, int32_t parts, float eps,
                                                       Planes X, int64_t ldx) {
    pdl_next();
    pdl_start();
    __shared__ float tile[kSplitM][kSplitN + 1];
    __shared__ double sh[kThreads / 32];
    const int64_t q = blockIdx.z;
    const bool tall = rows > cols;
    const int32_t m = tall ? cols : rows, n = tall ? rows : cols;
    const int32_t i0 = (int32_t)blockIdx.y * kSplitM, j0 = (int32_t)blockIdx.x * kSplitN;
    const auto u_at = [&](int64_t r, int64_t c) {
        float u = to_f(src.g[(q * rows + r) * src.ld + c]);
        if (src.mom_out) {
            const float mo = src.mom_out[(q * rows + r) * cols + c];
            u = src.nesterov ? u + src.mu * mo : mo;
        }
        return u;
    };
    float u[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {  // consecutive threads on consecutive columns of U
        const int e = k * kThreads + (int)threadIdx.x;
        const int i = tall ? e % kSplitM : e / kSplitN, j = tall ? e / kSplitM : e % kSplitN;
        u[k] = i0 + i < m && j0 + j < n ? (tall ? u_at(j0 + j, i0 + i) : u_at(i0 + i, j0 + j)) : 0.f;
    }
    double s = warp_sum((int)threadIdx.x < parts ? part[q * parts + threadIdx.x] : 0.0);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) s += sh[w];
    const float mul = kScale / (sqrtf((float)s) + eps);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int e = k * kThreads + (int)threadIdx.x;
        tile[tall ? e % kSplitM : e / kSplitN][tall ? e / kSplitM : e % kSplitN] = u[k] * mul;
    }
    __syncthreads();
    const int i = (int)threadIdx.x >> 3, j = ((int)threadIdx.x & 7) * 8;
    if (i0 + i >= m || j0 + j >= n) return;  // a row's padding (to a multiple of 8) takes zeros
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = tile[i][j + k];
    uint4 hi, lo;
    split8(v, hi, lo);
    const int64_t at = (q * m + i0 + i) * ldx + j0 + j;
    *reinterpret_cast<uint4*>(X.hi + at) = hi;
    *reinterpret_cast<uint4*>(X.lo + at) = lo;
}

// ----------------------------------------------------------------- products
// Instruction descriptor of kind::f16 with fp16 operands (formats 0), fp32
// accumulation (bits 4-5 = 1), B MN-major (bit 16) or not, N >> 3 in bits
// 17-22, M >> 4 (M = 128) in bits 24-28.
__host__ __device__ constexpr uint32_t desc_f16(bool b_mn, int n) {
    return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
}

struct PairMaps {
    CUtensorMap hi, lo;
};

// Ring of kStages stages of BYTES; a full and an empty barrier a stage.
template <int STAGES>
struct Ring {
    uint64_t full[STAGES], empty[STAGES];
    uint64_t sum[2], read[2];  // hi hi's accumulators: complete, and taken out
};

template <int STAGES>
__device__ __forceinline__ void ring_init(Ring<STAGES>& r) {
    for (int s = 0; s < STAGES; ++s) {
        mbar_init(&r.full[s], 1);
        mbar_init(&r.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
        mbar_init(&r.sum[b], 1);
        mbar_init(&r.read[b], kSumWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
}

// How hi hi is summed: kBufs accumulators of COLS columns in turn, kTurn K tiles
// (4 accumulations each) in each; the accumulator of the cross products is at
// column 512 - COLS.  A tile's hi hi comes first and its cross products while
// the turn's accumulator is read (at 256 columns there is room for one only).
template <int COLS>
constexpr int kBufs = COLS > 128 ? 1 : 2;
template <int COLS>
constexpr int kTurn = COLS > 128 ? 2 : 1;

// K tile i of the products: waits for its accumulator if it is the tile that
// begins a turn; returns it.
template <int COLS, int STAGES>
__device__ __forceinline__ uint32_t turn_begin(Ring<STAGES>& r, uint32_t tmem, int i, bool& ok) {
    const int turn = i / kTurn<COLS>, b = turn % kBufs<COLS>;
    if (i % kTurn<COLS> == 0 && turn >= kBufs<COLS> && !mbar_wait(&r.read[b], (uint32_t)(turn / kBufs<COLS> - 1) & 1u))
        ok = false;
    return tmem + (uint32_t)b * COLS;
}
template <int COLS, int STAGES>
__device__ __forceinline__ void turn_end(Ring<STAGES>& r, int i, int n_k) {
    if (i % kTurn<COLS> == kTurn<COLS> - 1 || i == n_k - 1) mma_commit(&r.sum[i / kTurn<COLS> % kBufs<COLS>]);
}

// The products' sum of this warp's 32 rows and COLS / 2 columns (warps w and
// w + 4 share tensor-memory lanes 32 (w % 4) ..), as the turns complete.
template <int COLS, int STAGES>
__device__ __forceinline__ void sum_turns(Ring<STAGES>& r, uint32_t tmem, int n_k, float (&acc)[COLS / 2]) {
    const int warp = (int)(threadIdx.x >> 5), lane = (int)(threadIdx.x & 31);
    const uint32_t at = ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)((warp >> 2) * (COLS / 2));
    const int turns = (n_k + kTurn<COLS> - 1) / kTurn<COLS>;
#pragma unroll
    for (int u = 0; u < COLS / 2; ++u) acc[u] = 0.f;
    const auto add = [&](uint32_t from) {
        if constexpr (COLS == 64) {
            float v[32];
            tmem_load_32(from + at, v);
#pragma unroll
            for (int u = 0; u < 32; ++u) acc[u] += v[u];
        } else {
#pragma unroll
            for (int c = 0; c < COLS / 2; c += 64) {
                uint32_t x[32], y[32];
                tmem_load_issue(from + at + (uint32_t)c, x);
                tmem_load_issue(from + at + (uint32_t)c + 32, y);
                tmem_load_wait(x);
                tmem_load_wait(y);
#pragma unroll
                for (int u = 0; u < 32; ++u) {
                    acc[c + u] += __uint_as_float(x[u]);
                    acc[c + 32 + u] += __uint_as_float(y[u]);
                }
            }
        }
    };
    for (int t = 0; t < turns; ++t) {
        const int b = t % kBufs<COLS>;
        if (!mbar_wait(&r.sum[b], (uint32_t)(t / kBufs<COLS>) & 1u) && lane == 0) dev_err(ERR_TIMEOUT);
        tmem_fence_after();
        add(tmem + (uint32_t)b * COLS);
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&r.read[b]);
    }
    if (turns) add(tmem + 512 - COLS);  // complete with the last turn
}

template <int COLS>
__device__ __forceinline__ void tmem_alloc(uint32_t* base) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_addr(base)), "r"(COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
}
template <int COLS>
__device__ __forceinline__ void tmem_free(uint32_t base) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(base), "r"(COLS) : "memory");
}

// Every load issued into the ring has landed (normally the MMA issuer has
// waited for them already).
template <int STAGES>
__device__ __forceinline__ void ring_drain(Ring<STAGES>& r, int issued) {
    for (int k = issued > STAGES ? issued - STAGES : 0; k < issued; ++k)
        if (!mbar_wait(&r.full[k % STAGES], (uint32_t)(k / STAGES) & 1u)) dev_err(ERR_TIMEOUT);
}

// Symmetric product: a 128 x 128 tile (i0, j0), j0 >= i0, of
//   GRAM    A = X X^T                      (K = n)
//   SQUARE  B = a I + b A + c A A          (K = m; A is symmetric, so A A = A A^T)
// both operands K-major rows of one matrix.  The tiles below the diagonal are
// written as mirror images.  The K tiles are split over the S CTAs of a
// cluster: each leaves its partial sum in shared memory, and CTA r adds
// columns [r, r + 1) 128 / S of all parts in rank order.
// 1024 x 4096: GRAM 18.0 us (144 CTAs, K split over 4; bound by the ring's loads
// and the emptying of accumulators), SQUARE 10.0 (a third of it the main loop: the
// rest is set-up, the exchange of parts and the writes).
constexpr int kSymStages = 3;
constexpr int kSymStage = 4 * kOperand;  // hi and lo of both operands: 64 KB
constexpr int kSymSmem = kSymStages * kSymStage + 1024;
enum { GRAM = 0, SQUARE = 1 };

template <int S, int KIND>
__global__ void __launch_bounds__(kProductThreads, 1)
    k_ns_sym(const __grid_constant__ PairMaps maps, int32_t m, int32_t K, float a, float b, float c, Planes in, Planes out,
             int64_t ld) {
    extern __shared__ uint8_t dsm[];
    __shared__ __align__(8) Ring<kSymStages> ring;
    __shared__ uint32_t tmem_base;
    pdl_next();
    const int warp = (int)(threadIdx.x >> 5), lane = (int)(threadIdx.x & 31);
    const int rank = (int)(blockIdx.x % S);
    const int32_t q = (int32_t)blockIdx.y;
    // tile t of the upper triangle, row by row
    const int32_t nt = (m + kTile - 1) / kTile;
    int32_t t = (int32_t)(blockIdx.x / S), ti = 0;
    while (t >= nt - ti) {
        t -= nt - ti;
        ++ti;
    }
    const int32_t i0 = ti * kTile, j0 = (ti + t) * kTile;
    const bool diag = t == 0;
    uint8_t* tiles = dsm + ((1024 - (smem_addr(dsm) & 1023)) & 1023);
    if (threadIdx.x == 0) {
        ring_init(ring);
        prefetch_map(&maps.hi);
        prefetch_map(&maps.lo);
    }
    if (warp == kSumWarps + 1) tmem_alloc<512>(&tmem_base);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = tmem_base, cross = tmem + 512 - kTile;
    pdl_start();
    const int n_kt = (K + kBK - 1) / kBK, per = (n_kt + S - 1) / S;
    const int kt0 = min(n_kt, rank * per), n_k = min(n_kt, kt0 + per) - kt0;
    float acc[kTile / 2];
    if (warp == kSumWarps && lane == 0) {
        int issued = 0;
        for (int i = 0; i < n_k; ++i) {
            const int s = i % kSymStages;
            if (i >= kSymStages && !mbar_wait(&ring.empty[s], (uint32_t)((i / kSymStages) - 1) & 1u)) {
                dev_err(ERR_TIMEOUT);
                break;
            }
            uint8_t* p = tiles + s * kSymStage;
            const int32_t x = (kt0 + i) * kBK;
            mbar_expect_tx(&ring.full[s], diag ? 2 * kOperand : 4 * kOperand);
            tma_load_3d(p, &maps.hi, x, i0, q, &ring.full[s]);
            tma_load_3d(p + kOperand, &maps.lo, x, i0, q, &ring.full[s]);
            if (!diag) {
                tma_load_3d(p + 2 * kOperand, &maps.hi, x, j0, q, &ring.full[s]);
                tma_load_3d(p + 3 * kOperand, &maps.lo, x, j0, q, &ring.full[s]);
            }
            ++issued;
        }
        ring_drain(ring, issued);
    } else if (warp == kSumWarps + 1 && lane == 0) {
        constexpr uint32_t idesc = desc_f16(false, kTile);
        for (int i = 0; i < n_k; ++i) {
            const int s = i % kSymStages;
            bool ok = true;
            const uint32_t main = turn_begin<kTile>(ring, tmem, i, ok);
            if (!ok || !mbar_wait(&ring.full[s], (uint32_t)(i / kSymStages) & 1u)) {
                dev_err(ERR_TIMEOUT);
                break;
            }
            tmem_fence_after();
            const uint32_t ah = smem_addr(tiles + s * kSymStage), al = ah + kOperand;
            const uint32_t bh = diag ? ah : ah + 2 * kOperand, bl = bh + kOperand;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                mma_issue(main, smem_desc_sw128(ah + kk * 32), smem_desc_sw128(bh + kk * 32), idesc,
                          (uint32_t)((i % kTurn<kTile> | kk) != 0), false);
            if (i + 1 < n_k) turn_end<kTile>(ring, i, n_k);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const uint32_t o = kk * 32;
                mma_issue(cross, smem_desc_sw128(ah + o), smem_desc_sw128(bl + o), idesc, (uint32_t)((i | kk) != 0), false);
                mma_issue(cross, smem_desc_sw128(al + o), smem_desc_sw128(bh + o), idesc, 1u, false);
            }
            mma_commit(&ring.empty[s]);
            if (i + 1 == n_k) turn_end<kTile>(ring, i, n_k);
        }
    } else if (warp < kSumWarps) {
        sum_turns<kTile>(ring, tmem, n_k, acc);
    }
    __syncwarp();
    __syncthreads();  // the producer has drained: the ring is free
    // SQUARE also adds b A: on its way while the parts are exchanged.  Thread t
    // takes 8 columns at a time of row t % 128.
    constexpr int kW = kTile / S, kTurns = kW / 16;  // columns of this CTA; turns of 16 of them
    const int row = (int)(threadIdx.x & 127);
    const int32_t i = i0 + row;
    const auto col_of = [&](int turn) { return rank * kW + turn * 16 + (int)(threadIdx.x >> 7) * 8; };
    uint4 ah[kTurns], al[kTurns];
    if (KIND == SQUARE && warp < kSumWarps) {
#pragma unroll
        for (int u = 0; u < kTurns; ++u) {
            const int32_t j = j0 + col_of(u);
            const int64_t at = ((int64_t)q * m + i) * ld + j;
            const bool in_range = i < m && j < m;
            ah[u] = in_range ? *reinterpret_cast<const uint4*>(in.hi + at) : make_uint4(0, 0, 0, 0);
            al[u] = in_range ? *reinterpret_cast<const uint4*>(in.lo + at) : make_uint4(0, 0, 0, 0);
        }
    }
    // partial sums to shared memory as [column / 4][row][4]
    float* dump = reinterpret_cast<float*>(tiles);
    if (warp < kSumWarps) {
        const int r = (warp & 3) * 32 + lane, c0 = (warp >> 2) * (kTile / 2);
#pragma unroll
        for (int u = 0; u < kTile / 2; u += 4)
            *reinterpret_cast<float4*>(dump + ((c0 + u) / 4 * kTile + r) * 4) =
                make_float4(acc[u], acc[u + 1], acc[u + 2], acc[u + 3]);
    }
    tmem_fence_before();
    if constexpr (S > 1) cluster_sync();
    else __syncthreads();
    if (warp == kSumWarps + 1) tmem_free<512>(tmem);
    if (warp >= kSumWarps) return;
    const uint32_t base = smem_addr(dump);
    float4 x[kTurns][S][2];  // 16 loads in flight, whatever S is
#pragma unroll
    for (int u = 0; u < kTurns; ++u)
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const uint32_t at = (uint32_t)((col_of(u) / 4 * kTile + row) * 16);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (S > 1) x[u][s][h] = ld_cluster4(map_rank(base, (uint32_t)s) + at + h * kTile * 16);
                else x[u][s][h] = *reinterpret_cast<const float4*>(dump + (col_of(u) / 4 + h) * kTile * 4 + row * 4);
            }
        }
    // (the loads above are volatile: they are issued before the arrival, and
    // used before the wait)
#pragma unroll
    for (int u = 0; u < kTurns; ++u) {
        float v[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float4 t = x[u][0][h];
#pragma unroll
            for (int s = 1; s < S; ++s) t.x += x[u][s][h].x, t.y += x[u][s][h].y, t.z += x[u][s][h].z, t.w += x[u][s][h].w;
            v[4 * h] = t.x, v[4 * h + 1] = t.y, v[4 * h + 2] = t.z, v[4 * h + 3] = t.w;
        }
        if (S > 1 && u == kTurns - 1) asm volatile("barrier.cluster.arrive.release;\n" ::: "memory");  // done reading
        const int32_t j = j0 + col_of(u);
        if (i >= m || j >= m) continue;
        if (KIND == GRAM) {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] *= 1.f / kScale;
        } else {
            const __half2* h2 = reinterpret_cast<const __half2*>(&ah[u]);
            const __half2* l2 = reinterpret_cast<const __half2*>(&al[u]);
            const float cs = c * (1.f / kScale);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 h = __half22float2(h2[k]), l = __half22float2(l2[k]);
                v[2 * k] = fmaf(b, h.x, fmaf(b, l.x, cs * v[2 * k]));
                v[2 * k + 1] = fmaf(b, h.y, fmaf(b, l.y, cs * v[2 * k + 1]));
            }
            if (diag && (i & ~7) == (j & ~7)) {
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] += i == j + k ? a * kScale : 0.f;
            }
        }
        uint4 hi, lo;
        split8(v, hi, lo);
        const int64_t at = ((int64_t)q * m + i) * ld + j;
        *reinterpret_cast<uint4*>(out.hi + at) = hi;
        *reinterpret_cast<uint4*>(out.lo + at) = lo;
        if (!diag) {
            const __half* ph = reinterpret_cast<const __half*>(&hi);
            const __half* pl = reinterpret_cast<const __half*>(&lo);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (j + k >= m) continue;
                const int64_t mir = ((int64_t)q * m + j + k) * ld + i;
                out.hi[mir] = ph[k];
                out.lo[mir] = pl[k];
            }
        }
    }
    // no CTA leaves while another reads its part
    if constexpr (S > 1) asm volatile("barrier.cluster.wait.acquire;\n" ::: "memory");
}

// X' = B X: a 128 x BN tile.  B's tile is K-major (B is m x m), X's MN-major
// (its rows are K, n contiguous).
// FINAL: out = keep w + step X', transposed back when tall; else X' as planes.
// 1024 x 4096 (128 tiles of 256 columns): 21.3 us, three quarters of them in the
// main loop, which the ring's loads bound (110 bytes/ns an SM, 96 KB a stage of
// 1,536 cycles of products).
struct FinalArgs {
    const void* w;
    void* out;
    float keep, step;
    int64_t ld_out;
    int32_t tall;
    int32_t vec;  // rows of w and out are on boundaries of 4 elements
};

template <int BN>
constexpr int kApplyStage = 2 * kOperand + 2 * BN * kBK * 2;
template <int BN>
constexpr int kApplyStages = BN == 256 ? 2 : BN == 128 ? 3 : 4;
template <int BN>
constexpr int kApplySmem = kApplyStages<BN> * kApplyStage<BN> + 1024;

struct ApplyMaps {
    CUtensorMap bhi, blo, xhi, xlo;
};

template <int BN, typename TW, bool FINAL>
__global__ void __launch_bounds__(kProductThreads, 1)
    k_ns_apply(const __grid_constant__ ApplyMaps maps, int32_t m, int32_t n, Planes out, int64_t ldx, FinalArgs fin) {
    constexpr int kStages = kApplyStages<BN>, kStage = kApplyStage<BN>, kBox = kBK * 128;  // 64 K rows of 64 columns
    extern __shared__ uint8_t dsm[];
    __shared__ __align__(8) Ring<kStages> ring;
    __shared__ uint32_t tmem_base;
    pdl_next();
    const int warp = (int)(threadIdx.x >> 5), lane = (int)(threadIdx.x & 31);
    const int32_t q = (int32_t)blockIdx.z, i0 = (int32_t)blockIdx.y * kTile, j0 = (int32_t)blockIdx.x * BN;
    uint8_t* tiles = dsm + ((1024 - (smem_addr(dsm) & 1023)) & 1023);
    if (threadIdx.x == 0) {
        ring_init(ring);
        prefetch_map(&maps.bhi);
        prefetch_map(&maps.blo);
        prefetch_map(&maps.xhi);
        prefetch_map(&maps.xlo);
    }
    if (warp == kSumWarps + 1) tmem_alloc<512>(&tmem_base);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = tmem_base, cross = tmem + 512 - BN;
    pdl_start();
    const int n_k = (m + kBK - 1) / kBK;
    float acc[BN / 2];
    if (warp == kSumWarps && lane == 0) {
        int issued = 0;
        for (int i = 0; i < n_k; ++i) {
            const int s = i % kStages;
            if (i >= kStages && !mbar_wait(&ring.empty[s], (uint32_t)((i / kStages) - 1) & 1u)) {
                dev_err(ERR_TIMEOUT);
                break;
            }
            uint8_t* p = tiles + s * kStage;
            mbar_expect_tx(&ring.full[s], kStage);
            tma_load_3d(p, &maps.bhi, i * kBK, i0, q, &ring.full[s]);
            tma_load_3d(p + kOperand, &maps.blo, i * kBK, i0, q, &ring.full[s]);
#pragma unroll
            for (int h = 0; h < BN / 64; ++h) {
                tma_load_3d(p + 2 * kOperand + h * kBox, &maps.xhi, j0 + h * 64, i * kBK, q, &ring.full[s]);
                tma_load_3d(p + 2 * kOperand + (BN / 64 + h) * kBox, &maps.xlo, j0 + h * 64, i * kBK, q, &ring.full[s]);
            }
            ++issued;
        }
        ring_drain(ring, issued);
    } else if (warp == kSumWarps + 1 && lane == 0) {
        constexpr uint32_t idesc = desc_f16(true, BN);
        for (int i = 0; i < n_k; ++i) {
            const int s = i % kStages;
            bool ok = true;
            const uint32_t main = turn_begin<BN>(ring, tmem, i, ok);
            if (!ok || !mbar_wait(&ring.full[s], (uint32_t)(i / kStages) & 1u)) {
                dev_err(ERR_TIMEOUT);
                break;
            }
            tmem_fence_after();
            const uint32_t bh = smem_addr(tiles + s * kStage), bl = bh + kOperand;
            const uint32_t xh = bh + 2 * kOperand, xl = xh + (BN / 64) * kBox;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)  // 16 K elements of a row; 16 K rows
                mma_issue(main, smem_desc_sw128(bh + kk * 32), smem_desc_mn_sw128(xh + kk * 2048, kBox), idesc,
                          (uint32_t)((i % kTurn<BN> | kk) != 0), false);
            if (i + 1 < n_k) turn_end<BN>(ring, i, n_k);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const uint32_t o = kk * 32, ox = kk * 2048;
                mma_issue(cross, smem_desc_sw128(bh + o), smem_desc_mn_sw128(xl + ox, kBox), idesc, (uint32_t)((i | kk) != 0),
                          false);
                mma_issue(cross, smem_desc_sw128(bl + o), smem_desc_mn_sw128(xh + ox, kBox), idesc, 1u, false);
            }
            mma_commit(&ring.empty[s]);
            if (i + 1 == n_k) turn_end<BN>(ring, i, n_k);
        }
    } else if (warp < kSumWarps) {
        sum_turns<BN>(ring, tmem, n_k, acc);
    }
    __syncwarp();
    __syncthreads();  // the producer has drained: the ring is free
    // the tile through shared memory, so that rows go out whole: [row][BN + 4]
    // (rows on 16-byte boundaries, 8 rows in different banks)
    float* dump = reinterpret_cast<float*>(tiles);
    constexpr int kLd = BN + 4;
    if (warp < kSumWarps) {
        const int row = (warp & 3) * 32 + lane, c0 = (warp >> 2) * (BN / 2);
#pragma unroll
        for (int u = 0; u < BN / 2; u += 4)
            *reinterpret_cast<float4*>(dump + row * kLd + c0 + u) = make_float4(acc[u], acc[u + 1], acc[u + 2], acc[u + 3]);
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == kSumWarps + 1) tmem_free<512>(tmem);
    if (warp >= kSumWarps) return;
    if constexpr (!FINAL) {
        constexpr int kLanes = BN / 8, kRows = kThreads / kLanes;  // 8 columns a lane; rows at a time
        const int c = (int)(threadIdx.x % kLanes) * 8;
        if (j0 + c < n) {
#pragma unroll 4
            for (int row = (int)threadIdx.x / kLanes; row < kTile; row += kRows) {
                if (i0 + row >= m) break;
                const float4 x = *reinterpret_cast<const float4*>(dump + row * kLd + c);
                const float4 y = *reinterpret_cast<const float4*>(dump + row * kLd + c + 4);
                constexpr float d = 1.f / kScale;
                const float v[8] = {x.x * d, x.y * d, x.z * d, x.w * d, y.x * d, y.y * d, y.z * d, y.w * d};
                uint4 hi, lo;
                split8(v, hi, lo);
                const int64_t at = ((int64_t)q * m + i0 + row) * ldx + j0 + c;
                *reinterpret_cast<uint4*>(out.hi + at) = hi;
                *reinterpret_cast<uint4*>(out.lo + at) = lo;
            }
        }
    } else {
        const float mul = fin.step * (1.f / (kScale * kScale));
        const TW* w = (const TW*)fin.w;
        TW* o = (TW*)fin.out;
        if (fin.tall) {  // element (i, j) of X is (j, i) of the matrix
            for (int c = warp; c < BN && j0 + c < n; c += kThreads / 32) {
                const int64_t at = ((int64_t)q * n + j0 + c) * fin.ld_out + i0;
                for (int row = lane; row < kTile && i0 + row < m; row += 32) {
                    const float x = mul * dump[row * kLd + c];
                    put(o + at + row, w ? fin.keep * to_f(w[at + row]) + x : x);
                }
            }
        } else {
            for (int row = warp; row < kTile && i0 + row < m; row += kThreads / 32) {
                const int64_t at = ((int64_t)q * m + i0 + row) * fin.ld_out + j0;
                for (int c = lane; c < BN && j0 + c < n; c += 32) {
                    const float x = mul * dump[row * kLd + c];
                    put(o + at + c, w ? fin.keep * to_f(w[at + c]) + x : x);
                }
            }
        }
    }
}

// out = keep w + step X of the planes (no steps at all)
template <typename TW>
__global__ void __launch_bounds__(kThreads) k_ns_store(Planes X, int64_t ldx, int32_t rows, int32_t cols, FinalArgs fin) {
    pdl_start();
    const int64_t q = blockIdx.y, total = (int64_t)rows * cols;
    const int32_t m = fin.tall ? cols : rows;
    const TW* w = (const TW*)fin.w;
    TW* o = (TW*)fin.out;
    for (int64_t t = blockIdx.x * (int64_t)kThreads + threadIdx.x; t < total; t += (int64_t)gridDim.x * kThreads) {
        const int64_t r = t / cols, c = t - r * cols;
        const int64_t p = (q * m + (fin.tall ? c : r)) * ldx + (fin.tall ? r : c);
        const float x = fin.step * ((__half2float(X.hi[p]) + __half2float(X.lo[p])) * (1.f / kScale));
        const int64_t at = (q * rows + r) * fin.ld_out + c;
        put(o + at, w ? fin.keep * to_f(w[at]) + x : x);
    }
}

// ------------------------------------------- m <= 128: one launch, on the chip
// A cluster of S CTAs holds one matrix for the whole call: CTA r keeps columns
// [r W, r W + W) of X in shared memory as fp16 pairs, in the swizzled layout
// that serves both as K-major rows (A = X X^T) and as an MN-major operand
// (X <- B X).  A step is
//   each CTA's partial X X^T (K = W), left in its shared memory as fp32;
//   CTA r adds its share of the parts' 8 x 8 blocks (half of A: it is
//   symmetric) and copies them, as pairs, to every CTA, which completes A;
//   every CTA forms B = a I + b A + c A A and X <- B X for its own columns.
// No iterate goes to memory: the call reads its input and writes the result.
// The time is a chain of latencies: two cluster barriers, three products and
// four passes over tensor memory a step.  Cycles of a step, 128 x 200 on one SM
// (48 us for five steps) / 128 x 2048 on 16 (58 us), before the passes' arithmetic
// was paired: partial Gram 3,800 / 2,800,
// taking it out 1,100 / 1,700 with the barrier, exchange - / 5,000 (8,500 with all
// blocks of A; distributed shared memory gives 16 bytes a clock an SM), square
// 2,800 / 2,700, B 1,700 / 2,300, B X 4,000 / 2,700, X 2,100 / 1,300.
constexpr int kFusedM = 128;
constexpr int kFusedMaxCtas = 16;
constexpr int kPairTile = kFusedM * 128;  // bytes of a 128 x 64 fp16 tile

// W = 256: one CTA for the whole matrix, of 512 threads; its A comes straight
// from tensor memory and needs no fp32 copy in shared memory.
template <int W>
constexpr int kFusedThreads = W == 256 ? 512 : kThreads;

// Address of 8 elements (columns 8 c ..) of row r of a [128 x 64 t] swizzled
// operand.
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    return (uint32_t)((c >> 3) * kPairTile + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// The exchange of A.  A is symmetric, so of its 16 x 16 blocks of 8 x 8 the
// kHalf blocks (g, g + d mod 16), d = 0 .. 8, of each row group g are enough;
// the pair (g, g + 8) = (g + 8, g) has two names, and owns_last picks one.
constexpr int kHalf = 9;
constexpr int kDumpBytes = kFusedM * kHalf * 8 * 4;   // partial sums: [d][half][row][4]
constexpr int kGroupBytes = 2 * kHalf * 128;          // a row group's sums as pairs: [plane][d][8][8]
constexpr int kStageBytes = kFusedM / 8 * kGroupBytes;
__device__ __forceinline__ bool owns_last(int g) { return ((g ^ (g >> 3)) & 1) == 0; }

template <int W>
constexpr int kFusedSmem = 2 * (W / 64) * kPairTile + 4 * kPairTile + (W == 256 ? 0 : kDumpBytes + kStageBytes) + 1024;

// The blocks of this rank's row groups from the S partial sums (da: their place,
// in every CTA), as pairs into this CTA's stage.  They are added in the order
// of ranks beginning with this one, so that not every CTA reads from the same one.
template <int S>
__device__ __forceinline__ void reduce_blocks(uint32_t da, uint32_t rank, uint8_t* stage) {
    constexpr int kGroups = kFusedM / 8 / S, kItems = kGroups * kHalf * 16;  // 4 columns of a block's row
    constexpr int kTurns = (kItems + kThreads - 1) / kThreads;
    float4 x[kTurns][S];
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        const int t = i * kThreads + (int)threadIdx.x, r = t % 8, c = t / 8 % (2 * kHalf), g = (int)rank * kGroups + t / (16 * kHalf);
        if (t < kItems && (c < 16 || owns_last(g))) {
#pragma unroll
            for (int s = 0; s < S; ++s)
                x[i][s] = ld_cluster4(map_rank(da, (rank + (uint32_t)s) % S) + (uint32_t)((c * kFusedM + 8 * g + r) * 16));
        }
    }
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        const int t = i * kThreads + (int)threadIdx.x, r = t % 8, c = t / 8 % (2 * kHalf), g = (int)rank * kGroups + t / (16 * kHalf);
        if (t < kItems && (c < 16 || owns_last(g))) {
            float4 v = x[i][0];
#pragma unroll
            for (int s = 1; s < S; ++s) v.x += x[i][s].x, v.y += x[i][s].y, v.z += x[i][s].z, v.w += x[i][s].w;
            uint32_t h0, l0, h1, l1;
            split2(pair(v.x * (1.f / kScale), v.y * (1.f / kScale)), h0, l0);
            split2(pair(v.z * (1.f / kScale), v.w * (1.f / kScale)), h1, l1);
            uint8_t* at = stage + g * kGroupBytes + c * 64 - (c & 1) * 56 + r * 16;
            *reinterpret_cast<uint2*>(at) = make_uint2(h0, h1);
            *reinterpret_cast<uint2*>(at + kHalf * 128) = make_uint2(l0, l1);
        }
    }
}

// A, both halves, from the staged blocks: four of them a warp at a time, as they
// are and transposed (a diagonal block: transposed only).  Both names of a pair
// write the same.
__device__ __forceinline__ void spread_blocks(uint32_t stage, uint32_t as) {
    const int lane = (int)(threadIdx.x & 31), r = lane & 7;
#pragma unroll 3
    for (int k = (int)(threadIdx.x >> 5); k < kHalf * 8; k += kThreads / 32) {
        const int p = k / (kHalf * 4), q = k % (kHalf * 4), d = q >> 2;
        int g = (q & 3) * 4 + (lane >> 3);
        if (d == 8 && !owns_last(g)) g ^= 8;
        const int c = (g + d) & 15;
        uint32_t x0, x1, x2, x3;
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];\n"
                     : "=r"(x0), "=r"(x1), "=r"(x2), "=r"(x3)
                     : "r"(stage + (uint32_t)(g * kGroupBytes + p * kHalf * 128 + d * 128 + r * 16))
                     : "memory");
        if (d != 0)
            asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};\n" ::"r"(
                             as + (uint32_t)(p * 2 * kPairTile) + chunk_at(8 * g + r, c)),
                         "r"(x0), "r"(x1), "r"(x2), "r"(x3)
                         : "memory");
        asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};\n" ::"r"(
                         as + (uint32_t)(p * 2 * kPairTile) + chunk_at(8 * c + r, g)),
                     "r"(x0), "r"(x1), "r"(x2), "r"(x3)
                     : "memory");
    }
}

// 8 consecutive elements, 16 bytes at a time.
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[2 * k] = __uint_as_float(w[k] << 16);
        v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&v)[4]) {
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(a.x << 16), v[1] = __uint_as_float(a.x & 0xFFFF0000u);
    v[2] = __uint_as_float(a.y << 16), v[3] = __uint_as_float(a.y & 0xFFFF0000u);
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

struct Steps {
    float coef[SG_MAX_NS_STEPS][3];
    int32_t count;
};

template <int W, typename TS, typename TW>
__global__ void __launch_bounds__(kFusedThreads<W>, 1)
    k_ns_fused(Source<TS> src, int32_t rows, int32_t cols, Steps steps, float eps, FinalArgs fin) {
    extern __shared__ uint8_t dsm[];
    __shared__ __align__(8) uint64_t done, full;  // products; the other CTAs' rows of A
    __shared__ uint32_t tmem_base;
    __shared__ float norm[kFusedMaxCtas];
    __shared__ float red[kFusedThreads<W> / 32];
    constexpr int kNT = kFusedThreads<W>, kWarps = kNT / 32, kXTiles = W / 64, kChunks = kFusedM * W / 8 / kNT;  // 16-byte chunks of X a thread handles
    pdl_start();
    const int warp = (int)(threadIdx.x >> 5), lane = (int)(threadIdx.x & 31);
    const uint32_t rank = cluster_rank();
    uint32_t S = 1;
    if constexpr (W < 256) asm volatile("mov.u32 %0, %%cluster_nctarank;\n" : "=r"(S));
    const int64_t q = blockIdx.y;
    const bool tall = rows > cols;
    const int32_t m = tall ? cols : rows, n = tall ? rows : cols, j0 = (int32_t)rank * W;
    uint8_t* base = dsm + ((1024 - (smem_addr(dsm) & 1023)) & 1023);
    uint8_t* xs = base;                          // X: hi tiles, then lo tiles
    uint8_t* as = xs + 2 * kXTiles * kPairTile;  // A, then B: hi tiles (2), lo tiles (2)
    float* dump = reinterpret_cast<float*>(as + 4 * kPairTile);
    [[maybe_unused]] uint8_t* stage = as + 4 * kPairTile + kDumpBytes;
    constexpr uint32_t kXLo = kXTiles * kPairTile, kALo = 2 * kPairTile;
    if (threadIdx.x == 0) {
        mbar_init(&done, 1);
        mbar_init(&full, 1);
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == 1) tmem_alloc<512>(&tmem_base);

    // U of this CTA's columns, in registers; the new momentum on the way.
    // Consecutive threads take consecutive addresses: columns of a row, or
    // (tall: X is the transpose) rows of X.
    const auto row_of = [&](int it) {
        const int e = it * kNT + (int)threadIdx.x;
        return tall ? e % kFusedM : e / (W / 8);
    };
    const auto chunk_of = [&](int it) {
        const int e = it * kNT + (int)threadIdx.x;
        return tall ? e / kFusedM : e % (W / 8);
    };
    const auto place = [&](int it, int64_t ld) {  // of the chunk's first element
        const int64_t j = j0 + chunk_of(it) * 8, i = row_of(it);
        return tall ? (q * rows + j) * ld + i : (q * rows + i) * ld + j;
    };
    const auto valid_of = [&](int it) { return row_of(it) < m ? n - j0 - chunk_of(it) * 8 : 0; };
    // Wide: every chunk is whole or empty and its rows may be read 16 bytes at a
    // time.  (Nothing else may write the registers of a load on its way, not
    // even for other lanes, or the loads wait for one another.)
    const bool wide = !tall && n % 8 == 0 && (src.vec & 1) && (!src.mom_out || (src.vec & 2));
    float u[kChunks][8];
    float sq = 0.f;
#pragma unroll
    for (int it = 0; it < kChunks; ++it)
#pragma unroll
        for (int k = 0; k < 8; ++k) u[it][k] = 0.f;
    constexpr int kBatch = 4;  // chunks whose momentum is in registers at once
    if (wide) {
#pragma unroll
        for (int it = 0; it < kChunks; ++it)
            if (valid_of(it) > 0) load8(src.g + place(it, src.ld), u[it]);
        if (src.mom_out) {
#pragma unroll
            for (int i0 = 0; i0 < kChunks; i0 += kBatch) {
                float mo[kBatch][8] = {};
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    if (valid_of(i0 + i) > 0) load8(src.mom + place(i0 + i, cols), mo[i]);
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        mo[i][k] = src.mu * mo[i][k] + u[i0 + i][k];
                        u[i0 + i][k] = src.nesterov ? u[i0 + i][k] + src.mu * mo[i][k] : mo[i][k];
                    }
                    if (valid_of(i0 + i) > 0) {
                        float* p = src.mom_out + place(i0 + i, cols);
                        *reinterpret_cast<float4*>(p) = make_float4(mo[i][0], mo[i][1], mo[i][2], mo[i][3]);
                        *reinterpret_cast<float4*>(p + 4) = make_float4(mo[i][4], mo[i][5], mo[i][6], mo[i][7]);
                    }
                }
            }
        }
    } else {
        const int64_t step_g = tall ? src.ld : 1, step_m = tall ? cols : 1;
#pragma unroll
        for (int it = 0; it < kChunks; ++it)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < valid_of(it)) u[it][k] = to_f(src.g[place(it, src.ld) + k * step_g]);
        if (src.mom_out) {
#pragma unroll
            for (int i0 = 0; i0 < kChunks; i0 += kBatch) {
                float mo[kBatch][8] = {};
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k < valid_of(i0 + i)) mo[i][k] = src.mom[place(i0 + i, cols) + k * step_m];
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        mo[i][k] = src.mu * mo[i][k] + u[i0 + i][k];
                        u[i0 + i][k] = src.nesterov ? u[i0 + i][k] + src.mu * mo[i][k] : mo[i][k];
                        if (k < valid_of(i0 + i)) src.mom_out[place(i0 + i, cols) + k * step_m] = mo[i][k];
                    }
            }
        }
    }
#pragma unroll
    for (int it = 0; it < kChunks; ++it) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) s += u[it][k] * u[it][k];
        sq += s;
    }
    sq = warp_sum(sq);
    if (lane == 0) red[warp] = sq;
    tmem_fence_before();
    cluster_sync();  // every CTA runs (and red, the barriers and tmem_base are set)
    tmem_fence_after();
    const uint32_t tmem = tmem_base;
    if (threadIdx.x < S) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kNT / 32; ++w) s += red[w];
        asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(map_rank(smem_addr(norm + rank), threadIdx.x)), "f"(s)
                     : "memory");
    }
    cluster_sync();
    {
        const float mul = kScale / (sqrtf(warp_sum(lane < (int)S ? norm[lane] : 0.f)) + eps);
#pragma unroll
        for (int it = 0; it < kChunks; ++it) {
#pragma unroll
            for (int k = 0; k < 8; ++k) u[it][k] *= mul;
            uint4 hi, lo;
            split8(u[it], hi, lo);
            *reinterpret_cast<uint4*>(xs + chunk_at(row_of(it), chunk_of(it))) = hi;
            *reinterpret_cast<uint4*>(xs + kXLo + chunk_at(row_of(it), chunk_of(it))) = lo;
        }
    }
    const uint32_t xa = smem_addr(xs), aa = smem_addr(as);
    const int row = (warp & 3) * 32 + lane;  // of tensor memory, in every pass over it
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    uint32_t phase = 0, a_phase = 0;
    const int km = (m + 15) / 16;  // 16-row pieces of X, and columns of A
    const int kx = max(1, (min(W, n - j0) + 15) / 16);  // 16-column pieces of X that are not empty
    const int part = warp >> 2;  // which columns this warp takes in a pass over tensor memory
    // runs `issue` on one thread once all shared memory is written, and waits for it
    const auto product = [&](auto issue) {
        tmem_fence_before();
        fence_async();
        __syncthreads();
        if (threadIdx.x == 0) {
            tmem_fence_after();
            fence_async();
            issue();
            mma_commit(&done);
        }
        __syncwarp();
        if (!mbar_wait(&done, phase) && lane == 0) dev_err(ERR_TIMEOUT);
        phase ^= 1u;
        tmem_fence_after();
    };
    // hi hi, and hi lo + lo hi, over K steps of 16; a and b give a step's
    // descriptors.  hi hi is dealt to `mains` accumulators: two of 128 columns, or
    // one of 256.
    const auto pairs = [&](int ksteps, int mains, int cols, uint32_t idesc, auto a, auto b) {
        const uint32_t cross = tmem + (uint32_t)(mains * cols);
        for (int k = 0; k < ksteps; ++k) {
            mma_issue(tmem + (uint32_t)(k % mains * cols), a(k, 0), b(k, 0), idesc, (uint32_t)(k >= mains), false);
            mma_issue(cross, a(k, 0), b(k, 1), idesc, (uint32_t)(k != 0), false);
            mma_issue(cross, a(k, 1), b(k, 0), idesc, 1u, false);
        }
    };
    // 32 columns of their sum, in pairs
    const auto load_sum = [&](int ksteps, int mains, int cols, uint32_t at, f2 (&v)[16]) {
        uint32_t x[32], y[32];
        const auto two = [](const uint32_t (&r)[32], int k) { return pair(__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1])); };
        tmem_load_issue(tmem + (uint32_t)(mains * cols) + at, x);
        tmem_load_issue(tmem + at, y);
        tmem_load_wait(x);
        tmem_load_wait(y);
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = add2(two(x, k), two(y, k));
        if (mains > 1 && ksteps > 1) {
            tmem_load_issue(tmem + (uint32_t)cols + at, x);
            tmem_load_wait(x);
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = add2(v[k], two(x, k));
        }
    };
    const auto load_sum_32 = [&](int ksteps, int mains, int cols, uint32_t at, float (&v)[32]) {
        f2 p[16];
        load_sum(ksteps, mains, cols, at, p);
#pragma unroll
        for (int k = 0; k < 16; ++k) unpair(p[k], v[2 * k], v[2 * k + 1]);
    };
    const f2 unscale = pair(1.f / kScale, 1.f / kScale);
    constexpr int kXMains = W == 256 ? 1 : 2, kXCols = W == 256 ? 256 : 128;  // of X <- B X
    const auto x_rows = [&](int k, int lo) {
        return smem_desc_sw128(xa + (lo ? kXLo : 0) + (uint32_t)((k >> 2) * kPairTile + (k & 3) * 32));
    };
    const auto a_rows = [&](int k, int lo) {
        return smem_desc_sw128(aa + (lo ? kALo : 0) + (uint32_t)((k >> 2) * kPairTile + (k & 3) * 32));
    };
    const auto x_cols = [&](int k, int lo) {
        return smem_desc_mn_sw128(xa + (lo ? kXLo : 0) + (uint32_t)(k * 16 * 128), kPairTile);
    };
    // the partial sums of all CTAs into A, in every CTA
    [[maybe_unused]] const auto gather = [&](bool last) {
        if (threadIdx.x == 0) mbar_expect_tx(&full, (uint32_t)kStageBytes / S * (S - 1));
        cluster_sync();
        // this CTA's row groups into its own stage, then to the others'.  (The
        // barrier: all partial sums are written, and all copies of the last
        // step have been waited for, so the stage may be written.)
        if (W == 128 || S == 16)
            reduce_blocks<16>(smem_addr(dump), rank, stage);
        else
            reduce_blocks<8>(smem_addr(dump), rank, stage);
        fence_async();
        __syncthreads();
        if (warp == 0 && lane < (int)S && lane != (int)rank) {  // lane: to whom
            const uint32_t bytes = (uint32_t)kStageBytes / S, from = smem_addr(stage) + rank * bytes;
            asm volatile(
                "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                    map_rank(from, (uint32_t)lane)),
                "r"(from), "r"(bytes), "r"(map_rank(smem_addr(&full), (uint32_t)lane))
                : "memory");
        }
        __syncwarp();
        // With every other CTA's blocks here, all of them have read this one's
        // partial sums, so those may be overwritten.
        if (!mbar_wait(&full, (uint32_t)a_phase) && lane == 0) dev_err(ERR_TIMEOUT);
        __syncwarp();
        a_phase ^= 1u;
        if (last) asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
        spread_blocks(smem_addr(stage), aa);
    };
#pragma unroll 1
    for (int step = 0; step < steps.count; ++step) {
        // partial A = X X^T
        product([&] { pairs(kx, 2, 128, desc_f16(false, kFusedM), x_rows, x_rows); });
        if constexpr (W == 256) {
            f2 v[16];
            load_sum(kx, 2, 128, lanes + (uint32_t)part * 32, v);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                f2 x[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) x[k] = mul2(v[4 * t + k], unscale);
                uint4 hi, lo;
                split8(x, hi, lo);
                *reinterpret_cast<uint4*>(as + chunk_at(row, part * 4 + t)) = hi;
                *reinterpret_cast<uint4*>(as + kALo + chunk_at(row, part * 4 + t)) = lo;
            }
        } else {
#pragma unroll 1
            for (int c0 = part * 64; c0 < part * 64 + 64; c0 += 32) {
                float v[32];
                load_sum_32(kx, 2, 128, lanes + (uint32_t)c0, v);
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    const int d = (c0 / 8 + t / 2 - row / 8) & 15;
                    if (d < kHalf)
                        *reinterpret_cast<float4*>(dump + ((d * 2 + t % 2) * kFusedM + row) * 4) =
                            make_float4(v[4 * t], v[4 * t + 1], v[4 * t + 2], v[4 * t + 3]);
                }
            }
            gather(step + 1 == steps.count);
        }
        // B = a I + b A + c A A, in A's place
        product([&] { pairs(km, 2, 128, desc_f16(false, kFusedM), a_rows, a_rows); });
        const float ca = steps.coef[step][0] * kScale, cb = steps.coef[step][1], cc = steps.coef[step][2] * (1.f / kScale);
        const f2 cb2 = pair(cb, cb), cc2 = pair(cc, cc);
#pragma unroll 1
        for (int c0 = part * (kFusedM * 4 / kWarps); c0 < (part + 1) * (kFusedM * 4 / kWarps); c0 += 32) {
            f2 v[16];
            load_sum(km, 2, 128, lanes + (uint32_t)c0, v);
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = mul2(v[k], cc2);
            if ((c0 >> 5) == (warp & 3)) {  // the diagonal: column c0 + lane of row `row`
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    v[k] = add2(v[k], pair(2 * k == lane ? ca : 0.f, 2 * k + 1 == lane ? ca : 0.f));
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                uint4* ph = reinterpret_cast<uint4*>(as + chunk_at(row, c0 / 8 + t));
                uint4* pl = reinterpret_cast<uint4*>(as + kALo + chunk_at(row, c0 / 8 + t));
                const uint4 h4 = *ph, l4 = *pl;
                const __half2* h2 = reinterpret_cast<const __half2*>(&h4);
                const __half2* l2 = reinterpret_cast<const __half2*>(&l4);
                f2 b[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 h = __half22float2(h2[k]), l = __half22float2(l2[k]);
                    b[k] = fma2(cb2, pair(h.x, h.y), fma2(cb2, pair(l.x, l.y), v[4 * t + k]));
                }
                uint4 hi, lo;
                split8(b, hi, lo);
                *ph = hi;
                *pl = lo;
            }
        }
        // X <- B X
        product([&] { pairs(km, kXMains, kXCols, desc_f16(true, 16 * kx), a_rows, x_cols); });
        if (step + 1 < steps.count) {
#pragma unroll 1
            for (int c0 = part * (W * 4 / kWarps); c0 < (part + 1) * (W * 4 / kWarps); c0 += 32) {
                f2 v[16];
                load_sum(km, kXMains, kXCols, lanes + (uint32_t)c0, v);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    f2 x[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[k] = mul2(v[4 * t + k], unscale);
                    uint4 hi, lo;
                    split8(x, hi, lo);
                    *reinterpret_cast<uint4*>(xs + chunk_at(row, c0 / 8 + t)) = hi;
                    *reinterpret_cast<uint4*>(xs + kXLo + chunk_at(row, c0 / 8 + t)) = lo;
                }
            }
        }
    }
    // out = keep w + step X, through shared memory so that rows go out whole;
    // the weights are all on their way before that
    const TW* w = (const TW*)fin.w;
    TW* o = (TW*)fin.out;
    const int32_t wn = min(W, n - j0);  // columns of X here
    const float mul = fin.step * (1.f / (kScale * kScale));
    float* tile = dump;  // A's place, and X's, are free too
    if constexpr (W == 128) tile = reinterpret_cast<float*>(as);
    if constexpr (W == 256) tile = reinterpret_cast<float*>(xs);
    constexpr int kCols = W * 4 / kWarps;  // columns a warp takes of tensor memory
    if (!tall && wn % 4 == 0 && fin.vec) {
        // 4 columns at a time: [row][W + 4]
        constexpr int kFours = kFusedM * W / 4 / kNT, kRow = W / 4;
        float wr[kFours][4] = {};
        if (w) {
#pragma unroll
            for (int e = 0; e < kFours; ++e) {
                const int t = e * kNT + (int)threadIdx.x, r = t / kRow, c = t % kRow * 4;
                if (r < m && c < wn) load4(w + (q * m + r) * fin.ld_out + j0 + c, wr[e]);
            }
        }
#pragma unroll 1
        for (int c0 = part * kCols; c0 < (part + 1) * kCols; c0 += 32) {
            float v[32];
            load_sum_32(km, kXMains, kXCols, lanes + (uint32_t)c0, v);
#pragma unroll
            for (int t = 0; t < 8; ++t)
                *reinterpret_cast<float4*>(tile + row * (W + 4) + c0 + 4 * t) =
                    make_float4(v[4 * t], v[4 * t + 1], v[4 * t + 2], v[4 * t + 3]);
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kFours; ++e) {
            const int t = e * kNT + (int)threadIdx.x, r = t / kRow, c = t % kRow * 4;
            if (r >= m || c >= wn) continue;
            const float4 x = *reinterpret_cast<const float4*>(tile + r * (W + 4) + c);
            float v[4] = {mul * x.x, mul * x.y, mul * x.z, mul * x.w};
            if (w) {
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = fin.keep * wr[e][k] + v[k];
            }
            store4(o + (q * m + r) * fin.ld_out + j0 + c, v);
        }
    } else {
        // one element at a time: [row][W + 1], or [column][129] when tall
        const int ld_row = tall ? 1 : W + 1, ld_col = tall ? kFusedM + 1 : 1;
#pragma unroll 1
        for (int c0 = part * kCols; c0 < (part + 1) * kCols; c0 += 32) {
            float v[32];
            load_sum_32(km, kXMains, kXCols, lanes + (uint32_t)c0, v);
#pragma unroll
            for (int t = 0; t < 32; ++t) tile[row * ld_row + (c0 + t) * ld_col] = v[t];
        }
        __syncthreads();
        const int lines = tall ? wn : m, width = tall ? m : wn;  // rows of the output here
        for (int l = warp; l < lines; l += kWarps) {
            const int64_t at = tall ? (q * n + j0 + l) * fin.ld_out : (q * m + l) * fin.ld_out + j0;
            const float* x = tile + l * (tall ? kFusedM + 1 : W + 1);
#pragma unroll 4
            for (int c = lane; c < width; c += 32) put(o + at + c, w ? fin.keep * to_f(w[at + c]) + mul * x[c] : mul * x[c]);
        }
    }
    tmem_fence_before();
    __syncthreads();
    // no CTA leaves before the others have its last blocks
    if constexpr (W < 256) asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
    if (warp == 1) tmem_free<512>(tmem);
}

// -------------------------------------------------------------------- host
size_t a256(size_t x) { return (x + 255) & ~(size_t)255; }

int64_t r8(int64_t x) { return (x + 7) & ~(int64_t)7; }

struct Layout {
    int64_t m, n, ldx, lda;
    size_t x[2][2], a[2], b[2], part, total;  // [buffer][plane]
};

Layout layout(int64_t count, int64_t rows, int64_t cols) {
    Layout L;
    L.m = rows < cols ? rows : cols;
    L.n = rows < cols ? cols : rows;
    L.ldx = r8(L.n);
    L.lda = r8(L.m);
    size_t o = 0;
    const auto place = [&o](int64_t bytes) {
        const size_t at = o;
        o += a256((size_t)bytes);
        return at;
    };
    for (int p = 0; p < 2; ++p) {
        L.x[0][p] = place(count * L.m * L.ldx * 2);
        L.x[1][p] = place(count * L.m * L.ldx * 2);
        L.a[p] = place(count * L.m * L.lda * 2);
        L.b[p] = place(count * L.m * L.lda * 2);
    }
    L.part = place(count * kNormParts * 8);
    L.total = o;
    return L;
}

// Map of `count` matrices [rows x cols] of fp16, ld elements a row, read in
// boxes of 64 columns x box_rows rows; reads past a matrix give zeros.
bool map_f16(CUtensorMap* map, const __half* base, int64_t cols, int64_t rows, int64_t count, int64_t ld, int box_rows) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)count};
    const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)(ld * rows) * 2};
    const cuuint32_t box[3] = {(cuuint32_t)kBK, (cuuint32_t)box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<__half*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Dependent launch of clusters of S CTAs along x.
template <int S, typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), dim3 grid, size_t smem, cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kProductThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = S;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

template <int S, int KIND>
sg_status launch_sym(const PairMaps& maps, int64_t tiles, int32_t count, int32_t m, int32_t K, const float* coef,
                     Planes in, Planes out, int64_t ld, cudaStream_t s) {
    static OncePerDevice set;
    SG_CUDA(allow_smem(set, k_ns_sym<S, KIND>, kSymSmem));
    SG_CUDA(launch_cluster<S>(k_ns_sym<S, KIND>, dim3((unsigned)(tiles * S), (unsigned)count), kSymSmem, s, maps, m, K,
                              coef[0], coef[1], coef[2], in, out, ld));
    return SG_OK;
}

// The upper triangle's tiles are few when m is small, and K is long: K is
// split over up to 8 CTAs while that many more still fit the SMs and each
// keeps two K tiles or more.  us for five steps, split 1 / 2 / 4 / 8 at most: 256 x
// 4096 324 / 213 / 162 / 142; 1024 x 4096 461 / 330 / 269 / -.
template <int KIND>
sg_status run_sym(const PairMaps& maps, int32_t count, int32_t m, int32_t K, const float* coef, Planes in, Planes out,
                  int64_t ld, cudaStream_t s) {
    const int64_t nt = cdiv(m, kTile), tiles = nt * (nt + 1) / 2, kt = cdiv(K, kBK);
    int split = 1;
    while (split < 8 && tiles * count * split * 2 <= num_sms() && kt >= split * 4) split *= 2;
    switch (split) {
        case 1: return launch_sym<1, KIND>(maps, tiles, count, m, K, coef, in, out, ld, s);
        case 2: return launch_sym<2, KIND>(maps, tiles, count, m, K, coef, in, out, ld, s);
        case 4: return launch_sym<4, KIND>(maps, tiles, count, m, K, coef, in, out, ld, s);
        default: return launch_sym<8, KIND>(maps, tiles, count, m, K, coef, in, out, ld, s);
    }
}

template <int BN, typename TW, bool FINAL>
sg_status launch_apply(const ApplyMaps& maps, int32_t count, int32_t m, int32_t n, Planes out, int64_t ldx,
                       const FinalArgs& fin, cudaStream_t s) {
    constexpr int smem = kApplySmem<BN>;
    static OncePerDevice set;
    SG_CUDA(allow_smem(set, k_ns_apply<BN, TW, FINAL>, smem));
    SG_CUDA(launch_pdl(k_ns_apply<BN, TW, FINAL>, dim3((unsigned)cdiv(n, BN), (unsigned)cdiv(m, kTile), (unsigned)count),
                       dim3(kProductThreads), smem, s, maps, m, n, out, ldx, fin));
    return SG_OK;
}

template <typename TW, bool FINAL>
sg_status run_apply(int bn, const ApplyMaps& maps, int32_t count, int32_t m, int32_t n, Planes out, int64_t ldx,
                    const FinalArgs& fin, cudaStream_t s) {
    if (bn == 256) return launch_apply<256, TW, FINAL>(maps, count, m, n, out, ldx, fin, s);
    if (bn == 128) return launch_apply<128, TW, FINAL>(maps, count, m, n, out, ldx, fin, s);
    return launch_apply<64, TW, FINAL>(maps, count, m, n, out, ldx, fin, s);
}

const float kCoef[3] = {3.4445f, -4.7750f, 2.0315f};

// The fused form: W columns a CTA, `ctas` of them (8 or 16; 1 for W = 256).
template <int W, typename TS, typename TW>
sg_status launch_fused(const Source<TS>& src, int32_t count, int32_t rows, int32_t cols, int ctas, const Steps& steps,
                       float eps, const FinalArgs& fin, cudaStream_t s) {
    static OncePerDevice set;
    SG_CUDA(once_on_device(set, [] {
        const auto kernel = k_ns_fused<W, TS, TW>;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kFusedSmem<W>);
        return e != cudaSuccess || W == 256 ? e : cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    }));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, (unsigned)count);
    cfg.blockDim = dim3(kFusedThreads<W>);
    cfg.dynamicSmemBytes = kFusedSmem<W>;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)ctas;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    SG_CUDA(cudaLaunchKernelEx(&cfg, k_ns_fused<W, TS, TW>, src, rows, cols, steps, eps, fin));
    return SG_OK;
}

// Whether the current device takes clusters of 16 CTAs with all of an SM's
// shared memory each (looked up once for each device).
bool clusters_of_16() {
    static OncePerDevice set;
    static std::atomic<uint64_t> yes{0};  // by device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        return false;
    }
    set(dev, [&] {
        const auto kernel = k_ns_fused<128, float, float>;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(16);
        cfg.blockDim = dim3(kFusedThreads<128>);
        cfg.dynamicSmemBytes = kFusedSmem<128>;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = 16;
        at[0].val.clusterDim.y = 1;
        at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        int n = 0;
        const bool ok = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kFusedSmem<128>) == cudaSuccess &&
                        cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n > 0;
        if (ok) yes.fetch_or((uint64_t)1 << dev);
        else cudaGetLastError();
        return 0;
    });
    return (yes.load() >> dev) & 1;
}

template <typename TS, typename TW>
sg_status run(Source<TS> src, int32_t count, int32_t rows, int32_t cols, int32_t steps, const float* coef, float eps,
              const TW* w, float keep, float step, TW* out, int64_t ld_out, char* ws, cudaStream_t s) {
    const Layout L = layout(count, rows, cols);
    const int32_t m = (int32_t)L.m, n = (int32_t)L.n;
    const FinalArgs fin = {w, out, keep, step, ld_out, rows > cols ? 1 : 0,
                           (((uintptr_t)w | (uintptr_t)out) % (4 * sizeof(TW)) == 0 && ld_out % 4 == 0) ? 1 : 0};
    // a matrix that the shared memory of one cluster holds is done in one
    // launch: up to 256 columns by one CTA, which has nothing to exchange; else
    // 64 columns a CTA while 16 CTAs reach, since each product and each pass
    // over tensor memory is then half as long.  us: 128 x 200 by 256 / 64 columns
    // a CTA 50 / 56; 128 x 1024 by 64 / 128 59 / 65.  With cold caches and against the
    // launches of products: 128 x 200 59 / 125, 128 x 2048 78 / 127
    if (m <= kFusedM && n <= kFusedMaxCtas * 128 && steps > 0 && (n <= 8 * 64 || clusters_of_16())) {
        Steps st;
        st.count = steps;
        for (int32_t k = 0; k < SG_MAX_NS_STEPS; ++k)
            for (int i = 0; i < 3; ++i) st.coef[k][i] = k < steps ? (coef ? coef[3 * k + i] : kCoef[i]) : 0.f;
        const int width = n <= 256 ? 256 : n <= kFusedMaxCtas * 64 ? 64 : 128;
        int ctas = 1;
        while (ctas * width < n) ctas *= 2;
        if (width == 256) return launch_fused<256, TS, TW>(src, count, rows, cols, 1, st, eps, fin, s);
        return width == 64 ? launch_fused<64, TS, TW>(src, count, rows, cols, ctas, st, eps, fin, s)
                           : launch_fused<128, TS, TW>(src, count, rows, cols, ctas, st, eps, fin, s);
    }
    Planes x[2], a, b;
    for (int i = 0; i < 2; ++i) x[i] = {(__half*)(ws + L.x[i][0]), (__half*)(ws + L.x[i][1])};
    a = {(__half*)(ws + L.a[0]), (__half*)(ws + L.a[1])};
    b = {(__half*)(ws + L.b[0]), (__half*)(ws + L.b[1])};
    double* part = (double*)(ws + L.part);
    // one part for every 8 row pieces of 512 columns (a warp each), up to kNormParts
    int64_t parts = cdiv((int64_t)rows * cdiv(cols, 512), 8);
    if (parts > kNormParts) parts = kNormParts;
    SG_CUDA(launch_pdl(k_ns_norm<TS>, dim3((unsigned)parts, (unsigned)count), dim3(kThreads), 0, s, src, rows, cols, part));
    SG_CUDA(launch_pdl(k_ns_split<TS>, dim3((unsigned)cdiv(n, kSplitN), (unsigned)cdiv(m, kSplitM), (unsigned)count),
                       dim3(kThreads), 0, s, src, rows, cols, (const double*)part, (int32_t)parts, eps, x[0], L.ldx));
    if (steps == 0) {
        const int64_t eb = cdiv((int64_t)rows * cols, kThreads) < 1024 ? cdiv((int64_t)rows * cols, kThreads) : 1024;
        SG_CUDA(launch_pdl(k_ns_store<TW>, dim3((unsigned)eb, (unsigned)count), dim3(kThreads), 0, s, x[0], L.ldx, rows,
                           cols, fin));
        return SG_OK;
    }
    PairMaps mx[2], ma;   // rows as 128-row K-major operands
    ApplyMaps mb[2];      // B K-major, X MN-major
    memset(mx, 0, sizeof(mx));
    memset(&ma, 0, sizeof(ma));
    memset(mb, 0, sizeof(mb));
    bool ok = map_f16(&ma.hi, a.hi, m, m, count, L.lda, kTile) && map_f16(&ma.lo, a.lo, m, m, count, L.lda, kTile);
    for (int i = 0; i < 2 && ok; ++i)
        ok = map_f16(&mx[i].hi, x[i].hi, n, m, count, L.ldx, kTile) &&
             map_f16(&mx[i].lo, x[i].lo, n, m, count, L.ldx, kTile) &&
             map_f16(&mb[i].bhi, b.hi, m, m, count, L.lda, kTile) &&
             map_f16(&mb[i].blo, b.lo, m, m, count, L.lda, kTile) &&
             map_f16(&mb[i].xhi, x[i].hi, n, m, count, L.ldx, kBK) &&
             map_f16(&mb[i].xlo, x[i].lo, n, m, count, L.ldx, kBK);
    if (!ok) return fail(SG_ERR_CUDA, "orthogonalise: tensor map encoding failed");
    // 256-column tiles read B least often, when they give three SMs of four a
    // tile; 64-column ones are the quickest when even they leave SMs idle.  us,
    // 64 / 128 / 256: 1001 x 603 148 / 154 / 185; 512 x 4096 188 / 163 / 184; 768 x
    // 2000 215 / 182 / 207; 1024 x 4096 398 / 302 / 273
    const int64_t bands = cdiv(m, kTile) * count;
    const int bn = cdiv(n, 256) * bands >= num_sms() * 3 / 4 ? 256 : cdiv(n, 64) * bands <= num_sms() ? 64 : 128;
    for (int32_t k = 0; k < steps; ++k) {
        const float* c = coef ? coef + 3 * k : kCoef;
        sg_status st = run_sym<GRAM>(mx[k & 1], count, m, n, c, a, a, L.lda, s);
        if (st == SG_OK) st = run_sym<SQUARE>(ma, count, m, m, c, a, b, L.lda, s);
        if (st != SG_OK) return st;
        const Planes to = x[(k & 1) ^ 1];
        st = k + 1 < steps ? run_apply<float, false>(bn, mb[k & 1], count, m, n, to, L.ldx, fin, s)
                           : run_apply<TW, true>(bn, mb[k & 1], count, m, n, to, L.ldx, fin, s);
        if (st != SG_OK) return st;
    }
    return SG_OK;
}

sg_status check(const char* what, int32_t count, int32_t rows, int32_t cols, int32_t steps, const void* ws,
                size_t ws_bytes) {
    if (count < 0 || count > 65535 || rows <= 0 || cols <= 0 || rows > 65536 || cols > 65536 ||
        (rows < cols ? rows : cols) > 8192)
        return fail(SG_ERR_INVALID_ARG, "%s: bad sizes", what);
    if (steps < 0 || steps > SG_MAX_NS_STEPS)
        return fail(SG_ERR_INVALID_ARG, "%s: steps must be 0 .. %d", what, SG_MAX_NS_STEPS);
    if (count == 0) return SG_OK;
    const size_t need = layout(count, rows, cols).total;
    if (!ws || (uintptr_t)ws % 256 || ws_bytes < need)
        return fail(SG_ERR_INVALID_ARG, "%s: workspace needs %zu bytes, 256-byte aligned", what, need);
    return SG_OK;
}

}  // namespace

extern "C" size_t sg_orthogonalise_workspace(int32_t count, int32_t rows, int32_t cols) {
    if (count <= 0 || count > 65535 || rows <= 0 || cols <= 0 || rows > 65536 || cols > 65536 ||
        (rows < cols ? rows : cols) > 8192)
        return 0;
    return layout(count, rows, cols).total;
}

extern "C" sg_status sg_orthogonalise(const void* d_g, int32_t dtype, int32_t count, int32_t rows, int32_t cols,
                                      int64_t ld, int32_t steps, const float* h_coef, float eps, float scale,
                                      void* d_out, int64_t ld_out, void* d_workspace, size_t workspace_bytes,
                                      sg_stream_t stream) {
    if (dtype != SG_F32 && dtype != SG_BF16) return fail(SG_ERR_UNSUPPORTED, "sg_orthogonalise: dtype");
    const sg_status st = check("sg_orthogonalise", count, rows, cols, steps, d_workspace, workspace_bytes);
    if (st != SG_OK || count == 0) return st;
    if (ld < cols || ld_out < cols) return fail(SG_ERR_INVALID_ARG, "sg_orthogonalise: a row stride is below cols");
    if (!d_g || !d_out) return fail(SG_ERR_INVALID_ARG, "sg_orthogonalise: NULL array");
    if (((uintptr_t)d_g | (uintptr_t)d_out) % (dtype == SG_F32 ? 4 : 2))
        return fail(SG_ERR_INVALID_ARG, "sg_orthogonalise: an array is not aligned to its elements");
    if (d_g == d_out && ld != ld_out) return fail(SG_ERR_INVALID_ARG, "sg_orthogonalise: in place needs ld_out = ld");
    cudaStream_t s = (cudaStream_t)stream;
    const int64_t elem = dtype == SG_F32 ? 4 : 2;
    if (dtype == SG_F32) {
        const Source<float> src = {(const float*)d_g, ld, nullptr, nullptr, 0.f, 0, (uintptr_t)d_g % 16 == 0 && ld * elem % 16 == 0};
        return run<float, float>(src, count, rows, cols, steps, h_coef, eps, nullptr, 0.f, scale, (float*)d_out, ld_out,
                                 (char*)d_workspace, s);
    }
    const Source<__nv_bfloat16> src = {(const __nv_bfloat16*)d_g, ld, nullptr, nullptr, 0.f, 0, (uintptr_t)d_g % 16 == 0 && ld * elem % 16 == 0};
    return run<__nv_bfloat16, __nv_bfloat16>(src, count, rows, cols, steps, h_coef, eps, nullptr, 0.f, scale,
                                             (__nv_bfloat16*)d_out, ld_out, (char*)d_workspace, s);
}

extern "C" sg_status sg_muon_step(const void* d_w, int32_t dtype_w, const float* d_g, const float* d_m, int32_t count,
                                  int32_t rows, int32_t cols, float rate, float momentum, int32_t nesterov,
                                  float weight_decay, float scale, int32_t steps, const float* h_coef, float eps,
                                  void* d_w_out, float* d_m_out, void* d_workspace, size_t workspace_bytes,
                                  sg_stream_t stream) {
    if (dtype_w != SG_F32 && dtype_w != SG_BF16) return fail(SG_ERR_UNSUPPORTED, "sg_muon_step: dtype");
    const sg_status st = check("sg_muon_step", count, rows, cols, steps, d_workspace, workspace_bytes);
    if (st != SG_OK || count == 0) return st;
    if (!d_w || !d_g || !d_m || !d_w_out || !d_m_out) return fail(SG_ERR_INVALID_ARG, "sg_muon_step: NULL array");
    if (((uintptr_t)d_w | (uintptr_t)d_w_out) % (dtype_w == SG_F32 ? 4 : 2) ||
        ((uintptr_t)d_g | (uintptr_t)d_m | (uintptr_t)d_m_out) % 4)
        return fail(SG_ERR_INVALID_ARG, "sg_muon_step: an array is not aligned to its elements");
    cudaStream_t s = (cudaStream_t)stream;
    const int32_t vec = cols % 4 ? 0 : ((uintptr_t)d_g % 16 == 0 ? 1 : 0) + (((uintptr_t)d_m | (uintptr_t)d_m_out) % 16 == 0 ? 2 : 0);
    const Source<float> src = {d_g, cols, d_m, d_m_out, momentum, nesterov, vec};
    const float keep = 1.f - rate * weight_decay, step = -rate * scale;
    if (dtype_w == SG_F32)
        return run<float, float>(src, count, rows, cols, steps, h_coef, eps, (const float*)d_w, keep, step,
                                 (float*)d_w_out, cols, (char*)d_workspace, s);
    return run<float, __nv_bfloat16>(src, count, rows, cols, steps, h_coef, eps, (const __nv_bfloat16*)d_w, keep, step,
                                     (__nv_bfloat16*)d_w_out, cols, (char*)d_workspace, s);
}
