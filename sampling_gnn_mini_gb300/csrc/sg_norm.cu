// Layer norm of rows x of dim values, and its gradient:
//   mu = mean x,  r = 1 / sqrt(mean (x - mu)^2 + eps),  h = (x - mu) r,  y = h w + b
//   u = g w:  dx = r (u - mean u - h mean(u h)),  dw = sum over rows of g h,  db = sum over rows of g
// Bound by memory: forward reads and writes a row once, backward reads two rows and
// writes one.  A row's values stay in the registers of a group of 4 to 32 lanes (up
// to 512 values) or of a block (up to 16,384): 16 a thread, so that the gradient of
// the weight and bias, 32 sums a thread, fits beside them.  The deviation is summed
// about the mean, in a second pass over the registers.
//
// Columns belong to threads.  In the gradient a block walks over its rows with the
// columns' sums in registers, writes them once to the workspace, and a second kernel
// adds up the blocks' sums in order: no float atomics, the same bits on every run.
//
// Values move in units of up to 16 bytes, the largest that every array and row
// stride is a multiple of (odd widths in bf16: single values).
#include "sg_internal.cuh"
#include "sg_rows.cuh"

using namespace sgi;

namespace {

constexpr int kHeld = 16;      // values of a row a thread holds
constexpr int kThreads = 256;  // of a block of warps' rows

// ------------------------------------------------- N values in one access
template <int BYTES>
struct Raw;
template <>
struct Raw<16> {
    typedef uint4 type;
};
template <>
struct Raw<8> {
    typedef uint2 type;
};
template <>
struct Raw<4> {
    typedef uint32_t type;
};
template <>
struct Raw<2> {
    typedef uint16_t type;
};
template <typename T, int N>
using raw_t = typename Raw<N * (int)sizeof(T)>::type;

template <typename T, int N>
__device__ __forceinline__ void values_of(const raw_t<T, N>& u, float (&f)[N]) {
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = to_f(e[i]);
}
template <typename T, int N>
__device__ __forceinline__ raw_t<T, N> raw_of(const float (&f)[N]) {
    raw_t<T, N> u;
    T* e = reinterpret_cast<T*>(&u);
#pragma unroll
    for (int i = 0; i < N; ++i) put(e + i, f[i]);
    return u;
}
// N values of a weight or bias at column c (fp32 or bf16; none: `none`)
template <int N>
__device__ __forceinline__ void load_param(const void* w, int32_t bf16, int32_t c, float none, float (&f)[N]) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = none;
    } else if (bf16) {
        values_of<__nv_bfloat16, N>(__ldg(reinterpret_cast<const raw_t<__nv_bfloat16, N>*>((const __nv_bfloat16*)w + c)), f);
    } else {
        constexpr int M = N < 4 ? N : 4;
#pragma unroll
        for (int k = 0; k < N; k += M) {
            float t[M];
            values_of<float, M>(__ldg(reinterpret_cast<const raw_t<float, M>*>((const float*)w + c + k)), t);
#pragma unroll
            for (int i = 0; i < M; ++i) f[k + i] = t[i];
        }
    }
}

// -------------------------------------------------------- sums over a group
// Sums of C values over the L threads that share a row, in every one of them.
// L > 32: the whole block; sh holds two sets of warps' sums, used in turn (a set is
// written again after the barrier of the other one, which follows its last reading).
template <int L, int C>
struct GroupSum {
    __device__ __forceinline__ static void of(float (&x)[C], float*, int&) {
#pragma unroll
        for (int d = L / 2; d > 0; d >>= 1)
#pragma unroll
            for (int c = 0; c < C; ++c) x[c] += __shfl_xor_sync(0xFFFFFFFFu, x[c], d);
    }
};
template <int L, int C>
__device__ __forceinline__ void group_sum(float (&x)[C], float* sh, int& turn) {
    if constexpr (L <= 32) {
        GroupSum<L, C>::of(x, sh, turn);
    } else {
        constexpr int W = L / 32;
        GroupSum<32, C>::of(x, sh, turn);
        float* to = sh + turn * 2 * W;
        turn ^= 1;
        if (lane_id() == 0)
#pragma unroll
            for (int c = 0; c < C; ++c) to[c * W + (threadIdx.x >> 5)] = x[c];
        __syncthreads();
#pragma unroll
        for (int c = 0; c < C; ++c) x[c] = (int)lane_id() < W ? to[c * W + lane_id()] : 0.f;
        GroupSum<(W < 32 ? W : 32), C>::of(x, sh, turn);
        if constexpr (W < 32) {
#pragma unroll
            for (int c = 0; c < C; ++c) x[c] = __shfl_sync(0xFFFFFFFFu, x[c], 0);
        }
    }
}

// ----------------------------------------------------------------- forward
template <typename T>
struct FwdArgs {
    const T* x;
    T* y;
    int64_t ld, ld_y;
    const void* weight;
    const void* bias;
    const int32_t* d_n;
    int32_t n_cap, dim, w_bf16;
    float eps;
    float* mean;
    float* rstd;
};

// R rows a group at once, their loads in flight together.
template <typename T, int N, int V, int L, int NT, int R>
__global__ void __launch_bounds__(NT) k_norm_fwd(FwdArgs<T> a) {
    pdl_start();
    constexpr int kRows = L <= 32 ? NT / L : 1;  // of a block at once
    __shared__ float sh[L > 32 ? 4 * (L / 32) : 1];
    int turn = 0;
    const int32_t n = rows_of(a.d_n, a.n_cap), units = a.dim / N;
    const int l = (int)threadIdx.x % L;
    const int64_t r0 = (int64_t)blockIdx.x * (kRows * R) + (int)threadIdx.x / L;
    if ((int64_t)blockIdx.x * (kRows * R) >= n) return;
    raw_t<T, N> x[R][V];
#pragma unroll
    for (int q = 0; q < R; ++q)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int32_t u = l + v * L;
            const int64_t r = r0 + q * kRows;
            if (r < n && u < units) x[q][v] = *reinterpret_cast<const raw_t<T, N>*>(a.x + r * a.ld + u * N);
            else x[q][v] = raw_t<T, N>{};
        }
    const float inv = 1.f / (float)a.dim;
#pragma unroll
    for (int q = 0; q < R; ++q) {
        const int64_t r = r0 + q * kRows;
        float f[V][N], s[1] = {0.f};
#pragma unroll
        for (int v = 0; v < V; ++v) {
            values_of<T, N>(x[q][v], f[v]);
#pragma unroll
            for (int i = 0; i < N; ++i) s[0] += f[v][i];
        }
        group_sum<L, 1>(s, sh, turn);
        const float mu = s[0] * inv;
        s[0] = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (l + v * L < units)
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    f[v][i] -= mu;
                    s[0] = fmaf(f[v][i], f[v][i], s[0]);
                }
        group_sum<L, 1>(s, sh, turn);
        const float rs = __frsqrt_rn(fmaf(s[0], inv, a.eps));
        if (r >= n) continue;
        if (l == 0) {
            if (a.mean) a.mean[r] = mu;
            if (a.rstd) a.rstd[r] = rs;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int32_t u = l + v * L;
            if (u >= units) continue;
            float w[N], b[N];
            load_param<N>(a.weight, a.w_bf16, u * N, 1.f, w);
            load_param<N>(a.bias, a.w_bf16, u * N, 0.f, b);
#pragma unroll
            for (int i = 0; i < N; ++i) f[v][i] = fmaf(f[v][i] * rs, w[i], b[i]);
            *reinterpret_cast<raw_t<T, N>*>(a.y + r * a.ld_y + u * N) = raw_of<T, N>(f[v]);
        }
    }
}

// ---------------------------------------------------------------- backward
template <typename T>
struct BwdArgs {
    const T* g;
    const T* x;
    T* dx;
    int64_t ld_g, ld, ld_dx;
    const void* weight;
    const float* mean;
    const float* rstd;
    const int32_t* d_n;
    int32_t n_cap, dim, w_bf16;
    float* parts;  // per block: sums of g h by column, then of g; NULL: not wanted
};

template <typename T, int N, int V, int L, int NT, int R>
__global__ void __launch_bounds__(NT) k_norm_bwd(BwdArgs<T> a) {
    pdl_start();
    constexpr int kRows = L <= 32 ? NT / L : 1;
    __shared__ float sh[L > 32 ? 4 * (L / 32) : 1];
    __shared__ float cols[L > 32 ? 1 : NT * V * N];  // the warps' sums of a column
    int turn = 0;
    const int32_t n = rows_of(a.d_n, a.n_cap), units = a.dim / N;
    const int l = (int)threadIdx.x % L;
    float sw[V][N], sb[V][N], w[V][N];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int i = 0; i < N; ++i) sw[v][i] = 0.f, sb[v][i] = 0.f, w[v][i] = 0.f;
        if (l + v * L < units) load_param<N>(a.weight, a.w_bf16, (l + v * L) * N, 1.f, w[v]);
    }
    const float inv = 1.f / (float)a.dim;
    const int64_t step = (int64_t)gridDim.x * (kRows * R);
    for (int64_t b0 = (int64_t)blockIdx.x * (kRows * R); b0 < n; b0 += step) {  // the same in the whole block
        const int64_t r0 = b0 + (int)threadIdx.x / L;
        raw_t<T, N> x[R][V], g[R][V];
        float mu[R], rs[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int64_t r = r0 + q * kRows;
            mu[q] = r < n ? __ldg(a.mean + r) : 0.f;
            rs[q] = r < n ? __ldg(a.rstd + r) : 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int32_t u = l + v * L;
                x[q][v] = raw_t<T, N>{};
                g[q][v] = raw_t<T, N>{};
                if (r < n && u < units) {
                    x[q][v] = *reinterpret_cast<const raw_t<T, N>*>(a.x + r * a.ld + u * N);
                    g[q][v] = *reinterpret_cast<const raw_t<T, N>*>(a.g + r * a.ld_g + u * N);
                }
            }
        }
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int64_t r = r0 + q * kRows;
            float h[V][N], f[V][N], s[2] = {0.f, 0.f};
#pragma unroll
            for (int v = 0; v < V; ++v) {
                values_of<T, N>(x[q][v], h[v]);
                values_of<T, N>(g[q][v], f[v]);
#pragma unroll
                for (int i = 0; i < N; ++i) {  // (values past the row's end: g = 0, w = 0)
                    h[v][i] = (h[v][i] - mu[q]) * rs[q];
                    sw[v][i] = fmaf(f[v][i], h[v][i], sw[v][i]);
                    sb[v][i] += f[v][i];
                    f[v][i] *= w[v][i];
                    s[0] += f[v][i];
                    s[1] = fmaf(f[v][i], h[v][i], s[1]);
                }
            }
            group_sum<L, 2>(s, sh, turn);
            if (r >= n) continue;
            const float mg = s[0] * inv, mh = s[1] * inv;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int32_t u = l + v * L;
                if (u >= units) continue;
#pragma unroll
                for (int i = 0; i < N; ++i) f[v][i] = rs[q] * (f[v][i] - fmaf(h[v][i], mh, mg));
                *reinterpret_cast<raw_t<T, N>*>(a.dx + r * a.ld_dx + u * N) = raw_of<T, N>(f[v]);
            }
        }
    }
    if (!a.parts) return;
    float* to = a.parts + (int64_t)blockIdx.x * 2 * a.dim;
    if constexpr (L > 32) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int32_t u = l + v * L;
            if (u >= units) continue;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                to[u * N + i] = sw[v][i];
                to[a.dim + u * N + i] = sb[v][i];
            }
        }
    } else {
        constexpr int W = L * V * N;  // columns of a group
        for (int p = 0; p < 2; ++p) {
            __syncthreads();
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int i = 0; i < N; ++i)
                    cols[((int)threadIdx.x / L) * W + (l + v * L) * N + i] = p ? sb[v][i] : sw[v][i];
            __syncthreads();
            for (int c = threadIdx.x; c < a.dim; c += NT) {
                float s = 0.f;
#pragma unroll 8
                for (int q = 0; q < kRows; ++q) s += cols[q * W + c];
                to[p * a.dim + c] = s;
            }
        }
    }
}

// The blocks' sums in order: 32 columns a block, a 32nd of the blocks' sums a warp.
__global__ void __launch_bounds__(1024) k_norm_join(const float* __restrict__ parts, int32_t count, int32_t dim,
                                                    void* dweight, void* dbias, int32_t bf16) {
    pdl_start();
    __shared__ float sh[32][33];
    const int lane = (int)lane_id(), warp = (int)(threadIdx.x >> 5);
    const int32_t c = (int32_t)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < 2 * dim) {
#pragma unroll 8
        for (int32_t p = warp; p < count; p += 32) s += parts[(int64_t)p * 2 * dim + c];
    }
    sh[warp][lane] = s;
    __syncthreads();
    s = warp_sum(sh[lane][warp]);  // column `warp` of the block
    const int32_t o = (int32_t)blockIdx.x * 32 + warp;
    if (lane != 0 || o >= 2 * dim) return;
    void* to = o < dim ? dweight : dbias;
    if (!to) return;
    const int32_t i = o < dim ? o : o - dim;
    if (bf16) put((__nv_bfloat16*)to + i, s);
    else put((float*)to + i, s);
}

// -------------------------------------------------------------------- host
constexpr int kMaxDim = SG_MAX_NORM_DIM;

// Blocks of the gradient at most: three of 256 threads an SM, one of 1024.
int64_t max_parts(int32_t dim) { return (int64_t)num_sms() * (dim <= 4096 ? 4 : dim <= 8192 ? 2 : 1); }

template <typename T, int N, int V, int L, int NT, int R>
sg_status go(const FwdArgs<T>& a, cudaStream_t s) {
    constexpr int kRows = (L <= 32 ? NT / L : 1) * R;
    SG_CUDA(launch_pdl(k_norm_fwd<T, N, V, L, NT, R>, dim3((unsigned)cdiv(a.n_cap, kRows)), dim3(NT), 0, s, a));
    return SG_OK;
}
template <typename T, int N, int V, int L, int NT, int R>
sg_status go(const BwdArgs<T>& a, cudaStream_t s, int64_t* count) {
    constexpr int kRows = (L <= 32 ? NT / L : 1) * R;
    int64_t blocks = cdiv(a.n_cap, kRows);
    if (blocks > max_parts(a.dim)) blocks = max_parts(a.dim);
    *count = blocks;
    SG_CUDA(launch_pdl(k_norm_bwd<T, N, V, L, NT, R>, dim3((unsigned)blocks), dim3(NT), 0, s, a));
    return SG_OK;
}

template <typename T, int N, typename A, typename... More>
sg_status by_size(const A& a, More... more) {
    constexpr int V = kHeld / N;
    const int32_t units = a.dim / N;
    if constexpr (N * sizeof(T) == 16) {
        if (units <= 4) return go<T, N, 1, 4, kThreads, 4>(a, more...);
        if (units <= 8) return go<T, N, 1, 8, kThreads, 4>(a, more...);
        if (units <= 16) return go<T, N, 1, 16, kThreads, 4>(a, more...);
        if (units <= 32) return go<T, N, 1, 32, kThreads, 4>(a, more...);
        if (units <= 64) return go<T, N, 2, 32, kThreads, 2>(a, more...);
    } else {
        if (a.dim <= 128) return go<T, N, 4 / N, 32, kThreads, 2>(a, more...);
    }
    if (a.dim <= 32 * kHeld) return go<T, N, V, 32, kThreads, 1>(a, more...);
    if (a.dim <= 64 * kHeld) return go<T, N, V, 64, 64, 1>(a, more...);
    if (a.dim <= 128 * kHeld) return go<T, N, V, 128, 128, 1>(a, more...);
    if (a.dim <= 256 * kHeld) return go<T, N, V, 256, 256, 1>(a, more...);
    if (a.dim <= 512 * kHeld) return go<T, N, V, 512, 512, 1>(a, more...);
    return go<T, N, V, 1024, 1024, 1>(a, more...);
}

// Values of a unit: the largest power of two that the width, the arrays (bits: all
// addresses and row strides in bytes) and the parameters (pbits) allow.
int unit_of(int32_t dim, uintptr_t bits, uintptr_t pbits, int e, int ew) {
    int n = 16 / e;
    const auto fits = [&](int k) {
        return dim % k == 0 && bits % (uintptr_t)(k * e) == 0 && pbits % (uintptr_t)(k * ew < 16 ? k * ew : 16) == 0;
    };
    while (n > 1 && !fits(n)) n /= 2;
    return n;
}

template <typename T, typename A, typename... More>
sg_status by_unit(int unit, const A& a, More... more) {
    if constexpr (sizeof(T) == 2)
        if (unit == 8) return by_size<T, 8>(a, more...);
    if (unit == 4) return by_size<T, 4>(a, more...);
    if (unit == 2) return by_size<T, 2>(a, more...);
    return by_size<T, 1>(a, more...);
}

bool known(int32_t dtype) { return dtype == SG_F32 || dtype == SG_BF16; }
int size_of(int32_t dtype) { return dtype == SG_F32 ? 4 : 2; }

template <typename T>
sg_status bwd(BwdArgs<T> a, int unit, void* dw, void* db, cudaStream_t s) {
    int64_t count = 0;
    if (a.n_cap > 0) {
        const sg_status st = by_unit<T>(unit, a, s, &count);
        if (st != SG_OK) return st;
    }
    if (!a.parts) return SG_OK;
    SG_CUDA(launch_pdl(k_norm_join, dim3((unsigned)cdiv(2 * (int64_t)a.dim, 32)), dim3(1024), 0, s, (const float*)a.parts,
                       (int32_t)count, a.dim, dw, db, a.w_bf16));
    return SG_OK;
}

}  // namespace

extern "C" sg_status sg_layernorm_fwd(const void* d_x, int32_t dtype, int32_t n_cap, const int32_t* d_n, int32_t dim,
                                      int64_t ld, const void* d_weight, const void* d_bias, int32_t dtype_w, float eps,
                                      void* d_y, int64_t ld_y, float* d_mean, float* d_rstd, sg_stream_t stream) {
    if (!known(dtype) || !known(dtype_w)) return fail(SG_ERR_UNSUPPORTED, "sg_layernorm_fwd: dtype");
    if (n_cap < 0 || dim <= 0 || dim > kMaxDim)
        return fail(SG_ERR_INVALID_ARG, "sg_layernorm_fwd: bad sizes (dim 1 to %d)", kMaxDim);
    if (!(eps > 0.f)) return fail(SG_ERR_INVALID_ARG, "sg_layernorm_fwd: eps must be above 0");
    if (ld < dim || ld_y < dim) return fail(SG_ERR_INVALID_ARG, "sg_layernorm_fwd: a row stride is below dim");
    if (n_cap > 0 && (!d_x || !d_y)) return fail(SG_ERR_INVALID_ARG, "sg_layernorm_fwd: NULL array");
    const int e = size_of(dtype), ew = size_of(dtype_w);
    if (((uintptr_t)d_x | (uintptr_t)d_y) % e || ((uintptr_t)d_weight | (uintptr_t)d_bias) % ew ||
        ((uintptr_t)d_mean | (uintptr_t)d_rstd) % 4)
        return fail(SG_ERR_INVALID_ARG, "sg_layernorm_fwd: an array is not aligned to its elements");
    if (d_x == d_y && ld != ld_y) return fail(SG_ERR_INVALID_ARG, "sg_layernorm_fwd: in place needs ld_y = ld");
    if (n_cap == 0) return SG_OK;
    cudaStream_t s = (cudaStream_t)stream;
    const int unit = unit_of(dim, (uintptr_t)d_x | (uintptr_t)d_y | (uintptr_t)(ld * e) | (uintptr_t)(ld_y * e),
                             (uintptr_t)d_weight | (uintptr_t)d_bias, e, ew);
    if (dtype == SG_F32) {
        const FwdArgs<float> a = {(const float*)d_x, (float*)d_y, ld, ld_y, d_weight, d_bias, d_n, n_cap, dim,
                                  dtype_w == SG_BF16, eps, d_mean, d_rstd};
        return by_unit<float>(unit, a, s);
    }
    const FwdArgs<__nv_bfloat16> a = {(const __nv_bfloat16*)d_x, (__nv_bfloat16*)d_y, ld, ld_y, d_weight, d_bias, d_n,
                                      n_cap, dim, dtype_w == SG_BF16, eps, d_mean, d_rstd};
    return by_unit<__nv_bfloat16>(unit, a, s);
}

extern "C" size_t sg_layernorm_bwd_workspace(int32_t n_cap, int32_t dim) {
    if (n_cap < 0 || dim <= 0 || dim > kMaxDim) return 0;
    int64_t parts = max_parts(dim);
    if (parts > n_cap) parts = n_cap;
    return (size_t)cdiv((parts > 0 ? parts : 1) * 2 * dim * 4, 256) * 256;
}

extern "C" sg_status sg_layernorm_bwd(const void* d_g, const void* d_x, int32_t dtype, int32_t n_cap, const int32_t* d_n,
                                      int32_t dim, int64_t ld_g, int64_t ld, const void* d_weight, int32_t dtype_w,
                                      const float* d_mean, const float* d_rstd, void* d_dx, int64_t ld_dx, void* d_dweight,
                                      void* d_dbias, void* d_workspace, size_t workspace_bytes, sg_stream_t stream) {
    if (!known(dtype) || !known(dtype_w)) return fail(SG_ERR_UNSUPPORTED, "sg_layernorm_bwd: dtype");
    if (n_cap < 0 || dim <= 0 || dim > kMaxDim)
        return fail(SG_ERR_INVALID_ARG, "sg_layernorm_bwd: bad sizes (dim 1 to %d)", kMaxDim);
    if (ld < dim || ld_g < dim || ld_dx < dim)
        return fail(SG_ERR_INVALID_ARG, "sg_layernorm_bwd: a row stride is below dim");
    if (n_cap > 0 && (!d_g || !d_x || !d_dx || !d_mean || !d_rstd))
        return fail(SG_ERR_INVALID_ARG, "sg_layernorm_bwd: NULL array");
    const size_t need = sg_layernorm_bwd_workspace(n_cap, dim);
    if (!d_workspace || (uintptr_t)d_workspace % 256 || workspace_bytes < need)
        return fail(SG_ERR_INVALID_ARG, "sg_layernorm_bwd: workspace needs %zu bytes, 256-byte aligned", need);
    const int e = size_of(dtype), ew = size_of(dtype_w);
    if (((uintptr_t)d_g | (uintptr_t)d_x | (uintptr_t)d_dx) % e ||
        ((uintptr_t)d_weight | (uintptr_t)d_dweight | (uintptr_t)d_dbias) % ew ||
        ((uintptr_t)d_mean | (uintptr_t)d_rstd) % 4)
        return fail(SG_ERR_INVALID_ARG, "sg_layernorm_bwd: an array is not aligned to its elements");
    if ((d_dx == d_g && ld_dx != ld_g) || (d_dx == d_x && ld_dx != ld))
        return fail(SG_ERR_INVALID_ARG, "sg_layernorm_bwd: in place needs equal row strides");
    cudaStream_t s = (cudaStream_t)stream;
    const int unit =
        unit_of(dim, (uintptr_t)d_g | (uintptr_t)d_x | (uintptr_t)d_dx | (uintptr_t)((ld | ld_g | ld_dx) * e),
                (uintptr_t)d_weight, e, ew);
    float* parts = d_dweight || d_dbias ? (float*)d_workspace : nullptr;
    if (dtype == SG_F32) {
        const BwdArgs<float> a = {(const float*)d_g, (const float*)d_x, (float*)d_dx, ld_g, ld, ld_dx, d_weight, d_mean,
                                  d_rstd, d_n, n_cap, dim, dtype_w == SG_BF16, parts};
        return bwd<float>(a, unit, d_dweight, d_dbias, s);
    }
    const BwdArgs<__nv_bfloat16> a = {(const __nv_bfloat16*)d_g, (const __nv_bfloat16*)d_x, (__nv_bfloat16*)d_dx, ld_g, ld,
                                      ld_dx, d_weight, d_mean, d_rstd, d_n, n_cap, dim, dtype_w == SG_BF16, parts};
    return bwd<__nv_bfloat16>(a, unit, d_dweight, d_dbias, s);
}
