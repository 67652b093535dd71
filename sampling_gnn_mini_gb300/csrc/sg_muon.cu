// Orthogonalised updates (the Muon optimiser's step) by Newton-Schulz products:
//   X = U / (||U||_F + eps), on the smaller side (transposed when rows > cols)
//   steps times:  A = X X^T;  B = a I + b A + c A A;  X <- B X
// with U the matrix itself (sg_orthogonalise) or the momentum update of
// sg_muon_step, and the weights updated from the result.
//
// Here m = min(rows, cols), n = max(rows, cols); X is held as m rows of n.
#include <cuda_bf16.h>
#include <string.h>

#include "sg_internal.cuh"

SGI_ERROR_WORD(muon)

using namespace sgi;

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 32;
constexpr int kNormBlocks = 64;  // partial sums of squares of a matrix

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// What enters: a matrix of type T (momentum NULL), or gradient and momentum.
template <typename T>
struct Source {
    const T* g;
    int64_t ld;
    const float* mom;
    float* mom_out;
    float mu;
    int32_t nesterov;
};

// U into X (transposed when tall) and partial sums of its squares.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_ns_load(Source<T> src, int32_t rows, int32_t cols, float* __restrict__ X,
                                                      double* __restrict__ part) {
    pdl_start();
    __shared__ double sh[kThreads / 32];
    const int64_t q = blockIdx.y, total = (int64_t)rows * cols;
    double sum = 0.0;
    for (int64_t t = blockIdx.x * (int64_t)kThreads + threadIdx.x; t < total; t += (int64_t)gridDim.x * kThreads) {
        const int64_t r = t / cols, c = t - r * cols;
        float u = to_f(src.g[(q * rows + r) * src.ld + c]);
        if (src.mom) {
            const float m = src.mu * src.mom[q * total + t] + u;
            src.mom_out[q * total + t] = m;
            u = src.nesterov ? u + src.mu * m : m;
        }
        X[q * total + (rows > cols ? c * rows + r : t)] = u;
        sum += (double)(u * u);
    }
    sum = warp_sum(sum);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kThreads / 32; ++w) sum += sh[w];
        part[q * gridDim.x + blockIdx.x] = sum;
    }
}

__global__ void __launch_bounds__(kThreads) k_ns_scale(float* __restrict__ X, int64_t total, const double* __restrict__ part,
                                                       int32_t parts, float eps) {
    pdl_start();
    const int64_t q = blockIdx.y;
    double s = 0.0;
    for (int i = 0; i < parts; ++i) s += part[q * parts + i];
    const float inv = 1.f / ((float)sqrt(s) + eps);
    for (int64_t t = blockIdx.x * (int64_t)kThreads + threadIdx.x; t < total; t += (int64_t)gridDim.x * kThreads)
        X[q * total + t] *= inv;
}

// D[i, j] = alpha * sum_k A[i, k] B(k, j) + beta * C[i, j] + gamma (i == j)
// with B(k, j) = B[j, k] (TB) or B[k, j]; row-major, one 32 x 32 tile a block.
template <bool TB>
__global__ void __launch_bounds__(kThreads) k_ns_mm(const float* __restrict__ A, const float* __restrict__ B,
                                                    const float* __restrict__ C, float* __restrict__ D, int32_t M,
                                                    int32_t N, int32_t K, float alpha, float beta, float gamma) {
    pdl_start();
    __shared__ float sa[kTile][kTile + 1], sb[kTile][kTile + 1];
    const int64_t q = blockIdx.z;
    A += q * (int64_t)M * K;
    B += q * (int64_t)N * K;
    D += q * (int64_t)M * N;
    if (C) C += q * (int64_t)M * N;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int32_t i0 = (int32_t)blockIdx.y * kTile, j0 = (int32_t)blockIdx.x * kTile;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int32_t k0 = 0; k0 < K; k0 += kTile) {
        for (int r = ty; r < kTile; r += 8) {
            sa[r][tx] = i0 + r < M && k0 + tx < K ? A[(int64_t)(i0 + r) * K + k0 + tx] : 0.f;
            if (TB) sb[r][tx] = j0 + r < N && k0 + tx < K ? B[(int64_t)(j0 + r) * K + k0 + tx] : 0.f;
            else sb[tx][r] = k0 + r < K && j0 + tx < N ? B[(int64_t)(k0 + r) * N + j0 + tx] : 0.f;
        }
        __syncthreads();
        for (int k = 0; k < kTile; ++k)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[r] += sa[ty + 8 * r][k] * sb[tx][k];
        __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int32_t i = i0 + ty + 8 * r, j = j0 + tx;
        if (i < M && j < N)
            D[(int64_t)i * N + j] = alpha * acc[r] + (C ? beta * C[(int64_t)i * N + j] : 0.f) + (i == j ? gamma : 0.f);
    }
}

// out = keep * w + step * X, transposed back (w NULL: out = step * X)
template <typename T>
__global__ void __launch_bounds__(kThreads) k_ns_store(const float* __restrict__ X, int32_t rows, int32_t cols,
                                                       const T* w, float keep, float step, T* out, int64_t ld_out) {
    pdl_start();
    const int64_t q = blockIdx.y, total = (int64_t)rows * cols;
    for (int64_t t = blockIdx.x * (int64_t)kThreads + threadIdx.x; t < total; t += (int64_t)gridDim.x * kThreads) {
        const int64_t r = t / cols, c = t - r * cols;
        const float x = step * X[q * total + (rows > cols ? c * rows + r : t)];
        const int64_t o = (q * rows + r) * ld_out + c;
        put(out + o, w ? keep * to_f(w[o]) + x : x);
    }
}

size_t a256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Layout {
    size_t x0, x1, a, b, part, total;
};

Layout layout(int64_t count, int64_t rows, int64_t cols) {
    const int64_t m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
    Layout L;
    size_t o = 0;
    const auto place = [&o](size_t bytes) {
        const size_t at = o;
        o += a256(bytes);
        return at;
    };
    L.x0 = place((size_t)(count * m * n) * 4);
    L.x1 = place((size_t)(count * m * n) * 4);
    L.a = place((size_t)(count * m * m) * 4);
    L.b = place((size_t)(count * m * m) * 4);
    L.part = place((size_t)(count * kNormBlocks) * 8);
    L.total = o;
    return L;
}

const float kCoef[3] = {3.4445f, -4.7750f, 2.0315f};

template <typename TS, typename TW>
sg_status run(Source<TS> src, int32_t count, int32_t rows, int32_t cols, int32_t steps, const float* coef, float eps,
              const TW* w, float keep, float step, TW* out, int64_t ld_out, char* ws, cudaStream_t s) {
    const Layout L = layout(count, rows, cols);
    const int32_t m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
    float* x = (float*)(ws + L.x0);
    float* x2 = (float*)(ws + L.x1);
    float* a = (float*)(ws + L.a);
    float* b = (float*)(ws + L.b);
    double* part = (double*)(ws + L.part);
    const int64_t total = (int64_t)rows * cols;
    const int64_t eb = cdiv(total, kThreads) < 1024 ? cdiv(total, kThreads) : 1024;
    const dim3 flat((unsigned)eb, (unsigned)count);
    SG_CUDA(launch_pdl(k_ns_load<TS>, dim3(kNormBlocks, (unsigned)count), dim3(kThreads), 0, s, src, rows, cols, x,
                       part));
    SG_CUDA(launch_pdl(k_ns_scale, flat, dim3(kThreads), 0, s, x, total, (const double*)part, (int32_t)kNormBlocks,
                       eps));
    const unsigned tm = (unsigned)cdiv(m, kTile), tn = (unsigned)cdiv(n, kTile);
    for (int32_t k = 0; k < steps; ++k) {
        const float* c = coef ? coef + 3 * k : kCoef;
        SG_CUDA(launch_pdl(k_ns_mm<true>, dim3(tm, tm, (unsigned)count), dim3(kThreads), 0, s, (const float*)x,
                           (const float*)x, (const float*)nullptr, a, m, m, n, 1.f, 0.f, 0.f));
        SG_CUDA(launch_pdl(k_ns_mm<true>, dim3(tm, tm, (unsigned)count), dim3(kThreads), 0, s, (const float*)a,
                           (const float*)a, (const float*)a, b, m, m, m, c[2], c[1], c[0]));
        SG_CUDA(launch_pdl(k_ns_mm<false>, dim3(tn, tm, (unsigned)count), dim3(kThreads), 0, s, (const float*)b,
                           (const float*)x, (const float*)nullptr, x2, m, n, m, 1.f, 0.f, 0.f));
        float* t = x;
        x = x2;
        x2 = t;
    }
    SG_CUDA(launch_pdl(k_ns_store<TW>, flat, dim3(kThreads), 0, s, (const float*)x, rows, cols, w, keep, step, out,
                       ld_out));
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
    if (dtype == SG_F32) {
        const Source<float> src = {(const float*)d_g, ld, nullptr, nullptr, 0.f, 0};
        return run<float, float>(src, count, rows, cols, steps, h_coef, eps, nullptr, 0.f, scale, (float*)d_out, ld_out,
                                 (char*)d_workspace, s);
    }
    const Source<__nv_bfloat16> src = {(const __nv_bfloat16*)d_g, ld, nullptr, nullptr, 0.f, 0};
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
    const Source<float> src = {d_g, cols, d_m, d_m_out, momentum, nesterov};
    const float keep = 1.f - rate * weight_decay, step = -rate * scale;
    if (dtype_w == SG_F32)
        return run<float, float>(src, count, rows, cols, steps, h_coef, eps, (const float*)d_w, keep, step,
                                 (float*)d_w_out, cols, (char*)d_workspace, s);
    return run<float, __nv_bfloat16>(src, count, rows, cols, steps, h_coef, eps, (const __nv_bfloat16*)d_w, keep, step,
                                     (__nv_bfloat16*)d_w_out, cols, (char*)d_workspace, s);
}
