// Softmax cross-entropy of rows of logits with its gradient:
//   loss[r] = log(z) + (m - x[r, label]),  m = max_c x[r, c],  z = sum_c exp(x[r, c] - m)
//   grad[r, c] = w (exp(x[r, c] - m) / z - (c == label))
// Bound by memory: the logits are read and the gradient is written once.
#include <cuda_bf16.h>

#include "sg_internal.cuh"

SGI_ERROR_WORD(loss)

using namespace sgi;

namespace {

constexpr int kThreads = 256;
constexpr int kTotalThreads = 1024;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ int32_t rows_of(const int32_t* d_n, int32_t n_cap) {
    return d_n ? min(max(*d_n, 0), n_cap) : n_cap;
}

// (m, z) of two parts of a row; a part without a finite logit is (-inf, 0)
__device__ __forceinline__ void join(float& m, float& z, float m2, float z2) {
    const float top = fmaxf(m, m2);
    if (top == -INFINITY) {
        z += z2;  // 0, or NaN
        return;
    }
    z = z * __expf(m - top) + z2 * __expf(m2 - top);
    m = top;
}

// Rows whose label is not -1, into *valid (one block).
__global__ void __launch_bounds__(kTotalThreads) k_xent_count(const int32_t* __restrict__ labels, int32_t n_cap,
                                                              const int32_t* __restrict__ d_n,
                                                              int32_t* __restrict__ valid) {
    pdl_start();
    __shared__ int32_t sh[kTotalThreads / 32 + 1];
    const int32_t n = rows_of(d_n, n_cap);
    int32_t v = 0;
    for (int32_t i = threadIdx.x; i < n; i += kTotalThreads) v += labels[i] != -1;
    v = block_sum<kTotalThreads, int32_t>(v, sh);
    if (threadIdx.x == 0) *valid = v;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_xent_row(const T* x, int32_t n_cap,
                                                       const int32_t* __restrict__ d_n, int32_t classes, int64_t ld,
                                                       const int32_t* __restrict__ labels, int32_t mean, float gs,
                                                       const int32_t* __restrict__ valid, float* __restrict__ loss,
                                                       T* grad, int64_t ld_grad) {
    pdl_start();
    __shared__ float sm[kThreads / 32], sz[kThreads / 32];
    const int32_t r = (int32_t)blockIdx.x;
    if (r >= rows_of(d_n, n_cap)) return;
    const T* row = x + (int64_t)r * ld;
    const int32_t y = labels[r];
    const bool ignored = y < 0 || y >= classes;
    if (ignored && y != -1 && threadIdx.x == 0) dev_err(ERR_INDEX);
    if (ignored) {
        if (threadIdx.x == 0) loss[r] = 0.f;
        if (grad)
            for (int32_t c = threadIdx.x; c < classes; c += kThreads) put(grad + (int64_t)r * ld_grad + c, 0.f);
        return;
    }
    const float xy = to_f(row[y]);
    float m = -INFINITY, z = 0.f;
    for (int32_t c = threadIdx.x; c < classes; c += kThreads) {
        const float v = to_f(row[c]);
        if (v != -INFINITY) join(m, z, v, v != v ? v : 1.f);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const float m2 = __shfl_xor_sync(0xFFFFFFFFu, m, d), z2 = __shfl_xor_sync(0xFFFFFFFFu, z, d);
        join(m, z, m2, z2);
    }
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = m, sz[threadIdx.x >> 5] = z;
    __syncthreads();
    m = sm[0], z = sz[0];
    for (int w = 1; w < kThreads / 32; ++w) join(m, z, sm[w], sz[w]);
    if (threadIdx.x == 0) loss[r] = xy == -INFINITY && z == z ? INFINITY : __logf(z) + (m - xy);
    if (!grad) return;
    const float w = mean ? gs / (float)max(1, *valid) : gs;
    for (int32_t c = threadIdx.x; c < classes; c += kThreads) {
        const float v = to_f(row[c]);
        const float p = v == -INFINITY ? 0.f : __expf(v - m) / z;
        const bool none = m == -INFINITY && z == 0.f;
        put(grad + (int64_t)r * ld_grad + c, none ? 0.f : fmaf(w, p, c == y ? -w : 0.f));
    }
}

// total = {sum of the losses in a fixed order (divided by the count with mean), count}
__global__ void __launch_bounds__(kTotalThreads) k_xent_total(const float* __restrict__ loss, int32_t n_cap,
                                                              const int32_t* __restrict__ d_n, int32_t mean,
                                                              const int32_t* __restrict__ valid,
                                                              float* __restrict__ total) {
    pdl_start();
    __shared__ float sh[kTotalThreads / 32 + 1];
    const int32_t n = rows_of(d_n, n_cap);
    float s = 0.f;
    for (int32_t i = threadIdx.x; i < n; i += kTotalThreads) s += loss[i];
    s = warp_sum(s);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x < 32) {
        s = warp_sum(sh[threadIdx.x]);
        if (threadIdx.x == 0) {
            total[0] = mean ? s / (float)max(1, *valid) : s;
            total[1] = (float)*valid;
        }
    }
}

template <typename T>
sg_status run(const T* x, int32_t n_cap, const int32_t* d_n, int32_t classes, int64_t ld, const int32_t* labels,
              int32_t mean, float gs, float* loss, float* total, T* grad, int64_t ld_grad, void* ws, cudaStream_t s) {
    int32_t* valid = (int32_t*)ws;
    SG_CUDA(launch_pdl(k_xent_count, dim3(1), dim3(kTotalThreads), 0, s, labels, n_cap, d_n, valid));
    if (n_cap > 0)
        SG_CUDA(launch_pdl(k_xent_row<T>, dim3((unsigned)n_cap), dim3(kThreads), 0, s, x, n_cap, d_n, classes, ld,
                           labels, mean, gs, (const int32_t*)valid, loss, grad, ld_grad));
    if (total)
        SG_CUDA(launch_pdl(k_xent_total, dim3(1), dim3(kTotalThreads), 0, s, (const float*)loss, n_cap, d_n, mean,
                           (const int32_t*)valid, total));
    return SG_OK;
}

size_t ws_bytes() { return 256; }

}  // namespace

extern "C" size_t sg_xent_workspace(int32_t n_cap, int32_t n_classes) {
    if (n_cap < 0 || n_classes <= 0) return 0;
    return ws_bytes();
}

extern "C" sg_status sg_xent(const void* d_logits, int32_t dtype, int32_t n_cap, const int32_t* d_n, int32_t n_classes,
                             int64_t ld, const int32_t* d_labels, int32_t mean, float grad_scale, float* d_loss,
                             float* d_total, void* d_grad, int64_t ld_grad, void* d_workspace, size_t workspace_bytes,
                             sg_stream_t stream) {
    if (dtype != SG_F32 && dtype != SG_BF16) return fail(SG_ERR_UNSUPPORTED, "sg_xent: dtype");
    if (n_cap < 0 || n_classes <= 0) return fail(SG_ERR_INVALID_ARG, "sg_xent: bad sizes");
    if (ld < n_classes || (d_grad && ld_grad < n_classes))
        return fail(SG_ERR_INVALID_ARG, "sg_xent: a row stride is below n_classes");
    if (n_cap > 0 && (!d_logits || !d_labels || !d_loss)) return fail(SG_ERR_INVALID_ARG, "sg_xent: NULL array");
    if (!d_workspace || (uintptr_t)d_workspace % 256 || workspace_bytes < ws_bytes())
        return fail(SG_ERR_INVALID_ARG, "sg_xent: workspace needs %zu bytes, 256-byte aligned", ws_bytes());
    const int e = dtype == SG_F32 ? 4 : 2;
    if ((uintptr_t)d_logits % e || (uintptr_t)d_grad % e || ((uintptr_t)d_labels | (uintptr_t)d_loss | (uintptr_t)d_total) % 4)
        return fail(SG_ERR_INVALID_ARG, "sg_xent: an array is not aligned to its elements");
    if (d_grad == d_logits && d_grad && ld_grad != ld)
        return fail(SG_ERR_INVALID_ARG, "sg_xent: in place needs ld_grad = ld");
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == SG_F32)
        return run<float>((const float*)d_logits, n_cap, d_n, n_classes, ld, d_labels, mean, grad_scale, d_loss, d_total,
                          (float*)d_grad, ld_grad, d_workspace, s);
    return run<__nv_bfloat16>((const __nv_bfloat16*)d_logits, n_cap, d_n, n_classes, ld, d_labels, mean, grad_scale,
                              d_loss, d_total, (__nv_bfloat16*)d_grad, ld_grad, d_workspace, s);
}
