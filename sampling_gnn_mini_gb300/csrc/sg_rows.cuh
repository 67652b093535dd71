// Rows of fp32 or bf16 values as the row kernels read and write them: 16-byte
// parts at any alignment, exponentials relative to a row's maximum, launches of
// clusters.
#pragma once

#include <cuda_bf16.h>

#include "sg_internal.cuh"

namespace sgi {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ int32_t rows_of(const int32_t* d_n, int32_t n_cap) {
    return d_n ? min(max(*d_n, 0), n_cap) : n_cap;
}

// 2^x; the hardware's approximation is within 2^-22 of the value, results
// below the normal range are 0
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// exp(x - m), m finite; with l = log2(e) / T, exp((x - m) / T)
__device__ __forceinline__ float exp_from(float x, float m, float l = kLog2e) { return ex2((x - m) * l); }

__device__ __forceinline__ float warp_max(float x) {
    float m;  // (without NaN, as fmaxf)
    asm volatile("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(m) : "f"(x));
    return m;
}

// --------------------------------------------------- 16-byte parts of a row
template <typename T>
constexpr int kE = 16 / (int)sizeof(T);  // elements of a vector

// A row as its elements before the first 16-byte boundary (head), its whole
// vectors, and its elements after the last of them.  Whole vectors are dealt
// to threads; the up to 7 + 7 others go to lanes 0.. and 8.. of one warp.
template <typename T>
struct RowParts {
    int32_t head, vecs, tail;
    __device__ __forceinline__ RowParts(const T* row, int32_t classes) {
        const int32_t off = (int32_t)(((uintptr_t)row & 15) / sizeof(T));
        head = off ? min(classes, kE<T> - off) : 0;
        vecs = (classes - head) / kE<T>;
        tail = classes - head - vecs * kE<T>;
    }
    // element of edge lane l, or -1
    __device__ __forceinline__ int32_t edge(int l) const {
        if (l < 8) return l < head ? l : -1;
        return l - 8 < tail ? head + vecs * kE<T> + l - 8 : -1;
    }
    // where element c sits: vector >= 0, or -1 - (edge lane)
    __device__ __forceinline__ int32_t place(int32_t c) const {
        if (c < head) return -1 - c;
        const int32_t v = (c - head) / kE<T>;
        return v < vecs ? v : -1 - (8 + c - head - vecs * kE<T>);
    }
};

template <typename T>
__device__ __forceinline__ bool same_phase(const T* a, const T* b) {
    return (((uintptr_t)a ^ (uintptr_t)b) & 15) == 0;
}

template <typename T>
__device__ __forceinline__ uint4 empty_part() {
    const uint32_t w = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;  // -inf
    return make_uint4(w, w, w, w);
}

__device__ __forceinline__ void pairs_of(const uint4& u, f2 (&p)[2]) {
    p[0] = pair(__uint_as_float(u.x), __uint_as_float(u.y));
    p[1] = pair(__uint_as_float(u.z), __uint_as_float(u.w));
}
__device__ __forceinline__ void pairs_of(const uint4& u, f2 (&p)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ uint4 part_of(const f2 (&p)[2]) {
    float a, b, c, d;
    unpair(p[0], a, b);
    unpair(p[1], c, d);
    return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
}
__device__ __forceinline__ uint4 part_of(const f2 (&p)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        unpair(p[i], a, b);
        const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
        w[i] = *reinterpret_cast<const uint32_t*>(&t);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Keeps the compiler from carrying a vector's unpacked elements (twice its
// registers) from one use to the next: they are unpacked again instead.
__device__ __forceinline__ void repack(uint4& u) {
    asm volatile("" : "+r"(u.x), "+r"(u.y), "+r"(u.z), "+r"(u.w));
}

template <typename T>
__device__ __forceinline__ float part_max(const uint4& u) {
    if constexpr (sizeof(T) == 2) {  // pairwise on the packed elements
        const auto h = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
        const __nv_bfloat162 m = __hmax2(__hmax2(h(u.x), h(u.y)), __hmax2(h(u.z), h(u.w)));
        return fmaxf(__low2float(m), __high2float(m));
    }
    return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
}

// Stores a vector at p; whole: p is on a 16-byte boundary.
template <typename T>
__device__ __forceinline__ void store_part(T* p, bool whole, const uint4& u) {
    if (whole) {
        *reinterpret_cast<uint4*>(p) = u;
        return;
    }
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int q = 0; q < kE<T>; ++q) p[q] = e[q];
}

// ------------------------------------------- a thread's own copies, ahead of use
// 16 bytes from global into shared memory (both addresses the address of a uint4 there).
__device__ __forceinline__ void copy_async(const uint4* to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from)
                 : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
// Waits for all groups of copies but the last N.
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

// Sum of n fp32 values in a fixed order, by one block of NT threads (in thread 0):
// 16 bytes and 8 loads a thread at a time (65,536 values one by one took 35 us).
template <int NT>
__device__ __forceinline__ float block_sum_fixed(const float* x, int32_t n) {
    __shared__ float sh[NT / 32];
    // a value or so before the first 16-byte boundary, whole vectors, the rest
    const int32_t head = min(n, (int32_t)((4 - ((uintptr_t)x >> 2 & 3)) & 3)), vecs = (n - head) / 4;
    const float4* v = reinterpret_cast<const float4*>(x + head);
    float s = 0.f;
    for (int32_t i0 = threadIdx.x; i0 < vecs; i0 += 8 * NT) {
        float4 y[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) y[u] = i0 + u * NT < vecs ? __ldcg(v + i0 + u * NT) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int u = 0; u < 8; ++u) s += (y[u].x + y[u].y) + (y[u].z + y[u].w);
    }
    const int32_t rest = n - 4 * vecs, i = (int32_t)threadIdx.x;  // head and tail together
    if (i < rest) s += __ldcg(x + (i < head ? i : i + 4 * vecs));
    s = warp_sum(s);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int w = 1; w < NT / 32; ++w) s += sh[w];
    return s;
}

// -------------------------------------------------------------------- host
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), unsigned grid, unsigned threads, unsigned cluster, cudaStream_t s,
                           int smem, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

}  // namespace sgi
