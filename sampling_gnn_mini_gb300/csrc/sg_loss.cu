// Softmax cross-entropy of rows of logits with its gradient:
//   loss[r] = log(z) + (m - x[r, label]),  m = max_c x[r, c],  z = sum_c exp(x[r, c] - m)
//   grad[r, c] = w (exp(x[r, c] - m) / z - (c == label))
// Bound by memory: the logits are read and the gradient is written once, so a
// row has to stay on the chip between the two.  It stays in registers, as the
// 16-byte vectors it was read in (up to kVecs a thread), spread over
//   a warp              rows of up to 32 kVecs vectors (k_xent_warp)
//   a cluster of CTAs   longer rows (k_xent_row): 1 to 8 CTAs of 256 or 512 threads
// Each warp reduces its part of the row to (m, z) relative to its own
// maximum; the parts meet once, in shared memory (of every CTA of the
// cluster), and a warp scales its exponentials by exp(m_warp - m) w / z, so a
// row costs one barrier.  Vectors past the registers' reach (rows above 65,536
// fp32 or 131,072 bf16 logits, or one vector of a misaligned row) are read
// again for the gradient, from L2.
//
// The mean needs the number of labelled rows before the first gradient:
// k_xent_count finds it, and the last block to finish sums the losses in
// a fixed order.  A small call does all of it in one cluster (k_xent_small).
//
// -inf logits: m and x - m are kept apart from -inf - -inf by taking m = 0 when
// a part has no finite logit (its exponentials are then 0); x - m is formed
// before the scaling by log2(e), so rows at a type's lowest value do not
// overflow.
#include <cuda_bf16.h>

#include "sg_internal.cuh"
#include "sg_tc.cuh"

SGI_ERROR_WORD(loss)

using namespace sgi;

namespace {

constexpr int kThreads = 256;
constexpr int kTotalThreads = 1024;
constexpr int kVecs = 8;              // 16-byte vectors of a row a thread holds
constexpr int kSmallCtas = 8;         // the one cluster of a small call
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ int32_t rows_of(const int32_t* d_n, int32_t n_cap) {
    return d_n ? min(max(*d_n, 0), n_cap) : n_cap;
}

// 2^x; the hardware's approximation is within 2^-22 of the value
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// exp(x - m), m finite
__device__ __forceinline__ float exp_from(float x, float m) { return ex2((x - m) * kLog2e); }

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, d));
    return x;
}

// --------------------------------------------------- 16-byte parts of a row
template <typename T>
constexpr int kE = 16 / (int)sizeof(T);  // elements of a vector

__device__ __forceinline__ void unpack(const uint4& u, float (&v)[4]) {
    v[0] = __uint_as_float(u.x), v[1] = __uint_as_float(u.y), v[2] = __uint_as_float(u.z), v[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void unpack(const uint4& u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint4 pack(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ uint4 pack(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&t);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Elements of the row before the 16-byte boundary at or below its start:
// vector v of the row holds elements v E - off .. v E - off + E - 1.
template <typename T>
__device__ __forceinline__ int32_t phase(const T* row) {
    return (int32_t)(((uintptr_t)row & 15) / sizeof(T));
}

// Vector at element e0; elements outside the row read as -inf.
template <typename T>
__device__ __forceinline__ uint4 load_part(const T* row, int32_t e0, int32_t classes) {
    if (e0 >= 0 && e0 + kE<T> <= classes) return *reinterpret_cast<const uint4*>(row + e0);
    float v[kE<T>];
#pragma unroll
    for (int q = 0; q < kE<T>; ++q) v[q] = e0 + q >= 0 && e0 + q < classes ? to_f(row[e0 + q]) : -INFINITY;
    return pack(v);
}

template <typename T>
__device__ __forceinline__ uint4 empty_part() {
    float v[kE<T>];
#pragma unroll
    for (int q = 0; q < kE<T>; ++q) v[q] = -INFINITY;
    return pack(v);
}

// Stores the vector at element e0; same: the gradient's row has the logits'
// 16-byte phase.
template <typename T>
__device__ __forceinline__ void store_part(T* row, int32_t e0, int32_t classes, bool same, const float (&v)[kE<T>]) {
    if (same && e0 >= 0 && e0 + kE<T> <= classes) {
        *reinterpret_cast<uint4*>(row + e0) = pack(v);
        return;
    }
#pragma unroll
    for (int q = 0; q < kE<T>; ++q)
        if (e0 + q >= 0 && e0 + q < classes) put(row + e0 + q, v[q]);
}

template <typename T>
__device__ __forceinline__ float part_max(const uint4& u) {
    float v[kE<T>];
    unpack(u, v);
    float m = v[0];
#pragma unroll
    for (int q = 1; q < kE<T>; ++q) m = fmaxf(m, v[q]);
    return m;
}

// Sum of exp(x - m); fp32 vectors keep the exponentials in place of x.
template <typename T>
__device__ __forceinline__ float part_exp(uint4& u, float m) {
    float v[kE<T>], s = 0.f;
    unpack(u, v);
#pragma unroll
    for (int q = 0; q < kE<T>; ++q) {
        v[q] = exp_from(v[q], m);
        s += v[q];
    }
    if constexpr (sizeof(T) == 4) u = pack(v);
    return s;
}

// The gradient (without its -w at the label) of a vector that part_exp saw.
template <typename T>
__device__ __forceinline__ void part_grad(const uint4& u, float m, float inv, float (&v)[kE<T>]) {
    unpack(u, v);
#pragma unroll
    for (int q = 0; q < kE<T>; ++q) v[q] = inv * (sizeof(T) == 4 ? v[q] : exp_from(v[q], m));
}

__device__ __forceinline__ float loss_of(float m, float z, float xy) {
    return xy == -INFINITY && z == z ? INFINITY : __logf(z) + (m - xy);
}

template <typename T>
struct RowArgs {
    const T* x;  // may be grad
    T* grad;
    int64_t ld, ld_grad;
    const int32_t* labels;
    const int32_t* d_n;
    int32_t n_cap, classes;
    int32_t mean;
    float gs;
    float* loss;
    float* total;
    int32_t* valid;  // [0] labelled rows, [1] rows or blocks that are done
};

// ------------------------------------------------------------ rows by warps
// R rows (r0, r0 + 1, ..) at once, each in NV vectors a lane; returns their
// losses (the same in every lane; 0 for rows past n).
template <typename T, int NV, int R>
__device__ __forceinline__ void warp_rows(const RowArgs<T>& a, int32_t r0, int32_t n, float w, float (&loss)[R]) {
    const int lane = (int)lane_id();
    uint4 x[R][NV];
    int32_t off[R], y[R];
    float xy[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        y[r] = r0 + r < n ? __ldg(a.labels + r0 + r) : -1;
        if (y[r] < -1 || y[r] >= a.classes) {
            if (lane == 0) dev_err(ERR_INDEX);
            y[r] = -1;
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const T* row = a.x + (int64_t)(r0 + r) * a.ld;
        off[r] = phase(row);
        xy[r] = 0.f;
        if (y[r] >= 0) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
                x[r][k] = load_part(row, (lane + 32 * k) * kE<T> - off[r], a.classes);
            if (((y[r] + off[r]) / kE<T>) % 32 == lane) xy[r] = to_f(row[y[r]]);
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        loss[r] = 0.f;
        if (r0 + r >= n) continue;  // the same in every lane
        T* out = a.grad ? a.grad + (int64_t)(r0 + r) * a.ld_grad : nullptr;
        if (y[r] < 0) {
            if (lane == 0) a.loss[r0 + r] = 0.f;
            if (out)
                for (int32_t c = lane; c < a.classes; c += 32) put(out + c, 0.f);
            continue;
        }
        float m = part_max<T>(x[r][0]);
#pragma unroll
        for (int k = 1; k < NV; ++k) m = fmaxf(m, part_max<T>(x[r][k]));
        m = warp_max(m);
        if (m == -INFINITY) m = 0.f;
        float z = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) z += part_exp<T>(x[r][k], m);
        z = warp_sum(z);
        const int owner = ((y[r] + off[r]) / kE<T>) % 32;
        const float at = __shfl_sync(0xFFFFFFFFu, xy[r], owner);
        loss[r] = loss_of(m, z, at);
        if (lane == owner) a.loss[r0 + r] = loss[r];
        if (!out) continue;
        const float inv = z == 0.f ? 0.f : w / z;
        const bool same = phase(out) == off[r];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float v[kE<T>];
            part_grad<T>(x[r][k], m, inv, v);
            store_part(out, (lane + 32 * k) * kE<T> - off[r], a.classes, same, v);
        }
        // this lane stored the label's element above: it may now replace it
        if (lane == owner) put(out + y[r], z == 0.f ? 0.f : fmaf(inv, exp_from(at, m), -w));
    }
}

// Sum of the losses in a fixed order, by the last block to finish.
template <int NT, typename T>
__device__ __forceinline__ void put_total(const RowArgs<T>& a, int32_t n) {
    __shared__ float sh[NT / 32];
    float s = 0.f;
    for (int32_t i = threadIdx.x; i < n; i += NT) s += __ldcg(a.loss + i);
    s = warp_sum(s);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < NT / 32; ++w) s += sh[w];
        a.total[0] = a.mean ? s / (float)max(1, *a.valid) : s;
    }
}

template <typename T, int NV, int R>
__global__ void __launch_bounds__(kThreads) k_xent_warp(RowArgs<T> a) {
    pdl_start();
    __shared__ bool last;
    constexpr int kRows = kThreads / 32 * R;  // rows of a block
    const int32_t n = rows_of(a.d_n, a.n_cap);
    const int64_t b0 = (int64_t)blockIdx.x * kRows;
    if (b0 >= n) return;
    const float w = a.mean ? a.gs / (float)max(1, *a.valid) : a.gs;
    float loss[R];
    warp_rows<T, NV, R>(a, (int32_t)b0 + (int)(threadIdx.x >> 5) * R, n, w, loss);
    if (!a.total) return;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(a.valid + 1, 1) == (n + kRows - 1) / kRows - 1;
    __syncthreads();
    if (last) put_total<kThreads>(a, n);
}

// The whole of a small call in one cluster: each CTA counts the labels, the
// cluster's warps take the rows in turn, the warps' sums meet in CTA 0.
template <typename T, int NV, int R>
__global__ void __launch_bounds__(kThreads) k_xent_small(RowArgs<T> a) {
    pdl_start();
    __shared__ int32_t sh[kThreads / 32 + 1];
    __shared__ float part[kThreads / 32];
    constexpr int kWarps = kThreads / 32;
    const int warp = (int)(threadIdx.x >> 5);
    const int32_t n = rows_of(a.d_n, a.n_cap);
    int32_t v = 0;
    for (int32_t i = threadIdx.x; i < n; i += kThreads) v += __ldg(a.labels + i) != -1;
    v = block_sum<kThreads, int32_t>(v, sh);
    const float w = a.mean ? a.gs / (float)max(1, v) : a.gs;
    float sum = 0.f;
    for (int32_t r0 = ((int32_t)blockIdx.x * kWarps + warp) * R; r0 < n; r0 += kSmallCtas * kWarps * R) {
        float loss[R];
        warp_rows<T, NV, R>(a, r0, n, w, loss);
#pragma unroll
        for (int r = 0; r < R; ++r) sum += loss[r];
    }
    if ((threadIdx.x & 31) == 0) part[warp] = sum;
    cluster_sync();
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.total) {
        float s = 0.f;
        for (int c = 0; c < kSmallCtas; ++c)
            for (int i = 0; i < kWarps; ++i) s += ld_cluster(map_rank(smem_addr(part + i), (uint32_t)c));
        a.total[0] = a.mean ? s / (float)max(1, v) : s;
        a.total[1] = (float)v;
    }
    cluster_sync();  // the parts stay until they are read
}

// --------------------------------------------------------- rows by clusters
template <typename T, int NT, int S>
__global__ void __launch_bounds__(NT, 1024 / NT) k_xent_row(RowArgs<T> a) {
    pdl_start();
    constexpr int kWarps = NT / 32, kParts = S * kWarps;
    __shared__ float pm[kParts], pz[kParts];  // (m, z) of every warp of the cluster
    __shared__ bool last;
    const int warp = (int)(threadIdx.x >> 5), lane = (int)lane_id();
    const int32_t r = (int32_t)(blockIdx.x / S), rank = (int32_t)(blockIdx.x % S);
    const int32_t n = rows_of(a.d_n, a.n_cap);
    if (r >= n) return;  // the whole cluster
    if constexpr (S > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");
    if (threadIdx.x == 0) last = false;
    const T* row = a.x + (int64_t)r * a.ld;
    T* out = a.grad ? a.grad + (int64_t)r * a.ld_grad : nullptr;
    const int32_t off = phase(row), classes = a.classes;
    const bool same = out && phase(out) == off;
    const int32_t nv = (classes + off + kE<T> - 1) / kE<T>, per = (nv + S - 1) / S;
    const int32_t v0 = rank * per, v1 = min(nv, v0 + per);
    int32_t y = __ldg(a.labels + r);
    if (y < -1 || y >= classes) {
        if (rank == 0 && threadIdx.x == 0) dev_err(ERR_INDEX);
        y = -1;
    }
    const bool used = y >= 0;  // the same in the whole cluster
    const int32_t vy = used ? (y + off) / kE<T> : 0;
    const bool owner = vy >= v0 && vy < v0 + per && (vy - v0) % NT == (int32_t)threadIdx.x;
    uint4 x[kVecs];
    float m = -INFINITY, z = 0.f, xy = 0.f;
    if (used) {
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const int32_t v = v0 + (int32_t)threadIdx.x + k * NT;
            x[k] = v < v1 ? load_part(row, v * kE<T> - off, classes) : empty_part<T>();
        }
        if (owner) xy = to_f(row[y]);
#pragma unroll
        for (int k = 0; k < kVecs; ++k) m = fmaxf(m, part_max<T>(x[k]));
        float mr = -INFINITY, zr = 0.f;  // the part past the registers
        for (int32_t v = v0 + (int32_t)threadIdx.x + kVecs * NT; v < v1; v += NT) {
            uint4 u = load_part(row, v * kE<T> - off, classes);
            const float top = fmaxf(mr, part_max<T>(u)), base = top == -INFINITY ? 0.f : top;
            zr = zr * exp_from(mr, base) + part_exp<T>(u, base);
            mr = top;
        }
        m = warp_max(fmaxf(m, mr));
        if (m == -INFINITY) m = 0.f;
        if (zr != 0.f) z = zr * exp_from(mr == -INFINITY ? 0.f : mr, m);
#pragma unroll
        for (int k = 0; k < kVecs; ++k) z += part_exp<T>(x[k], m);
        z = warp_sum(z);
    }
    if constexpr (S > 1) {
        asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");  // every CTA runs: its shared memory may be written
        if (lane < S) {
            const uint32_t slot = (uint32_t)(rank * kWarps + warp) * 4;
            asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(map_rank(smem_addr(pm) + slot, (uint32_t)lane)), "f"(m)
                         : "memory");
            asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(map_rank(smem_addr(pz) + slot, (uint32_t)lane)), "f"(z)
                         : "memory");
        }
        cluster_sync();
    } else {
        if (lane == 0) pm[warp] = m, pz[warp] = z;
        __syncthreads();
    }
    if (used) {
        // the row's (M, Z): parts without a finite logit have m = 0, z = 0 and
        // are left out of the maximum
        float M = -INFINITY, Z = 0.f;
#pragma unroll
        for (int i = lane; i < kParts; i += 32)
            if (pz[i] != 0.f) M = fmaxf(M, pm[i]);
        M = warp_max(M);
        if (M == -INFINITY) M = 0.f;
#pragma unroll
        for (int i = lane; i < kParts; i += 32)
            if (pz[i] != 0.f) Z += pz[i] * exp_from(pm[i], M);
        Z = warp_sum(Z);
        const float w = a.mean ? a.gs / (float)max(1, *a.valid) : a.gs;
        if (out) {
            const float inv = z == 0.f || Z == 0.f ? 0.f : w / Z * exp_from(m, M);
#pragma unroll
            for (int k = 0; k < kVecs; ++k) {
                const int32_t v = v0 + (int32_t)threadIdx.x + k * NT;
                if (v >= v1) continue;
                float g[kE<T>];
                part_grad<T>(x[k], m, inv, g);
                store_part(out, v * kE<T> - off, classes, same, g);
            }
            for (int32_t v = v0 + (int32_t)threadIdx.x + kVecs * NT; v < v1; v += NT) {
                uint4 u = load_part(row, v * kE<T> - off, classes);
                float g[kE<T>];
                part_exp<T>(u, m);
                part_grad<T>(u, m, inv, g);
                store_part(out, v * kE<T> - off, classes, same, g);
            }
            // this thread stored the label's element above: it may now replace it
            if (owner) put(out + y, Z == 0.f ? 0.f : fmaf(w / Z, exp_from(xy, M), -w));
        }
        if (owner) a.loss[r] = loss_of(M, Z, xy);
    } else {
        if (owner) a.loss[r] = 0.f;
        if (out) {
            const float none[kE<T>] = {};
            for (int32_t v = v0 + (int32_t)threadIdx.x; v < v1; v += NT)
                store_part(out, v * kE<T> - off, classes, same, none);
        }
    }
    if (!a.total) return;
    if (owner) {
        __threadfence();
        if (atomicAdd(a.valid + 1, 1) == n - 1) last = true;
    }
    __syncthreads();
    if (last) {
        __threadfence();
        put_total<NT>(a, n);
    }
}

// Rows whose label is not -1 (one block); clears the count of finished blocks.
__global__ void __launch_bounds__(kTotalThreads) k_xent_count(const int32_t* __restrict__ labels, int32_t n_cap,
                                                              const int32_t* __restrict__ d_n,
                                                              int32_t* __restrict__ valid, float* __restrict__ total) {
    pdl_start();
    __shared__ int32_t sh[kTotalThreads / 32 + 1];
    const int32_t n = rows_of(d_n, n_cap);
    int32_t v = 0;
#pragma unroll 8
    for (int32_t i = threadIdx.x; i < n; i += kTotalThreads) v += labels[i] != -1;
    v = block_sum<kTotalThreads, int32_t>(v, sh);
    if (threadIdx.x == 0) {
        valid[0] = v;
        valid[1] = 0;
        if (total) total[0] = 0.f, total[1] = (float)v;
    }
}

// -------------------------------------------------------------------- host
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), unsigned grid, unsigned threads, unsigned cluster, cudaStream_t s,
                           Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
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

template <typename T, int NV, int R>
sg_status run_warp(const RowArgs<T>& a, bool small, cudaStream_t s) {
    if (small)
        SG_CUDA(launch_cluster(k_xent_small<T, NV, R>, kSmallCtas, kThreads, kSmallCtas, s, a));
    else
        SG_CUDA(launch_pdl(k_xent_warp<T, NV, R>, dim3((unsigned)cdiv(a.n_cap, kThreads / 32 * R)), dim3(kThreads), 0, s, a));
    return SG_OK;
}

template <typename T, int NT, int S>
sg_status run_row(const RowArgs<T>& a, cudaStream_t s) {
    SG_CUDA(launch_cluster(k_xent_row<T, NT, S>, (unsigned)((int64_t)a.n_cap * S), NT, S, s, a));
    return SG_OK;
}

template <typename T>
sg_status run(RowArgs<T> a, cudaStream_t s) {
    const int64_t nv = cdiv((int64_t)a.classes + kE<T> - 1, kE<T>);  // vectors of a row, at any phase
    const bool by_warp = nv <= 32 * kVecs;
    // one cluster serves a call whose vectors its warps hold in a few turns
    const bool small = by_warp && a.n_cap <= 1024 && a.n_cap * nv <= kSmallCtas * kThreads * kVecs;
    if (!small)
        SG_CUDA(launch_pdl(k_xent_count, dim3(1), dim3(kTotalThreads), 0, s, a.labels, a.n_cap, a.d_n, a.valid, a.total));
    if (a.n_cap == 0 && !small) return SG_OK;
    if (by_warp) {
        if (nv <= 32) return run_warp<T, 1, 4>(a, small, s);
        if (nv <= 64) return run_warp<T, 2, 2>(a, small, s);
        if (nv <= 128) return run_warp<T, 4, 2>(a, small, s);
        return run_warp<T, 8, 1>(a, small, s);
    }
    // smallest cluster whose registers hold the row, widened while the rows do
    // not fill the SMs; 512 threads when 8 CTAs of 256 do not hold it
    int split = 1;
    while (split < 8 && nv > (int64_t)split * kThreads * kVecs) split *= 2;
    if (nv > 8 * kThreads * kVecs) return run_row<T, 512, 8>(a, s);
    while (split < 8 && (int64_t)a.n_cap * split * 2 <= 2 * num_sms() && nv >= split * 2 * kThreads) split *= 2;
    switch (split) {
        case 1: return run_row<T, kThreads, 1>(a, s);
        case 2: return run_row<T, kThreads, 2>(a, s);
        case 4: return run_row<T, kThreads, 4>(a, s);
        default: return run_row<T, kThreads, 8>(a, s);
    }
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
    if ((int64_t)n_cap * 8 > 2147483647LL) return fail(SG_ERR_INVALID_ARG, "sg_xent: more than 2^28 rows");
    if (n_classes > 2147483647 - 64) return fail(SG_ERR_INVALID_ARG, "sg_xent: n_classes out of range");
    if (dtype == SG_F32) {
        const RowArgs<float> a = {(const float*)d_logits, (float*)d_grad, ld, ld_grad, d_labels, d_n, n_cap, n_classes,
                                  mean ? 1 : 0, grad_scale, d_loss, d_total, (int32_t*)d_workspace};
        return run(a, s);
    }
    const RowArgs<__nv_bfloat16> a = {(const __nv_bfloat16*)d_logits, (__nv_bfloat16*)d_grad, ld, ld_grad, d_labels, d_n,
                                      n_cap, n_classes, mean ? 1 : 0, grad_scale, d_loss, d_total, (int32_t*)d_workspace};
    return run(a, s);
}
