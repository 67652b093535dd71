// Softmax cross-entropy of rows of logits with its gradient:
//   loss[r] = log(z) + (m - x[r, label]),  m = max_c x[r, c],  z = sum_c exp(x[r, c] - m)
//   grad[r, c] = w (exp(x[r, c] - m) / z - (c == label))
// Bound by memory: the logits are read and the gradient is written once, so a
// row has to stay on the chip between the two.  It stays in registers, as the
// 16-byte vectors it was read in (up to kVecs a thread), spread over
//   a thread            rows of up to 16 classes (k_xent_thread)
//   a warp              rows of up to 32 kVecs vectors (k_xent_warp)
//   a cluster of CTAs   longer rows (k_xent_row): 1 to 8 CTAs of 256 or 512 threads
// Each warp reduces its part of the row to (m, z) relative to its own
// maximum; the parts meet once, in shared memory (of every CTA of the
// cluster), and a warp scales its exponentials by exp(m_warp - m) w / z, so a
// row costs one barrier.  Vectors past the registers' reach (rows above 131,072
// fp32 or 262,144 bf16 logits, or one vector of a misaligned row) are read
// again for the gradient, from L2.  Many long rows are streamed through shared
// memory instead, ahead of their use (k_xent_stream).
//
// The mean needs the number of labelled rows before the first gradient:
// k_xent_count finds it, and the last block to finish sums the losses in
// a fixed order.  A small call does all of it in one cluster (k_xent_small).
//
// -inf logits: m and x - m are kept apart from -inf - -inf by taking m = 0 when
// a part has no finite logit (its exponentials are then 0); x - m is formed
// before the scaling by log2(e), so rows at a type's lowest value do not
// overflow and a row's common level costs no accuracy.
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

// 2^x; the hardware's approximation is within 2^-22 of the value, results
// below the normal range are 0
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// exp(x - m), m finite
__device__ __forceinline__ float exp_from(float x, float m) { return ex2((x - m) * kLog2e); }

// (logf, once a row: z is just above 1 in a row that is sure of its label, and the
// fast logarithm is off by up to 2^-21 there, whatever the loss)
__device__ __forceinline__ float loss_of(float m, float z, float xy) {
    return xy == -INFINITY && z == z ? INFINITY : logf(z) + (m - xy);
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, d));
    return x;
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

// exp(x - m) of values and pairs, the difference taken first, as in exp_from():
// it is exact near m, so the largest logit's exponential is 1 whatever its level.
// (One fused operation, x log2(e) - m log2(e), leaves the rounding of the second
// product in every exponential: at |m| = 1e6 they are off by 1.5 %, at 1e10 by
// more than the type's range.)
struct Base {
    f2 l, b;
    float m;
    __device__ __forceinline__ explicit Base(float m_) : m(m_) {
        l = pair(kLog2e, kLog2e);
        b = pair(-m_, -m_);
    }
    __device__ __forceinline__ float of(float x) const { return exp_from(x, m); }
    __device__ __forceinline__ f2 of(f2 x) const {
        float a, c;
        unpair(mul2(add2(x, b), l), a, c);
        return pair(ex2(a), ex2(c));
    }
};

// Adds exp(x - m) to sum; fp32 vectors keep the exponentials in place of x.
template <typename T>
__device__ __forceinline__ void part_exp(uint4& u, const Base& m, f2& sum) {
    f2 p[kE<T> / 2];
    pairs_of(u, p);
#pragma unroll
    for (int i = 0; i < kE<T> / 2; ++i) {
        p[i] = m.of(p[i]);
        sum = add2(sum, p[i]);
    }
    if constexpr (sizeof(T) == 4) u = part_of(p);
}

// The gradient (without its -w at the label) of a vector that part_exp saw.
template <typename T>
__device__ __forceinline__ uint4 part_grad(const uint4& u, const Base& m, f2 inv) {
    f2 p[kE<T> / 2];
    pairs_of(u, p);
#pragma unroll
    for (int i = 0; i < kE<T> / 2; ++i) p[i] = mul2(inv, sizeof(T) == 4 ? p[i] : m.of(p[i]));
    return part_of(p);
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
template <int R>
__device__ __forceinline__ void load_labels(const int32_t* labels, int32_t r0, int32_t n, int32_t (&y)[R]) {
#pragma unroll
    for (int r = 0; r < R; ++r) y[r] = r0 + r < n ? __ldg(labels + r0 + r) : -1;
}

// R rows (r0, r0 + 1, ..) with labels y at once, each in NV vectors a lane;
// returns row r0 + r's loss in lane r, 0 in the lanes from R (one logarithm for all
// of them: kernels' us for 65,536 rows of 128 fp32 with one a row 27.3, so 26.1).  The
// labels of the rows at r_next are loaded into y on the way.
template <typename T, int NV, int R>
__device__ __forceinline__ float warp_rows(const RowArgs<T>& a, int32_t r0, int32_t n, float w, int32_t r_next,
                                           int32_t (&y_next)[R]) {
    const int lane = (int)lane_id();
    float m_of = 0.f, z_of = 1.f, xy_of = 0.f;  // lane r: of row r0 + r (these: a loss of 0)
    uint4 x[R][NV];
    float xe[R], xy[R];  // this lane's edge element; the label's logit
    int32_t y[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        y[r] = y_next[r];
        xe[r] = -INFINITY;
        xy[r] = 0.f;
        if (y[r] < -1 || y[r] >= a.classes) {
            if (lane == 0) dev_err(ERR_INDEX);
            y[r] = -1;
        }
        const T* row = a.x + (int64_t)(r0 + r) * a.ld;
        const RowParts<T> part(row, a.classes);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int32_t v = lane + 32 * k;
            x[r][k] = y[r] >= 0 && v < part.vecs ? *reinterpret_cast<const uint4*>(row + part.head + v * kE<T>)
                                                 : empty_part<T>();
        }
        const int32_t e = part.edge(lane);
        if (y[r] >= 0) {
            if (e >= 0) xe[r] = to_f(row[e]);
            xy[r] = to_f(row[y[r]]);
        }
    }
    load_labels(a.labels, r_next, n, y_next);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (r0 + r >= n) continue;  // the same in every lane
        T* out = a.grad ? a.grad + (int64_t)(r0 + r) * a.ld_grad : nullptr;
        if (y[r] < 0) {
            if (out)
                for (int32_t c = lane; c < a.classes; c += 32) put(out + c, 0.f);
            continue;
        }
        float m = xe[r];
#pragma unroll
        for (int k = 0; k < NV; ++k) m = fmaxf(m, part_max<T>(x[r][k]));
        m = warp_max(m);
        if (m == -INFINITY) m = 0.f;
        const Base base(m);
        f2 sum = pair(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < NV; ++k) part_exp<T>(x[r][k], base, sum);
        float z, z1;
        unpair(sum, z, z1);
        z = warp_sum(z + z1 + base.of(xe[r]));
        if (lane == r) m_of = m, z_of = z, xy_of = xy[r];
        if (!out) continue;
        const T* row = a.x + (int64_t)(r0 + r) * a.ld;
        const RowParts<T> part(row, a.classes);
        const bool same = same_phase(row, (const T*)out);
        const float inv = z == 0.f ? 0.f : w / z;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int32_t v = lane + 32 * k;
            if (v < part.vecs)
                store_part(out + part.head + v * kE<T>, same, part_grad<T>(x[r][k], base, pair(inv, inv)));
        }
        const int32_t e = part.edge(lane), at = part.place(y[r]);
        if (e >= 0) put(out + e, inv * base.of(xe[r]));
        // the lane that stored the label's element above may now replace it
        if ((at < 0 ? -1 - at : at % 32) == lane) put(out + y[r], z == 0.f ? 0.f : fmaf(inv, exp_from(xy[r], m), -w));
    }
    const float loss = loss_of(m_of, z_of, xy_of);
    if (lane < R && r0 + lane < n) a.loss[r0 + lane] = loss;
    return loss;
}

// Sum of the losses in a fixed order, by the last block to finish: 16 bytes and
// 8 loads a thread at a time (65,536 rows one by one took 35 us).
template <int NT, typename T>
__device__ __forceinline__ void put_total(const RowArgs<T>& a, int32_t n) {
    __shared__ float sh[NT / 32];
    // a row or so before the first 16-byte boundary, whole vectors, the rest
    const int32_t head = min(n, (int32_t)((4 - ((uintptr_t)a.loss >> 2 & 3)) & 3)), vecs = (n - head) / 4;
    const float4* v = reinterpret_cast<const float4*>(a.loss + head);
    float s = 0.f;
    for (int32_t i0 = threadIdx.x; i0 < vecs; i0 += 8 * NT) {
        float4 x[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) x[u] = i0 + u * NT < vecs ? __ldcg(v + i0 + u * NT) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int u = 0; u < 8; ++u) s += (x[u].x + x[u].y) + (x[u].z + x[u].w);
    }
    const int32_t rest = n - 4 * vecs, i = (int32_t)threadIdx.x;  // head and tail together
    if (i < rest) s += __ldcg(a.loss + (i < head ? i : i + 4 * vecs));
    s = warp_sum(s);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < NT / 32; ++w) s += sh[w];
        a.total[0] = a.mean ? s / (float)max(1, *a.valid) : s;
    }
}

// Blocks of k_xent_warp an SM: by the registers of what a lane holds.
template <int NV, int R>
constexpr int kWarpBlocks = NV * R > 4 ? 2 : 3;

// Each warp walks over its rows with the next rows' labels a turn ahead (65,536
// rows of 128 fp32: 27 us for the call; with a block for every 32 rows 33).
template <typename T, int NV, int R>
__global__ void __launch_bounds__(kThreads, kWarpBlocks<NV, R>) k_xent_warp(RowArgs<T> a) {
    pdl_start();
    __shared__ bool last;
    constexpr int kRows = kThreads / 32 * R;  // rows of a block's turn
    const int32_t n = rows_of(a.d_n, a.n_cap);
    const int32_t blocks = min((int32_t)gridDim.x, (n + kRows - 1) / kRows);  // that have rows
    if ((int32_t)blockIdx.x >= blocks) return;
    const float w = a.mean ? a.gs / (float)max(1, *a.valid) : a.gs;
    const int32_t step = (int32_t)gridDim.x * kRows;
    int32_t r0 = (int32_t)blockIdx.x * kRows + (int)(threadIdx.x >> 5) * R;
    int32_t y[R];
    load_labels(a.labels, r0, n, y);
    for (; r0 < n; r0 += step) warp_rows<T, NV, R>(a, r0, n, w, r0 + step, y);
    if (!a.total) return;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(a.valid + 1, 1) == blocks - 1;
    __syncthreads();
    if (last) put_total<kThreads>(a, n);
}

// Many rows of a few classes: a thread a row.  65,536 rows of 4 / 16 classes 11 /
// 17 us, by warps 25 / 25.
constexpr int kFewClasses = 16;
template <typename T>
__global__ void __launch_bounds__(kThreads) k_xent_thread(RowArgs<T> a) {
    pdl_start();
    __shared__ bool last;
    const int32_t n = rows_of(a.d_n, a.n_cap), blocks = (n + kThreads - 1) / kThreads;
    if ((int32_t)blockIdx.x >= blocks) return;
    const int32_t r = (int32_t)blockIdx.x * kThreads + (int32_t)threadIdx.x;
    if (r < n) {
        const T* row = a.x + (int64_t)r * a.ld;
        T* out = a.grad ? a.grad + (int64_t)r * a.ld_grad : nullptr;
        int32_t y = __ldg(a.labels + r);
        if (y < -1 || y >= a.classes) {
            dev_err(ERR_INDEX);
            y = -1;
        }
        float x[kFewClasses], m = -INFINITY, xy = 0.f, z = 0.f, loss = 0.f;
#pragma unroll
        for (int c = 0; c < kFewClasses; ++c) x[c] = y >= 0 && c < a.classes ? to_f(row[c]) : -INFINITY;
#pragma unroll
        for (int c = 0; c < kFewClasses; ++c) {
            m = fmaxf(m, x[c]);
            if (c == y) xy = x[c];
        }
        if (m == -INFINITY) m = 0.f;
#pragma unroll
        for (int c = 0; c < kFewClasses; ++c) {
            x[c] = exp_from(x[c], m);
            z += x[c];
        }
        const float w = a.mean ? a.gs / (float)max(1, *a.valid) : a.gs;
        const float inv = y < 0 || z == 0.f ? 0.f : w / z;
        if (y >= 0) loss = loss_of(m, z, xy);
        a.loss[r] = loss;
        if (out) {
#pragma unroll
            for (int c = 0; c < kFewClasses; ++c)
                if (c < a.classes) put(out + c, y < 0 || z == 0.f ? 0.f : fmaf(inv, x[c], c == y ? -w : 0.f));
        }
    }
    if (!a.total) return;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(a.valid + 1, 1) == blocks - 1;
    __syncthreads();
    if (last) put_total<kThreads>(a, n);
}

// The whole of a small call in one cluster: each CTA counts the labels, the
// cluster's warps take the rows in turn, the warps' sums meet in CTA 0.  256
// rows of 128 fp32: 6.5 us with the host's time, which bounds it (5.1 without).
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
    int32_t r0 = ((int32_t)blockIdx.x * kWarps + warp) * R;
    int32_t y[R];
    load_labels(a.labels, r0, n, y);
    for (; r0 < n; r0 += kSmallCtas * kWarps * R)
        sum += warp_rows<T, NV, R>(a, r0, n, w, r0 + kSmallCtas * kWarps * R, y);
    sum = warp_sum(sum);
    if ((threadIdx.x & 31) == 0) part[warp] = sum;
    cluster_sync();
    if (blockIdx.x == 0 && warp == 0 && a.total) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < kSmallCtas * kWarps; k += 32) {
            const int t = k + (int)threadIdx.x;
            s += ld_cluster(map_rank(smem_addr(part + t % kWarps), (uint32_t)(t / kWarps)));
        }
        s = warp_sum(s);
        if (threadIdx.x == 0) {
            a.total[0] = a.mean ? s / (float)max(1, v) : s;
            a.total[1] = (float)v;
        }
    }
    cluster_sync();  // the parts stay until they are read
}

// --------------------------------------------------------- rows by clusters
// What a thread holds of a row: up to kVecs vectors of its CTA's slice, NT
// apart, and for the lanes of warp 0 of CTA 0 an edge element.
template <typename T, int NT>
struct Held {
    uint4 x[kVecs];
    float xe;
    float m, z;  // of this warp: z = sum of exp(x - m)
};

// (m, z) of the warp from its vectors and, when given, the part (mr, zr) of
// each thread that is not held.
template <typename T, int NT>
__device__ __forceinline__ void reduce_held(Held<T, NT>& h, int32_t count, float mr, float zr) {
    float m = fmaxf(h.xe, mr);
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
        if ((int32_t)threadIdx.x + k * NT < count) m = fmaxf(m, part_max<T>(h.x[k]));
    m = warp_max(m);
    if (m == -INFINITY) m = 0.f;
    h.m = m;
    const Base base(m);
    f2 sum = pair(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
        if ((int32_t)threadIdx.x + k * NT < count) {
            repack(h.x[k]);
            part_exp<T>(h.x[k], base, sum);
        }
    float z, z1;
    unpair(sum, z, z1);
    z += z1 + base.of(h.xe);
    if (zr != 0.f) z += zr * exp_from(mr == -INFINITY ? 0.f : mr, m);
    h.z = warp_sum(z);
}

// The warps' (m, z) into every CTA of the cluster, and a barrier.
template <int NT, int S>
__device__ __forceinline__ void share_parts(float2* parts, int32_t rank, float m, float z) {
    const int warp = (int)(threadIdx.x >> 5), lane = (int)lane_id();
    if constexpr (S > 1) {
        if (lane < S)
            asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};\n" ::"r"(
                             map_rank(smem_addr(parts + rank * (NT / 32) + warp), (uint32_t)lane)),
                         "f"(m), "f"(z)
                         : "memory");
        cluster_sync();
    } else {
        if (lane == 0) parts[warp] = make_float2(m, z);
        __syncthreads();
    }
}

// The row's (M, Z); parts without a finite logit (z = 0) take no part.
template <int PARTS>
__device__ __forceinline__ void join_parts(const float2* parts, float& M, float& Z) {
    const int lane = (int)lane_id();
    M = -INFINITY, Z = 0.f;
#pragma unroll
    for (int i = lane; i < PARTS; i += 32)
        if (parts[i].y != 0.f) M = fmaxf(M, parts[i].x);
    M = warp_max(M);
    if (M == -INFINITY) M = 0.f;
#pragma unroll
    for (int i = lane; i < PARTS; i += 32)
        if (parts[i].y != 0.f) Z += parts[i].y * exp_from(parts[i].x, M);
    Z = warp_sum(Z);
}

// What a warp's exponentials, relative to its own m, are multiplied by in the
// gradient.  A warp without a finite logit (z = 0; its m says nothing) has
// exponentials of 0: any finite factor will do, but a row with NaN has NaN there too.
__device__ __forceinline__ float held_scale(float m, float z, float w, float M, float Z) {
    if (Z == 0.f) return 0.f;
    return z == 0.f ? w / Z : w / Z * exp_from(m, M);
}

// Gradient of what the thread holds; first: the slice's first vector.
template <typename T, int NT>
__device__ __forceinline__ void store_held(Held<T, NT>& h, T* first, int32_t count, bool same, float inv) {
    const Base base(h.m);
    const f2 inv2 = pair(inv, inv);
    T* p = first + (int32_t)threadIdx.x * kE<T>;
    if (same) {
#pragma unroll
        for (int k = 0; k < kVecs; ++k)
            if ((int32_t)threadIdx.x + k * NT < count) {
                repack(h.x[k]);
                *reinterpret_cast<uint4*>(p + k * NT * kE<T>) = part_grad<T>(h.x[k], base, inv2);
            }
    } else {
#pragma unroll
        for (int k = 0; k < kVecs; ++k)
            if ((int32_t)threadIdx.x + k * NT < count) {
                repack(h.x[k]);
                store_part(p + k * NT * kE<T>, false, part_grad<T>(h.x[k], base, inv2));
            }
    }
}

// A zero gradient for this CTA's part of an ignored row.
template <typename T, int NT>
__device__ __forceinline__ void zero_row(T* out, int32_t classes, int32_t rank, int32_t ctas) {
    const int32_t per = (classes + ctas - 1) / ctas, c1 = min(classes, (rank + 1) * per);
    for (int32_t c = rank * per + (int32_t)threadIdx.x; c < c1; c += NT) put(out + c, 0.f);
}

template <typename T, int NT, int S>
__global__ void __launch_bounds__(NT, 1024 / NT) k_xent_row(RowArgs<T> a) {
    pdl_start();
    constexpr int kParts = S * NT / 32;
    __shared__ __align__(8) float2 parts[kParts];  // (m, z) of every warp of the cluster
    __shared__ bool last;
    const int32_t r = (int32_t)(blockIdx.x / S), rank = (int32_t)(blockIdx.x % S);
    const int32_t n = rows_of(a.d_n, a.n_cap), classes = a.classes;
    if (r >= n) return;  // the whole cluster
    if constexpr (S > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");
    if (threadIdx.x == 0) last = false;
    const T* row = a.x + (int64_t)r * a.ld;
    T* out = a.grad ? a.grad + (int64_t)r * a.ld_grad : nullptr;
    int32_t y = __ldg(a.labels + r);
    if (y < -1 || y >= classes) {
        if (rank == 0 && threadIdx.x == 0) dev_err(ERR_INDEX);
        y = -1;
    }
    const bool used = y >= 0;  // the same in the whole cluster
    const RowParts<T> part(row, classes);
    const int32_t per = (part.vecs + S - 1) / S, v0 = min(part.vecs, rank * per), count = min(part.vecs, v0 + per) - v0;
    const int32_t edge = rank == 0 && threadIdx.x < 32 ? part.edge((int)threadIdx.x) : -1;
    // the thread that holds the label's element
    const int32_t at = used ? part.place(y) : -1;
    const bool owner = at < 0 ? rank == 0 && (int32_t)threadIdx.x == -1 - at
                              : at >= v0 && at < v0 + count && (at - v0) % NT == (int32_t)threadIdx.x;
    const T* p = row + part.head + (v0 + (int32_t)threadIdx.x) * kE<T>;
    Held<T, NT> h;
    h.m = 0.f, h.z = 0.f;
    float xy = 0.f;
    if (used) {
#pragma unroll
        for (int k = 0; k < kVecs; ++k)
            h.x[k] = (int32_t)threadIdx.x + k * NT < count ? *reinterpret_cast<const uint4*>(p + k * NT * kE<T>)
                                                           : empty_part<T>();
        h.xe = edge >= 0 ? to_f(row[edge]) : -INFINITY;
        if (owner) xy = to_f(row[y]);
        float mr = -INFINITY, zr = 0.f;  // the part past the registers
        for (int32_t i = (int32_t)threadIdx.x + kVecs * NT; i < count; i += NT) {
            const T* q = row + part.head + (v0 + i) * kE<T>;
            const float top = fmaxf(mr, part_max<T>(*reinterpret_cast<const uint4*>(q)));
            const float b = top == -INFINITY ? 0.f : top;
            zr *= exp_from(mr, b);
#pragma unroll
            for (int e = 0; e < kE<T>; ++e) zr += exp_from(to_f(q[e]), b);
            mr = top;
        }
        reduce_held(h, count, mr, zr);
    }
    // every CTA runs: its shared memory may be written
    if constexpr (S > 1) asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");
    share_parts<NT, S>(parts, rank, h.m, h.z);
    if (used) {
        float M, Z;
        join_parts<kParts>(parts, M, Z);
        const float w = a.mean ? a.gs / (float)max(1, *a.valid) : a.gs;
        if (out) {
            const bool same = same_phase(row, (const T*)out);
            const float inv = held_scale(h.m, h.z, w, M, Z);
            store_held(h, out + part.head + v0 * kE<T>, count, same, inv);
            if (edge >= 0) put(out + edge, inv * Base(h.m).of(h.xe));
            for (int32_t i = (int32_t)threadIdx.x + kVecs * NT; i < count; i += NT) {
                const int32_t c = part.head + (v0 + i) * kE<T>;
                float g[kE<T>];
#pragma unroll
                for (int e = 0; e < kE<T>; ++e) g[e] = Z == 0.f ? 0.f : w / Z * exp_from(to_f(row[c + e]), M);
#pragma unroll
                for (int e = 0; e < kE<T>; ++e) put(out + c + e, g[e]);
            }
            // this thread stored the label's element above: it may now replace it
            if (owner) put(out + y, Z == 0.f ? 0.f : fmaf(w / Z, exp_from(xy, M), -w));
        }
        if (owner) a.loss[r] = loss_of(M, Z, xy);
    } else {
        if (owner) a.loss[r] = 0.f;
        if (out) zero_row<T, NT>(out, classes, rank, S);
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

// Many long rows: the same, with each cluster walking over its rows and the
// next two rows' slices on their way into shared memory (one bulk copy of a
// slice's vectors) while the current row is worked on.  4096 x 50,257 bf16:
// 138 us, 6.0 TB/s; memory bounds it, with 67 % of the issue slots taken.
constexpr int kStreamVecs = 3500;  // of a CTA's slice: two buffers of it, two CTAs an SM

template <typename T, int NT, int S>
__global__ void __launch_bounds__(NT, 1024 / NT) k_xent_stream(RowArgs<T> a, int32_t slots) {
    extern __shared__ __align__(128) uint8_t dsm[];
    pdl_start();
    constexpr int kParts = S * NT / 32;
    __shared__ __align__(8) float2 parts[2][kParts];  // (m, z) of every warp of the cluster, of used rows in turn
    __shared__ __align__(8) uint64_t full[2], met[2];  // buffers; parts
    __shared__ bool last;
    const int32_t rank = (int32_t)(blockIdx.x % S), first = (int32_t)(blockIdx.x / S), step = (int32_t)(gridDim.x / S);
    const int32_t n = rows_of(a.d_n, a.n_cap), classes = a.classes;
    if (first >= n) return;  // the whole cluster
    if (threadIdx.x == 0) {
        last = false;
        mbar_init(&full[0], 1);
        mbar_init(&full[1], 1);
        mbar_init(&met[0], 1);
        mbar_init(&met[1], 1);
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    __syncthreads();
    if constexpr (S > 1) cluster_sync();  // every CTA runs: its shared memory may be written
    const auto label = [&](int32_t r) { return r < n ? __ldg(a.labels + r) : -1; };
    // copies this CTA's slice of row r into buffer b (thread 0)
    const auto fetch = [&](int32_t r, int32_t y, int b) {
        if (r >= n || y < 0 || y >= classes) return;
        const T* row = a.x + (int64_t)r * a.ld;
        const RowParts<T> part(row, classes);
        const int32_t per = (part.vecs + S - 1) / S, v0 = min(part.vecs, rank * per);
        const uint32_t bytes = (uint32_t)(min(part.vecs, v0 + per) - v0) * 16;
        mbar_expect_tx(&full[b], bytes);
        if (bytes)
            asm volatile(
                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                    smem_addr(dsm) + (uint32_t)(b * slots) * 16),
                "l"(row + part.head + (int64_t)v0 * kE<T>), "r"(bytes), "r"(smem_addr(&full[b]))
                : "memory");
    };
    int32_t y = label(first), y1 = label(first + step), y2;
    if (threadIdx.x == 0) {
        fetch(first, y, 0);
        fetch(first + step, y1, 1);
    }
    const float w = a.mean ? a.gs / (float)max(1, *a.valid) : a.gs;
    uint32_t phases = 0;  // bits 0, 1: parity of the next phase of full[0], full[1]; bits 2, 3: of met[0], met[1]
    int32_t par = 0;      // the row's buffer: alternates over all rows
    int32_t slot = 0;     // its parts and met: alternate over the used rows only
    for (int32_t r = first; r < n; r += step, par ^= 1, y = y1, y1 = y2) {
        y2 = label(r + 2 * step);
        const T* row = a.x + (int64_t)r * a.ld;
        T* out = a.grad ? a.grad + (int64_t)r * a.ld_grad : nullptr;
        if (y < 0 || y >= classes) {  // the same in the whole cluster
            if (rank == 0 && threadIdx.x == 0) {
                if (y != -1) dev_err(ERR_INDEX);
                a.loss[r] = 0.f;
            }
            if (out) zero_row<T, NT>(out, classes, rank, S);
            if (threadIdx.x == 0) fetch(r + 2 * step, y2, par);  // this row's buffer was not filled
            continue;
        }
        const RowParts<T> part(row, classes);
        const int32_t per = (part.vecs + S - 1) / S, v0 = min(part.vecs, rank * per), count = min(part.vecs, v0 + per) - v0;
        const int32_t edge = rank == 0 && threadIdx.x < 32 ? part.edge((int)threadIdx.x) : -1;
        const int32_t at = part.place(y);
        const bool owner = at < 0 ? rank == 0 && (int32_t)threadIdx.x == -1 - at
                                  : at >= v0 && at < v0 + count && (at - v0) % NT == (int32_t)threadIdx.x;
        Held<T, NT> h;
        h.xe = edge >= 0 ? to_f(row[edge]) : -INFINITY;
        const float xy = owner ? to_f(row[y]) : 0.f;
        if (!mbar_wait(&full[par], (phases >> par) & 1u) && lane_id() == 0) dev_err(ERR_TIMEOUT);
        const uint4* buf = reinterpret_cast<const uint4*>(dsm) + par * slots + threadIdx.x;
#pragma unroll
        for (int k = 0; k < kVecs; ++k)
            h.x[k] = (int32_t)threadIdx.x + k * NT < count ? buf[k * NT] : empty_part<T>();
        reduce_held(h, count, -INFINITY, 0.f);
        // The parts meet by asynchronous stores that complete on the receiver's
        // barrier.  (A cluster barrier here would first wait for this row's
        // predecessor's gradient to be stored: with one, 144 us and the memory
        // fence the largest stall.)  A slot is written again two used rows later,
        // by a warp that has met the used row between: to that one every reader
        // of the slot has sent its part, after it had read.  (Ignored rows exchange
        // nothing, so the slots may not go by the rows' own parity.)
        if (threadIdx.x == 0) mbar_expect_tx(&met[slot], kParts * 8);
        if (lane_id() < S) {
            const uint32_t to = smem_addr(&parts[slot][rank * (NT / 32) + (threadIdx.x >> 5)]);
            asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];\n" ::"r"(
                             map_rank(to, lane_id())),
                         "f"(h.m), "f"(h.z), "r"(map_rank(smem_addr(&met[slot]), lane_id()))
                         : "memory");
        }
        __syncwarp();
        if (!mbar_wait(&met[slot], (phases >> (2 + slot)) & 1u) && lane_id() == 0) dev_err(ERR_TIMEOUT);
        phases ^= (1u << par) | (4u << slot);
        // every thread has its vectors in registers: the buffer is free
        if (threadIdx.x == 0) fetch(r + 2 * step, y2, par);
        float M, Z;
        join_parts<kParts>(parts[slot], M, Z);
        slot ^= 1;
        if (out) {
            const float inv = held_scale(h.m, h.z, w, M, Z);
            store_held(h, out + part.head + v0 * kE<T>, count, same_phase(row, (const T*)out), inv);
            if (edge >= 0) put(out + edge, inv * Base(h.m).of(h.xe));
            // this thread stored the label's element above: it may now replace it
            if (owner) put(out + y, Z == 0.f ? 0.f : fmaf(w / Z, exp_from(xy, M), -w));
        }
        if (owner) a.loss[r] = loss_of(M, Z, xy);
    }
    __threadfence();
    if constexpr (S > 1) cluster_sync();
    else __syncthreads();
    if (!a.total) return;
    if (rank == 0 && threadIdx.x == 0) {
        __threadfence();
        last = atomicAdd(a.valid + 1, 1) == min(step, n) - 1;
    }
    __syncthreads();
    if (last) {
        __threadfence();
        put_total<NT>(a, n);
    }
}

// Rows whose label is not -1 (one cluster: one block, or kCountCtas when there
// are many); clears the count of finished blocks.  us for the whole call, one block /
// a cluster: 8,192 rows of 128 8.7 / 9.7, 16,384 12.6 / 12.3, 65,536 32 / 27.
constexpr int kCountCtas = 8, kCountMany = 8192;
__global__ void __launch_bounds__(kTotalThreads) k_xent_count(const int32_t* __restrict__ labels, int32_t n_cap,
                                                              const int32_t* __restrict__ d_n,
                                                              int32_t* __restrict__ valid, float* __restrict__ total) {
    pdl_start();
    __shared__ int32_t sh[kTotalThreads / 32 + 1];
    __shared__ float part;  // a count's bits
    const int32_t n = rows_of(d_n, n_cap), stride = (int32_t)(gridDim.x * kTotalThreads);
    int32_t v = 0;
    for (int32_t i0 = (int32_t)(blockIdx.x * kTotalThreads + threadIdx.x); i0 < n; i0 += 8 * stride) {
        int32_t y[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int32_t i = i0 + u * stride;
            y[u] = i < n ? __ldg(labels + i) : -1;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) v += y[u] != -1;
    }
    v = block_sum<kTotalThreads, int32_t>(v, sh);
    if (threadIdx.x == 0) part = __int_as_float(v);
    cluster_sync();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        v = 0;
        for (uint32_t c = 0; c < gridDim.x; ++c) v += __float_as_int(ld_cluster(map_rank(smem_addr(&part), c)));
        valid[0] = v;
        valid[1] = 0;
        if (total) total[0] = 0.f, total[1] = (float)v;
    }
    cluster_sync();  // the parts stay until they are read
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

template <typename T, int NV, int R>
sg_status run_warp(const RowArgs<T>& a, bool small, cudaStream_t s) {
    if (small) {
        SG_CUDA(launch_cluster(k_xent_small<T, NV, R>, kSmallCtas, kThreads, kSmallCtas, s, 0, a));
        return SG_OK;
    }
    int64_t blocks = cdiv(a.n_cap, kThreads / 32 * R);
    if (blocks > (int64_t)num_sms() * kWarpBlocks<NV, R>) blocks = (int64_t)num_sms() * kWarpBlocks<NV, R>;
    SG_CUDA(launch_pdl(k_xent_warp<T, NV, R>, dim3((unsigned)blocks), dim3(kThreads), 0, s, a));
    return SG_OK;
}

template <typename T, int NT, int S>
sg_status run_row(const RowArgs<T>& a, cudaStream_t s) {
    SG_CUDA(launch_cluster(k_xent_row<T, NT, S>, (unsigned)((int64_t)a.n_cap * S), NT, S, s, 0, a));
    return SG_OK;
}

template <typename T, int NT, int S>
sg_status run_stream(const RowArgs<T>& a, int64_t nv, cudaStream_t s) {
    const int32_t slots = (int32_t)cdiv(nv, S);  // of a buffer
    const int smem = 2 * slots * 16;
    static OncePerDevice set;
    SG_CUDA(allow_smem(set, k_xent_stream<T, NT, S>, 2 * kStreamVecs * 16));
    int64_t clusters = (int64_t)num_sms() * (1024 / NT) / S;
    if (clusters > a.n_cap) clusters = a.n_cap;
    SG_CUDA(launch_cluster(k_xent_stream<T, NT, S>, (unsigned)(clusters * S), NT, S, s, smem, a, slots));
    return SG_OK;
}

template <typename T>
sg_status run(RowArgs<T> a, cudaStream_t s) {
    const int64_t nv = cdiv((int64_t)a.classes, kE<T>);  // vectors of a row, at most
    const bool by_warp = nv <= 32 * kVecs;
    // one cluster serves a call whose rows its warps hold in a turn or two; a
    // turn costs as much as the second launch saves (fp32, cluster / two
    // launches, us on the device: 256 rows of 40 or 128 classes 5.1 / 7.4, 384 of
    // 128 7.6 / 7.6, 1,000 of 40 12.5 / 7.7; 256 of 200 5.6 / 6.6; 128 of 400 4.5 /
    // 7.0; 64 of 1000 4.3 / 6.8)
    const bool small = by_warp && a.n_cap <= 256 && a.n_cap * nv <= kSmallCtas * kThreads * kVecs;
    if (!small) {
        if (a.n_cap > kCountMany)
            SG_CUDA(launch_cluster(k_xent_count, kCountCtas, kTotalThreads, kCountCtas, s, 0, a.labels, a.n_cap, a.d_n,
                                   a.valid, a.total));
        else
            SG_CUDA(launch_pdl(k_xent_count, dim3(1), dim3(kTotalThreads), 0, s, a.labels, a.n_cap, a.d_n, a.valid, a.total));
    }
    if (a.n_cap == 0 && !small) return SG_OK;
    if (!small && a.classes <= kFewClasses) {
        SG_CUDA(launch_pdl(k_xent_thread<T>, dim3((unsigned)cdiv(a.n_cap, kThreads)), dim3(kThreads), 0, s, a));
        return SG_OK;
    }
    if (by_warp) {
        if (nv <= 32) return run_warp<T, 1, 4>(a, small, s);
        if (nv <= 64) return run_warp<T, 2, 2>(a, small, s);
        if (nv <= 128) return run_warp<T, 4, 2>(a, small, s);
        return run_warp<T, 8, 1>(a, small, s);
    }
    // rows for several turns of every cluster are streamed: one and a half turns
    // are enough for clusters of one or two CTAs, three for wider ones, which
    // idle together in a last turn (bf16, streamed / in registers, us: 1,300
    // rows of 10,000 18.5 / 19.3, 450 of 20,000 14.6 / 16.1, 300 of 50,257 20.4
    // / 21.5, but 200 17.0 / 17.3 and 100 11.9 / 9.7; 170 of 100,000 26.5 / 23.1;
    // 4,096 of 50,257 140 / 178)
    const int wide = nv <= 7 * kThreads ? 1 : nv <= kStreamVecs ? 2 : nv <= 2 * kStreamVecs ? 4 : nv <= 4 * kStreamVecs ? 8 : 16;
    if (nv <= 8 * kStreamVecs && (int64_t)a.n_cap * wide >= (wide <= 4 ? 6 : 12) * num_sms()) {
        switch (wide) {
            case 1: return run_stream<T, kThreads, 1>(a, nv, s);
            case 2: return run_stream<T, 512, 1>(a, nv, s);
            case 4: return run_stream<T, 512, 2>(a, nv, s);
            case 8: return run_stream<T, 512, 4>(a, nv, s);
            default: return run_stream<T, 512, 8>(a, nv, s);
        }
    }
    // smallest cluster whose registers hold the row, widened while the rows do
    // not fill the SMs (20 rows of 20,000 fp32: 7.3 us, 7.8 unwidened); 512
    // threads when 8 CTAs of 256 do not hold it
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
