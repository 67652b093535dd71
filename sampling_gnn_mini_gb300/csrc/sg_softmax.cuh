// Softmax of a row whose vectors stay in registers between reading and writing:
// each warp reduces its part to (m, z) relative to its own maximum, the parts meet
// once, in shared memory of every CTA of the row's cluster, and a warp scales its
// exponentials by exp(m_warp - m) / z.  (l: log2(e), divided by the temperature.)
#pragma once

#include "sg_rows.cuh"
#include "sg_tc.cuh"

namespace sgi {

constexpr int kVecs = 8;  // 16-byte vectors of a row a thread holds

// exp(x - m) of values and pairs, the difference taken first, as in exp_from():
// it is exact near m, so the largest logit's exponential is 1 whatever its level.
// (One fused operation, x log2(e) - m log2(e), leaves the rounding of the second
// product in every exponential: at |m| = 1e6 they are off by 1.5 %, at 1e10 by
// more than the type's range.)
// With l = log2(e) / T: exp((x - m) / T).
struct Base {
    f2 l, b;
    float m, l1;
    __device__ __forceinline__ explicit Base(float m_, float l_ = kLog2e) : m(m_), l1(l_) {
        l = pair(l_, l_);
        b = pair(-m_, -m_);
    }
    __device__ __forceinline__ float of(float x) const { return exp_from(x, m, l1); }
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
__device__ __forceinline__ void reduce_held(Held<T, NT>& h, int32_t count, float mr, float zr, float l = kLog2e) {
    float m = fmaxf(h.xe, mr);
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
        if ((int32_t)threadIdx.x + k * NT < count) m = fmaxf(m, part_max<T>(h.x[k]));
    m = warp_max(m);
    if (m == -INFINITY) m = 0.f;
    h.m = m;
    const Base base(m, l);
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
    if (zr != 0.f) z += zr * exp_from(mr == -INFINITY ? 0.f : mr, m, l);
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
__device__ __forceinline__ void join_parts(const float2* parts, float& M, float& Z, float l = kLog2e) {
    const int lane = (int)lane_id();
    M = -INFINITY, Z = 0.f;
#pragma unroll
    for (int i = lane; i < PARTS; i += 32)
        if (parts[i].y != 0.f) M = fmaxf(M, parts[i].x);
    M = warp_max(M);
    if (M == -INFINITY) M = 0.f;
#pragma unroll
    for (int i = lane; i < PARTS; i += 32)
        if (parts[i].y != 0.f) Z += parts[i].y * exp_from(parts[i].x, M, l);
    Z = warp_sum(Z);
}

// What a warp's exponentials, relative to its own m, are multiplied by in the
// gradient.  A warp without a finite logit (z = 0; its m says nothing) has
// exponentials of 0: any finite factor will do, but a row with NaN has NaN there too.
__device__ __forceinline__ float held_scale(float m, float z, float w, float M, float Z, float l = kLog2e) {
    if (Z == 0.f) return 0.f;
    return z == 0.f ? w / Z : w / Z * exp_from(m, M, l);
}

// Gradient of what the thread holds; first: the slice's first vector.
template <typename T, int NT>
__device__ __forceinline__ void store_held(Held<T, NT>& h, T* first, int32_t count, bool same, float inv, float l = kLog2e) {
    const Base base(h.m, l);
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

}  // namespace sgi
