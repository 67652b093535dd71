// Layer norm of rows x of dim values, and its gradient:
//   mu = mean x,  r = 1 / sqrt(mean (x - mu)^2 + eps),  h = (x - mu) r,  y = h w + b
//   u = g w:  dx = r (u - mean u - h mean(u h)),  dw = sum over rows of g h,  db = sum over rows of g
// Bound by memory: forward reads and writes a row once, backward reads two rows and
// writes one.  A row belongs to a group of 4 to 32 lanes or to a block, 4 to 32 values a
// thread.  Short rows go from global memory into registers, the next ones ahead; longer
// ones through a ring in shared memory that every thread fills with its own vectors,
// rows ahead, and with 16 (24) values a thread the gradient of the weight and bias, two sums a
// value, still fits beside them.  The deviation is summed about the mean, in a second
// pass over the values on the chip.
//
// Columns belong to threads.  In the gradient a block walks over its rows with the
// columns' sums in registers, writes them once to the workspace, and a second kernel
// adds up the blocks' sums in order: no float atomics, the same bits on every run.
//
// Values move in vectors of 16 bytes at any alignment of the rows: the up to 7 + 7
// values before a row's first 16-byte boundary and after its last one go to the
// group's first lanes, one each.  A group meets only rows that start at the same place
// within 16 bytes (rows a multiple of 8 apart), so a thread's columns stay the same.
// Arrays whose rows do not start alike are moved value by value.  30,011 x 1001 bf16
// forward: 26 us, all in single values 50.
#include <type_traits>

#include "sg_internal.cuh"
#include "sg_rows.cuh"
#include "sg_tc.cuh"

using namespace sgi;

namespace {

constexpr int kHeld = 16;      // values of a row a thread holds
constexpr int kThreads = 256;  // of a block of groups' rows

// -------------------------------------------------------- sums over a group
// Sums of C values over the L threads that share a row, in every one of them.  L > 32: a
// block of L threads, 0: a block of any size; sh holds two sets of warps' sums, used in turn (a set is written
// again after the barrier of the other one, which follows its last reading).
constexpr int kSums = 2 * 2 * 32;  // of sh
template <int L, int C>
__device__ __forceinline__ void lane_sum(float (&x)[C]) {
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1)
#pragma unroll
        for (int c = 0; c < C; ++c) x[c] += __shfl_xor_sync(0xFFFFFFFFu, x[c], d);
}
template <int L, int C>
__device__ __forceinline__ void group_sum(float (&x)[C], float* sh, int& turn) {
    if constexpr (L > 0 && L <= 32) {
        lane_sum<L, C>(x);
    } else {
        lane_sum<32, C>(x);
        float* to = sh + turn * 2 * 32;
        turn ^= 1;
        if (lane_id() == 0)
#pragma unroll
            for (int c = 0; c < C; ++c) to[c * 32 + (threadIdx.x >> 5)] = x[c];
        __syncthreads();
        if constexpr (L > 0) {
            constexpr int W = L / 32;
#pragma unroll
            for (int c = 0; c < C; ++c) x[c] = to[c * 32 + (int)lane_id() % W];
            lane_sum<W, C>(x);
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c) x[c] = lane_id() < blockDim.x / 32 ? to[c * 32 + lane_id()] : 0.f;
            lane_sum<32, C>(x);
        }
    }
}

// This thread's group in its block.
template <int L>
__device__ __forceinline__ int group_of() {
    return L ? (int)threadIdx.x / (L ? L : 1) : 0;
}

// ------------------------------------------------- a thread's part of a row
// A vector's values one by one, in a loop that takes few registers.
__device__ __forceinline__ void push_front(uint4& v, float x) { v = make_uint4(__float_as_uint(x), v.x, v.y, v.z); }
__device__ __forceinline__ void push_front(uint4& v, __nv_bfloat16 x) {
    v = make_uint4((uint32_t)__bfloat16_as_ushort(x) | v.x << 16, __funnelshift_l(v.x, v.y, 16), __funnelshift_l(v.y, v.z, 16),
                   __funnelshift_l(v.z, v.w, 16));
}
__device__ __forceinline__ void pop_front(uint4& v, float& x) {
    x = __uint_as_float(v.x);
    v = make_uint4(v.y, v.z, v.w, 0);
}
__device__ __forceinline__ void pop_front(uint4& v, __nv_bfloat16& x) {
    x = __ushort_as_bfloat16((unsigned short)v.x);
    v = make_uint4(__funnelshift_r(v.x, v.y, 16), __funnelshift_r(v.y, v.z, 16), __funnelshift_r(v.z, v.w, 16), v.w >> 16);
}

// What thread l of a group of L (0: the block) holds of each of its rows: vectors l, l +
// L, .. (V of them at most) and ends l, l + L, .. (of 16: 8 for the head, 8 for the tail).
// alike: every array's rows start at the same place within 16 bytes; if not, all
// vectors are moved by values and the ends are the tail's.
template <typename T, int V, int L>
struct Part {
    static constexpr int P = kE<T> / 2;                // pairs of a vector
    static constexpr int NE = L == 0 || L >= 16 ? 1 : 16 / L;  // ends of a thread
    int32_t head, vecs, l;
    int32_t ends[NE];  // columns, or -1
    bool alike;
    // rows of x from r on, 8 apart
    __device__ __forceinline__ Part(const T* x, int64_t ld, int64_t r, int32_t dim, bool alike_)
        : l(L ? (int)threadIdx.x % (L ? L : 1) : (int)threadIdx.x), alike(alike_) {
        const RowParts<T> part(alike ? x + r * ld : (const T*)nullptr, dim);
        head = part.head;
        vecs = part.vecs;
#pragma unroll
        for (int e = 0; e < NE; ++e) ends[e] = l + e * L < 16 ? part.edge(l + e * L) : -1;
    }
    __device__ __forceinline__ int stride() const { return L ? L : (int)blockDim.x; }
    __device__ __forceinline__ bool has(int v) const { return l + v * stride() < vecs; }
    __device__ __forceinline__ int32_t column(int v) const { return head + (l + v * stride()) * kE<T>; }
    __device__ __forceinline__ uint4 load(const T* row, int v) const {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (!has(v)) return u;
        const T* p = row + column(v);
        if (alike) return *reinterpret_cast<const uint4*>(p);
#pragma unroll 1
        for (int i = kE<T> - 1; i >= 0; --i) push_front(u, p[i]);
        return u;
    }
    // (as it is: its conversion would wait for the load)
    __device__ __forceinline__ T load_end(const T* row, int e) const { return ends[e] >= 0 ? row[ends[e]] : T(0.f); }
    __device__ __forceinline__ void store(T* row, int v, const f2 (&f)[P]) const {
        if (!has(v)) return;
        T* p = row + column(v);
        uint4 u = part_of(f);
        if (alike) {
            *reinterpret_cast<uint4*>(p) = u;
            return;
        }
#pragma unroll 1
        for (int i = 0; i < kE<T>; ++i) {
            T x;
            pop_front(u, x);
            p[i] = x;
        }
    }
    __device__ __forceinline__ void store_end(T* row, int e, float x) const {
        if (ends[e] >= 0) put(row + ends[e], x);
    }
};
// A weight or bias (fp32 or bf16; none: `none`); 0 where the thread has no value
__device__ __forceinline__ float param_at(const void* w, int32_t bf16, int32_t c, float none) {
    return !w ? none : bf16 ? to_f(((const __nv_bfloat16*)w)[c]) : __ldg((const float*)w + c);
}
template <typename T, int V, int L>
struct Param {
    f2 f[V][kE<T> / 2];
    float end[Part<T, V, L>::NE];
    __device__ __forceinline__ Param(const Part<T, V, L>& p, const void* w, int32_t bf16, float none) {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < kE<T> / 2; ++i) {
                const int32_t c = p.column(v) + 2 * i;
                f[v][i] = p.has(v) ? pair(param_at(w, bf16, c, none), param_at(w, bf16, c + 1, none)) : pair(0.f, 0.f);
            }
#pragma unroll
        for (int e = 0; e < Part<T, V, L>::NE; ++e) end[e] = p.ends[e] >= 0 ? param_at(w, bf16, p.ends[e], none) : 0.f;
    }
};
__device__ __forceinline__ float total_of(f2 a) {
    float x, y;
    unpair(a, x, y);
    return x + y;
}
__device__ __forceinline__ f2 both(float x) { return pair(x, x); }

// ----------------------------------------------------------------- forward
template <typename T>
struct FwdArgs {
    const T* x;
    T* y;
    int64_t ld, ld_y;
    const void* weight;
    const void* bias;
    const int32_t* d_n;
    int32_t n_cap, dim, w_bf16, alike;
    float eps;
    float* mean;
    float* rstd;
};

// One row, from its vectors (get(v)) and ends.
template <typename T, int V, int L, typename Get>
__device__ __forceinline__ void norm_row(const FwdArgs<T>& a, const Part<T, V, L>& p, const Param<T, V, L>& w,
                                         const Param<T, V, L>& b, int64_t r, int32_t n, float inv, float* sh, int& turn,
                                         const T (&ends)[Part<T, V, L>::NE], Get get) {
    constexpr int P = kE<T> / 2, NE = Part<T, V, L>::NE;
    f2 f[V][P], t = both(0.f);
    float fe[NE], s[1] = {0.f};
#pragma unroll
    for (int v = 0; v < V; ++v) {
        pairs_of(get(v), f[v]);
#pragma unroll
        for (int i = 0; i < P; ++i) t = add2(t, f[v][i]);
    }
#pragma unroll
    for (int e = 0; e < NE; ++e) s[0] += fe[e] = to_f(ends[e]);
    s[0] += total_of(t);
    group_sum<L, 1>(s, sh, turn);
    const float mu = s[0] * inv;
    t = both(0.f);
    s[0] = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (p.has(v)) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                f[v][i] = add2(f[v][i], both(-mu));
                t = fma2(f[v][i], f[v][i], t);
            }
        }
#pragma unroll
    for (int e = 0; e < NE; ++e)
        if (p.ends[e] >= 0) {
            fe[e] -= mu;
            s[0] = fmaf(fe[e], fe[e], s[0]);
        }
    s[0] += total_of(t);
    group_sum<L, 1>(s, sh, turn);
    const float rs = rsqrtf(fmaf(s[0], inv, a.eps));
    if (r >= n) return;
    if (p.l == 0) {
        if (a.mean) a.mean[r] = mu;
        if (a.rstd) a.rstd[r] = rs;
    }
    T* to = a.y + r * a.ld_y;
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int i = 0; i < P; ++i) f[v][i] = fma2(mul2(f[v][i], both(rs)), w.f[v][i], b.f[v][i]);
        p.store(to, v, f[v]);
    }
#pragma unroll
    for (int e = 0; e < NE; ++e) p.store_end(to, e, fmaf(fe[e] * rs, w.end[e], b.end[e]));
}

// Blocks walk over their rows, R rows a group at once, with the next rows' values on
// their way into registers.
template <typename T, int V, int L, int NT, int R>
__global__ void __launch_bounds__(NT, NT == kThreads ? 4 : 1) k_norm_fwd(FwdArgs<T> a) {
    pdl_start();
    constexpr int kRows = L ? NT / (L ? L : 1) : 1;  // of a block at once
    constexpr int NE = Part<T, V, L>::NE;
    __shared__ float sh[L == 0 || L > 32 ? kSums : 1];
    int turn = 0;
    const int32_t n = rows_of(a.d_n, a.n_cap);
    const int64_t step = (int64_t)gridDim.x * (kRows * R);
    int64_t b0 = (int64_t)blockIdx.x * (kRows * R);
    if (b0 >= n) return;
    const Part<T, V, L> p(a.x, a.ld, b0 + group_of<L>(), a.dim, a.alike != 0);
    const Param<T, V, L> w(p, a.weight, a.w_bf16, 1.f), b(p, a.bias, a.w_bf16, 0.f);
    struct Rows {
        uint4 x[R][V];
        T ends[R][NE];
    } next;
    const auto load = [&](int64_t b1, Rows& o) {
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int64_t r = b1 + q * kRows + group_of<L>();
#pragma unroll
            for (int v = 0; v < V; ++v) o.x[q][v] = r < n ? p.load(a.x + r * a.ld, v) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < NE; ++e) o.ends[q][e] = r < n ? p.load_end(a.x + r * a.ld, e) : T(0.f);
        }
    };
    const float inv = 1.f / (float)a.dim;
    load(b0, next);
    for (; b0 < n; b0 += step) {  // the same in the whole block
        const Rows cur = next;
        load(b0 + step, next);
#pragma unroll
        for (int q = 0; q < R; ++q)
            norm_row<T, V, L>(a, p, w, b, b0 + q * kRows + group_of<L>(), n, inv, sh, turn, cur.ends[q],
                              [&](int v) { return cur.x[q][v]; });
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
    int32_t n_cap, dim, w_bf16, alike;
    float* parts;  // per block: sums of g h, then of g, kLead before the first vector's; NULL: not wanted
    void* dweight;
    void* dbias;
};
// A block's sums of dim columns: kLead - head before the head's first, so that vectors
// are on 16 bytes; the two rows are `pitch` apart.
constexpr int kLead = 8;
__host__ __device__ constexpr int32_t pitch_of(int32_t dim) { return (dim + kLead + 3) / 4 * 4; }

// A thread's columns' sums over its rows.
template <typename T, int V, int L>
struct Sums {
    f2 w[V][kE<T> / 2], b[V][kE<T> / 2];
    float we[Part<T, V, L>::NE], be[Part<T, V, L>::NE];
    __device__ __forceinline__ Sums() {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < kE<T> / 2; ++i) w[v][i] = b[v][i] = both(0.f);
#pragma unroll
        for (int e = 0; e < Part<T, V, L>::NE; ++e) we[e] = be[e] = 0.f;
    }
    // one of the two into o[column + lead], which is 16-byte aligned at vectors if `wide`
    template <bool wide>
    __device__ __forceinline__ void put(const Part<T, V, L>& p, bool bias, float* o) const {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (p.has(v))
#pragma unroll
                for (int i = 0; i < kE<T> / 2; i += 2) {
                    float4 q;
                    unpair(bias ? b[v][i] : w[v][i], q.x, q.y);
                    unpair(bias ? b[v][i + 1] : w[v][i + 1], q.z, q.w);
                    float* to = o + p.column(v) + 2 * i;
                    if constexpr (wide) {
                        *reinterpret_cast<float4*>(to) = q;
                    } else {
                        to[0] = q.x, to[1] = q.y, to[2] = q.z, to[3] = q.w;
                    }
                }
#pragma unroll
        for (int e = 0; e < Part<T, V, L>::NE; ++e)
            if (p.ends[e] >= 0) o[p.ends[e]] = bias ? be[e] : we[e];
    }
    // a block's two rows of sums (L: the whole block)
    __device__ __forceinline__ void put_block(const Part<T, V, L>& p, const BwdArgs<T>& a) const {
        if (!a.parts) return;
        float* to = a.parts + (int64_t)blockIdx.x * 2 * pitch_of(a.dim) + kLead - p.head;
        put<true>(p, false, to);
        put<true>(p, true, to + pitch_of(a.dim));
    }
};

// The sums of a block's groups of L threads, added up in order: into the workspace or,
// SMALL, with those of the cluster's other blocks.  cols: room for a group's columns
// each, not in use.
constexpr int kSmallCtas = 8, kSmallTurns = 8;  // turns of a cluster's groups at most
template <typename T, int V, int L>
constexpr int kGroupColumns = L * V * kE<T> + 16;

template <typename T, int V, int L, int NT, bool SMALL>
__device__ __forceinline__ void join_groups(const Sums<T, V, L>& sums, const Part<T, V, L>& p, const BwdArgs<T>& a, float* cols) {
    if (!SMALL && !a.parts) return;
    constexpr int W = kGroupColumns<T, V, L>;
    __shared__ float block[SMALL ? 2 * W : 1];
    float* to = SMALL ? block : a.parts + (int64_t)blockIdx.x * 2 * pitch_of(a.dim) + kLead;
    const int32_t pitch = SMALL ? W : pitch_of(a.dim);
    for (int k = 0; k < 2; ++k) {
        __syncthreads();
        sums.template put<false>(p, k != 0, cols + (group_of<L>()) * W);
        __syncthreads();
        for (int c = threadIdx.x; c < a.dim; c += NT) {
            float s = 0.f;
#pragma unroll 8
            for (int q = 0; q < NT / L; ++q) s += cols[q * W + c];
            to[k * pitch + c] = s;
        }
    }
    if constexpr (SMALL) {
        cluster_sync();
        for (int32_t o = (int32_t)(blockIdx.x * NT + threadIdx.x); o < 2 * a.dim; o += kSmallCtas * NT) {
            const int k = o >= a.dim, c = o - k * a.dim;
            float s = 0.f;
            for (uint32_t q = 0; q < kSmallCtas; ++q) s += ld_cluster(map_rank(smem_addr(block + k * W + c), q));
            void* d = k ? a.dbias : a.dweight;
            if (!d) continue;
            if (a.w_bf16) put((__nv_bfloat16*)d + c, s);
            else put((float*)d + c, s);
        }
        cluster_sync();  // the sums stay until they are read
    }
}

// One row: the columns' sums and dx.  The row's values are asked for twice (x(v), g(v)
// and the ends): held over the sums they would take the registers of half the threads.
// between(): called when the group's sums are there.
template <typename T, int V, int L, typename GetX, typename GetG, typename Between>
__device__ __forceinline__ void grad_row(const BwdArgs<T>& a, const Part<T, V, L>& p, const Param<T, V, L>& w,
                                         Sums<T, V, L>& sums, int64_t r, int32_t n, float inv, float* sh, int& turn,
                                         float mean, float rstd, const T (&x_ends)[Part<T, V, L>::NE],
                                         const T (&g_ends)[Part<T, V, L>::NE], GetX x, GetG g, Between between) {
    constexpr int P = kE<T> / 2, NE = Part<T, V, L>::NE;
    float xe[NE], ge[NE];
#pragma unroll
    for (int e = 0; e < NE; ++e) xe[e] = to_f(x_ends[e]), ge[e] = to_f(g_ends[e]);
    const f2 mu = both(-mean), rs = both(rstd);
    f2 t0 = both(0.f), t1 = both(0.f);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        f2 h[P], f[P];
        pairs_of(x(v), h);
        pairs_of(g(v), f);
#pragma unroll
        for (int i = 0; i < P; ++i) {  // (a vector that is not there: g = 0, w = 0)
            h[i] = mul2(add2(h[i], mu), rs);
            sums.w[v][i] = fma2(f[i], h[i], sums.w[v][i]);
            sums.b[v][i] = add2(sums.b[v][i], f[i]);
            f[i] = mul2(f[i], w.f[v][i]);
            t0 = add2(t0, f[i]);
            t1 = fma2(f[i], h[i], t1);
        }
    }
    float s[2] = {total_of(t0), total_of(t1)}, he[NE];
#pragma unroll
    for (int e = 0; e < NE; ++e) {
        he[e] = (xe[e] - mean) * rstd;
        sums.we[e] = fmaf(ge[e], he[e], sums.we[e]);
        sums.be[e] += ge[e];
        s[0] = fmaf(ge[e], w.end[e], s[0]);
        s[1] = fmaf(ge[e] * w.end[e], he[e], s[1]);
    }
    group_sum<L, 2>(s, sh, turn);
    between();
    if (r >= n) return;
    // dx = rstd (g w - s0 / dim - h s1 / dim)
    const float cg = -s[0] * inv, ch = -s[1] * inv;
    T* to = a.dx + r * a.ld_dx;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        f2 h[P], f[P];
        pairs_of(x(v), h);
        pairs_of(g(v), f);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            f[i] = mul2(fma2(f[i], w.f[v][i], fma2(mul2(add2(h[i], mu), rs), both(ch), both(cg))), rs);
        }
        p.store(to, v, f);
    }
#pragma unroll
    for (int e = 0; e < NE; ++e) p.store_end(to, e, fmaf(ge[e], w.end[e], fmaf((xe[e] - mean) * rstd, ch, cg)) * rstd);
}

// Blocks an SM: bf16 vectors hold twice the values.
template <typename T, int NT>
constexpr int kBwdBlocks = NT == kThreads ? (sizeof(T) == 2 ? 2 : 3) : 1;

// SMALL: the whole of a small call in one cluster, whose CTAs' sums meet in distributed
// shared memory (1,024 x 128 fp32: 9.8 us with the host's time, with a second
// launch for the sums 11.3; twice the rows, 16 turns of its groups, 17.5, 11.0).
template <typename T, int V, int L, int NT, int R, bool SMALL>
__global__ void __launch_bounds__(NT, kBwdBlocks<T, NT>) k_norm_bwd(BwdArgs<T> a) {
    pdl_start();
    constexpr int kRows = L ? NT / (L ? L : 1) : 1;
    constexpr int NE = Part<T, V, L>::NE;
    __shared__ float sh[L == 0 || L > 32 ? kSums : 1];
    __shared__ float cols[L ? kRows * kGroupColumns<T, V, L> : 1];
    int turn = 0;
    const int32_t n = rows_of(a.d_n, a.n_cap);
    const int64_t step = (int64_t)gridDim.x * (kRows * R);
    int64_t b0 = (int64_t)blockIdx.x * (kRows * R);
    const Part<T, V, L> p(a.x, a.ld, b0 + group_of<L>(), a.dim, a.alike != 0);
    const Param<T, V, L> w(p, a.weight, a.w_bf16, 1.f);
    Sums<T, V, L> sums;
    struct Rows {
        uint4 x[R][V], g[R][V];
        T xe[R][NE], ge[R][NE];
        float mu[R], rs[R];
    } next;
    const auto load = [&](int64_t b1, Rows& o) {
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int64_t r = b1 + q * kRows + group_of<L>();
            o.mu[q] = r < n ? __ldg(a.mean + r) : 0.f;
            o.rs[q] = r < n ? __ldg(a.rstd + r) : 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                o.x[q][v] = r < n ? p.load(a.x + r * a.ld, v) : make_uint4(0, 0, 0, 0);
                o.g[q][v] = r < n ? p.load(a.g + r * a.ld_g, v) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int e = 0; e < NE; ++e) {
                o.xe[q][e] = r < n ? p.load_end(a.x + r * a.ld, e) : T(0.f);
                o.ge[q][e] = r < n ? p.load_end(a.g + r * a.ld_g, e) : T(0.f);
            }
        }
    };
    const float inv = 1.f / (float)a.dim;
    load(b0, next);
    for (; b0 < n; b0 += step) {  // the same in the whole block
        Rows cur = next;
        load(b0 + step, next);
#pragma unroll
        for (int q = 0; q < R; ++q)
            grad_row<T, V, L>(
                a, p, w, sums, b0 + q * kRows + group_of<L>(), n, inv, sh, turn, cur.mu[q], cur.rs[q], cur.xe[q], cur.ge[q],
                [&](int v) { return cur.x[q][v]; }, [&](int v) { return cur.g[q][v]; },
                [&] {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        repack(cur.x[q][v]);
                        repack(cur.g[q][v]);
                    }
                });
    }
    if constexpr (L == 0 || L > 32) {
        sums.put_block(p, a);
    } else {
        join_groups<T, V, L, NT, SMALL>(sums, p, a, cols);
    }
}

// ------------------------------------------------------ long rows by blocks
// Each thread copies its own vectors of the block's next rows into a ring of slots in
// shared memory, asynchronously, and waits for its own copies alone; the ends are
// loaded a row ahead.
// A group is a warp (L = 32, blocks of NT = 256 threads) or the block: of L threads, or (L
// = 0) of as many, up to NT, as the row needs.  The constant size is worth its
// instances: 19,531 x 4096 bf16 forward 61 us, of any size 64.
constexpr int kRingBytes = 208 * 1024;  // of an SM
// Threads an SM, by the registers for HELD values of a row a thread (NT = 1024: 64).  A:
// arrays that are read (1 forward, 2 backward).  Backward, 16 values a thread: 512 of
// 128 registers 80 us for 16,384 x 4096 bf16, 768 of 80 105, 1,024 of 64 140.
template <int HELD, int A, int NT>
constexpr int kRingThreads = NT == 1024 ? 1024 : A == 1 && HELD <= 16 ? 768 : A == 1 || HELD <= 16 ? 512 : 384;
// Slots: as many as there is room for, four at most.
template <typename T, int V, int A, int NT>
constexpr int kRoom = kRingBytes / (kRingThreads<V * kE<T>, A, NT> * V * A * 16);
template <typename T, int V, int A, int NT>
constexpr int kDepth = kRoom<T, V, A, NT> > 4 ? 4 : kRoom<T, V, A, NT> > 0 ? kRoom<T, V, A, NT> : 1;
// Threads of the longest rows' blocks: 16 values each.
template <int A>
constexpr int kBlockThreads = A == 1 ? 384 : 512;  // two blocks or one an SM; above: 1024

template <typename T, int V, int L, int NT>
__global__ void __launch_bounds__(NT, kRingThreads<V * kE<T>, 1, NT> / NT) k_norm_fwd_ring(FwdArgs<T> a) {
    extern __shared__ __align__(128) uint4 ring[];
    pdl_start();
    constexpr int D = kDepth<T, V, 1, NT>, kRows = L == 32 ? NT / 32 : 1;  // kRows: of a block at once
    __shared__ float sh[L == 0 || L > 32 ? kSums : 1];
    int turn = 0;
    const int32_t n = rows_of(a.d_n, a.n_cap), first = (int32_t)blockIdx.x * kRows + group_of<L>();
    const int32_t step = (int32_t)gridDim.x * kRows;
    if (first >= n) return;  // whole groups
    const Part<T, V, L> p(a.x, a.ld, first, a.dim, true);
    const auto slot = [&](int at, int v) { return ring + (at * V + v) * (L > 32 ? L : (int)blockDim.x) + (int)threadIdx.x; };
    const auto fetch = [&](int64_t r, int at) {
        if (r < n) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (p.has(v)) copy_async(slot(at, v), a.x + r * a.ld + p.column(v));
        }
        copies_end();
    };
#pragma unroll
    for (int i = 0; i < D - 1; ++i) fetch(first + (int64_t)i * step, i);
    const Param<T, V, L> w(p, a.weight, a.w_bf16, 1.f), b(p, a.bias, a.w_bf16, 0.f);
    const float inv = 1.f / (float)a.dim;
    int at = 0;
    T next = p.load_end(a.x + first * a.ld, 0);
    for (int64_t r = first; r < n; r += step) {
        fetch(r + (int64_t)(D - 1) * step, at ? at - 1 : D - 1);
        const T end[1] = {next};
        if (r + step < n && p.ends[0] >= 0) next = a.x[(r + step) * a.ld + p.ends[0]];
        copies_wait<D - 1>();
        norm_row<T, V, L>(a, p, w, b, r, n, inv, sh, turn, end,
                          [&](int v) { return p.has(v) ? *slot(at, v) : make_uint4(0, 0, 0, 0); });
        if (++at == D) at = 0;
    }
}

template <typename T, int V, int L, int NT>
__global__ void __launch_bounds__(NT, kRingThreads<V * kE<T>, 2, NT> / NT) k_norm_bwd_ring(BwdArgs<T> a) {
    extern __shared__ __align__(128) uint4 ring[];
    pdl_start();
    constexpr int D = kDepth<T, V, 2, NT>, kRows = L == 32 ? NT / 32 : 1;
    __shared__ float sh[L == 0 || L > 32 ? kSums : 1];
    int turn = 0;
    const int32_t n = rows_of(a.d_n, a.n_cap), first = (int32_t)blockIdx.x * kRows + group_of<L>();
    const int32_t step = (int32_t)gridDim.x * kRows;
    const Part<T, V, L> p(a.x, a.ld, first, a.dim, true);
    const auto slot = [&](int at, int v) { return ring + (at * 2 * V + v) * (L > 32 ? L : (int)blockDim.x) + (int)threadIdx.x; };  // (g: v + V)
    const auto fetch = [&](int64_t r, int at) {
        if (r < n) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (p.has(v)) {
                    copy_async(slot(at, v), a.x + r * a.ld + p.column(v));
                    copy_async(slot(at, v + V), a.g + r * a.ld_g + p.column(v));
                }
        }
        copies_end();
    };
#pragma unroll
    for (int i = 0; i < D - 1; ++i) fetch(first + (int64_t)i * step, i);
    const Param<T, V, L> w(p, a.weight, a.w_bf16, 1.f);
    Sums<T, V, L> sums;
    const float inv = 1.f / (float)a.dim;
    int at = 0;
    struct Next {
        float mu, rs;
        T xe, ge;
    } next = {};
    const auto load = [&](int64_t r) {
        if (r < n) next = {__ldg(a.mean + r), __ldg(a.rstd + r), p.load_end(a.x + r * a.ld, 0), p.load_end(a.g + r * a.ld_g, 0)};
    };
    load(first);
    for (int64_t r = first; r < n; r += step) {  // (the same in the whole group)
        fetch(r + (int64_t)(D - 1) * step, at ? at - 1 : D - 1);
        const Next cur = next;
        load(r + step);
        copies_wait<D - 1>();
        const T xe[1] = {cur.xe}, ge[1] = {cur.ge};
        grad_row<T, V, L>(
            a, p, w, sums, r, n, inv, sh, turn, cur.mu, cur.rs, xe, ge,
            [&](int v) { return p.has(v) ? *slot(at, v) : make_uint4(0, 0, 0, 0); },
            [&](int v) { return p.has(v) ? *slot(at, v + V) : make_uint4(0, 0, 0, 0); }, [] {});
        if (++at == D) at = 0;
    }
    if constexpr (L == 0 || L > 32) sums.put_block(p, a);
    else join_groups<T, V, L, NT, false>(sums, p, a, reinterpret_cast<float*>(ring));  // (its copies are all used)
}

// The blocks' sums in order: 32 columns a block, a 32nd of the blocks' sums a warp.
// heads: block p's vectors begin at the head of row p (x, its row stride in bytes).
__global__ void __launch_bounds__(1024) k_norm_join(const float* __restrict__ parts, int32_t count, int32_t dim, void* dweight,
                                                    void* dbias, int32_t bf16, uintptr_t x, int64_t ld_bytes, int32_t size,
                                                    int32_t heads) {
    pdl_start();
    __shared__ float sh[32][33];
    const int lane = (int)lane_id(), warp = (int)(threadIdx.x >> 5);
    const int32_t pitch = pitch_of(dim), o0 = (int32_t)blockIdx.x * 32, o = o0 + lane;
    float s = 0.f;
    if (o < 2 * dim) {
        const int32_t at = o < dim ? o : o - dim + pitch;
#pragma unroll 8
        for (int32_t p = warp; p < count; p += 32) {
            const int32_t off = heads ? (int32_t)((x + (uintptr_t)(p * ld_bytes)) & 15) : 0;
            s += parts[(int64_t)p * 2 * pitch + kLead - (off ? (16 - off) / size : 0) + at];
        }
    }
    sh[warp][lane] = s;
    __syncthreads();
    s = warp_sum(sh[lane][warp]);  // column `warp` of the block
    const int32_t i = o0 + warp < dim ? o0 + warp : o0 + warp - dim;
    if (lane != 0 || o0 + warp >= 2 * dim) return;
    void* to = o0 + warp < dim ? dweight : dbias;
    if (!to) return;
    if (bf16) put((__nv_bfloat16*)to + i, s);
    else put((float*)to + i, s);
}

// -------------------------------------------------------------------- host
constexpr int kMaxDim = SG_MAX_NORM_DIM;

// Blocks that fill the device, a multiple of 8.
int64_t all_blocks(int per_sm) { return (int64_t)num_sms() * per_sm / 8 * 8; }
// Blocks of the gradient at most, whatever the form: the workspace has room for them.
// (By the widths where by_size() changes its forms, which go by whole vectors: up to 7
// values more.  4,097 to 4,608 columns run two blocks an SM: 9,746 x 4104 fp32 79 us, with
// room for one 94; 19,526 x 4097 bf16 97, 124.)
int64_t max_parts(int32_t dim) { return all_blocks(dim < 1032 ? 12 : dim < 2056 ? 6 : dim < 4616 ? 3 : 1); }
unsigned grid_of(int64_t rows, int per_sm) {
    const int64_t most = all_blocks(per_sm);
    return (unsigned)(rows < most ? rows : most);
}
template <typename T>
unsigned grid_of(const BwdArgs<T>& a, int64_t rows, int per_sm) {
    const unsigned blocks = grid_of(rows, per_sm);
    return blocks < max_parts(a.dim) ? blocks : (unsigned)max_parts(a.dim);
}

template <typename T, int V, int L, int NT, int R>
sg_status go(const FwdArgs<T>& a, cudaStream_t s) {
    const unsigned blocks = grid_of(cdiv(a.n_cap, (L ? NT / (L ? L : 1) : 1) * R), NT == kThreads ? 4 : 1);
    SG_CUDA(launch_pdl(k_norm_fwd<T, V, L, NT, R>, dim3(blocks), dim3(NT), 0, s, a));
    return SG_OK;
}
template <typename T, int V, int L, int NT, int R>
sg_status go(const BwdArgs<T>& a, cudaStream_t s, int64_t* count, int32_t* heads) {
    constexpr int kRows = (L ? NT / (L ? L : 1) : 1) * R;
    *heads = 0;  // (by columns, or rows that are moved value by value)
    if constexpr (L > 0)
        if (a.n_cap <= kSmallTurns * kSmallCtas * kRows && a.parts) {
            *count = 0;  // the sums are done
            SG_CUDA(launch_cluster(k_norm_bwd<T, V, L, NT, R, true>, kSmallCtas, NT, kSmallCtas, s, 0, a));
            return SG_OK;
        }
    const unsigned blocks = grid_of(a, cdiv(a.n_cap, kRows), kBwdBlocks<T, NT>);
    *count = blocks;
    SG_CUDA(launch_pdl(k_norm_bwd<T, V, L, NT, R, false>, dim3(blocks), dim3(NT), 0, s, a));
    return SG_OK;
}

// Threads and shared memory of a ring's block, and blocks an SM.
struct Ring {
    int threads, bytes, per_sm;
};
template <typename T, int V, int L, int NT, int A>
Ring ring_of(int32_t dim) {
    const int vecs = dim / kE<T>, t = L == 32 ? NT : L ? L : (int)cdiv(vecs, 32 * V) * 32;  // (vectors at most)
    return {t, t * kDepth<T, V, A, NT> * V * A * 16, kRingThreads<V * kE<T>, A, NT> / t};
}
template <typename T, int V, int L, int NT>
sg_status go_ring(const FwdArgs<T>& a, cudaStream_t s) {
    const Ring r = ring_of<T, V, L, NT, 1>(a.dim);
    static OncePerDevice set;
    SG_CUDA(allow_smem(set, k_norm_fwd_ring<T, V, L, NT>, NT * kDepth<T, V, 1, NT> * V * 16));
    SG_CUDA(launch_pdl(k_norm_fwd_ring<T, V, L, NT>, dim3(grid_of(cdiv(a.n_cap, L == 32 ? NT / 32 : 1), r.per_sm)),
                       dim3(r.threads), r.bytes, s, a));
    return SG_OK;
}
template <typename T, int V, int L, int NT>
sg_status go_ring(const BwdArgs<T>& a, cudaStream_t s, int64_t* count, int32_t* heads) {
    const Ring r = ring_of<T, V, L, NT, 2>(a.dim);
    constexpr int kBytes = NT * kDepth<T, V, 2, NT> * V * 2 * 16;
    static_assert(L != 32 || NT / 32 * kGroupColumns<T, V, L> * 4 <= kBytes, "room for the groups' sums");
    static OncePerDevice set;
    SG_CUDA(allow_smem(set, k_norm_bwd_ring<T, V, L, NT>, kBytes));
    const unsigned blocks = grid_of(a, cdiv(a.n_cap, L == 32 ? NT / 32 : 1), r.per_sm);
    *count = blocks;
    *heads = L != 32;
    SG_CUDA(launch_pdl(k_norm_bwd_ring<T, V, L, NT>, dim3(blocks), dim3(r.threads), r.bytes, s, a));
    return SG_OK;
}

// The smallest group that holds a row's vectors.
template <typename T, typename A, typename... More>
sg_status by_size(const A& a, More... more) {
    constexpr int V = kHeld / kE<T>;
    const int32_t vecs = a.dim / kE<T> > 0 ? a.dim / kE<T> : 1;  // at most
    if (vecs <= 4) return go<T, 1, 4, kThreads, 1>(a, more...);
    if (vecs <= 8) return go<T, 1, 8, kThreads, 1>(a, more...);
    if (vecs <= 16) return go<T, 1, 16, kThreads, 2>(a, more...);
    if (vecs <= 32) return go<T, 1, 32, kThreads, 2>(a, more...);
    if (!a.alike) {
        if (vecs <= 64) return go<T, 2, 32, kThreads, 1>(a, more...);
        return go<T, V, 0, 1024, 1>(a, more...);
    }
    // a warp a row while there are rows for all warps: no barrier (us, by warps / by
    // blocks: backward 2000 x 400 fp32 11.9 / 14.5, 9000 x 400 11.9 / 21.0, 1000 x 400 12.2 /
    // 11.3; forward 5000 x 1000 fp32 9.4 / 8.6, 9000 x 1000 15.1 / 15.2)
    const bool many = a.n_cap >= (std::is_same_v<A, FwdArgs<T>> ? 64 : 8) * num_sms();
    if constexpr (std::is_same_v<A, FwdArgs<T>>) {
        if (vecs <= 64) return go_ring<T, 2, 32, kThreads>(a, more...);
        if (vecs <= 48 * V && many) return go_ring<T, 3 * V / 2, 32, kThreads>(a, more...);
        if (vecs <= 64 * V && many) return go_ring<T, 2 * V, 32, kThreads>(a, more...);
        if (vecs <= 64 * V && vecs > 48 * V) return go_ring<T, V, 64, kBlockThreads<1>>(a, more...);
        if (vecs <= 128 * V && vecs > 96 * V) return go_ring<T, V, 128, kBlockThreads<1>>(a, more...);
        if (vecs <= 256 * V && vecs > 192 * V) return go_ring<T, V, 256, kBlockThreads<1>>(a, more...);
        if (vecs <= kBlockThreads<1> * V) return go_ring<T, V, 0, kBlockThreads<1>>(a, more...);
    } else {
        if (vecs <= 64 && !many) return go<T, 2, 32, kThreads, 1>(a, more...);
        if (vecs <= 64) return go_ring<T, 2, 32, kThreads>(a, more...);
        if (vecs <= 32 * V && many) return go_ring<T, V, 32, kThreads>(a, more...);
        if (vecs <= 64 * V && vecs > 48 * V) return go_ring<T, V, 64, kBlockThreads<2>>(a, more...);
        if (vecs <= 128 * V && vecs > 96 * V) return go_ring<T, V, 128, kBlockThreads<2>>(a, more...);
        if (vecs <= 256 * V && vecs > 192 * V) return go_ring<T, V, 256, kBlockThreads<2>>(a, more...);
        if (vecs <= 512 * V && vecs > 384 * V) return go_ring<T, V, 512, kBlockThreads<2>>(a, more...);
        // (24 values a thread leave room for two blocks: 9,746 x 4104 fp32 79 us, by one of 16 140)
        if (vecs <= 288 * V && vecs > 256 * V) return go_ring<T, 3 * V / 2, 0, 192>(a, more...);
        if (vecs <= kBlockThreads<2> * V) return go_ring<T, V, 0, kBlockThreads<2>>(a, more...);
    }
    return go_ring<T, V, 0, 1024>(a, more...);
}

bool known(int32_t dtype) { return dtype == SG_F32 || dtype == SG_BF16; }
int size_of(int32_t dtype) { return dtype == SG_F32 ? 4 : 2; }

template <typename T>
sg_status bwd(const BwdArgs<T>& a, cudaStream_t s) {
    int64_t count = 0;
    int32_t heads = 0;
    if (a.n_cap > 0) {
        const sg_status st = by_size<T>(a, s, &count, &heads);
        if (st != SG_OK || count == 0) return st;
    }
    if (!a.parts) return SG_OK;
    SG_CUDA(launch_pdl(k_norm_join, dim3((unsigned)cdiv(2 * (int64_t)a.dim, 32)), dim3(1024), 0, s, (const float*)a.parts,
                       (int32_t)count, a.dim, a.dweight, a.dbias, a.w_bf16, (uintptr_t)a.x, a.ld * (int64_t)sizeof(T),
                       (int32_t)sizeof(T), heads));
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
    const int32_t alike = ((((uintptr_t)d_x - (uintptr_t)d_y) | (uintptr_t)((ld - ld_y) * e)) & 15) == 0;
    if (dtype == SG_F32) {
        const FwdArgs<float> a = {(const float*)d_x, (float*)d_y, ld, ld_y, d_weight, d_bias, d_n, n_cap, dim,
                                  dtype_w == SG_BF16, alike, eps, d_mean, d_rstd};
        return by_size<float>(a, s);
    }
    const FwdArgs<__nv_bfloat16> a = {(const __nv_bfloat16*)d_x, (__nv_bfloat16*)d_y, ld, ld_y, d_weight, d_bias, d_n,
                                      n_cap, dim, dtype_w == SG_BF16, alike, eps, d_mean, d_rstd};
    return by_size<__nv_bfloat16>(a, s);
}

extern "C" size_t sg_layernorm_bwd_workspace(int32_t n_cap, int32_t dim) {
    if (n_cap < 0 || dim <= 0 || dim > kMaxDim) return 0;
    int64_t parts = max_parts(dim);
    if (parts > n_cap) parts = n_cap;
    return (size_t)cdiv((parts > 0 ? parts : 1) * 2 * pitch_of(dim) * 4, 256) * 256;
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
    const int32_t alike = ((((uintptr_t)d_x - (uintptr_t)d_g) | ((uintptr_t)d_x - (uintptr_t)d_dx) |
                            (uintptr_t)((ld - ld_g) * e) | (uintptr_t)((ld - ld_dx) * e)) & 15) == 0;
    float* parts = d_dweight || d_dbias ? (float*)d_workspace : nullptr;
    if (dtype == SG_F32) {
        const BwdArgs<float> a = {(const float*)d_g, (const float*)d_x, (float*)d_dx, ld_g, ld, ld_dx, d_weight, d_mean,
                                  d_rstd, d_n, n_cap, dim, dtype_w == SG_BF16, alike, parts, d_dweight, d_dbias};
        return bwd<float>(a, s);
    }
    const BwdArgs<__nv_bfloat16> a = {(const __nv_bfloat16*)d_g, (const __nv_bfloat16*)d_x, (__nv_bfloat16*)d_dx, ld_g, ld,
                                      ld_dx, d_weight, d_mean, d_rstd, d_n, n_cap, dim, dtype_w == SG_BF16, alike, parts, d_dweight, d_dbias};
    return bwd<__nv_bfloat16>(a, s);
}
