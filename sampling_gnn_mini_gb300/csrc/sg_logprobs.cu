// What a model answers: per row of logits x the log probability of a given
// class, the entropy, and the k most probable classes.  With m = max_c x[c],
// d_c = m - x[c], z = sum_c exp(-d_c), t = sum_c exp(-d_c) (-d_c):
//   logp = -d_label - log z,  entropy = log z - t / z,
//   the k largest by (x descending, class ascending) with their log probabilities.
// The logits are read once and next to nothing is written; beside the bytes an
// exponential a logit counts (16 a cycle and SM: at 2 bytes a logit three quarters of the
// copy rate's time).
//
// Many rows of up to 128 classes go through shared memory to a thread each
// (k_logprobs_few).  Rows of up to 2,048 vectors of 16 bytes stay in the registers of 1,
// 2 or 4 warps (k_logprobs_warp).  Longer ones stream past 128 or 256 threads, or a
// cluster of 2 to 8 such CTAs when rows are few (k_logprobs_row): each thread copies its
// own vectors asynchronously, those of the next row already while this row's classes are
// chosen, and keeps (m, z, t) of what it has seen, relative to its own running maximum.
//
// The k best are chosen through a bound: the k-th largest of some maxima (of lanes,
// threads or groups of vectors) is a lower bound of the k-th largest logit, so only
// vectors that reach it are read again (from L2), and only the logits that reach it
// become candidates: about k of them, whatever the row's length.  Where they are more
// than the list holds (equal logits, masks by one value), the bound is raised by bisection
// over the row, and logits equal to it are taken in order.
//
// Logits of -inf take no part.  x - m is formed before the scaling by log2(e), so
// a row's level costs no accuracy, and exponents are cut off at -200, where the
// exponential is 0, so that 0 * (-inf) never arises.
#include <type_traits>

#include "sg_internal.cuh"
#include "sg_rows.cuh"
#include "sg_tc.cuh"

SGI_ERROR_WORD(logprobs)

using namespace sgi;

namespace {

constexpr int kThreads = 256;  // of a block of warps' rows
constexpr int kTurn = 4;      // vectors a thread takes at a time
constexpr int kRing = 2;      // turns of them in shared memory
constexpr int kGroups = 16;   // groups of a thread's vectors, at most
// Candidates that a CTA of NT threads holds, and groups it reads again.
template <int NT>
constexpr int kCap = NT < 256 ? 2 * SG_MAX_TOP : 4 * SG_MAX_TOP;
constexpr int kWarpCap = 256; // candidates a warp holds
constexpr float kNone = -200.f;  // 2^x is 0 from here on

template <typename T>
struct Args {
    const T* x;
    int64_t ld;
    const int32_t* labels;
    const int32_t* d_n;
    int32_t n_cap, classes, k;
    float* logp;
    float* entropy;
    int32_t* top_ids;
    float* top_logp;
};

// The larger of two, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Order of values as whole numbers (-0 with 0; no NaN).
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
constexpr uint32_t kOrderNone = 0x007FFFFFu;  // of -inf
// A candidate: the larger one is the better (larger logit, then lower class).
__device__ __forceinline__ unsigned long long entry_of(uint32_t order, int32_t c) {
    return (unsigned long long)order << 32 | (0xFFFFFFFFu - (uint32_t)c);
}
__device__ __forceinline__ int32_t class_of(unsigned long long e) { return (int32_t)(0xFFFFFFFFu - (uint32_t)e); }

// z = sum exp(x - m), t = sum exp(x - m) (x - m) log2(e) of a part of a row; m = -inf: nothing yet
struct Stat {
    float m, z, t;
};
__device__ __forceinline__ float finite_base(float m) { return m == -INFINITY ? 0.f : m; }
// s relative to the maximum m >= s.m
__device__ __forceinline__ void rebase(Stat& s, float m) {
    const float a = fmaxf((s.m - finite_base(m)) * kLog2e, kNone), e = ex2(a);
    s.t = e * fmaf(a, s.z, s.t);
    s.z *= e;
    s.m = m;
}
__device__ __forceinline__ Stat stat_of(float x) {
    return {x, x == -INFINITY ? 0.f : 1.f + (x - x), 0.f};  // (NaN and +inf: z = NaN)
}
// Adds a vector; s.m is at least its maximum.
template <typename T>
__device__ __forceinline__ void add_part(const uint4& u, f2 base, f2& z, f2& t) {
    f2 p[kE<T> / 2];
    pairs_of(u, p);
    const f2 l = pair(kLog2e, kLog2e);
#pragma unroll
    for (int i = 0; i < kE<T> / 2; ++i) {
        float a, c;
        unpair(mul2(add2(p[i], base), l), a, c);
        a = max_nan(a, kNone);
        c = max_nan(c, kNone);
        const f2 e = pair(ex2(a), ex2(c));
        z = add2(z, e);
        t = fma2(e, pair(a, c), t);
    }
}
__device__ __forceinline__ Stat warp_join(Stat s) {
    rebase(s, warp_max(s.m));
    s.z = warp_sum(s.z);
    s.t = warp_sum(s.t);
    return s;
}
__device__ __forceinline__ float logp_of(float x, float m, float log_z) {
    return (x - finite_base(m)) - log_z;
}

// The row's label, -1 if there is none.
template <typename T>
__device__ __forceinline__ int32_t label_of(const Args<T>& a, int32_t r) {
    const int32_t y = a.labels ? __ldg(a.labels + r) : -1;
    if (y >= -1 && y < a.classes) return y;
    dev_err(ERR_INDEX);
    return -1;
}

// One thread: the row's own numbers.
template <typename T>
__device__ __forceinline__ void put_row(const Args<T>& a, int32_t r, const Stat& s, float log_z, int32_t y, float xy) {
    if (a.logp) a.logp[r] = y < 0 ? 0.f : s.z == 0.f ? -INFINITY : logp_of(xy, s.m, log_z);
    if (a.entropy) a.entropy[r] = s.z == 0.f ? 0.f : log_z - s.t / s.z * 0.69314718055994531f;
}

// Descending over the warp's lanes.
__device__ __forceinline__ float warp_sort(float x) {
    const int lane = (int)lane_id();
#pragma unroll
    for (int size = 2; size <= 32; size *= 2)
#pragma unroll
        for (int d = size / 2; d > 0; d /= 2) {
            const float o = __shfl_xor_sync(0xFFFFFFFFu, x, d);
            const bool larger = ((lane & d) == 0) == ((lane & size) == 0);  // this lane keeps the larger one
            x = larger ? fmaxf(x, o) : fminf(x, o);
        }
    return x;
}

// The largest element of several vectors (bf16: pairwise on the packed elements).
template <typename T, int N>
__device__ __forceinline__ float parts_max(const uint4 (&u)[N]) {
    if constexpr (sizeof(T) == 2) {
        const auto h = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
        __nv_bfloat162 m = __hmax2(__hmax2(h(u[0].x), h(u[0].y)), __hmax2(h(u[0].z), h(u[0].w)));
#pragma unroll
        for (int k = 1; k < N; ++k) m = __hmax2(m, __hmax2(__hmax2(h(u[k].x), h(u[k].y)), __hmax2(h(u[k].z), h(u[k].w))));
        return fmaxf(__low2float(m), __high2float(m));
    }
    float m = part_max<T>(u[0]);
#pragma unroll
    for (int k = 1; k < N; ++k) m = fmaxf(m, part_max<T>(u[k]));
    return m;
}
// Elements of a vector, one at a time.
template <typename T>
__device__ __forceinline__ void unpack(const uint4& u, float (&f)[kE<T>]) {
    f2 p[kE<T> / 2];
    pairs_of(u, p);
#pragma unroll
    for (int i = 0; i < kE<T> / 2; ++i) unpair(p[i], f[2 * i], f[2 * i + 1]);
}

// ------------------------------------------------------------ rows by threads
// kFewRows rows of up to kFewClasses classes to a block, in shared memory, then a
// thread a row.  A thread's top K sit in registers in order: a logit moves in where it
// is larger, so that equal ones stay in the order of their classes.  For K > 1 only the
// logits that reach the K-th largest of 8 or 16 groups' maxima are tried, some K + 2 of
// them: the pass that finds the row's maximum finds the groups', the pass that adds up the
// exponentials marks them (us, 200,001 x 47 fp32 k = 3 15.3, each logit tried 17.9; k = 8
// 24, 32).  The rows are copied
//   by vectors when every row is on 16 bytes, at an odd pitch of vectors, filled up
//              with -inf (threads that read a vector each meet different banks);
//   whole      when they follow one another from a 16-byte boundary (threads that
//              read one element each meet at most in twos: the length is no multiple
//              of 16 bytes);
//   by values  if neither, at an odd pitch (up to kFewByValues classes: the index
//              arithmetic costs more than a warp a row from there on).
// us, fp32, this / a warp a row: 200,000 x 47 k = 1 13 / 80, k = 3 15 / 102, k = 8 24 /
// 115; 100,000 x 128 k = 1 15 / 42, k = 5 24 / 54; 25,000 x 128 k = 1 7.3 / 11, k = 8 11 / 15.
// It does not matter how many rows a block has (32 to 192).
constexpr int kFewRows = 64, kFewClasses = 128, kFewByValues = 64, kFewTop = 8;
enum Few { kWhole, kByVectors, kByValues };

// Rows in shared memory: elements to f(value, class), in order.
template <typename T, Few HOW, typename F>
__device__ __forceinline__ void few_each(const uint4* smem, int32_t pitch, int32_t classes, F f) {
    if constexpr (HOW == kByVectors) {
        const uint4* row = smem + (int32_t)threadIdx.x * pitch;
#pragma unroll 2
        for (int32_t v = 0; v * kE<T> < classes; ++v) {
            float e[kE<T>];
            unpack<T>(row[v], e);
#pragma unroll
            for (int i = 0; i < kE<T>; ++i) f(e[i], v * kE<T> + i);
        }
    } else {
        typedef std::conditional_t<HOW == kWhole, T, float> M;
        const M* row = reinterpret_cast<const M*>(smem) + (int32_t)threadIdx.x * pitch;
#pragma unroll 4
        for (int32_t c = 0; c < classes; ++c) f(to_f(row[c]), c);
    }
}

// This thread's element of a class.
template <typename T, Few HOW>
__device__ __forceinline__ float few_at(const uint4* smem, int32_t pitch, int32_t c) {
    typedef std::conditional_t<HOW == kByValues, float, T> M;
    return to_f(reinterpret_cast<const M*>(smem)[(int32_t)threadIdx.x * pitch * (HOW == kByVectors ? kE<T> : 1) + c]);
}
// Elements to f(value, class mod G).
template <typename T, Few HOW, int G, typename F>
__device__ __forceinline__ void few_groups(const uint4* smem, int32_t pitch, int32_t classes, F f) {
    int32_t c = 0;
    if constexpr (HOW == kByVectors) {
        const uint4* row = smem + (int32_t)threadIdx.x * pitch;
        for (; c < classes; c += G)
#pragma unroll
            for (int v = 0; v < G / kE<T>; ++v) {
                if (v > 0 && c + v * kE<T> >= classes) break;
                float e[kE<T>];
                unpack<T>(row[c / kE<T> + v], e);
#pragma unroll
                for (int i = 0; i < kE<T>; ++i) f(e[i], v * kE<T> + i);
            }
    } else {
        for (; c + G <= classes; c += G)
#pragma unroll
            for (int j = 0; j < G; ++j) f(few_at<T, HOW>(smem, pitch, c + j), j);
#pragma unroll
        for (int j = 0; j < G; ++j)
            if (c + j < classes) f(few_at<T, HOW>(smem, pitch, c + j), j);
    }
}
// Elements to take(value); those for which it is true to f(value, class), in order.
template <typename T, Few HOW, typename Take, typename F>
__device__ __forceinline__ void few_bits(const uint4* smem, int32_t pitch, int32_t classes, Take take, F f) {
    for (int32_t c0 = 0; c0 < classes; c0 += 32) {
        uint32_t bits = 0;
        const int32_t most = min(32, classes - c0);
        if constexpr (HOW == kByVectors) {
            const uint4* row = smem + (int32_t)threadIdx.x * pitch + c0 / kE<T>;
            for (int32_t q = 0; q < most; q += 8) {
                uint32_t part = 0;
#pragma unroll
                for (int v = 0; v < 8 / kE<T>; ++v) {
                    if (v > 0 && q + v * kE<T> >= most) break;
                    float e[kE<T>];
                    unpack<T>(row[q / kE<T> + v], e);
#pragma unroll
                    for (int i = 0; i < kE<T>; ++i)
                        if (take(e[i])) part |= 1u << (v * kE<T> + i);
                }
                bits |= part << q;
            }
        } else {
            int32_t q = 0;
            for (; q + 8 <= most; q += 8) {
                uint32_t part = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (take(few_at<T, HOW>(smem, pitch, c0 + q + i))) part |= 1u << i;
                bits |= part << q;
            }
            for (; q < most; ++q)
                if (take(few_at<T, HOW>(smem, pitch, c0 + q))) bits |= 1u << q;
        }
        while (bits) {
            const int32_t c = c0 + __ffs((int)bits) - 1;
            bits &= bits - 1;
            f(few_at<T, HOW>(smem, pitch, c), c);
        }
    }
}

// pitch: of rows in shared memory (vectors or elements); magic: ceil(2^32 / d), d > 1 the
// whole vectors or the elements of a row (i / d is exact for the i < 2^14 here)
template <typename T, int K, Few HOW>
__global__ void __launch_bounds__(kFewRows) k_logprobs_few(Args<T> a, int32_t pitch, uint32_t magic) {
    extern __shared__ __align__(16) uint4 few_smem[];
    pdl_start();
    const int32_t n = rows_of(a.d_n, a.n_cap), r0 = (int32_t)blockIdx.x * kFewRows, classes = a.classes;
    if (r0 >= n) return;
    const int32_t rows = min(kFewRows, n - r0);
    const T* x = a.x + (int64_t)r0 * a.ld;
    if constexpr (HOW == kWhole) {
        T* to = reinterpret_cast<T*>(few_smem);
        const int32_t all = rows * classes, vecs = all / kE<T>;
        for (int32_t i = (int32_t)threadIdx.x; i < vecs; i += kFewRows) copy_async(few_smem + i, x + i * kE<T>);
        const int32_t i = vecs * kE<T> + (int32_t)threadIdx.x;
        if (i < all) to[i] = x[i];
    } else if constexpr (HOW == kByVectors) {
        const int32_t vecs = classes / kE<T>, all = rows * vecs;
        for (int32_t i = (int32_t)threadIdx.x; i < all; i += kFewRows) {
            const int32_t row = vecs == 1 ? i : (int32_t)__umulhi((uint32_t)i, magic), v = i - row * vecs;
            copy_async(few_smem + row * pitch + v, x + row * a.ld + v * kE<T>);
        }
        if (vecs * kE<T> < classes && (int32_t)threadIdx.x < rows) {  // a thread's own row
            uint4 u = empty_part<T>();
            T* e = reinterpret_cast<T*>(&u);
#pragma unroll
            for (int i = 0; i < kE<T>; ++i)
                if (vecs * kE<T> + i < classes) e[i] = x[(int32_t)threadIdx.x * a.ld + vecs * kE<T> + i];
            few_smem[(int32_t)threadIdx.x * pitch + vecs] = u;
        }
    } else {
        float* to = reinterpret_cast<float*>(few_smem);
        const int32_t all = rows * classes;
        for (int32_t i0 = (int32_t)threadIdx.x; i0 < all; i0 += 8 * kFewRows) {
            T v[8];
            int32_t at[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int32_t i = i0 + u * kFewRows;
                const int32_t row = (int32_t)__umulhi((uint32_t)i, magic), c = i - row * classes;
                at[u] = i < all ? row * pitch + c : -1;
                if (i < all) v[u] = x[row * a.ld + c];
            }
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (at[u] >= 0) to[at[u]] = to_f(v[u]);
        }
    }
    copies_end();
    copies_wait<0>();
    __syncthreads();
    const int32_t r = r0 + (int32_t)threadIdx.x;
    if (r >= n) return;
    const int32_t y = label_of(a, r);
    const float xy = y >= 0 ? to_f(a.x[(int64_t)r * a.ld + y]) : 0.f;
    float top[K];
    int32_t at[K];
#pragma unroll
    for (int j = 0; j < K; ++j) top[j] = -INFINITY, at[j] = -1;
    const auto insert = [&](float v, int32_t c) {
        if (v > top[K - 1]) {  // the entries below it move down, equal ones above it stay
#pragma unroll
            for (int j = K - 1; j > 0; --j) {
                const bool down = v > top[j - 1], here = v > top[j];
                at[j] = down ? at[j - 1] : here ? c : at[j];
                top[j] = down ? top[j - 1] : here ? v : top[j];
            }
            if (v > top[0]) top[0] = v, at[0] = c;
        }
    };
    Stat s = {-INFINITY, 0.f, 0.f};
    if constexpr (K == 1) {
        few_each<T, HOW>(few_smem, pitch, classes, insert);
        s.m = top[0];
        const float b = finite_base(s.m);
        few_each<T, HOW>(few_smem, pitch, classes, [&](float v, int32_t) {
            const float d = max_nan((v - b) * kLog2e, kNone), e = ex2(d);
            s.z += e;
            s.t = fmaf(e, d, s.t);
        });
    } else {
        constexpr int G = K <= 4 ? 8 : 16;
        float g[G];
#pragma unroll
        for (int j = 0; j < G; ++j) g[j] = -INFINITY;
        few_groups<T, HOW, G>(few_smem, pitch, classes, [&](float v, int j) { g[j] = fmaxf(g[j], v); });
#pragma unroll
        for (int size = 2; size <= G; size *= 2)
#pragma unroll
            for (int d = size / 2; d > 0; d /= 2)
#pragma unroll
                for (int i = 0; i < G; ++i)
                    if ((i & d) == 0) {
                        const float x = g[i], y = g[i + d];
                        g[i] = (i & size) == 0 ? fmaxf(x, y) : fminf(x, y);
                        g[i + d] = (i & size) == 0 ? fminf(x, y) : fmaxf(x, y);
                    }
        s.m = g[0];
        const float b = finite_base(s.m), bound = fmaxf(g[K - 1], -3.402823466e38f);
        few_bits<T, HOW>(few_smem, pitch, classes, [&](float v) {
            const float d = max_nan((v - b) * kLog2e, kNone), e = ex2(d);
            s.z += e;
            s.t = fmaf(e, d, s.t);
            return v >= bound;
        }, insert);
    }
    const float log_z = logf(s.z);
    put_row(a, r, s, log_z, y, xy);
    const bool bad = s.z != s.z;
    int32_t* ids = a.top_ids + (int64_t)r * a.k;
    float* lps = a.top_logp + (int64_t)r * a.k;
#pragma unroll
    for (int j = 0; j < K; ++j)
        if (j < a.k) {
            ids[j] = bad ? -1 : at[j];
            lps[j] = bad ? s.z : at[j] < 0 ? -INFINITY : logp_of(top[j], s.m, log_z);
        }
}

// -------------------------------------------------------------- rows by warps
// A candidate as a number (the larger one is the better): the value's order, then the
// class from the last one on.  bf16 values have 16 bits, rows of warps fewer than 2^16
// classes.
template <typename T>
using Key = std::conditional_t<sizeof(T) == 2, uint32_t, unsigned long long>;
template <typename T>
__device__ __forceinline__ Key<T> key_of(float x, int32_t c) {
    if constexpr (sizeof(T) == 2) return (order_of(x) & 0xFFFF0000u) | (0xFFFFu - (uint32_t)c);
    else return entry_of(order_of(x), c);
}
__device__ __forceinline__ int32_t key_class(uint32_t e) { return (int32_t)(0xFFFFu - (e & 0xFFFFu)); }
__device__ __forceinline__ int32_t key_class(unsigned long long e) { return class_of(e); }
// (a negative value's order has ones below its 16 bits)
__device__ __forceinline__ float key_value(uint32_t e) { return value_of(e & 0x80000000u ? e & 0xFFFF0000u : e | 0xFFFFu); }
__device__ __forceinline__ float key_value(unsigned long long e) { return value_of((uint32_t)(e >> 32)); }

// The maxima of a lane's vectors' parts of PER elements, G in all, as orders.
template <typename T, int PER, int NV, int G>
__device__ __forceinline__ void group_orders(const uint4 (&x)[NV], uint32_t (&g)[G]) {
    constexpr int EACH = kE<T> / PER;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        float f[kE<T>];
        unpack<T>(x[k], f);
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            float m = f[i * PER];
#pragma unroll
            for (int e = 1; e < PER; ++e) m = fmaxf(m, f[i * PER + e]);
            g[k * EACH + i] = order_of(m);
        }
    }
}
// A lower bound of the k-th largest order: the largest found by bisection that at
// least k of the lanes' G maxima reach (the lowest order if they are fewer).
template <int G>
__device__ __forceinline__ uint32_t bound_of(const uint32_t (&g)[G], int32_t k, uint32_t top) {
    const auto reach = [&](uint32_t o) {
        int32_t c = 0;
#pragma unroll
        for (int i = 0; i < G; ++i) c += g[i] >= o;
        return __reduce_add_sync(0xFFFFFFFFu, c);
    };
    uint32_t lo = g[0], hi = top + 1;
#pragma unroll
    for (int i = 1; i < G; ++i) lo = min(lo, g[i]);
    lo = __reduce_min_sync(0xFFFFFFFFu, lo);
    if (lo <= kOrderNone) {
        lo = kOrderNone + 1;
        if (reach(lo) < k) return lo;
    }
    while (hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        const int32_t c = reach(mid);
        if (c < k) {
            hi = mid;
        } else {
            lo = mid;
            if (c <= k + k / 8) break;
        }
    }
    return lo;
}

// The k best of a row of which more than kWarpCap logits have order o and above, as
// keys in `list`, which they fit; returns their number.  top: an order that none is
// above.  Each pass reads the row again.
template <typename T>
__device__ __noinline__ int32_t select_by_warp(const T* row, int32_t classes, int32_t k, uint32_t o, uint32_t top, Key<T>* list) {
    const int lane = (int)lane_id();
    const uint32_t below = (1u << lane) - 1u;
    const auto order_at = [&](int32_t c) { return c < classes ? order_of(to_f(row[c])) : 0u; };
    const auto count = [&](uint32_t from) {
        int32_t c = 0;
#pragma unroll 4
        for (int32_t i = lane; i < classes; i += 32) c += order_at(i) >= from;
        return __reduce_add_sync(0xFFFFFFFFu, c);
    };
    uint32_t lo = o, hi = top + 1;  // at least k from lo on, fewer from hi on
    int32_t have = kWarpCap + 1;
    for (uint32_t mid = lo + 1; have > kWarpCap && hi - lo > 1; mid = lo + (hi - lo) / 2) {
        const int32_t c = count(mid);
        if (c >= k) lo = mid, have = c;
        else hi = mid;
    }
    // all from lo on or, of those that are equal to lo, the lowest classes
    const bool all = have <= kWarpCap;
    int32_t found = 0;
    for (int pass = 0; pass < (all ? 1 : 2); ++pass)
        for (int32_t c0 = 0; c0 < classes && (pass == 0 || found < k); c0 += 32) {
            const uint32_t at = order_at(c0 + lane);
            const bool take = all ? at >= lo : pass == 0 ? at > lo : at == lo;
            const uint32_t mask = __ballot_sync(0xFFFFFFFFu, take);
            const int32_t to = found + __popc(mask & below);
            if (take && to < (pass ? k : kWarpCap)) list[to] = key_of<T>(value_of(at), c0 + lane);
            found += __popc(mask);
        }
    __syncwarp();
    return all ? found : min(found, k);
}

// Room in a list for a warp's entries, `mine` of them this lane's: where they begin.
__device__ __forceinline__ int32_t reserve(int32_t mine, int32_t* count) {
    const int32_t upto = warp_incl_scan(mine), all = __shfl_sync(0xFFFFFFFFu, upto, 31);
    int32_t at = 0;
    if (lane_id() == 0 && all > 0) at = atomicAdd(count, all);
    return __shfl_sync(0xFFFFFFFFu, at, 0) + upto - mine;
}

// A warp's list in order, P keys a lane (bitonic; key lane P + i in e[i]), its first k
// written.
template <typename T, int P>
__device__ __forceinline__ void put_sorted(const Key<T>* list, int32_t found, int32_t k, float m, float log_z, int32_t* ids,
                                           float* lps) {
    const int lane = (int)lane_id();
    Key<T> e[P];
#pragma unroll
    for (int i = 0; i < P; ++i) e[i] = lane * P + i < found ? list[lane * P + i] : 0;
#pragma unroll
    for (int size = 2; size <= 32 * P; size *= 2)
#pragma unroll
        for (int d = size / 2; d > 0; d /= 2) {
            if (d >= P) {
                const bool larger = ((lane & d / P) == 0) == ((lane * P & size) == 0);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const Key<T> o = __shfl_xor_sync(0xFFFFFFFFu, e[i], d / P);
                    e[i] = larger == (o > e[i]) ? o : e[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < P; ++i)
                    if ((i & d) == 0) {
                        const bool down = ((lane * P + i) & size) == 0;
                        const Key<T> x = e[i], y = e[i + d];
                        e[i] = down == (x > y) ? x : y;
                        e[i + d] = down == (x > y) ? y : x;
                    }
            }
        }
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int32_t j = lane * P + i;
        if (j < min(found, k)) {
            ids[j] = key_class(e[i]);
            lps[j] = logp_of(key_value(e[i]), m, log_z);
        }
    }
}

// W warps a row, in NV vectors a lane.  The bound of the k best: each warp's k-th of
// its lanes' maxima is one, and the lowest of the warps' ceil(k / W)-th is one, by a
// sort for up to kBySort, else by bisection over a warp's 256 or 512 groups' maxima.
// The vectors that reach the better one are read again, a lane each, and their logits
// that do are listed and put in order.  us, 40,000 x 2000 bf16: 33 without top classes, 43
// for 1, 49 for 5, 58 for 20, 126 for 100 (taken one by one from orders of all logits in
// registers, at half the warps an SM: 69, 119, 174, 210, 429).  By bisection 20 take
// 72, by a sort 32 take 122 (78): too many logits reach the lowest of 32 maxima.
constexpr int kBySort = 24;
template <int W>
constexpr int kWarpThreads = W == 1 ? kThreads : 32 * W;  // of a block: 8 rows or one

template <typename T, int NV, int W>
__global__ void __launch_bounds__(kWarpThreads<W>, (NV <= 2 ? 48 : NV == 4 ? 40 : NV == 8 ? 32 : NV == 12 ? 28 : 24) * 32 / kWarpThreads<W>)
    k_logprobs_warp(Args<T> a) {
    pdl_start();
    constexpr int kRows = kWarpThreads<W> / 32 / W;
    __shared__ Key<T> lists[kRows][kWarpCap];
    __shared__ uint16_t hit_lists[kRows * W][32 * NV];
    __shared__ float4 parts[W];
    __shared__ float2 bounds[W];
    __shared__ int32_t counts[kRows];
    const int lane = (int)lane_id(), warp = (int)(threadIdx.x >> 5), rank = W == 1 ? 0 : warp;
    const int32_t n = rows_of(a.d_n, a.n_cap), r = (int32_t)blockIdx.x * kRows + warp / W;
    if (r >= n) return;  // all of the row's warps
    const T* row = a.x + (int64_t)r * a.ld;
    const RowParts<T> part(row, a.classes);
    const int32_t first = rank * 32 + lane;  // vector of x[0], the others 32 W apart
    uint4 x[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int32_t v = first + 32 * W * k;
        x[k] = v < part.vecs ? *reinterpret_cast<const uint4*>(row + part.head + v * kE<T>) : empty_part<T>();
    }
    const int32_t ce = rank == 0 ? part.edge(lane) : -1;
    const float xe = ce >= 0 ? to_f(row[ce]) : -INFINITY;
    int32_t y = -1;
    float xy = 0.f;
    if (rank == 0 && lane == 0) {
        counts[warp / W] = 0;
        y = label_of(a, r);
        if (y >= 0) xy = to_f(row[y]);
    }
    Stat s = stat_of(xe);
    float vm[NV], top = xe;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        vm[k] = part_max<T>(x[k]);
        top = fmaxf(top, vm[k]);
    }
    rebase(s, warp_max(top));
    f2 z = pair(s.z, 0.f), t = pair(s.t, 0.f);
    const float b = -finite_base(s.m);
#pragma unroll
    for (int k = 0; k < NV; ++k) add_part<T>(x[k], pair(b, b), z, t);
    float z0, z1, t0, t1;
    unpair(z, z0, z1);
    unpair(t, t0, t1);
    s.z = warp_sum(z0 + z1);
    s.t = warp_sum(t0 + t1);
    const int32_t need = (a.k + W - 1) / W;
    float tau = s.m;
    const auto bisect = [&] {
        constexpr int PER = NV > 8 ? kE<T> : kE<T> * NV >= 8 ? kE<T> * NV / 8 : 1;
        uint32_t g[kE<T> * NV / PER];
        if constexpr (PER == kE<T>) {
#pragma unroll
            for (int k = 0; k < NV; ++k) g[k] = order_of(vm[k]);
        } else {
#pragma unroll
            for (int k = 0; k < NV; ++k) repack(x[k]);
            group_orders<T, PER>(x, g);
        }
        g[0] = max(g[0], order_of(xe));
        tau = value_of(bound_of(g, need, order_of(s.m)));
    };
    if constexpr (W > 1) {
        float other = -INFINITY;  // the other bound
        if (a.k > 1) {
            const float in_order = warp_sort(top);
            if (a.k <= 32) other = __shfl_sync(0xFFFFFFFFu, in_order, a.k - 1);
            if (need <= kBySort) tau = __shfl_sync(0xFFFFFFFFu, in_order, need - 1);
            else bisect();
        } else {
            other = s.m;
        }
        if (lane == 0) {
            parts[rank] = make_float4(s.m, s.z, s.t, 0.f);
            bounds[rank] = make_float2(tau, other);
        }
        __syncthreads();
        s = {-INFINITY, 0.f, 0.f};
        tau = INFINITY, other = -INFINITY;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const float4 p = parts[i];
            Stat o = {p.x, p.y, p.z};
            const float m = fmaxf(s.m, o.m);
            rebase(s, m);
            rebase(o, m);
            s.z += o.z;
            s.t += o.t;
            tau = fminf(tau, bounds[i].x);
            other = fmaxf(other, bounds[i].y);
        }
        tau = fmaxf(tau, other);
    }
    const float log_z = logf(s.z);
    if (rank == 0 && lane == 0) put_row(a, r, s, log_z, y, xy);
    if (a.k == 0) return;
    int32_t* ids = a.top_ids + (int64_t)r * a.k;
    float* lps = a.top_logp + (int64_t)r * a.k;
    if (s.z != s.z) {
        if (rank == 0)
            for (int32_t i = lane; i < a.k; i += 32) ids[i] = -1, lps[i] = s.z;
        return;
    }
    if (W == 1 && a.k > 1) {
        if (a.k > kBySort) bisect();
        else tau = __shfl_sync(0xFFFFFFFFu, warp_sort(top), a.k - 1);
    }
    tau = fmaxf(tau, -3.402823466e38f);  // (-inf takes no part)
    uint16_t* hits = hit_lists[warp];
    Key<T>* list = lists[warp / W];
    int32_t hit = 0, found = 0;  // found: of this warp, W = 1
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, vm[k] >= tau);
        if (vm[k] >= tau) hits[hit + __popc(mask & ((1u << lane) - 1u))] = (uint16_t)(first + 32 * W * k);
        hit += __popc(mask);
    }
    const auto room = [&](int32_t mine) {
        if constexpr (W > 1) return reserve(mine, &counts[0]);
        const int32_t upto = warp_incl_scan(mine), at = found + upto - mine;
        found += __shfl_sync(0xFFFFFFFFu, upto, 31);
        return at;
    };
    if (rank == 0 && part.head + part.tail > 0) {
        const int32_t at = room(xe >= tau);
        if (xe >= tau && at < kWarpCap) list[at] = key_of<T>(xe, ce);
    }
    __syncwarp();
    for (int32_t q = 0; q < hit; q += 32) {
        uint4 u = empty_part<T>();
        int32_t c = 0;
        if (q + lane < hit) {
            c = part.head + hits[q + lane] * kE<T>;
            u = *reinterpret_cast<const uint4*>(row + c);
        }
        float f[kE<T>];
        unpack<T>(u, f);
        int32_t mine = 0;
#pragma unroll
        for (int e = 0; e < kE<T>; ++e) mine += f[e] >= tau;
        int32_t at = room(mine);
#pragma unroll
        for (int e = 0; e < kE<T>; ++e)
            if (f[e] >= tau) {
                if (at < kWarpCap) list[at] = key_of<T>(f[e], c + e);
                ++at;
            }
    }
    if constexpr (W == 1) {
        __syncwarp();
    } else {
        __syncthreads();
        if (rank != 0) return;
        found = counts[0];
    }
    if (found > kWarpCap) found = select_by_warp<T>(row, a.classes, a.k, order_of(tau), order_of(s.m), list);
    if (found <= 32) {  // by counting: a lane's key and the ones before it
        const Key<T> e = lane < found ? list[lane] : 0;
        int32_t before = 0;
#pragma unroll 4
        for (int32_t q = 0; q < found; ++q) before += list[q] > e;
        if (lane < found && before < a.k) {
            ids[before] = key_class(e);
            lps[before] = logp_of(key_value(e), s.m, log_z);
        }
    } else if (found <= 64) {
        put_sorted<T, 2>(list, found, a.k, s.m, log_z, ids, lps);
    } else if (found <= 128) {
        put_sorted<T, 4>(list, found, a.k, s.m, log_z, ids, lps);
    } else {
        put_sorted<T, 8>(list, found, a.k, s.m, log_z, ids, lps);
    }
    for (int32_t i = found + lane; i < a.k; i += 32) ids[i] = -1, lps[i] = -INFINITY;
}

// --------------------------------------------------------- rows by clusters
// The candidates of a CTA's part of a row.
template <int CAP>
struct Candidates {
    unsigned long long __align__(16) e[CAP];
    int32_t count;
};
template <int CAP>
__device__ __forceinline__ void offer(Candidates<CAP>& l, float x, int32_t c) {
    const int32_t at = atomicAdd(&l.count, 1);
    if (at < CAP) l.e[at] = entry_of(order_of(x), c);
}

// A CTA's part of a row: vectors v0 .. v0 + count - 1, and for warp 0 of CTA 0 the
// edge elements.
template <typename T>
struct Slice {
    const T* row;
    RowParts<T> part;
    int32_t v0, count, edge;
    float xe;
    __device__ __forceinline__ int32_t first(int32_t i) const { return part.head + (v0 + i) * kE<T>; }
    __device__ __forceinline__ uint4 load(int32_t i) const { return *reinterpret_cast<const uint4*>(row + first(i)); }
};

// Logits of the slice of order o and above (o above that of -inf), over the block.
template <int NT, typename T>
__device__ __noinline__ int32_t count_from(const Slice<T>& s, uint32_t o, int32_t* sh) {
    int32_t c = s.edge >= 0 && order_of(s.xe) >= o;
    for (int32_t i = threadIdx.x; i < s.count; i += NT) {
        float f[kE<T>];
        unpack<T>(s.load(i), f);
#pragma unroll
        for (int e = 0; e < kE<T>; ++e) c += order_of(f[e]) >= o;
    }
    return block_sum<NT, int32_t>(c, sh);
}
template <int NT, typename T, int CAP>
__device__ __noinline__ void offer_from(const Slice<T>& s, uint32_t o, Candidates<CAP>& l) {
    if (s.edge >= 0 && order_of(s.xe) >= o) offer(l, s.xe, s.edge);
    for (int32_t i = threadIdx.x; i < s.count; i += NT) {
        float f[kE<T>];
        unpack<T>(s.load(i), f);
#pragma unroll
        for (int e = 0; e < kE<T>; ++e)
            if (order_of(f[e]) >= o) offer(l, f[e], s.first(i) + e);
    }
}

// The slice's k best when more than CAP of its logits have order o and above:
// l.count is k at the end.  top: an order that none is above.  Each pass reads the
// slice from L2.
template <int NT, typename T, int CAP>
__device__ __noinline__ void select_exactly(const Slice<T>& s, int32_t rank, uint32_t o, uint32_t top, int32_t k,
                                            Candidates<CAP>& l, int32_t* sh) {
    uint32_t lo = o;               // at least k from here on
    int32_t have = CAP + 1;       // how many (or more)
    const int32_t above = count_from<NT>(s, lo + 1, sh);
    uint32_t hi = lo + 1;          // fewer than k from here on
    if (above >= k) {
        lo = lo + 1;
        have = above;
        hi = top + 1;
        while (have > CAP && hi - lo > 1) {
            const uint32_t mid = lo + (hi - lo) / 2;
            const int32_t c = count_from<NT>(s, mid, sh);
            if (c >= k) lo = mid, have = c;
            else hi = mid;
        }
    }
    if (threadIdx.x == 0) l.count = 0;
    __syncthreads();
    if (have <= CAP) {
        offer_from<NT>(s, lo, l);
        __syncthreads();
        return;
    }
    offer_from<NT>(s, lo + 1, l);  // fewer than k
    __syncthreads();
    // the others are equal to lo: the lowest classes of them
    int32_t filled = l.count;
    __syncthreads();
    const int32_t begin[2] = {rank == 0 ? 0 : s.first(0), s.part.head + s.part.vecs * kE<T>};
    const int32_t end[2] = {s.first(s.count), rank == 0 ? s.part.head + s.part.vecs * kE<T> + s.part.tail : begin[1]};
    for (int p = 0; p < 2; ++p)
        for (int32_t c0 = begin[p]; c0 < end[p] && filled < k; c0 += NT) {
            const int32_t c = c0 + (int32_t)threadIdx.x;
            const bool eq = c < end[p] && order_of(to_f(s.row[c])) == lo;
            int32_t total;
            const int32_t at = filled + block_excl_scan<NT, int32_t>(eq, sh, total);
            if (eq && at < k) l.e[at] = entry_of(lo, c);
            filled += total;
        }
    if (threadIdx.x == 0) l.count = min(filled, k);
    __syncthreads();
}

constexpr int kRefine = 16;  // classes a warp from which the bound is refined
// Maxima of a row that take part in its bound, W warps' (k <= 32 W): each gives 32 at
// most.
template <int W>
constexpr int kTops = 32 * W < 256 ? 32 * W : 256;

template <typename T, int NT, int S>
__global__ void __launch_bounds__(NT, 1024 / NT) k_logprobs_row(Args<T> a, int32_t turns) {
    extern __shared__ __align__(16) uint4 ring[];  // kRing turns, in the end CTA 0's candidates of all; the groups' maxima
    pdl_start();
    constexpr int kWarps = NT / 32, W = S * kWarps, CAP = kCap<NT>;
    __shared__ __align__(16) float4 parts[W];
    __shared__ __align__(16) float tops[kTops<W>];
    __shared__ Candidates<CAP> list;
    __shared__ int32_t hits[CAP], hit_count;
    __shared__ float bound;
    __shared__ int32_t reach[3];  // groups that reach a bound, counted in turn
    __shared__ int32_t scan[NT / 32 + 1];
    const int warp = (int)(threadIdx.x >> 5), lane = (int)lane_id();
    const int32_t first = (int32_t)(blockIdx.x / S), rank = (int32_t)(blockIdx.x % S), step = (int32_t)(gridDim.x / S);
    const int32_t n = rows_of(a.d_n, a.n_cap);
    if (first >= n) return;  // the whole cluster
    if constexpr (S > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");
    float* gmax = reinterpret_cast<float*>(ring + (S > 1 && S * CAP > 2 * kRing * kTurn * NT ? S * CAP / 2 : kRing * kTurn * NT)) + threadIdx.x;
    const auto slice_of = [&](int32_t r) {
        const T* row = a.x + (int64_t)r * a.ld;
        const RowParts<T> part(row, a.classes);
        const int32_t per = (part.vecs + S - 1) / S, v0 = min(part.vecs, rank * per);
        return Slice<T>{row, part, v0, min(part.vecs, v0 + per) - v0, -1, -INFINITY};
    };
    // The copies run ahead: turn ft of row fr is the next one to be copied.
    int32_t fr = first, ft = 0, fcount;
    const T* from;
    const auto enter = [&] {
        if (fr >= n) return;
        const Slice<T> sl = slice_of(fr);
        from = sl.row + sl.first((int32_t)threadIdx.x);
        fcount = sl.count - (int32_t)threadIdx.x;
    };
    const auto fetch = [&](int at) {
        if (fr < n) {
            const bool whole = (ft + 1) * kTurn * NT <= fcount + (int32_t)threadIdx.x;  // the same in the whole block
#pragma unroll
            for (int k = 0; k < kTurn; ++k) {
                const int32_t i = (ft * kTurn + k) * NT;
                if (whole || i < fcount) copy_async(ring + (at * kTurn + k) * NT + threadIdx.x, from + i * kE<T>);
            }
            if (++ft * kTurn * NT >= fcount + (int32_t)threadIdx.x) {  // the same in the whole block
                fr += step;
                ft = 0;
                enter();
            }
        }
        copies_end();
    };
    enter();
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) fetch(i);
    int at = 0;
    for (int32_t r = first; r < n; r += step) {
        Slice<T> sl = slice_of(r);
        if (rank == 0 && warp == 0) sl.edge = sl.part.edge(lane);
        if (sl.edge >= 0) sl.xe = to_f(sl.row[sl.edge]);
        int32_t y = -1;
        float xy = 0.f;
        if (rank == 0 && threadIdx.x == 0) {
            y = label_of(a, r);
            if (y >= 0) xy = to_f(sl.row[y]);
        }
        Stat s = stat_of(sl.xe);
        float most = sl.xe;
        const int32_t span = turns * kTurn * NT;  // vectors of a group, over the block
        for (int32_t g0 = 0, g = 0; g0 < sl.count; g0 += span, ++g) {
            float gm = -INFINITY;
            for (int32_t i0 = g0; i0 < min(sl.count, g0 + span); i0 += kTurn * NT) {
                fetch(at ? at - 1 : kRing - 1);
                copies_wait<kRing - 1>();
                uint4 u[kTurn];
                if (i0 + kTurn * NT <= sl.count) {  // a whole turn
#pragma unroll
                    for (int k = 0; k < kTurn; ++k) u[k] = ring[(at * kTurn + k) * NT + threadIdx.x];
                } else {
#pragma unroll
                    for (int k = 0; k < kTurn; ++k)
                        u[k] = i0 + k * NT + (int32_t)threadIdx.x < sl.count ? ring[(at * kTurn + k) * NT + threadIdx.x] : empty_part<T>();
                }
                if (++at == kRing) at = 0;
                const float top = parts_max<T>(u);
                gm = fmaxf(gm, top);
                rebase(s, fmaxf(s.m, top));
                f2 z = pair(s.z, 0.f), t = pair(s.t, 0.f);
                const float b = -finite_base(s.m);
#pragma unroll
                for (int k = 0; k < kTurn; ++k) {
                    repack(u[k]);
                    add_part<T>(u[k], pair(b, b), z, t);
                }
                float z1, t1;
                unpair(z, s.z, z1);
                unpair(t, s.t, t1);
                s.z += z1;
                s.t += t1;
            }
            gmax[g * NT] = gm;
            most = fmaxf(most, gm);
        }
        s = warp_join(s);
        // the warp's j largest of its lanes' maxima: half as many again as k needs, so that
        // an uneven share of the warps does not lower the bound (M is a multiple of 4)
        const int32_t need = (a.k + W - 1) / W;
        int32_t j = min(need + (need + 1) / 2, kTops<W> / W);
        const int32_t M = W * j;
        if (j == 1) most = s.m;
        else if (j > 1) most = warp_sort(most);
        const int32_t w = rank * kWarps + warp;
        if constexpr (S > 1) {
            asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");  // every CTA runs (a cluster has one row)
            if (lane < S)
                st_cluster4(map_rank(smem_addr(parts + w), (uint32_t)lane),
                            make_uint4(__float_as_uint(s.m), __float_as_uint(s.z), __float_as_uint(s.t), 0u));
            if (lane < j)
                for (uint32_t q = 0; q < S; ++q)
                    asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(map_rank(smem_addr(tops + w * j + lane), q)),
                                 "f"(most)
                                 : "memory");
            cluster_sync();
        } else {
            if (lane == 0) parts[w] = make_float4(s.m, s.z, s.t, 0.f);
            if (lane < j) tops[w * j + lane] = most;
            __syncthreads();
        }
        // the whole row's, in every warp
        s = {-INFINITY, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < (W + 31) / 32; ++i)
            if (lane + 32 * i < W) {
                const float4 p = parts[lane + 32 * i];
                Stat o = {p.x, p.y, p.z};
                const float m = fmaxf(s.m, o.m);
                rebase(s, m);
                rebase(o, m);
                s.z += o.z;
                s.t += o.t;
            }
        s = warp_join(s);
        const float log_z = logf(s.z);
        if (rank == 0 && threadIdx.x == 0) put_row(a, r, s, log_z, y, xy);
        if (a.k == 0) {
            __syncthreads();  // before the next row's parts
            continue;
        }
        for (int32_t i0 = (int32_t)threadIdx.x; i0 < M; i0 += NT) {  // the k-th largest of tops
            const float v = tops[i0];
            int32_t before = 0;
#pragma unroll 2
            for (int32_t q = 0; q < M; q += 4) {
                const float4 o = *reinterpret_cast<const float4*>(tops + q);
                const int32_t i = i0 - q;
                before += (o.x > v || (o.x == v && i > 0)) + (o.y > v || (o.y == v && i > 1)) +
                          (o.z > v || (o.z == v && i > 2)) + (o.w > v || (o.w == v && i > 3));
            }
            if (before == a.k - 1) bound = v;
        }
        if (threadIdx.x == 0) list.count = hit_count = reach[0] = 0;
        __syncthreads();
        float tau = bound;
        const bool bad = s.z != s.z;
        if constexpr (S == 1) {
            // For many classes the threads' maxima are too few for a close bound: more
            // groups' maxima, by bisection (4096 x 50,257 bf16: k = 128 150 us, without
            // it 650; k = 100 140, 200; k = 80 134, 129)
            if (a.k > kRefine * W && !bad && tau < s.m) {
                uint32_t lo = order_of(tau), hi = order_of(s.m) + 1;
                for (int i = 0; i < 24 && hi - lo > 1; ++i) {
                    const uint32_t mid = lo + (hi - lo) / 2;
                    const float v = value_of(mid);
                    int32_t c = 0;
                    for (int32_t g0 = 0, g = 0; g0 < sl.count; g0 += span, ++g) c += gmax[g * NT] >= v;
                    c = __reduce_add_sync(0xFFFFFFFFu, c);
                    if (lane == 0) atomicAdd(&reach[i % 3], c);
                    if (threadIdx.x == 0) reach[(i + 1) % 3] = 0;  // (read two barriers ago)
                    __syncthreads();
                    c = reach[i % 3];
                    if (c < a.k) {
                        hi = mid;
                    } else {
                        lo = mid;
                        if (c <= a.k + a.k / 8) break;
                    }
                }
                tau = value_of(lo);
            }
        }
        const float lowest = fmaxf(tau, -3.402823466e38f);  // (-inf takes no part)
        if (!bad) {
            if (sl.xe >= lowest) offer(list, sl.xe, sl.edge);
            uint32_t reached = 0;  // of the thread's groups
            for (int32_t g0 = 0, g = 0; g0 < sl.count; g0 += span, ++g) reached |= gmax[g * NT] >= lowest ? 1u << g : 0u;
            for (int32_t to = reserve(__popc(reached), &hit_count); reached; ++to, reached &= reached - 1)
                if (to < CAP) hits[to] = (__ffs((int)reached) - 1) * NT + (int32_t)threadIdx.x;
        }
        __syncthreads();
        // the groups that reach the bound, their vectors over all threads
        const int32_t each = turns * kTurn, items = min(hit_count, CAP) * each;
        for (int32_t q = (int32_t)threadIdx.x; q < items; q += NT) {
            const int32_t h = hits[q / each];
            const int32_t i = (h / NT * each + q % each) * NT + h % NT;
            if (i >= sl.count) continue;
            const uint4 u = sl.load(i);
            if (part_max<T>(u) < tau) continue;
            float f[kE<T>];
            unpack<T>(u, f);
#pragma unroll
            for (int e = 0; e < kE<T>; ++e)
                if (f[e] >= lowest) offer(list, f[e], sl.first(i) + e);
        }
        __syncthreads();
        if (list.count > CAP || hit_count > CAP)
            select_exactly<NT>(sl, rank, max(order_of(tau), kOrderNone + 1), order_of(s.m), a.k, list, scan);
        const unsigned long long* all = list.e;
        int32_t total = list.count;
        if constexpr (S > 1) {  // CTA 0 takes everybody's
            cluster_sync();
            if (rank == 0) {
                unsigned long long* to = reinterpret_cast<unsigned long long*>(ring);
                total = 0;
                for (uint32_t q = 0; q < S; ++q) {
                    const int32_t c = __float_as_int(ld_cluster(map_rank(smem_addr(&list.count), q)));
                    for (int32_t i = threadIdx.x; i < c; i += NT) {
                        const uint32_t src = map_rank(smem_addr(&list.e[i]), q);
                        asm volatile("ld.shared::cluster.b64 %0, [%1];\n" : "=l"(to[total + i]) : "r"(src) : "memory");
                    }
                    total += c;
                }
                all = to;
            }
            cluster_sync();  // the lists stay until they are read
            if (rank != 0) return;
        }
        int32_t* ids = a.top_ids + (int64_t)r * a.k;
        float* lps = a.top_logp + (int64_t)r * a.k;
        for (int32_t i = threadIdx.x; i < total; i += NT) {
            const unsigned long long e = all[i];
            int32_t before = total % 2 && all[total - 1] > e;
#pragma unroll 4
            for (int32_t q = 0; q + 1 < total; q += 2) {
                const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(all + q);
                before += (o.x > e) + (o.y > e);
            }
            if (before < a.k) {
                ids[before] = class_of(e);
                lps[before] = logp_of(value_of((uint32_t)(e >> 32)), s.m, log_z);
            }
        }
        for (int32_t i = total + (int32_t)threadIdx.x; i < a.k; i += NT) {
            ids[i] = -1;
            lps[i] = bad ? s.z : -INFINITY;
        }
    }
}

// -------------------------------------------------------------------- host
template <typename T, int NV, int W = 1>
sg_status run_warp(const Args<T>& a, cudaStream_t s) {
    const int64_t rows = kWarpThreads<W> / 32 / W;  // of a block
    SG_CUDA(launch_pdl(k_logprobs_warp<T, NV, W>, dim3((unsigned)cdiv(a.n_cap, rows)), dim3(kWarpThreads<W>), 0, s, a));
    return SG_OK;
}

template <typename T, int NT, int S>
sg_status run_row(const Args<T>& a, int64_t nv, cudaStream_t s) {
    const int64_t per = cdiv(nv, S), all_turns = cdiv(per, kTurn * NT);
    const int64_t turns = all_turns > kGroups ? cdiv(all_turns, kGroups) : 1;
    int64_t lists = kRing * kTurn * NT * 16;
    if (S > 1 && lists < S * kCap<NT> * 8) lists = S * kCap<NT> * 8;
    const int64_t smem = lists + cdiv(all_turns, turns) * NT * 4;
    static OncePerDevice set;
    SG_CUDA(allow_smem(set, k_logprobs_row<T, NT, S>, (int)(lists + kGroups * NT * 4)));
    int64_t clusters = a.n_cap;  // a cluster of several CTAs has one row
    if (S == 1 && clusters > (1024 / NT) * num_sms()) clusters = (1024 / NT) * num_sms();
    SG_CUDA(launch_cluster(k_logprobs_row<T, NT, S>, (unsigned)(clusters * S), NT, S, s, (int)smem, a, (int32_t)turns));
    return SG_OK;
}

// How rows of few classes reach shared memory.
template <typename T>
Few few_of(const Args<T>& a) {
    const bool on16 = (uintptr_t)a.x % 16 == 0;
    if (on16 && a.ld % kE<T> == 0) return kByVectors;
    return on16 && a.ld == a.classes ? kWhole : kByValues;
}

template <typename T, int K, Few HOW>
sg_status run_few_as(const Args<T>& a, cudaStream_t s) {
    const int32_t vecs = (int32_t)cdiv(a.classes, kE<T>);
    const int32_t pitch = HOW == kWhole ? a.classes : HOW == kByVectors ? vecs | 1 : a.classes | 1;
    const size_t smem = kFewRows * (size_t)pitch * (HOW == kWhole ? sizeof(T) : HOW == kByVectors ? 16 : 4);
    const int32_t d = HOW == kByVectors ? a.classes / kE<T> : a.classes;
    const uint32_t magic = d > 1 ? (uint32_t)((((uint64_t)1 << 32) + d - 1) / d) : 0;  // (1: not used)
    static OncePerDevice set;
    SG_CUDA(allow_smem(set, k_logprobs_few<T, K, HOW>, kFewRows * (kFewClasses / 4 + 1) * 16));
    SG_CUDA(launch_pdl(k_logprobs_few<T, K, HOW>, dim3((unsigned)cdiv(a.n_cap, kFewRows)), dim3(kFewRows), smem, s, a, pitch,
                       magic));
    return SG_OK;
}
template <typename T, int K>
sg_status run_few(const Args<T>& a, cudaStream_t s) {
    switch (few_of(a)) {
        case kWhole: return run_few_as<T, K, kWhole>(a, s);
        case kByVectors: return run_few_as<T, K, kByVectors>(a, s);
        default: return run_few_as<T, K, kByValues>(a, s);
    }
}

template <typename T>
sg_status run(const Args<T>& a, cudaStream_t s) {
    if (a.n_cap == 0) return SG_OK;
    // (a block for every SM at least)
    if (a.classes > 1 && a.classes <= (few_of(a) == kByValues ? kFewByValues : kFewClasses) && a.k <= kFewTop &&
        a.n_cap >= kFewRows * num_sms()) {
        switch (a.k) {
            case 0:
            case 1: return run_few<T, 1>(a, s);
            case 2: return run_few<T, 2>(a, s);
            case 3: return run_few<T, 3>(a, s);
            case 4: return run_few<T, 4>(a, s);
            case 5: return run_few<T, 5>(a, s);
            case 6: return run_few<T, 6>(a, s);
            case 7: return run_few<T, 7>(a, s);
            default: return run_few<T, 8>(a, s);
        }
    }
    const int64_t nv = cdiv((int64_t)a.classes, kE<T>);  // vectors of a row, at most
    // In registers, as few as hold the row: 12 a lane where 16 would leave a quarter and
    // more of them empty (us, k = 5: 25,000 x 3000 bf16 43, with 16 53), the fewest warps
    // (20,000 x 4000 bf16 k = 20 by 1 x 16 52, by 2 x 8 55).  By CTAs of 64 threads from the
    // ring 16,000 x 5000 bf16 k = 1, 20, 100 take 74, 102, 291 (45, 56, 114), by 128 threads
    // 8000 x 10,000 k = 1, 20, 100 53, 63, 148 (42, 52, 96).  8 warps lose: 3000 x 30,000 k = 1
    // 48, by the ring 43.
    if (nv <= 32) return run_warp<T, 1>(a, s);
    if (nv <= 64) return run_warp<T, 2>(a, s);
    if (nv <= 128) return run_warp<T, 4>(a, s);
    if (nv <= 256) return run_warp<T, 8>(a, s);
    if (nv <= 384) return run_warp<T, 12>(a, s);
    if (nv <= 512) return run_warp<T, 16>(a, s);
    if (nv <= 768) return run_warp<T, 12, 2>(a, s);
    if (nv <= 1024) return run_warp<T, 16, 2>(a, s);
    if (nv <= 1536) return run_warp<T, 12, 4>(a, s);
    if (nv <= 2048) return run_warp<T, 16, 4>(a, s);
    // half the threads a CTA from two rows an SM on: what every warp does for a row, and
    // its barriers, cost less (4096 x 50,257 bf16 k = 64: 112 us, by 256 threads 122; 800 x
    // 20,000 k = 20 13, 17; 400 x 30,000 fp32 the same; 220 x 150,000 bf16 24, 20)
    if (a.n_cap >= 2 * num_sms()) return run_row<T, 128, 1>(a, nv, s);
    // clusters while the rows leave SMs idle and every CTA has a turn to do
    int split = 1;
    while (split < 8 && (int64_t)a.n_cap * split * 2 <= 2 * num_sms() && nv >= split * 2 * kThreads) split *= 2;
    switch (split) {
        case 1: return run_row<T, 256, 1>(a, nv, s);
        case 2: return run_row<T, 256, 2>(a, nv, s);
        case 4: return run_row<T, 256, 4>(a, nv, s);
        default: return run_row<T, 256, 8>(a, nv, s);
    }
}

}  // namespace

extern "C" sg_status sg_logprobs(const void* d_logits, int32_t dtype, int32_t n_cap, const int32_t* d_n, int32_t n_classes,
                                 int64_t ld, const int32_t* d_labels, int32_t k, float* d_logp, float* d_entropy,
                                 int32_t* d_top_ids, float* d_top_logp, sg_stream_t stream) {
    if (dtype != SG_F32 && dtype != SG_BF16) return fail(SG_ERR_UNSUPPORTED, "sg_logprobs: dtype");
    if (n_cap < 0 || n_cap > 1 << 27 || n_classes <= 0 || n_classes > 2147483647 - 1024)
        return fail(SG_ERR_INVALID_ARG, "sg_logprobs: bad sizes");
    if (k < 0 || k > SG_MAX_TOP) return fail(SG_ERR_INVALID_ARG, "sg_logprobs: k must be 0 to %d", SG_MAX_TOP);
    if (ld < n_classes) return fail(SG_ERR_INVALID_ARG, "sg_logprobs: the row stride is below n_classes");
    if (n_cap > 0 && !d_logits) return fail(SG_ERR_INVALID_ARG, "sg_logprobs: NULL logits");
    if (n_cap > 0 && !d_labels != !d_logp) return fail(SG_ERR_INVALID_ARG, "sg_logprobs: labels and logp come together");
    if (n_cap > 0 && k > 0 && (!d_top_ids || !d_top_logp))
        return fail(SG_ERR_INVALID_ARG, "sg_logprobs: k above 0 needs top_ids and top_logp");
    if (k == 0 && (d_top_ids || d_top_logp)) return fail(SG_ERR_INVALID_ARG, "sg_logprobs: top arrays with k = 0");
    const int e = dtype == SG_F32 ? 4 : 2;
    if ((uintptr_t)d_logits % e ||
        ((uintptr_t)d_labels | (uintptr_t)d_logp | (uintptr_t)d_entropy | (uintptr_t)d_top_ids | (uintptr_t)d_top_logp) % 4)
        return fail(SG_ERR_INVALID_ARG, "sg_logprobs: an array is not aligned to its elements");
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == SG_F32) {
        const Args<float> a = {(const float*)d_logits, ld, d_labels, d_n, n_cap, n_classes, k, d_logp, d_entropy, d_top_ids,
                               d_top_logp};
        return run(a, s);
    }
    const Args<__nv_bfloat16> a = {(const __nv_bfloat16*)d_logits, ld, d_labels, d_n, n_cap, n_classes, k, d_logp,
                                   d_entropy, d_top_ids, d_top_logp};
    return run(a, s);
}
