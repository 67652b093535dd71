// Distillation from a teacher's top logits: per row of the student's logits x and
// the teacher's k entries (id_j, v_j), with q = softmax(v / T) over the entries and
// p = softmax(x / T) over all classes,
//   loss[r]    = T^2 sum_j q_j (log q_j - log p[id_j])
//   grad[r, c] = w T (p[c] - sum of q_j over id_j = c)
// Bound by memory: the logits are read and the gradient is written once.  As in the
// cross-entropy a row stays in registers in between, spread over a warp
// (k_distill_warp) or a cluster of CTAs (k_distill_row), and many long rows are
// streamed through shared memory ahead of their use (k_distill_stream).
//
// The entries are a row's small part.  One warp of a CTA takes a row's (up to 4 a lane)
// and forms q while the row is on its way: the row's own warp, the first of a cluster's
// CTAs, or in the streaming form extra warps that do nothing else.  The vectors' w T p
// is stored first; then the entries' classes are written again, from their own logits.
// An entry adds up all q of its class where classes occur more than once (a match over
// the warp for up to 32 entries, a table for more, tells whether any does), so they are
// right whichever of them writes last (they write the same).
//
// Above a temperature of 4 the loss needs more care than its definition takes
// (k_distill_loss, which then follows and writes it).
#include "sg_internal.cuh"
#include "sg_rows.cuh"
#include "sg_softmax.cuh"
#include "sg_tc.cuh"

SGI_ERROR_WORD(distill)

using namespace sgi;

namespace {

constexpr int kThreads = 256;
constexpr int kCountThreads = 1024;
constexpr int kPer = SG_MAX_TOP / 32;  // entries of a lane

template <typename T>
struct Args {
    const T* x;
    T* grad;
    int64_t ld, ld_grad;
    const int32_t* ids;
    const float* values;
    const int32_t* d_n;
    int32_t n_cap, classes, k;
    int32_t mean;
    float gs, temp, inv_temp, l;  // l = log2(e) / temp
    float* loss;
    float* total;
    int32_t* done;   // rows or blocks that are done; then `counts` counts of rows with a teacher
    int32_t counts;
    float2* stats;  // rows' maximum and sum for k_distill_loss, or NULL
};

// Whether a row has a teacher: its first entry says so.
__device__ __forceinline__ bool is_used(int32_t id, float v, int32_t classes) {
    return id >= 0 && id < classes && v != -INFINITY;
}
template <typename T>
__device__ __forceinline__ bool row_used(const Args<T>& a, int32_t r) {
    return is_used(__ldg(a.ids + (int64_t)r * a.k), __ldg(a.values + (int64_t)r * a.k), a.classes);
}

// Rows with a teacher (a whole warp).
template <typename T>
__device__ __forceinline__ int32_t valid_of(const Args<T>& a) {
    int32_t v = 0;
    for (int32_t i = (int32_t)lane_id(); i < a.counts; i += 32) v += a.done[1 + i];
    return warp_sum(v);
}
// What the gradient's softmax is multiplied by (a whole warp).
template <typename T>
__device__ __forceinline__ float weight_of(const Args<T>& a) {
    const float w = a.gs * a.temp;
    return a.mean ? w / (float)max(1, valid_of(a)) : w;
}

// A row's entries in shared memory, for the threads that write their classes.
struct Entries {
    int32_t __align__(16) id[SG_MAX_TOP];  // -1: none, from k on as well
    float v[SG_MAX_TOP], x[SG_MAX_TOP], q[SG_MAX_TOP];
};
// Whether classes occur more than once: a table of 256 places for up to SG_MAX_TOP
// classes, cleared beforehand.  (A comparison of every two entries took longer than
// the row's other work from 64 entries on.)
constexpr int kPlaces = 256;
struct Table {
    int32_t place[kPlaces];  // -1: free
    __device__ __forceinline__ void clear(int t, int threads) {
        for (int i = t; i < kPlaces; i += threads) place[i] = -1;
    }
    // true if the class was there (for one of two at least)
    __device__ __forceinline__ bool insert(int32_t id) {
        uint32_t at = (uint32_t)id * 0x9E3779B1u >> 24;
        for (int i = 0; i < kPlaces; ++i, at = (at + 1) & (kPlaces - 1)) {
            const int32_t was = atomicCAS(&place[at], -1, id);
            if (was == -1) return false;
            if (was == id) return true;
        }
        return false;
    }
};
// Entry j of row r (-1 and -inf: none); report: names one out of range in the error word
template <typename T>
__device__ __forceinline__ void load_entry(const Args<T>& a, int32_t r, int32_t j, bool report, int32_t& id, float& v) {
    id = -1;
    v = -INFINITY;
    if (j >= a.k) return;
    const int32_t i = __ldg(a.ids + (int64_t)r * a.k + j);
    const float w = __ldg(a.values + (int64_t)r * a.k + j);
    if (i >= 0 && i < a.classes) id = i, v = w;
    else if (i != -1 && report) dev_err(ERR_INDEX);
}

// One warp: max v and sum exp((v - max) / T) with its logarithm, once the entries are
// there; q is put beside them (a used row: at least one value is above -inf)
struct Scale {
    float m, log_zq, zq;
};
template <typename T>
__device__ __forceinline__ Scale scale_entries(const Args<T>& a, Entries& n) {
    const int lane = (int)lane_id();
    float m = -INFINITY, z = 0.f, q[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        if (32 * e >= a.k) break;  // (the same in every lane)
        q[e] = lane + 32 * e < a.k ? n.v[lane + 32 * e] : -INFINITY;
        m = fmaxf(m, q[e]);
    }
    m = warp_max(m);
    if (m == -INFINITY) m = 0.f;  // all of them NaN
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        if (32 * e >= a.k) break;
        q[e] = exp_from(q[e], m, a.l);
        z += q[e];
    }
    z = warp_sum(z);
    const float inv = 1.f / z;
#pragma unroll
    for (int e = 0; e < kPer; ++e)
        if (lane + 32 * e < a.k) n.q[lane + 32 * e] = q[e] * inv;
    return {m, logf(z), z};
}
// The row's loss (one warp, the same in every lane), from the row's maximum M and sum Z:
// T^2 (log q - log p) as T (difference of the logits) + T^2 (difference of the logarithms).
// (A difference over T first is past fp32 for a class at the type's lowest value and T < 1.)
template <typename T>
__device__ __forceinline__ float loss_of(const Args<T>& a, const Scale& c, const Entries& n, float M, float Z) {
    const int lane = (int)lane_id();
    const float apart = (logf(Z) - c.log_zq) * (a.temp * a.temp);
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const int32_t j = lane + 32 * e;
        if (j >= a.k) break;
        const float q = n.q[j], x = n.x[j];
        if (q == 0.f) continue;
        if (x == -INFINITY && q > 0.f && Z == Z) s += INFINITY;  // (not with NaN)
        else s = fmaf(q, fmaf(a.temp, (n.v[j] - c.m) - (x - M), apart), s);
    }
    return warp_sum(s);
}
// One lane of a used row: its loss, and its statistics where they are asked for.
template <typename T>
__device__ __forceinline__ void put_loss(const Args<T>& a, int32_t r, float loss, float M, float Z) {
    a.loss[r] = loss;
    if (a.stats) a.stats[r] = make_float2(M, Z);
}
// One warp: all entries of the R rows r, r + step, .. below n, for itself.
template <int R, typename T>
__device__ __forceinline__ void load_entries(const Args<T>& a, int32_t r, int32_t step, int32_t n, Entries* to, bool report = true) {
    const int lane = (int)lane_id();
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        if (32 * e >= a.k) {  // (the same in every lane)
#pragma unroll
            for (int q = 0; q < R; ++q) to[q].id[lane + 32 * e] = -1;
            continue;
        }
        int32_t id[R];
        float v[R], x[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            id[q] = -1, v[q] = -INFINITY;
            if (r + q * step < n) load_entry(a, r + q * step, lane + 32 * e, report, id[q], v[q]);
        }
#pragma unroll
        for (int q = 0; q < R; ++q) x[q] = id[q] >= 0 ? to_f(a.x[(int64_t)(r + q * step) * a.ld + id[q]]) : 0.f;
#pragma unroll
        for (int q = 0; q < R; ++q) to[q].id[lane + 32 * e] = id[q], to[q].v[lane + 32 * e] = v[q], to[q].x[lane + 32 * e] = x[q];
    }
}
// One warp: whether a class occurs more than once.
template <typename T>
__device__ __forceinline__ bool any_twice(const Args<T>& a, const Entries& n, Table& table) {
    const int lane = (int)lane_id();
    if (a.k <= 32) {
        const int32_t id = n.id[lane];
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, id);  // (by every lane)
        return __any_sync(0xFFFFFFFFu, id >= 0 && __popc(same) > 1);
    }
    table.clear(lane, 32);
    __syncwarp();
    bool twice = false;
    for (int32_t j = lane; j < a.k; j += 32)
        if (n.id[j] >= 0) twice |= table.insert(n.id[j]);
    return __any_sync(0xFFFFFFFFu, twice);
}
// The gradient at entry j's class; false where there is none.  twice: classes may occur
// more than once; w_z: w / Z
template <typename T>
__device__ __forceinline__ bool entry_grad(const Args<T>& a, const Entries& n, int32_t j, bool twice, float w, float w_z, float M,
                                           float Z, float& g) {
    const int32_t id = n.id[j];
    if (id < 0) return false;
    float q = n.q[j];
    if (twice) {
        q = 0.f;
        for (int32_t i = 0; i < a.k; ++i)
            if (n.id[i] == id) q += n.q[i];
    }
    g = Z == 0.f ? 0.f : fmaf(w_z, exp_from(n.x[j], M, a.l), -w * q);
    return true;
}

// The total, by the last block to finish.
template <int NT, typename T>
__device__ __forceinline__ void put_total(const Args<T>& a, int32_t n) {
    const float s = block_sum_fixed<NT>(a.loss, n);
    if (threadIdx.x >= 32) return;
    const int32_t v = valid_of(a);
    if (threadIdx.x == 0) {
        a.total[0] = a.mean ? s / (float)max(1, v) : s;
        a.total[1] = (float)v;
    }
}

// ------------------------------------------------------------ rows by warps
// A row in NV vectors a lane, as loaded.
template <int NV>
struct WarpRow {
    uint4 x[NV];
    float xe;  // this lane's edge element
    bool used;
};
template <typename T, int NV>
__device__ __forceinline__ void load_row(const Args<T>& a, int32_t r, WarpRow<NV>& d) {
    const int lane = (int)lane_id();
    const T* row = a.x + (int64_t)r * a.ld;
    const RowParts<T> part(row, a.classes);
    d.used = row_used(a, r);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int32_t v = lane + 32 * k;
        d.x[k] = v < part.vecs ? *reinterpret_cast<const uint4*>(row + part.head + v * kE<T>) : empty_part<T>();
    }
    const int32_t ce = part.edge(lane);
    d.xe = ce >= 0 ? to_f(row[ce]) : -INFINITY;
}
// The row's loss (in every lane) and gradient; mine: its entries.
template <typename T, int NV>
__device__ __forceinline__ float finish_row(const Args<T>& a, int32_t r, float w, WarpRow<NV>& d, Entries& mine, Table& table) {
    const int lane = (int)lane_id();
    const T* row = a.x + (int64_t)r * a.ld;
    T* out = a.grad ? a.grad + (int64_t)r * a.ld_grad : nullptr;
    if (!d.used) {
        if (lane == 0) a.loss[r] = 0.f;
        if (out)
            for (int32_t c = lane; c < a.classes; c += 32) put(out + c, 0.f);
        return 0.f;
    }
    const RowParts<T> part(row, a.classes);
    const Scale scale = scale_entries(a, mine);  // (each lane's own entries)
    float m = d.xe;
#pragma unroll
    for (int k = 0; k < NV; ++k) m = fmaxf(m, part_max<T>(d.x[k]));
    m = warp_max(m);
    if (m == -INFINITY) m = 0.f;
    const Base base(m, a.l);
    f2 sum = pair(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < NV; ++k) part_exp<T>(d.x[k], base, sum);
    float z, z1;
    unpair(sum, z, z1);
    z = warp_sum(z + z1 + base.of(d.xe));
    const float loss = loss_of(a, scale, mine, m, z);
    if (lane == 0) put_loss(a, r, loss, m, z);
    if (!out) return loss;
    const bool same = same_phase(row, (const T*)out);
    const float inv = z == 0.f ? 0.f : w / z;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int32_t v = lane + 32 * k;
        if (v < part.vecs)
            store_part(out + part.head + v * kE<T>, same, part_grad<T>(d.x[k], base, pair(inv, inv)));
    }
    const int32_t ce = part.edge(lane);
    if (ce >= 0) put(out + ce, inv * base.of(d.xe));
    __syncwarp();  // the entries are there, the vectors stored
    const bool twice = any_twice(a, mine, table);
    for (int32_t j = lane; j < a.k; j += 32) {
        float g;
        if (entry_grad(a, mine, j, twice, w, inv, m, z, g)) put(out + mine.id[j], g);
    }
    __syncwarp();  // before the next row's entries
    return loss;
}

// A warp a row, with as many vectors a lane as hold it.  Rows of few classes are bound by
// instructions, some 500 of them in 700 issue slots a row whatever its length: 200,000 x 47
// fp32, k = 20: 122 us, 15.8 for the bytes.  The next row's loads ahead in registers take 130, six
// blocks an SM 126.  us, k = 20: 60,000 x 400 fp32 53 (floor 30), 40,000 x 2000 bf16 74 (48),
// 20,000 x 4000 bf16 76 (by blocks of 256 threads from shared memory 123, of 64 from
// registers 124).
template <int NV>
constexpr int kWarpBlocks = NV <= 2 ? 5 : NV == 4 ? 4 : NV == 8 ? 3 : 2;  // an SM

template <typename T, int NV>
__global__ void __launch_bounds__(kThreads, kWarpBlocks<NV>) k_distill_warp(Args<T> a) {
    pdl_start();
    constexpr int kWarps = kThreads / 32;
    __shared__ Entries entries[kWarps];
    __shared__ Table tables[kWarps];
    __shared__ bool last;
    const int warp = (int)(threadIdx.x >> 5);
    const int32_t n = rows_of(a.d_n, a.n_cap), blocks = min((int32_t)gridDim.x, (n + kWarps - 1) / kWarps);
    if ((int32_t)blockIdx.x >= blocks) return;
    const float w = weight_of(a);
    for (int32_t r = (int32_t)blockIdx.x * kWarps + warp; r < n; r += (int32_t)gridDim.x * kWarps) {
        WarpRow<NV> d;
        load_row(a, r, d);
        load_entries<1>(a, r, 0, n, &entries[warp]);
        finish_row(a, r, w, d, entries[warp], tables[warp]);
    }
    if (!a.total) return;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(a.done, 1) == blocks - 1;
    __syncthreads();
    if (last) {
        __threadfence();
        put_total<kThreads>(a, n);
    }
}

// The whole of a small call in one cluster: each CTA counts the rows with a teacher, the
// cluster's warps take up to R rows each, all their loads in flight together, the
// warps' sums meet in CTA 0.  256 rows of 128 fp32, 8 entries: 8.0 us with the
// host's time (by two launches, and a row after the other, 9.7).
constexpr int kSmallCtas = 8;
constexpr int kSmallThreads = 512;
template <int NV>
constexpr int kSmallRows = NV <= 2 ? 2 : 1;  // a warp's
template <int NV>
constexpr int kSmallBytes = kSmallThreads / 32 * kSmallRows<NV> * (int)sizeof(Entries);

template <typename T, int NV>
__global__ void __launch_bounds__(kSmallThreads) k_distill_small(Args<T> a) {
    extern __shared__ __align__(128) uint8_t dsm[];
    pdl_start();
    constexpr int kWarps = kSmallThreads / 32, R = kSmallRows<NV>;
    __shared__ Table tables[kWarps];
    __shared__ int32_t sh[kWarps + 1];
    __shared__ float part[kWarps];
    const int warp = (int)(threadIdx.x >> 5);
    Entries* entries = reinterpret_cast<Entries*>(dsm) + warp * R;
    const int32_t n = rows_of(a.d_n, a.n_cap), r0 = (int32_t)blockIdx.x * kWarps + warp, step = kSmallCtas * kWarps;
    int32_t v = 0;
    for (int32_t i = (int32_t)threadIdx.x; i < n; i += kSmallThreads) v += row_used(a, i);
    WarpRow<NV> d[R];
#pragma unroll
    for (int q = 0; q < R; ++q)
        if (r0 + q * step < n) load_row(a, r0 + q * step, d[q]);
    load_entries<R>(a, r0, step, n, entries);
    v = block_sum<kSmallThreads, int32_t>(v, sh);
    const float w = a.gs * a.temp / (a.mean ? (float)max(1, v) : 1.f);
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < R; ++q)
        if (r0 + q * step < n) sum += finish_row(a, r0 + q * step, w, d[q], entries[q], tables[warp]);
    if (lane_id() == 0) part[warp] = sum;
    cluster_sync();
    if (a.stats && blockIdx.x == 0 && threadIdx.x == 0) a.done[0] = 0, a.done[1] = v;
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
// This CTA's entries of a row whose vectors have been stored: the classes of its
// vectors and, for CTA 0, the edge elements.
template <typename T>
__device__ __forceinline__ void put_entries(const Args<T>& a, const Entries& n, T* out, const RowParts<T>& part, int32_t v0,
                                            int32_t count, int32_t rank, int32_t j, bool twice, float w, float M,
                                            float Z) {
    if (j >= a.k || n.id[j] < 0) return;
    const int32_t at = part.place(n.id[j]);
    if (at < 0 ? rank != 0 : at < v0 || at >= v0 + count) return;
    float g;
    if (entry_grad(a, n, j, twice, w, w / Z, M, Z, g)) put(out + n.id[j], g);
}

template <typename T, int NT, int S>
__global__ void __launch_bounds__(NT, 1024 / NT) k_distill_row(Args<T> a) {
    pdl_start();
    constexpr int kParts = S * NT / 32;
    __shared__ __align__(8) float2 parts[kParts];  // (m, z) of every warp of the cluster
    __shared__ Entries entries;
    __shared__ Table table;
    __shared__ bool last, twice;
    const int32_t r = (int32_t)(blockIdx.x / S), rank = (int32_t)(blockIdx.x % S);
    const int32_t n = rows_of(a.d_n, a.n_cap), classes = a.classes;
    if (r >= n) return;  // the whole cluster
    if constexpr (S > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");
    if (threadIdx.x == 0) last = false;
    const T* row = a.x + (int64_t)r * a.ld;
    T* out = a.grad ? a.grad + (int64_t)r * a.ld_grad : nullptr;
    const bool used = row_used(a, r);  // the same in the whole cluster
    const RowParts<T> part(row, classes);
    const int32_t per = (part.vecs + S - 1) / S, v0 = min(part.vecs, rank * per), count = min(part.vecs, v0 + per) - v0;
    const int32_t edge = rank == 0 && threadIdx.x < 32 ? part.edge((int)threadIdx.x) : -1;
    const T* p = row + part.head + (v0 + (int32_t)threadIdx.x) * kE<T>;
    const bool mine = threadIdx.x < 32 && (rank == 0 || out);  // the warp of the entries
    Scale scale = {0.f, 0.f};
    Held<T, NT> h;
    h.m = 0.f, h.z = 0.f;
    if (mine) load_entries<1>(a, r, 0, n, &entries, rank == 0);
    if (used) {
#pragma unroll
        for (int k = 0; k < kVecs; ++k)
            h.x[k] = (int32_t)threadIdx.x + k * NT < count ? *reinterpret_cast<const uint4*>(p + k * NT * kE<T>)
                                                           : empty_part<T>();
        h.xe = edge >= 0 ? to_f(row[edge]) : -INFINITY;
        if (mine) {
            scale = scale_entries(a, entries);
            __syncwarp();
            const bool t = out && any_twice(a, entries, table);
            if (threadIdx.x == 0) twice = t;
        }
        float mr = -INFINITY, zr = 0.f;  // the part past the registers
        for (int32_t i = (int32_t)threadIdx.x + kVecs * NT; i < count; i += NT) {
            const T* q = row + part.head + (v0 + i) * kE<T>;
            const float top = fmaxf(mr, part_max<T>(*reinterpret_cast<const uint4*>(q)));
            const float b = top == -INFINITY ? 0.f : top;
            zr *= exp_from(mr, b, a.l);
#pragma unroll
            for (int e = 0; e < kE<T>; ++e) zr += exp_from(to_f(q[e]), b, a.l);
            mr = top;
        }
        reduce_held(h, count, mr, zr, a.l);
    }
    // every CTA runs: its shared memory may be written
    if constexpr (S > 1) asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");
    share_parts<NT, S>(parts, rank, h.m, h.z);
    if (used) {
        float M, Z;
        join_parts<kParts>(parts, M, Z, a.l);
        const float w = weight_of(a);
        if (out) {
            const float inv = held_scale(h.m, h.z, w, M, Z, a.l);
            store_held(h, out + part.head + v0 * kE<T>, count, same_phase(row, (const T*)out), inv, a.l);
            if (edge >= 0) put(out + edge, inv * Base(h.m, a.l).of(h.xe));
            for (int32_t i = (int32_t)threadIdx.x + kVecs * NT; i < count; i += NT) {
                const int32_t c = part.head + (v0 + i) * kE<T>;
#pragma unroll
                for (int e = 0; e < kE<T>; ++e)
                    put(out + c + e, Z == 0.f ? 0.f : w / Z * exp_from(to_f(row[c + e]), M, a.l));
            }
        }
        if (rank == 0 && threadIdx.x < 32) {
            const float loss = loss_of(a, scale, entries, M, Z);
            if (threadIdx.x == 0) put_loss(a, r, loss, M, Z);
        }
        __syncthreads();  // the vectors are stored
        if (out) put_entries(a, entries, out, part, v0, count, rank, (int32_t)threadIdx.x, twice, w, M, Z);
    } else {
        if (rank == 0 && threadIdx.x == 0) a.loss[r] = 0.f;
        if (out) zero_row<T, NT>(out, classes, rank, S);
    }
    if (!a.total || rank != 0) return;
    if (threadIdx.x == 0) {
        __threadfence();
        if (atomicAdd(a.done, 1) == n - 1) last = true;
    }
    __syncthreads();
    if (last) {
        __threadfence();
        put_total<NT>(a, n);
    }
}

// Many long rows: the same, with each cluster walking over its rows and the next two
// rows' slices on their way into shared memory while the current row is worked on.
//
// The last warps of a block (3 of 16 or 2 of 8) do nothing but the entries, beside the
// others and a row each in turn: the classes and their logits are loaded while the row
// before is worked on, q is formed while the row is reduced, and the entries' classes are
// written once the row's vectors are stored (`stored`), while the other warps are at the
// next row.  us, 4096 x 50,257 bf16 and 64 entries: 151 (by one such warp 163); by the
// warps that hold vectors, at the row's start, 284; loaded ahead, with a barrier a row, 198,
// with a barrier for the entries' warps alone the same: every row waits for the longest
// warp.  Without entries at all, the cross-entropy, 139.
constexpr int kStreamVecs = 3200;  // of a CTA's slice: two buffers of it and the entries, two CTAs an SM
template <int NT>
constexpr int kEntryWarps = NT == 512 ? 3 : 2;
template <int NT>
constexpr int kVecThreads = NT - 32 * kEntryWarps<NT>;  // kVecs vectors each: 3,328 or 1,536

// A count in shared memory: set by one thread, waited for by others (false after kSpins
// polls).
__device__ __forceinline__ void set_count(uint32_t* c, uint32_t v) {
    asm volatile("st.release.cta.shared.u32 [%0], %1;\n" ::"r"(smem_addr(c)), "r"(v) : "memory");
}
__device__ __forceinline__ bool wait_count(const uint32_t* c, uint32_t v) {
    for (int i = 0; i < kSpins; ++i) {
        uint32_t x;
        asm volatile("ld.acquire.cta.shared.u32 %0, [%1];\n" : "=r"(x) : "r"(smem_addr(c)) : "memory");
        if (x >= v) return true;
        __nanosleep(32);
    }
    return false;
}

template <typename T, int NT, int S>
__global__ void __launch_bounds__(NT, 1024 / NT) k_distill_stream(Args<T> a, int32_t slots) {
    extern __shared__ __align__(128) uint8_t dsm[];
    pdl_start();
    constexpr int NV = kVecThreads<NT>, EW = kEntryWarps<NT>;
    constexpr int kParts = S * NV / 32;
    __shared__ __align__(8) float2 parts[2][kParts];  // (m, z) of every warp of the cluster, of used rows in turn
    __shared__ __align__(8) uint64_t full[2], met[2];  // buffers; parts
    __shared__ __align__(8) uint64_t stored[2], read[2];  // a row's vectors are stored; its entries' warps have met it
    __shared__ Entries entries[EW];
    __shared__ Table tables[EW];
    __shared__ uint32_t seen;  // used rows whose parts their entries' warp has met, in order
    __shared__ bool last;
    const int32_t rank = (int32_t)(blockIdx.x % S), first = (int32_t)(blockIdx.x / S), step = (int32_t)(gridDim.x / S);
    const int32_t n = rows_of(a.d_n, a.n_cap), classes = a.classes;
    if (first >= n) return;  // the whole cluster
    if (threadIdx.x == 0) {
        last = false;
        seen = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&met[i], 1);
            mbar_init(&stored[i], NV / 32);
            mbar_init(&read[i], S);
        }
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    __syncthreads();
    if constexpr (S > 1) cluster_sync();  // every CTA runs: its shared memory may be written
    const auto has = [&](int32_t r) { return r < n && row_used(a, r); };
    const float w = weight_of(a);
    // of the used rows so far: row u uses slot u % 2, for the (u / 2)-th time
    uint32_t used = 0;
    if (threadIdx.x < NV) {
        // copies this CTA's slice of row r into buffer b (thread 0)
        const auto fetch = [&](int32_t r, bool u, int b) {
            if (!u) return;
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
        bool u0 = has(first), u1 = has(first + step), u2;
        if (threadIdx.x == 0) {
            fetch(first, u0, 0);
            fetch(first + step, u1, 1);
        }
        uint32_t phases = 0;  // bits 0, 1: parity of the next phase of full[0], full[1]
        int32_t par = 0;      // the row's buffer: alternates over all rows
        for (int32_t r = first; r < n; r += step, par ^= 1, u0 = u1, u1 = u2) {
            u2 = has(r + 2 * step);
            const T* row = a.x + (int64_t)r * a.ld;
            T* out = a.grad ? a.grad + (int64_t)r * a.ld_grad : nullptr;
            if (!u0) {  // the same in the whole cluster
                if (rank == 0 && threadIdx.x == 0) a.loss[r] = 0.f;
                if (out) zero_row<T, NV>(out, classes, rank, S);
                if (threadIdx.x == 0) fetch(r + 2 * step, u2, par);  // this row's buffer was not filled
                continue;
            }
            const uint32_t slot = used & 1u, turn = (used >> 1) & 1u;
            const RowParts<T> part(row, classes);
            const int32_t per = (part.vecs + S - 1) / S, v0 = min(part.vecs, rank * per),
                          count = min(part.vecs, v0 + per) - v0;
            const int32_t edge = rank == 0 && threadIdx.x < 32 ? part.edge((int)threadIdx.x) : -1;
            Held<T, NV> h;
            h.xe = edge >= 0 ? to_f(row[edge]) : -INFINITY;
            if (!mbar_wait(&full[par], (phases >> par) & 1u) && lane_id() == 0) dev_err(ERR_TIMEOUT);
            const uint4* buf = reinterpret_cast<const uint4*>(dsm) + par * slots + threadIdx.x;
#pragma unroll
            for (int k = 0; k < kVecs; ++k)
                h.x[k] = (int32_t)threadIdx.x + k * NV < count ? buf[k * NV] : empty_part<T>();
            reduce_held(h, count, -INFINITY, 0.f, a.l);
            // The parts meet by asynchronous stores that complete on the receiver's
            // barrier.  A slot is written again two used rows later: by then its
            // readers have read it, the warps with vectors before they sent their part
            // of the used row between, the entries' warps before they arrived at `read`.
            if (used >= 2 && !mbar_wait(&read[slot], turn ^ 1u) && lane_id() == 0) dev_err(ERR_TIMEOUT);
            if (threadIdx.x == 0) mbar_expect_tx(&met[slot], kParts * 8);
            if (lane_id() < S) {
                const uint32_t to = smem_addr(&parts[slot][rank * (NV / 32) + (threadIdx.x >> 5)]);
                asm volatile(
                    "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];\n" ::"r"(
                        map_rank(to, lane_id())),
                    "f"(h.m), "f"(h.z), "r"(map_rank(smem_addr(&met[slot]), lane_id()))
                    : "memory");
            }
            __syncwarp();
            if (!mbar_wait(&met[slot], turn) && lane_id() == 0) dev_err(ERR_TIMEOUT);
            phases ^= 1u << par;
            ++used;
            // every thread has its vectors in registers: the buffer is free
            if (threadIdx.x == 0) fetch(r + 2 * step, u2, par);
            if (!out) continue;
            float M, Z;
            join_parts<kParts>(parts[slot], M, Z, a.l);
            const float inv = held_scale(h.m, h.z, w, M, Z, a.l);
            store_held(h, out + part.head + v0 * kE<T>, count, same_phase(row, (const T*)out), inv, a.l);
            if (edge >= 0) put(out + edge, inv * Base(h.m, a.l).of(h.xe));
            __syncwarp();
            if (lane_id() == 0) mbar_arrive(&stored[slot]);
        }
    } else {
        const int e = ((int)threadIdx.x - NV) / 32, lane = (int)lane_id();
        const bool mine = rank == 0 || a.grad;
        Entries& entry = entries[e];
        // the cluster's rows g, g + step, .. of which this warp has the e-th: which are used
        const auto used_of = [&](int32_t g) { return lane < EW && has(g + lane * step); };
        uint32_t flags = __ballot_sync(0xFFFFFFFFu, used_of(first));
        if (mine && first + e * step < n) load_entries<1>(a, first + e * step, 0, n, &entry, rank == 0);
        for (int32_t g = first; g < n; g += EW * step) {
            const int32_t r = g + e * step;
            const bool after = used_of(g + EW * step);
            if (flags >> e & 1u) {
                const uint32_t u = used + (uint32_t)__popc(flags & ((1u << e) - 1u)), slot = u & 1u, turn = (u >> 1) & 1u;
                T* out = a.grad ? a.grad + (int64_t)r * a.ld_grad : nullptr;
                Scale scale = {0.f, 0.f};
                bool twice = false;
                if (mine) {
                    scale = scale_entries(a, entry);
                    __syncwarp();
                    twice = any_twice(a, entry, tables[e]);
                }
                // (a phase of the barrier can be told from the one two before it only when
                // that one is over: rows are met in order)
                if (!wait_count(&seen, u) && lane == 0) dev_err(ERR_TIMEOUT);
                if (!mbar_wait(&met[slot], turn) && lane == 0) dev_err(ERR_TIMEOUT);
                __syncwarp();
                if (lane == 0) set_count(&seen, u + 1);
                float M, Z;
                join_parts<kParts>(parts[slot], M, Z, a.l);
                if (rank == 0) {
                    const float loss = loss_of(a, scale, entry, M, Z);
                    if (lane == 0) put_loss(a, r, loss, M, Z);
                }
                if (out && !mbar_wait(&stored[slot], turn) && lane == 0) dev_err(ERR_TIMEOUT);
                __syncwarp();
                if (lane < S)  // in every CTA of the cluster
                    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(
                                     map_rank(smem_addr(&read[slot]), (uint32_t)lane))
                                 : "memory");
                if (out) {
                    const T* row = a.x + (int64_t)r * a.ld;
                    const RowParts<T> part(row, classes);
                    const int32_t per = (part.vecs + S - 1) / S, v0 = min(part.vecs, rank * per),
                                  count = min(part.vecs, v0 + per) - v0;
                    for (int32_t j = lane; j < a.k; j += 32) put_entries(a, entry, out, part, v0, count, rank, j, twice, w, M, Z);
                }
                __syncwarp();  // before the next row's entries
            }
            used += (uint32_t)__popc(flags);
            flags = __ballot_sync(0xFFFFFFFFu, after);
            if (mine && r + EW * step < n) load_entries<1>(a, r + EW * step, 0, n, &entry, rank == 0);
        }
    }
    __threadfence();
    if constexpr (S > 1) cluster_sync();
    else __syncthreads();
    if (!a.total) return;
    if (rank == 0 && threadIdx.x == 0) {
        __threadfence();
        last = atomicAdd(a.done, 1) == min(step, n) - 1;
    }
    __syncthreads();
    if (last) {
        __threadfence();
        put_total<NT>(a, n);
    }
}

// Counts the rows with a teacher, a part of them a block, and clears the count of
// finished blocks.
constexpr int kCounts = 256;  // blocks at most
__global__ void __launch_bounds__(kCountThreads) k_distill_count(const int32_t* __restrict__ ids,
                                                                 const float* __restrict__ values, int32_t k,
                                                                 int32_t classes, int32_t n_cap,
                                                                 const int32_t* __restrict__ d_n,
                                                                 int32_t* __restrict__ done, float* __restrict__ total) {
    pdl_start();
    __shared__ int32_t sh[kCountThreads / 32 + 1];
    const int32_t n = rows_of(d_n, n_cap), stride = (int32_t)gridDim.x * kCountThreads;
    int32_t v = 0;
#pragma unroll 4
    for (int32_t i = (int32_t)(blockIdx.x * kCountThreads + threadIdx.x); i < n; i += stride)
        v += is_used(__ldg(ids + (int64_t)i * k), __ldg(values + (int64_t)i * k), classes);
    v = block_sum<kCountThreads, int32_t>(v, sh);
    if (threadIdx.x != 0) return;
    done[1 + blockIdx.x] = v;
    if (blockIdx.x != 0) return;
    done[0] = 0;
    if (total && n == 0) total[0] = 0.f, total[1] = 0.f;  // nobody else writes it
}

// ------------------------------------------------ the loss above a temperature
// T^2 sum q (log q - log p), as it is defined, is off by the rounding of the two
// logarithms, some 2^-22, times T^2.  Up to T = 4 that is 2^-18; but the higher T, the
// closer are q and p, and the sum shrinks like 1 / T^2 where the entries have (nearly)
// all of p: with 128 classes and 128 entries the loss was off by 1e-3 of itself at T =
// 100 and by 9e-2 at T = 1000 (now 3e-7).
//
// So it is made of parts that cannot be below 0 (where no class occurs twice).  With u =
// log q - log p, p = q exp(-u), and as q and p sum to 1 each,
//   sum q u = sum q (u + exp(-u) - 1) + rest,  rest = 1 - sum of p over the entries.
// The bracket is a series in u near 0, and q times it is q (u - 1) + p elsewhere.  What
// every u is off by alike (log z_q, log z) counts times the rest and its own square now.
// The rest is the difference it is defined by where the loss is large beside the
// difference's rounding.  Where it is not, the row is read once more: the rest is the
// exponentials' sum over the row less the entries', with what each addition rounds off
// carried along, so that an entry's exponential, the same bits in both, leaves nothing.
//
// A warp a row, from the maximum and sum that the row's own kernel left.  A row of up to
// kByWarp classes is read again by its warp, a longer one by the block (us, by warps / by
// blocks: 100,000 x 128 fp32, all of them read again, 247 / 378; 5000 x 4000 87 / 104; 1000
// x 4000 29 / 38).
constexpr float kPlainTemp = 4.f;
constexpr int kByWarp = 4096;
constexpr float kSmallLoss = 0.125f;  // over T^2 (1 - sum p is off by 2^-20 at most: 8e-6 of it)

// A sum and what its additions rounded off (Knuth's two-sum).
struct Exact {
    float s, off;
    __device__ __forceinline__ void add(float x) {
        const float t = s + x, b = t - s;
        off += (s - (t - b)) + (x - b);
        s = t;
    }
    __device__ __forceinline__ void add(const Exact& o) {
        off += o.off;
        add(o.s);
    }
    __device__ __forceinline__ void add_lanes() {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            add(Exact{__shfl_xor_sync(0xFFFFFFFFu, s, d), __shfl_xor_sync(0xFFFFFFFFu, off, d)});
    }
};

// Adds up a row's exponentials and `sum`, over n threads of which this is t; each warp's sum
// in all its lanes.
template <typename T>
__device__ __forceinline__ Exact sum_part(const Args<T>& a, int32_t r, float M, int32_t t, int32_t n, Exact sum) {
    const T* row = a.x + (int64_t)r * a.ld;
    const RowParts<T> part(row, a.classes);
    const int32_t ce = t < 32 ? part.edge(t) : -1;
    if (ce >= 0) sum.add(exp_from(to_f(row[ce]), M, a.l));
#pragma unroll 4
    for (int32_t v = t; v < part.vecs; v += n) {
        const uint4 u = *reinterpret_cast<const uint4*>(row + part.head + v * kE<T>);
        f2 f[kE<T> / 2];
        pairs_of(u, f);
#pragma unroll
        for (int i = 0; i < kE<T> / 2; ++i) {
            float x, y;
            unpair(f[i], x, y);
            sum.add(exp_from(x, M, a.l));
            sum.add(exp_from(y, M, a.l));
        }
    }
    sum.add_lanes();
    return sum;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_distill_loss(Args<T> a) {
    pdl_start();
    constexpr int kWarps = kThreads / 32;
    __shared__ Entries entries[kWarps];
    struct Again {
        float s, m, z;
        Exact out;  // less the entries' exponentials
        bool is;
    };
    __shared__ Again again[kWarps];
    __shared__ Exact sums[kWarps];
    __shared__ bool last;
    const int warp = (int)(threadIdx.x >> 5), lane = (int)lane_id();
    const int32_t n = rows_of(a.d_n, a.n_cap), groups = (n + kWarps - 1) / kWarps, blocks = min((int32_t)gridDim.x, groups);
    const float square = a.temp * a.temp;
    if (n == 0 && a.total && blockIdx.x == 0 && threadIdx.x == 0) a.total[0] = a.total[1] = 0.f;
    if ((int32_t)blockIdx.x >= blocks) return;
    Entries& e = entries[warp];
    for (int32_t g = (int32_t)blockIdx.x; g < groups; g += (int32_t)gridDim.x) {
        const int32_t r = g * kWarps + warp;
        bool small = false;
        if (r < n && row_used(a, r)) {
            const float2 st = __ldcg(a.stats + r);
            const float M = st.x, Z = st.y;
            load_entries<1>(a, r, 0, n, &e, false);
            const Scale c = scale_entries(a, e);  // (each lane's own entries)
            const float apart = logf(Z / c.zq);
            float s = 0.f, sum = 0.f;
            Exact out = {0.f, 0.f};
            for (int32_t j = lane; j < a.k; j += 32) {
                const float q = e.q[j], x = e.x[j];
                if (q == 0.f) continue;
                if (x == -INFINITY && q > 0.f && Z == Z) {
                    s += INFINITY;
                    continue;
                }
                const float u = fmaf((e.v[j] - c.m) - (x - M), a.inv_temp, apart), ex = exp_from(x, M, a.l), p = ex / Z;
                if (fabsf(u) < 0.5f) {  // (what the series leaves out is below 2^-24 of it)
                    float f = 1.f / 40320.f;
                    f = fmaf(-u, f, 1.f / 5040.f);
                    f = fmaf(-u, f, 1.f / 720.f);
                    f = fmaf(-u, f, 1.f / 120.f);
                    f = fmaf(-u, f, 1.f / 24.f);
                    f = fmaf(-u, f, 1.f / 6.f);
                    f = fmaf(-u, f, 0.5f);
                    s = fmaf(q * f, u * u, s);
                } else {
                    s += fmaf(q, u - 1.f, p);
                }
                sum += p;
                out.add(-ex);
            }
            s = warp_sum(s);
            float loss = s + (1.f - warp_sum(sum));
            if (loss < kSmallLoss) {
                if (a.classes <= kByWarp) {
                    const Exact all = sum_part(a, r, M, lane, 32, out);
                    loss = s + (all.s + all.off) / Z;
                } else {
                    small = true;
                    out.add_lanes();
                    if (lane == 0) again[warp] = {s, M, Z, out, true};
                }
            }
            if (!small && lane == 0) a.loss[r] = loss * square;
        }
        if (a.classes <= kByWarp) continue;
        if (!small && lane == 0) again[warp].is = false;
        if (!__syncthreads_or(small)) continue;
        for (int w = 0; w < kWarps; ++w) {
            if (!again[w].is) continue;
            Exact all = sum_part(a, g * kWarps + w, again[w].m, (int32_t)threadIdx.x, kThreads, Exact{0.f, 0.f});
            if (lane == 0) sums[warp] = all;
            __syncthreads();
            if (threadIdx.x == 0) {
                for (int i = 1; i < kWarps; ++i) all.add(sums[i]);
                all.add(again[w].out);
                a.loss[g * kWarps + w] = (again[w].s + (all.s + all.off) / again[w].z) * square;
            }
            __syncthreads();
        }
    }
    if (!a.total) return;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(a.done, 1) == blocks - 1;
    __syncthreads();
    if (last) {
        __threadfence();
        put_total<kThreads>(a, n);
    }
}

// -------------------------------------------------------------------- host
template <typename T, int NV>
sg_status run_warp(const Args<T>& a, bool small, cudaStream_t s) {
    if constexpr (NV <= 8) if (small) {
        static OncePerDevice set;
        SG_CUDA(allow_smem(set, k_distill_small<T, NV>, kSmallBytes<NV>));
        SG_CUDA(launch_cluster(k_distill_small<T, NV>, kSmallCtas, kSmallThreads, kSmallCtas, s, kSmallBytes<NV>, a));
        return SG_OK;
    }
    int64_t blocks = cdiv(a.n_cap, kThreads / 32);
    if (blocks > (int64_t)num_sms() * kWarpBlocks<NV>) blocks = (int64_t)num_sms() * kWarpBlocks<NV>;
    SG_CUDA(launch_pdl(k_distill_warp<T, NV>, dim3((unsigned)blocks), dim3(kThreads), 0, s, a));
    return SG_OK;
}

template <typename T, int NT, int S>
sg_status run_row(const Args<T>& a, cudaStream_t s) {
    SG_CUDA(launch_cluster(k_distill_row<T, NT, S>, (unsigned)((int64_t)a.n_cap * S), NT, S, s, 0, a));
    return SG_OK;
}

template <typename T, int NT, int S>
sg_status run_stream(const Args<T>& a, int64_t nv, cudaStream_t s) {
    const int32_t slots = (int32_t)cdiv(nv, S);  // of a buffer
    static OncePerDevice set;
    SG_CUDA(allow_smem(set, k_distill_stream<T, NT, S>, 2 * kStreamVecs * 16));
    int64_t clusters = (int64_t)num_sms() * (1024 / NT) / S;
    if (clusters > a.n_cap) clusters = a.n_cap;
    SG_CUDA(launch_cluster(k_distill_stream<T, NT, S>, (unsigned)(clusters * S), NT, S, s, 2 * slots * 16, a, slots));
    return SG_OK;
}

template <typename T>
sg_status run_rows(const Args<T>& a, bool small, int64_t nv, cudaStream_t s) {
    if (nv <= 32) return run_warp<T, 1>(a, small, s);
    if (nv <= 64) return run_warp<T, 2>(a, small, s);
    if (nv <= 128) return run_warp<T, 4>(a, small, s);
    if (nv <= 256) return run_warp<T, 8>(a, small, s);
    // (fewer rows leave warps idle; 700 x 4000 bf16: 12 us, by blocks 14)
    if (a.n_cap >= 4 * num_sms()) {
        if (nv <= 384) return run_warp<T, 12>(a, false, s);
        if (nv <= 512) return run_warp<T, 16>(a, false, s);
    }
    const int wide = nv <= kVecThreads<kThreads> * kVecs ? 1 : nv <= kStreamVecs ? 2 : nv <= 2 * kStreamVecs ? 4 : nv <= 4 * kStreamVecs ? 8 : 16;
    // from shared memory while each CTA has some rows to stream (us, streamed / not: 900 x
    // 6000 fp32 14.9 / 17.4, 500 x 6000 12.2 / 11.5; 300 x 20,000 16.7 / 21.0; 120 x 50,257 20 /
    // 18; 220 x 100,000 55 / 57, 115 x 100,000 37 / 35)
    if (nv <= 8 * kStreamVecs && (int64_t)a.n_cap * wide >= (wide <= 4 ? 4 : 12) * num_sms()) {
        switch (wide) {
            case 1: return run_stream<T, kThreads, 1>(a, nv, s);
            case 2: return run_stream<T, 512, 1>(a, nv, s);
            case 4: return run_stream<T, 512, 2>(a, nv, s);
            case 8: return run_stream<T, 512, 4>(a, nv, s);
            default: return run_stream<T, 512, 8>(a, nv, s);
        }
    }
    // smallest cluster whose registers hold the row, widened while the rows do not
    // fill the SMs; 512 threads when 8 CTAs of 256 do not hold it
    if (nv > 8 * kThreads * kVecs) return run_row<T, 512, 8>(a, s);
    int split = 1;
    while (split < 8 && nv > (int64_t)split * kThreads * kVecs) split *= 2;
    while (split < 8 && (int64_t)a.n_cap * split * 2 <= 2 * num_sms() && nv >= split * 2 * kThreads) split *= 2;
    switch (split) {
        case 1: return run_row<T, kThreads, 1>(a, s);
        case 2: return run_row<T, kThreads, 2>(a, s);
        case 4: return run_row<T, kThreads, 4>(a, s);
        default: return run_row<T, kThreads, 8>(a, s);
    }
}

template <typename T>
sg_status run(Args<T> a, cudaStream_t s) {
    const int64_t nv = cdiv((int64_t)a.classes, kE<T>);  // vectors of a row, at most
    const bool by_warp = nv <= 256;
    // one cluster serves a call whose rows its warps hold at once (4 rows a warp, so that
    // it would serve twice as many, are slower than two launches)
    const int64_t rows = kSmallCtas * (kSmallThreads / 32) * (nv <= 64 ? kSmallRows<2> : kSmallRows<8>);
    const bool small = by_warp && a.n_cap <= rows;
    float* const total = a.total;
    if (a.temp > kPlainTemp) a.total = nullptr;  // the losses are not there yet
    else a.stats = nullptr;
    if (!small) {
        a.counts = (int32_t)cdiv(a.n_cap, 2 * kCountThreads);
        if (a.counts < 1) a.counts = 1;
        if (a.counts > kCounts) a.counts = kCounts;
        SG_CUDA(launch_pdl(k_distill_count, dim3((unsigned)a.counts), dim3(kCountThreads), 0, s, a.ids, a.values, a.k,
                           a.classes, a.n_cap, a.d_n, a.done, total));
        if (a.n_cap == 0) return SG_OK;
    }
    const sg_status st = run_rows<T>(a, small, nv, s);
    if (st != SG_OK || !a.stats) return st;
    if (small) a.counts = 1;
    a.total = total;
    int64_t blocks = cdiv(a.n_cap, kThreads / 32);
    if (blocks < 1) blocks = 1;  // (the total)
    if (blocks > 8 * (int64_t)num_sms()) blocks = 8 * (int64_t)num_sms();
    SG_CUDA(launch_pdl(k_distill_loss<T>, dim3((unsigned)blocks), dim3(kThreads), 0, s, a));
    return SG_OK;
}

// (1 + kCounts) counts; rows' maxima and sums
constexpr size_t kCountBytes = 2048;
size_t ws_bytes(int32_t n_cap) { return kCountBytes + (size_t)n_cap * sizeof(float2); }

}  // namespace

extern "C" size_t sg_distill_workspace(int32_t n_cap, int32_t n_classes) {
    if (n_cap < 0 || n_classes <= 0) return 0;
    return ws_bytes(n_cap);
}

extern "C" sg_status sg_distill(const void* d_logits, int32_t dtype, int32_t n_cap, const int32_t* d_n, int32_t n_classes,
                                int64_t ld, const int32_t* d_ids, const float* d_values, int32_t k, float temperature,
                                int32_t mean, float grad_scale, float* d_loss, float* d_total, void* d_grad,
                                int64_t ld_grad, void* d_workspace, size_t workspace_bytes, sg_stream_t stream) {
    if (dtype != SG_F32 && dtype != SG_BF16) return fail(SG_ERR_UNSUPPORTED, "sg_distill: dtype");
    if (n_cap < 0 || n_cap > 1 << 27 || n_classes <= 0 || n_classes > 2147483647 - 1024)
        return fail(SG_ERR_INVALID_ARG, "sg_distill: bad sizes");
    if (k < 1 || k > SG_MAX_TOP) return fail(SG_ERR_INVALID_ARG, "sg_distill: k must be 1 to %d", SG_MAX_TOP);
    if (!(temperature >= 1e-3f && temperature <= 1e3f))
        return fail(SG_ERR_INVALID_ARG, "sg_distill: the temperature must be 0.001 to 1000");
    if (ld < n_classes || (d_grad && ld_grad < n_classes))
        return fail(SG_ERR_INVALID_ARG, "sg_distill: a row stride is below n_classes");
    if (n_cap > 0 && (!d_logits || !d_ids || !d_values || !d_loss)) return fail(SG_ERR_INVALID_ARG, "sg_distill: NULL array");
    if (!d_workspace || (uintptr_t)d_workspace % 256 || workspace_bytes < ws_bytes(n_cap))
        return fail(SG_ERR_INVALID_ARG, "sg_distill: workspace needs %zu bytes, 256-byte aligned", ws_bytes(n_cap));
    const int e = dtype == SG_F32 ? 4 : 2;
    if ((uintptr_t)d_logits % e || (uintptr_t)d_grad % e ||
        ((uintptr_t)d_ids | (uintptr_t)d_values | (uintptr_t)d_loss | (uintptr_t)d_total) % 4)
        return fail(SG_ERR_INVALID_ARG, "sg_distill: an array is not aligned to its elements");
    if (d_grad == d_logits && d_grad) return fail(SG_ERR_INVALID_ARG, "sg_distill: the gradient may not replace the logits");
    cudaStream_t s = (cudaStream_t)stream;
    const float l = kLog2e / temperature;
    float2* const stats = (float2*)((char*)d_workspace + kCountBytes);
    if (dtype == SG_F32) {
        const Args<float> a = {(const float*)d_logits, (float*)d_grad, ld, ld_grad, d_ids, d_values, d_n, n_cap, n_classes,
                               k, mean ? 1 : 0, grad_scale, temperature, 1.f / temperature, l, d_loss, d_total, (int32_t*)d_workspace, 0, stats};
        return run(a, s);
    }
    const Args<__nv_bfloat16> a = {(const __nv_bfloat16*)d_logits, (__nv_bfloat16*)d_grad, ld, ld_grad, d_ids, d_values,
                                   d_n, n_cap, n_classes, k, mean ? 1 : 0, grad_scale, temperature, 1.f / temperature, l, d_loss, d_total,
                                   (int32_t*)d_workspace, 0, stats};
    return run(a, s);
}
