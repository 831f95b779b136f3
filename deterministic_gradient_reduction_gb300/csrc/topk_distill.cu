// Distillation from a teacher's top logits: loss and gradient.
//
// For a row with student logits z [V] and the teacher's list (ids, t) [K], at
// temperature tau:
//   p = softmax(z / tau);
//   q_k = softmax(t / tau) over the list, or, with the teacher's logsumexp L_T
//   of all its logits, q_k = exp(t_k / tau - L_T) and q_r = 1 - sum_k q_k left
//   for the tokens outside the list (p_r: the student's mass there);
//   L = sum_k q_k (ln q_k - ln p_k) [+ q_r (ln q_r - ln p_r)];
//   loss = scale sum_t w_t L_t;
//   dz_j = dloss scale w / tau (S p_j - sum of the list's q at j      in the list,
//                               p_j (S - q_r / p_r)                   outside),
//   S the sum of all q that L counts: 1, but where q_r is left out (no logit
//   outside the list above -inf) or the list's q exceed 1.
// A row of weight 0 is not read; it and one whose list is empty have loss 0
// and gradient 0.
//
// A row is read twice: once for maximum and sum, once (out of L2) for the
// gradient. It lies across a cluster of CTAs, few enough rows at a time that
// they stay in L2 between the two (below), and few CTAs a row, as each has to
// do what there is to do for the list. The CTAs of a row exchange a (maximum,
// sum) pair a warp through shared memory of the cluster.
//
// With q_r the list's tokens (a bit an element in shared memory) are left out
// of that maximum and sum and have their own, so that p_r is a sum and not a
// difference from 1; the gradient outside is then
//   exp(z_j / tau - m) (S exp(m - lse) - q_r / s),  m, s: maximum and sum outside,
// which stays finite however small p_r is. Exponentials are taken to base 2
// (k = log2(e) / tau): with m a running maximum every one is ex2(z k - fl(m k)),
// sums meet by ex2(fl(m k) - fl(m' k)), so the roundings of these products
// cancel between numerator and sum. A maximum times k below -2^24 counts as -2^24
// there, so that a thread that meets nothing but a mask's values has a sum that
// is small and not infinite; where the maximum outside the list or in it times k
// is beyond 2^24 the row is done again with each of the two subtracted from its
// own elements first. Both sums are then at least 1, however far apart they lie.
//
// Deterministic: a row's sums go over threads, warps, CTAs of the cluster in a
// fixed order set by the type, V, T, K, the alignment, whether there is a tail
// and, for rows of more than 128 KB, whether there is a gradient; the rows'
// losses over one CTA in a fixed order.
//
// Measured: 4096 x 131072 bf16, loss and gradient (2.15 GB) 452 us = 4.75 TB/s;
// what a CTA does once a row (list, exchange, factors) takes about half of a
// row's time and is hidden in part by the SM's other CTAs.
#include <type_traits>

#include "dgr_diag.h"
#include "row_common.cuh"

namespace dgr {
namespace {

using namespace row;

constexpr int kMaxList = 1024;
constexpr int kMaxVocab = 1 << 20;
constexpr int kMaxCluster = 8;
constexpr int kWhereId = 311;
constexpr float kLn2 = 0.69314718055994531f;
// x k - fl(m k) carries the rounding of m k, up to half a unit of its size: up
// to 1/2 below this bound, where it cancels between an exponential and its sum;
// at 1e10 it is in the hundreds, and ex2 would give infinity or 0.
constexpr float kFar = 16777216.0f;

struct DistillParams {
    const void *z;
    int64_t ld;
    int32_t T, V, K;
    const int32_t *ids;
    int64_t ld_ids;
    const float *teacher;
    int64_t ld_t;
    const float *teacher_lse, *weights, *dloss;
    float inv_tau, k2, scale;  // k2 = log2(e) / tau
    float *row_loss, *loss;
    void *dz;
    int64_t ld_dz;
    int32_t per;         // vectors of a row a CTA
    WsHeader *hdr;       // pad[0]: clusters done
    Sched sched;
};

// ---- cluster and copy instructions ---------------------------------------------

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// All threads of the cluster's CTAs; what was written before is seen after.
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(const void *p, uint32_t rank) {
    uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}
__device__ __forceinline__ void remote_store(uint32_t a, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ void remote_store(uint32_t a, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
// ---- a row's parts -------------------------------------------------------------

// A row as whole 16-byte vectors between a few single elements; CTA `rank` of
// its cluster has `per` vectors from rank * per on (fewer at the row's end),
// CTA 0 the singles too.
template <typename T>
struct RowView {
    static constexpr int VEC = 16 / static_cast<int>(sizeof(T));
    int head, n_vec, n_single, first, count;
    __host__ __device__ __forceinline__ RowView(const T *z, int V, int rank, int per) {
        const int off = static_cast<int>(reinterpret_cast<uintptr_t>(z) & 15) / static_cast<int>(sizeof(T));
        head = off ? VEC - off : 0;
        head = head < V ? head : V;
        n_vec = (V - head) / VEC;
        n_single = V - n_vec * VEC;
        first = rank * per < n_vec ? rank * per : n_vec;
        count = per < n_vec - first ? per : n_vec - first;
        if (rank != 0) n_single = 0;
    }
    // element of single i: before the vectors, then behind them
    __device__ __forceinline__ int single(int i) const { return i < head ? i : n_vec * VEC + i; }
    // where element j lies in this CTA: an element of its vectors, kSingle + i, or -1
    static constexpr int kSingle = 1 << 24;
    __device__ __forceinline__ int place(int j) const {
        const int e = j - head;
        if (e >= 0 && e < n_vec * VEC) {
            const int mine = e - first * VEC;
            return mine >= 0 && mine < count * VEC ? mine : -1;
        }
        return n_single ? kSingle + (e < 0 ? j : j - n_vec * VEC) : -1;
    }
};

// A CTA's part of the gradient's row, `elements` long from `own` on: `lead`
// elements before its first 16-byte boundary, then n_out whole vectors. With a
// lead they lie across the logits' vectors, and vector v is made of the logits'
// vectors v and v + 1; without one of v alone, and v + 1 is not read: behind the
// last vector of the last row there may be no memory.
template <typename T>
struct GradView {
    static constexpr int VEC = 16 / static_cast<int>(sizeof(T));
    int lead, n_out;
    __host__ __device__ __forceinline__ GradView(const T *own, int elements) {
        const int off = static_cast<int>(reinterpret_cast<uintptr_t>(own) & 15) / static_cast<int>(sizeof(T));
        lead = off ? VEC - off : 0;
        lead = lead < elements ? lead : elements;
        n_out = (elements - lead) / VEC;
    }
    __host__ __device__ __forceinline__ bool has(int v) const { return v < n_out; }
    __host__ __device__ __forceinline__ bool takes_next(int v) const { return v < n_out && lead != 0; }
};

// fl(m k), at least -kFar: elements further below give little or 0, never inf - inf.
__device__ __forceinline__ float scaled_max(float m, float k) { return fmaxf(__fmul_rn(m, k), -kFar); }

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, s));
    return v;
}

// A maximum and the sum of exp2(x k - fl(m k)); the warp's from the lanes'.
struct Pair {
    float m, s;
    __device__ __forceinline__ void over_warp(float k) {
        const float top = warp_max(m);
        s = warp_sum(__fmul_rn(s, ex2(__fadd_rn(scaled_max(m, k), -scaled_max(top, k)))));
        m = top;
    }
};

// Maximum of a vector's elements (a NaN is passed over: it shows in the sum).
template <typename T, int U>
__device__ __forceinline__ float max_of(const uint4 (&r)[U]) {
    if constexpr (sizeof(T) == 2) {
        auto h = [](uint32_t v) { return *reinterpret_cast<const __nv_bfloat162 *>(&v); };
        __nv_bfloat162 m = h(r[0].x);
#pragma unroll
        for (int u = 0; u < U; ++u) m = __hmax2(m, __hmax2(__hmax2(h(r[u].x), h(r[u].y)), __hmax2(h(r[u].z), h(r[u].w))));
        return fmaxf(__low2float(m), __high2float(m));
    } else {
        float m = -INFINITY;
#pragma unroll
        for (int u = 0; u < U; ++u)
            m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(r[u].x), __uint_as_float(r[u].y)), fmaxf(__uint_as_float(r[u].z), __uint_as_float(r[u].w))));
        return m;
    }
}

// Running maximum m, c = fl(m k) and sum of exp2(x k - c) of a thread's elements.
struct Running {
    float m = -INFINITY, c = -kFar;
    float2 s = make_float2(0.0f, 0.0f);
    __device__ __forceinline__ void raise(float top, float k) {
        if (top > m) {
            m = top;
            const float to = scaled_max(top, k), down = ex2(__fadd_rn(c, -to));
            s = mul2(s, make_float2(down, down));
            c = to;
        }
    }
    template <int N>
    __device__ __forceinline__ void add(float (&x)[N], float k) {
        vec_fma(x, k, -c);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            s.x = __fadd_rn(s.x, ex2(x[i]));
            s.y = __fadd_rn(s.y, ex2(x[i + 1]));
        }
    }
};

// The list's bytes: ids, then teacher logits.
__host__ __device__ inline size_t list_bytes(int K) { return (static_cast<size_t>(K) * 8 + 15) / 16 * 16; }

// Vectors of a row a CTA, batches of 4 of a thread's in them (2 or 8 in flight
// are slower: 544 us instead of 461 for 4096 x 131072 bf16; 60 instead of 56 for
// 2048 x 32768 fp32); the list's bits have a word for each batch.
inline int vectors(int V, int size, int es) { return (V / (16 / es) + size - 1) / size; }
__host__ __device__ inline int batches(int per, int threads) { return (per + threads * 4 - 1) / (threads * 4); }

// Dynamic shared memory: the lists of this row and the next, the student's
// logits at the entries, their places [K], and the list's bits.
size_t distill_smem(int K, int V, int threads, int size, int es) {
    return 2 * list_bytes(K) + static_cast<size_t>(K) * 8 + static_cast<size_t>(batches(vectors(V, size, es), threads)) * threads * 4;
}

// At most 57,344 bytes: lists of 1024, and a row of 2^20 32-bit logits over 8 CTAs.
constexpr size_t kMostSmem = 56 * 1024;

template <typename T, int NT, bool TAIL>
__global__ void __launch_bounds__(NT, 1024 / NT) distill_rows(const DistillParams p) {
    using View = RowView<T>;
    constexpr int VEC = View::VEC, W = NT / 32, U = 4;  // U vectors of a thread in flight, one word of bits
    extern __shared__ __align__(16) char smem[];
    __shared__ float4 s_pair[2][kMaxCluster * W];  // the cluster's warps, by row parity: outside the list, in it
    __shared__ float s_loss[2][kMaxCluster * W];   // likewise their parts of a row's loss
    __shared__ float3 s_list;                      // ln of the list's normaliser in two parts (one sum of them
                                                   // would be rounded at its own size), sum of its q
    __shared__ float s_base;                       // subtracted from the logits at the list's entries before scaling
    __shared__ int s_any, last;
    __shared__ uint32_t s_twice;                   // the row (item + 1) in whose list an id came twice
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int size = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
    const uint32_t n_clusters = gridDim.x / size, T_rows = static_cast<uint32_t>(p.T);
    const int K = p.K;
    auto ids_of = [&](uint32_t n) { return reinterpret_cast<int32_t *>(smem + (n & 1) * list_bytes(K)); };
    float *s_z = reinterpret_cast<float *>(smem + 2 * list_bytes(K));      // [K]
    int32_t *s_copy = reinterpret_cast<int32_t *>(s_z + K);                // [K]: place, with kCopy where the id came before
    uint32_t *s_bits = reinterpret_cast<uint32_t *>(s_copy + K);           // [batches][NT]
    constexpr int kCopy = 1 << 30;

    auto row_of = [&](uint32_t i) { return static_cast<int64_t>(sched_item(p.sched, i)); };
    auto weight_of = [&](uint32_t i) { return i < T_rows ? (p.weights ? __ldg(p.weights + row_of(i)) : 1.0f) : 0.0f; };
    // the list of item i, the n-th of this cluster, on its way
    auto fetch_list = [&](uint32_t i, uint32_t n, float weight) {
        if (i < T_rows && weight != 0.0f) {
            const int64_t row = row_of(i);
            int32_t *ids = ids_of(n);
            for (int k = tid; k < K; k += NT) {
                copy_async<4>(ids + k, p.ids + row * p.ld_ids + k);
                copy_async<4>(ids + K + k, p.teacher + row * p.ld_t + k);
            }
        }
        copy_commit();
    };
    // ln of an entry's q. The list's own maximum is subtracted before 1 / tau, as
    // it may be out of range after it; the logsumexp is given at temperature tau.
    auto log_q = [&](float t, float2 base) {
        return __fadd_rn(TAIL ? __fadd_rn(__fmul_rn(t, p.inv_tau), -base.x) : __fmul_rn(__fadd_rn(t, -base.x), p.inv_tau), -base.y);
    };
    const int list_warps = min(W, (K + 31) / 32);  // warps that hold entries
    int64_t loss_row = -1;      // CTA 0, last warp: a row whose loss waits for the other CTAs' parts
    float loss_tail = 0.0f;
    uint32_t live_n = 0;        // rows worked on: the exchange's parity
    auto finish_loss = [&]() {  // their parts have come with the last cluster barrier
        if (loss_row < 0) return;
        float L = 0.0f;
        for (int j = lane; j < size * list_warps; j += 32) L = __fadd_rn(L, s_loss[(live_n & 1) ^ 1][j]);
        L = __fadd_rn(loss_tail, warp_sum(L));
        if (lane == 0) p.row_loss[loss_row] = L;
        loss_row = -1;
    };

    uint32_t item = blockIdx.x / size;
    float weight = weight_of(item), weight_next = weight_of(item + n_clusters);
    if (tid == 0) s_twice = 0;
    for (int j = tid; j < batches(p.per, NT) * NT; j += NT) s_bits[j] = 0;
    fetch_list(item, 0, weight);
    __syncthreads();
    for (uint32_t n = 0; item < T_rows; ++n, item += n_clusters) {
        const int64_t row = row_of(item);
        const T *z = static_cast<const T *>(p.z) + row * p.ld;
        T *dz = static_cast<T *>(p.dz) + row * p.ld_dz;
        const View view(z, p.V, rank, p.per);
        const char *first = reinterpret_cast<const char *>(z + view.head) + static_cast<int64_t>(view.first) * 16;
        int32_t *ids = ids_of(n);
        const float *teacher = reinterpret_cast<const float *>(ids + K);
        copy_wait();  // each thread's own part of the list
        const float weight_2 = weight_of(item + 2 * n_clusters);
        float a = 0.0f, c_rest = 0.0f, f = 0.0f, c_all = 0.0f, inv_mass = 0.0f, total = 1.0f;
        float shift = 0.0f;                // subtracted before scaling outside the list
        float rest_s = 0.0f, left = 0.0f;  // sum outside the list, q left for it
        bool live = false;
        if (weight != 0.0f) {
            // the list's entries in this CTA: where they lie, their bits. An
            // entry whose bit is set already is a copy (without a tail it does not
            // matter which of the two: the other writes the sum of both).
            for (int k = tid; k < K; k += NT) {
                const int id = ids[k];
                int at = id >= 0 && id < p.V ? view.place(id) : -1;
                if (at >= View::kSingle) {
                    for (int j = 0; j < k; ++j)
                        if (__ldg(p.ids + row * p.ld_ids + j) == id) at |= kCopy;
                } else if (at >= 0) {
                    const int v = at / VEC, j = v / NT;  // vector j of its thread
                    const uint32_t bit = 1u << (j % U * VEC + at % VEC);
                    if (atomicOr(&s_bits[j / U * NT + v % NT], bit) & bit) at |= kCopy;
                }
                if (at >= 0 && (at & kCopy)) s_twice = item + 1;
                s_copy[k] = at;
                if (k >= NT && at >= 0) s_z[k] = to_f32(z[id]);
            }
            // the student's logit at this thread's first entry, on its way during the pass
            raw_t<T, 1> z_raw = 0;
            if (tid < K) load_if<false>(z_raw, z + max(ids[tid], 0), s_copy[tid] >= 0);
            __syncthreads();
            fetch_list(item + n_clusters, n + 1, weight_next);
            if (w == W - 1) {  // the list's sums (read behind the cluster barrier)
                float top = -INFINITY, sum = 0.0f;
                const float lse_t = TAIL ? __ldg(p.teacher_lse + row) : 0.0f;
                bool any = false, bad = false;
                for (int k = lane; k < K; k += 32) {
                    const int id = ids[k];
                    bad |= id >= p.V;
                    if (id < 0 || id >= p.V) continue;
                    any |= TAIL || !(teacher[k] == -INFINITY);
                    if (TAIL) sum = __fadd_rn(sum, expf(__fadd_rn(__fmul_rn(teacher[k], p.inv_tau), -lse_t)));
                    else top = fmaxf(top, teacher[k]);
                }
                if (!TAIL) {
                    top = warp_max(top);
                    if (!(top > -INFINITY)) top = 0.0f;
                    for (int k = lane; k < K; k += 32)
                        if (ids[k] >= 0 && ids[k] < p.V) sum = __fadd_rn(sum, expf(__fmul_rn(__fadd_rn(teacher[k], -top), p.inv_tau)));
                }
                sum = warp_sum(sum);
                any = __any_sync(0xffffffffu, any);
                if (__any_sync(0xffffffffu, bad) && rank == 0 && lane == 0) record_error(p.hdr, DGR_ERR_INVALID_ARG, kWhereId);
                if (lane == 0) {
                    s_any = any;
                    s_list = TAIL ? make_float3(lse_t, 0.0f, sum) : make_float3(top, logf(sum), 1.0f);
                }
            }
            float shift_in = 0.0f;  // subtracted in the list's sum
            for (bool again = false;; again = true) {  // a second time only where k times a maximum is out of range
                Running run;
                auto pass = [&](auto shifted) {
                    const char *src = first + tid * 16;
                    int b = tid;
                    for (int v = tid; v < view.count; v += U * NT, src += static_cast<size_t>(U) * NT * 16, b += NT) {
                        uint4 r[U];
                        constexpr uint32_t low = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;  // -inf
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            r[u] = make_uint4(low, low, low, low);
                            load_if<false>(r[u], src + u * NT * 16, v + u * NT < view.count);
                        }
                        const uint32_t bits = TAIL ? s_bits[b] : 0;
                        if (bits) {
#pragma unroll
                            for (int u = 0; u < U; ++u) {
                                uint32_t q[4] = {r[u].x, r[u].y, r[u].z, r[u].w};
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    if constexpr (sizeof(T) == 4) {
                                        if (bits >> (u * 4 + i) & 1) q[i] = low;
                                    } else {
                                        const uint32_t two = bits >> (u * 8 + 2 * i) & 3;
                                        if (two & 1) q[i] = (q[i] & 0xffff0000u) | 0xff80u;
                                        if (two & 2) q[i] = (q[i] & 0xffffu) | 0xff800000u;
                                    }
                                }
                                r[u] = make_uint4(q[0], q[1], q[2], q[3]);
                            }
                        }
                        const float top = max_of<T, U>(r);
                        run.raise(shifted.value ? __fadd_rn(top, -shift) : top, p.k2);
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            float x[VEC];
                            unpack<T, VEC>(r[u], x);
                            if constexpr (shifted.value)
#pragma unroll
                                for (int i = 0; i < VEC; ++i) x[i] = __fadd_rn(x[i], -shift);
                            run.add(x, p.k2);
                        }
                    }
                };
                if (shift == 0.0f) pass(std::false_type{});
                else pass(std::true_type{});
                if (tid < view.n_single) {
                    const int j = view.single(tid);
                    bool listed = false;
                    if (TAIL)
                        for (int k = 0; k < K; ++k) listed |= ids[k] == j;
                    if (!listed) {
                        const float x = __fadd_rn(to_f32(z[j]), -shift);
                        run.raise(x, p.k2);
                        run.s.x = __fadd_rn(run.s.x, ex2(__fmaf_rn(x, p.k2, -run.c)));
                    }
                }
                Pair rest{run.m, __fadd_rn(run.s.x, run.s.y)}, in{-INFINITY, 0.0f};
                rest.over_warp(p.k2);
                if (tid < K) {
                    float one[1];
                    unpack<T, 1>(z_raw, one);
                    s_z[tid] = one[0];
                }
                if (TAIL && w < list_warps) {  // the list's tokens in this CTA, each once
                    // which of two threads set a bit first is chance, and the sum would
                    // take the entry of one or the other: the first in the list counts
                    if (s_twice == item + 1)
                        for (int k = tid; k < K; k += NT)
                            if (s_copy[k] >= 0) {
                                int at = s_copy[k] & ~kCopy;
                                for (int j = 0; j < k; ++j)
                                    if (ids[j] == ids[k]) at |= kCopy;
                                s_copy[k] = at;
                            }
                    for (int k = tid; k < K; k += NT)
                        if (s_copy[k] >= 0 && !(s_copy[k] & kCopy)) in.m = fmaxf(in.m, __fadd_rn(s_z[k], -shift_in));
                    const float ci = scaled_max(in.m, p.k2);
                    for (int k = tid; k < K; k += NT)
                        if (s_copy[k] >= 0 && !(s_copy[k] & kCopy)) in.s = __fadd_rn(in.s, ex2(__fmaf_rn(__fadd_rn(s_z[k], -shift_in), p.k2, -ci)));
                    in.over_warp(p.k2);
                }
                __syncwarp();
                if (lane < size) remote_store(remote(&s_pair[live_n & 1][rank * W + w], lane), make_float4(rest.m, rest.s, in.m, in.s));
                __syncwarp();
                if (size > 1) cluster_barrier();
                else __syncthreads();
                rest = Pair{-INFINITY, 0.0f};
                in = Pair{-INFINITY, 0.0f};
                for (int j = lane; j < size * W; j += 32) {
                    const float4 got = s_pair[live_n & 1][j];
                    rest.m = fmaxf(rest.m, got.x);
                    in.m = fmaxf(in.m, got.z);
                }
                rest.m = warp_max(rest.m);
                if (TAIL) in.m = warp_max(in.m);
                c_rest = scaled_max(rest.m, p.k2);
                const float c_in = scaled_max(in.m, p.k2);
                for (int j = lane; j < size * W; j += 32) {
                    const float4 got = s_pair[live_n & 1][j];
                    rest.s = __fadd_rn(rest.s, __fmul_rn(got.y, ex2(__fadd_rn(scaled_max(got.x, p.k2), -c_rest))));
                    if (TAIL) in.s = __fadd_rn(in.s, __fmul_rn(got.w, ex2(__fadd_rn(scaled_max(got.z, p.k2), -c_in))));
                }
                rest.s = warp_sum(rest.s);
                if (TAIL) in.s = warp_sum(in.s);
                auto far = [&](float m) { return fabsf(m) < INFINITY && fabsf(__fmul_rn(m, p.k2)) >= kFar; };
                if (!again && (far(rest.m) || (TAIL && far(in.m)))) {  // the same in every warp of the cluster
                    if (far(rest.m)) shift = rest.m;
                    if (TAIL && far(in.m)) shift_in = in.m;
                    if (size > 1) cluster_barrier();  // before the pairs are written over
                    else __syncthreads();
                    continue;
                }
                // the two maxima's exponents below the row's own maximum
                float gap = 0.0f, gap_in = 0.0f, base_z = 0.0f;
                if (!again) {
                    c_all = TAIL ? scaled_max(fmaxf(rest.m, in.m), p.k2) : c_rest;
                    gap = __fadd_rn(c_rest, -c_all);
                    gap_in = __fadd_rn(c_in, -c_all);
                } else {  // a maximum that was subtracted is 0 now
                    const float m_rest = shift != 0.0f ? shift : rest.m, m_in = shift_in != 0.0f ? shift_in : in.m;
                    base_z = TAIL ? fmaxf(m_rest, m_in) : m_rest;
                    gap = __fmul_rn(__fadd_rn(m_rest, -base_z), p.k2);
                    gap_in = __fmul_rn(__fadd_rn(m_in, -base_z), p.k2);
                    c_all = 0.0f;
                }
                live = s_any != 0;
                const float sum_q = s_list.z;
                const float down = ex2(gap);
                total = TAIL ? __fmaf_rn(rest.s, down, __fmul_rn(in.s, ex2(gap_in))) : rest.s;
                const float inv = 1.0f / total;
                const float q_rest = TAIL && rest.m != -INFINITY ? fmaxf(__fadd_rn(1.0f, -sum_q), 0.0f) : 0.0f;
                inv_mass = __fmul_rn(inv, !TAIL || q_rest > 0.0f ? 1.0f : sum_q);
                f = __fmul_rn(__fmul_rn(__fmul_rn(p.scale, weight), p.inv_tau), p.dloss ? __ldg(p.dloss) : 1.0f);
                a = __fmul_rn(TAIL ? __fadd_rn(__fmul_rn(down, inv_mass), q_rest > 0.0f ? -q_rest / rest.s : 0.0f) : inv, f);
                if (tid == 0) s_base = base_z;
                rest_s = rest.s;
                left = q_rest;
                break;
            }
        } else {
            fetch_list(item + n_clusters, n + 1, weight_next);
        }
        if (p.dz) {
            // the gradient of four words' elements
            auto gradient = [&](uint4 r, auto shifted) {
                float x[VEC];
                unpack<T, VEC>(r, x);
                if constexpr (shifted.value)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) x[i] = __fadd_rn(x[i], -shift);
                vec_fma(x, p.k2, -c_rest);
#pragma unroll
                for (int i = 0; i < VEC; ++i) x[i] = ex2(x[i]);
                vec_scale(x, a);
                return pack<T, VEC>(x);
            };
            T *own = dz + view.head + static_cast<int64_t>(view.first) * VEC;  // this CTA's part of the gradient's row
            // elements before its first 16-byte boundary: its vectors are then
            // made of two neighbouring ones of the logits
            const GradView<T> out(own, view.count * VEC);
            const int lead = out.lead, n_out = out.n_out;
            auto pass = [&](auto shifted, auto aligned_too) {
                constexpr int F = aligned_too.value ? U : 2;
                for (int v = tid; v < n_out; v += F * NT) {
                    const char *src = first + static_cast<int64_t>(v) * 16;
                    uint4 r[F], next[F];
#pragma unroll
                    for (int u = 0; u < F; ++u) {
                        r[u] = next[u] = make_uint4(0, 0, 0, 0);
                        load_if<false>(r[u], src + u * NT * 16, out.has(v + u * NT));
                        if constexpr (!aligned_too.value) load_if<false>(next[u], src + u * NT * 16 + 16, out.takes_next(v + u * NT));
                    }
#pragma unroll
                    for (int u = 0; u < F; ++u) {
                        if constexpr (!aligned_too.value) {
                            const int by = lead * static_cast<int>(sizeof(T)) * 8;
                            uint32_t q[8] = {r[u].x, r[u].y, r[u].z, r[u].w, next[u].x, next[u].y, next[u].z, next[u].w};
                            if (by & 64)
#pragma unroll
                                for (int i = 0; i < 6; ++i) q[i] = q[i + 2];
                            if (by & 32)
#pragma unroll
                                for (int i = 0; i < 5; ++i) q[i] = q[i + 1];
                            r[u] = make_uint4(__funnelshift_r(q[0], q[1], by & 31), __funnelshift_r(q[1], q[2], by & 31),
                                              __funnelshift_r(q[2], q[3], by & 31), __funnelshift_r(q[3], q[4], by & 31));
                        }
                        if (out.has(v + u * NT)) reinterpret_cast<uint4 *>(own + lead)[v + u * NT] = gradient(r[u], shifted);
                    }
                }
            };
            if (!live) {  // zeros, whatever the row holds
                for (int v = tid; v < n_out; v += NT) reinterpret_cast<uint4 *>(own + lead)[v] = make_uint4(0, 0, 0, 0);
            } else if (shift != 0.0f) {
                pass(std::true_type{}, std::false_type{});
            } else if (lead == 0) {
                pass(std::false_type{}, std::true_type{});
            } else {
                pass(std::false_type{}, std::false_type{});
            }
            if (tid < view.count * VEC - n_out * VEC) {  // elements around the vectors
                const int j = tid < lead ? tid : n_out * VEC + tid;
                const float in = to_f32(reinterpret_cast<const T *>(first)[j]);
                const float x = live ? __fmul_rn(ex2(__fmaf_rn(__fadd_rn(in, -shift), p.k2, -c_rest)), a) : 0.0f;
                *reinterpret_cast<raw_t<T, 1> *>(own + j) = pack<T, 1>(&x);
            }
            if (tid < view.n_single) {
                const int j = view.single(tid);
                const float x = live ? __fmul_rn(ex2(__fmaf_rn(__fadd_rn(to_f32(z[j]), -shift), p.k2, -c_rest)), a) : 0.0f;
                *reinterpret_cast<raw_t<T, 1> *>(dz + j) = pack<T, 1>(&x);
            }
        }
        if (weight != 0.0f) {
            __syncthreads();
            if (p.row_loss && rank == 0 && w == W - 1) {
                finish_loss();
                loss_row = row;
                loss_tail = 0.0f;
                if (left > 0.0f && live) {
                    loss_tail = __fmul_rn(left, __fadd_rn(logf(left), -__fadd_rn(__fmaf_rn(__fadd_rn(c_rest, -c_all), kLn2, logf(rest_s)), -logf(total))));
                    // what was subtracted, times q_r before 1 / tau: the exponent alone may be out of range
                    const float apart = __fadd_rn(s_base, -shift);
                    if (apart != 0.0f) loss_tail = __fmaf_rn(__fmul_rn(left, apart), p.inv_tau, loss_tail);
                }
            }
            // the list's entries: their part of the loss, their tokens' gradient
            if (w < list_warps) {
                float part = 0.0f;
                const float2 base = make_float2(s_list.x, s_list.y);
                const float ln_total = logf(total), base_z = s_base;
                for (int k = tid; k < K; k += NT) {
                    const int at = s_copy[k] & ~kCopy;
                    if (s_copy[k] < 0) continue;
                    if (at < View::kSingle) s_bits[at / VEC / NT / U * NT + at / VEC % NT] = 0;  // free again
                    if (!live) continue;
                    const float lq = log_q(teacher[k], base);
                    float q = expf(lq);
                    const float below = __fadd_rn(s_z[k], -base_z);
                    const float x = __fmaf_rn(below, p.k2, -c_all);  // log2 of p times the total
                    if (q != 0.0f) {
                        if (x > -1e30f || !(fabsf(below) < INFINITY)) part = __fmaf_rn(q, __fadd_rn(lq, -__fmaf_rn(x, kLn2, -ln_total)), part);
                        else part = __fmaf_rn(-__fmul_rn(q, below), p.inv_tau, part);  // x may be out of range; the rest is nothing beside it
                    }
                    if (!p.dz || (s_copy[k] & kCopy)) continue;
                    const int id = ids[k];
                    if (s_twice == item + 1) {
                        q = 0.0f;
                        for (int j = 0; j < K; ++j)
                            if (ids[j] == id) q = __fadd_rn(q, expf(log_q(teacher[j], base)));
                    }
                    const float g = __fmul_rn(__fmaf_rn(ex2(x), inv_mass, -q), f);
                    *reinterpret_cast<raw_t<T, 1> *>(dz + id) = pack<T, 1>(&g);
                }
                if (p.row_loss) {
                    part = warp_sum(part);
                    // read behind the next cluster barrier
                    if (lane == 0) remote_store(remote(&s_loss[live_n & 1][rank * list_warps + w], 0), part);
                }
            }
            ++live_n;
        }
        __syncthreads();
        weight = weight_next;
        weight_next = weight_2;
    }
    copy_wait();
    __syncwarp();
    if (size > 1) cluster_barrier();  // the last row's parts; no CTA leaves before its shared memory is read
    else __syncthreads();
    if (rank != 0) return;
    if (w == W - 1) finish_loss();
    // rows without weight: no loss
    if (p.row_loss && p.weights)
        for (uint32_t i = blockIdx.x / size + tid * n_clusters; i < T_rows; i += NT * n_clusters)
            if (weight_of(i) == 0.0f) p.row_loss[row_of(i)] = 0.0f;
    if (!p.loss) return;
    // the cluster that ends last adds the rows' losses
    __syncthreads();
    if (tid == 0) {
        __threadfence();
        last = atomicAdd(&p.hdr->pad[0], 1) == static_cast<int>(n_clusters) - 1;
        __threadfence();
    }
    __syncthreads();
    if (!last) return;
    float s[1] = {0.0f};
    for (int t = tid; t < p.T; t += NT) {
        const float wt = p.weights ? __ldg(p.weights + t) : 1.0f;
        // scaled first: the sum is out of range only where the loss is
        if (wt != 0.0f) s[0] = __fmaf_rn(__fmul_rn(p.scale, wt), __ldcg(p.row_loss + t), s[0]);
    }
    float *buf = reinterpret_cast<float *>(s_pair);  // free by now
    block_sum<1>(s, buf, W);
    if (tid == 0) {
        *p.loss = s[0];
        p.hdr->pad[0] = 0;  // ready for the next call
    }
}

// Host side -------------------------------------------------------------------

template <typename T, int NT, bool TAIL>
dgr_status launch_rows(DistillParams &p, int cluster, int sms, cudaStream_t s) {
    auto *k = distill_rows<T, NT, TAIL>;
    p.per = vectors(p.V, cluster, sizeof(T));
    const size_t smem = distill_smem(p.K, p.V, NT, cluster, sizeof(T));
    const dgr_status st = allow_smem(k, smem, kMostSmem);
    if (st != DGR_OK) return st;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(cluster);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    // One wave: as many clusters as the device holds at once (a cluster's CTAs
    // share a part of the SMs, so this is less than the SMs over its size; a
    // few clusters more would each take their share of the rows afterwards:
    // 4096 x 131072 bf16 over 4 CTAs a row 855 us without this, 575 with). An SM
    // holds at least two of the CTAs, so clusters of no more CTAs than there are
    // SMs fit without asking (0.4 us on the host).
    int clusters = p.T > 0 ? p.T : 1;
    if (static_cast<int64_t>(p.T) * cluster > sms &&
        (cudaOccupancyMaxActiveClusters(&clusters, k, &cfg) != cudaSuccess || clusters < 1))
        return DGR_ERR_CUDA;
    const int within = sms * (1024 / NT) / cluster;  // a green context's, or the test's cap
    if (clusters > within) clusters = within > 0 ? within : 1;
    if (clusters > p.T) clusters = p.T > 0 ? p.T : 1;
    const unsigned capped = sched_grid(static_cast<unsigned>(clusters * cluster)) / cluster;
    cfg.gridDim = dim3((capped > 0 ? capped : 1) * cluster);
    return cudaLaunchKernelEx(&cfg, k, p) == cudaSuccess ? DGR_OK : DGR_ERR_CUDA;
}

template <typename T, bool TAIL>
dgr_status launch_size(DistillParams &p, int sms, cudaStream_t s) {
    if (p.V < 8192) return launch_rows<T, 128, TAIL>(p, 1, sms, s);
    // A CTA does a list's work for every row it has a part of, so few CTAs a
    // row. With a gradient a row of up to 128 KB has one, a longer one more, so
    // that the CTAs of the device hold no more than about 80 MB at a time and
    // the second reading finds most of it in L2: 1021 x 50001 bf16 (100 KB) 53
    // us with 1, 58 with 2. Longer rows have CTAs of 512 threads (4096 x 131072
    // bf16, 2 CTAs a row: 464 us with 512, 486 with 256), others of 256 (2048 x
    // 32768 fp32 forward 56 us with 256, 66 with 512). A loss alone reads its rows
    // once and does best with one CTA of 256 up to 256 KB (at 640 KB 117 us, 109
    // with one of 512: 800 x 160000 fp32), though a
    // loss has other bits then than with its gradient: 4096 x 131072 bf16 199 us
    // so, 218 with one of 512, 283 as with the gradient; the gradient takes 498,
    // 476 and 464.
    const bool is_long = p.dz && static_cast<int64_t>(p.V) * static_cast<int64_t>(sizeof(T)) > (128 << 10);
    int cluster = 1;
    while (is_long && cluster < kMaxCluster && static_cast<int64_t>(p.V) * static_cast<int64_t>(sizeof(T)) > (128 << 10) * cluster) cluster <<= 1;
    // few rows: a row over more CTAs, down to 4096 elements each
    while (cluster < kMaxCluster && static_cast<int64_t>(p.T) * cluster * 2 <= 304 && p.V >= 4096 * cluster * 2) cluster <<= 1;
    // the list's bits leave room for four CTAs an SM
    while (cluster < kMaxCluster && distill_smem(p.K, p.V, 256, cluster, sizeof(T)) > 48 * 1024) cluster <<= 1;
    return is_long ? launch_rows<T, 512, TAIL>(p, cluster, sms, s) : launch_rows<T, 256, TAIL>(p, cluster, sms, s);
}

// The end, in elements from the row's start, of the vectors that the gradient
// pass reads in a row of V elements at z with its gradient at dz, over `ctas`
// CTAs (the walk of distill_rows, by the same RowView and GradView).
template <typename T>
int64_t gradient_reads(int V, const T *z, const T *dz, int ctas) {
    constexpr int VEC = RowView<T>::VEC;
    int64_t end = 0;
    for (int rank = 0; rank < ctas; ++rank) {
        const RowView<T> view(z, V, rank, vectors(V, ctas, sizeof(T)));
        const int64_t first = view.head + static_cast<int64_t>(view.first) * VEC;
        const GradView<T> out(dz + first, view.count * VEC);
        for (int v = 0; out.has(v); ++v) {
            const int64_t e = first + static_cast<int64_t>(v + (out.takes_next(v) ? 2 : 1)) * VEC;
            if (e > end) end = e;
        }
    }
    return end;
}

size_t extent(int64_t T, int64_t W, int64_t ld, int64_t es) { return T > 0 ? static_cast<size_t>(((T - 1) * ld + W) * es) : 0; }

}  // namespace
}  // namespace dgr

using namespace dgr;

extern "C" size_t dgr_topk_distill_workspace_bytes(int64_t T) { return T < 0 || T > INT32_MAX ? 0 : sizeof(WsHeader); }

extern "C" dgr_status dgr_diag_distill_reads(int32_t dtype, int64_t V, int32_t z_at, int32_t dz_at, int32_t ctas, int64_t *end) {
    if ((dtype != DGR_DTYPE_BF16 && dtype != DGR_DTYPE_F32) || V < 1 || V > kMaxVocab || ctas < 1 || ctas > kMaxCluster || !end)
        return DGR_ERR_INVALID_ARG;
    const int vec = dtype == DGR_DTYPE_BF16 ? 8 : 4;
    if (z_at < 0 || z_at >= vec || dz_at < 0 || dz_at >= vec) return DGR_ERR_INVALID_ARG;
    auto walk = [&](auto *base) { return gradient_reads(static_cast<int>(V), base + z_at, base + dz_at, ctas); };
    // addresses only, never read; both 16-byte boundaries
    *end = vec == 8 ? walk(reinterpret_cast<const bf16 *>(uintptr_t{4096})) : walk(reinterpret_cast<const float *>(uintptr_t{4096}));
    return DGR_OK;
}

extern "C" dgr_status dgr_topk_distill(const void *logits, int32_t dtype, int64_t T, int64_t V, int64_t ld, const int32_t *ids,
                                       int64_t ld_ids, const float *teacher, int64_t ld_teacher, int32_t K, float tau,
                                       const float *teacher_lse, const float *weights, float scale, const float *dloss,
                                       float *row_loss, float *loss, void *dlogits, int64_t ld_d, void *ws, size_t ws_bytes,
                                       void *stream) {
    if (dtype != DGR_DTYPE_BF16 && dtype != DGR_DTYPE_F32) return DGR_ERR_INVALID_ARG;
    if (T < 0 || V < 1 || K < 1 || ld < V || ld_ids < K || ld_teacher < K || (dlogits && ld_d < V) || !(tau > 0.0f)) return DGR_ERR_INVALID_ARG;
    if (!ws || (T > 0 && (!logits || !ids || !teacher || (!loss && !row_loss && !dlogits) || (loss && !row_loss)))) return DGR_ERR_INVALID_ARG;
    if (T > INT32_MAX || V > kMaxVocab || K > kMaxList) return DGR_ERR_UNSUPPORTED;
    const float inv_tau = static_cast<float>(1.0 / static_cast<double>(tau));
    if (!(inv_tau > 0.0f) || inv_tau > 1e30f) return DGR_ERR_INVALID_ARG;
    const int es = dtype == DGR_DTYPE_BF16 ? 2 : 4;
    if (!aligned(logits, es) || !aligned(dlogits, es)) return DGR_ERR_MISALIGNED;
    for (const void *q : {static_cast<const void *>(ids), static_cast<const void *>(teacher), static_cast<const void *>(teacher_lse),
                          static_cast<const void *>(weights), static_cast<const void *>(dloss), static_cast<const void *>(row_loss),
                          static_cast<const void *>(loss)})
        if (!aligned(q, 4)) return DGR_ERR_MISALIGNED;
    if (ws_bytes < sizeof(WsHeader)) return DGR_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned(ws, kAlign)) return DGR_ERR_MISALIGNED;
    struct Range { const void *q; size_t n; };
    const size_t rows = static_cast<size_t>(T) * 4;
    const Range ins[] = {{logits, extent(T, V, ld, es)}, {ids, extent(T, K, ld_ids, 4)}, {teacher, extent(T, K, ld_teacher, 4)},
                         {teacher_lse, rows}, {weights, rows}, {dloss, 4}};
    const Range outs[] = {{dlogits, extent(T, V, ld_d, es)}, {row_loss, rows}, {loss, 4}, {ws, sizeof(WsHeader)}};
    for (const Range &o : outs) {
        for (const Range &i : ins)
            if (ranges_overlap(o.q, o.n, i.q, i.n) && !(o.q == dlogits && i.q == logits && dlogits == logits && ld == ld_d)) return DGR_ERR_ALIAS;
        for (const Range &b : outs)
            if (&o < &b && ranges_overlap(o.q, o.n, b.q, b.n)) return DGR_ERR_ALIAS;
    }
    dgr_status st = check_device();
    if (st != DGR_OK) return st;
    if (T == 0 && !loss) return DGR_OK;
    DistillParams p{};
    p.z = logits, p.ld = ld, p.T = static_cast<int32_t>(T), p.V = static_cast<int32_t>(V), p.K = K;
    p.ids = ids, p.ld_ids = ld_ids, p.teacher = teacher, p.ld_t = ld_teacher;
    p.teacher_lse = teacher_lse, p.weights = weights, p.dloss = dloss;
    p.inv_tau = inv_tau, p.k2 = static_cast<float>(1.4426950408889634 / static_cast<double>(tau)), p.scale = scale;
    p.row_loss = row_loss, p.loss = loss, p.dz = dlogits, p.ld_dz = ld_d;
    p.hdr = static_cast<WsHeader *>(ws);
    p.sched = sched_for(static_cast<uint32_t>(T));
    int sms = 0;
    if ((st = usable_sms(&sms)) != DGR_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (es == 2) return teacher_lse ? launch_size<bf16, true>(p, sms, s) : launch_size<bf16, false>(p, sms, s);
    return teacher_lse ? launch_size<float, true>(p, sms, s) : launch_size<float, false>(p, sms, s);
}
