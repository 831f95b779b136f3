// Log probabilities of given tokens, with entropy, logsumexp and the top
// alternatives, and their gradient.
//
// For a row of logits z [V] at temperature tau, with m its maximum:
//   ln p_j = (z_j - m) / tau - ln s,   s = sum_j exp((z_j - m) / tau);
//   logp   = ln p_id,  lse = m / tau + ln s;
//   H      = -sum_j p_j ln p_j = ln s - (1 / s) sum_j e_j (z_j - m) / tau  (both terms >= 0);
//   dz_j   = (dlogp (1[j = id] - p_j) - dentropy p_j (ln p_j + H)) / tau.
//
// Forward: the row is read once, by one CTA or, where there are few rows, by a
// cluster of them; every thread keeps a running maximum, the sum of 2^t and the
// sum of 2^t t, t = z k - fl(m k), k = log2(e) / tau. Two such triples meet by
// a <- 2^d (a + d s), s <- 2^d s with d the difference of their fl(m k); the
// rounding of fl(m k) is the same in both sums and cancels in p and H. Elements
// below -1e30 (masks, -inf) count as -1e30: their 2^t is 0 either way and
// 2^t t stays finite. Where m k is beyond 2^24 the row is read again with m
// subtracted first.
// Alternatives: the K-th largest of the threads' maxima is a lower bound of the
// row's K-th largest element, and few elements lie above it. Each thread keeps
// the maxima of a few parts of its share; the parts that reach the bound are
// read again (out of L2) and their elements above it collected; each element's
// rank among those is counted, by value and then by the lower index. Where so
// many are equal that they do not fit, one CTA finds the K-th by its digits.
// Backward: one pass from the stored m, ln s and H, no sum over the row.
//
// Deterministic: sums go over threads, warps and CTAs in a fixed order set by the
// type, T, V, the alignment and K; the collected elements' order is chance, their
// ranks are not.
#include "row_common.cuh"

namespace dgr {
namespace {

using namespace row;

constexpr int kMaxTop = 256;
constexpr int kMaxVocab = 1 << 20;
constexpr int kMaxCluster = 8;
constexpr int kParts = 16;          // parts of a thread's share with a maximum of their own
constexpr int kCandidates = 2048;   // collected elements
constexpr int kWhereId = 440;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kFar = 16777216.0f;
constexpr float kMasked = -1e30f;

struct LogpParams {
    const void *z;
    int64_t ld;
    int32_t T, V, K, per;  // per: vectors of a row a CTA
    const int32_t *ids;
    float inv_tau, k2;     // k2 = log2(e) / tau
    float *logp, *entropy, *lse, *stats;
    int32_t *top_ids;
    float *top_logits, *top_logp;
    WsHeader *hdr;
    Sched sched;
};

// ---- cluster -------------------------------------------------------------------

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
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(const void *p, uint32_t rank) {
    uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}
__device__ __forceinline__ void remote_store(uint32_t a, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ void remote_store(uint32_t a, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ void remote_store(uint32_t a, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ int remote_add(uint32_t a, int v) {
    int r;
    asm volatile("atom.shared::cluster.add.s32 %0, [%1], %2;" : "=r"(r) : "r"(a), "r"(v) : "memory");
    return r;
}

// ---- a row ---------------------------------------------------------------------

// A row as whole 16-byte vectors between a few single elements; CTA `rank` has
// `per` vectors from rank * per on (fewer at the row's end), CTA 0 the singles too.
template <typename T>
struct RowView {
    static constexpr int VEC = 16 / static_cast<int>(sizeof(T));
    int head, n_vec, n_single, first, count;
    __device__ __forceinline__ RowView(const T *z, int V, int rank, int per) {
        const int off = static_cast<int>(reinterpret_cast<uintptr_t>(z) & 15) / static_cast<int>(sizeof(T));
        head = off ? VEC - off : 0;
        head = head < V ? head : V;
        n_vec = (V - head) / VEC;
        n_single = rank == 0 ? V - n_vec * VEC : 0;
        first = rank * per < n_vec ? rank * per : n_vec;
        count = per < n_vec - first ? per : n_vec - first;
    }
    // element of single i: before the vectors, then behind them
    __device__ __forceinline__ int single(int i) const { return i < head ? i : n_vec * VEC + i; }
};

// fl(m k), at least -kFar: elements further below give 0, never inf - inf.
__device__ __forceinline__ float scaled_max(float m, float k) { return fmaxf(__fmul_rn(m, k), -kFar); }

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, s));
    return v;
}

// max(v, low), a NaN kept.
__device__ __forceinline__ float at_least(float v, float low) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(low));
    return r;
}
__device__ __forceinline__ float at_least_masked(float v) { return at_least(v, kMasked); }
__device__ __forceinline__ uint32_t at_least_masked2(uint32_t v) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0xf14af14au));  // -1e30 rounded to bf16
    return r;
}

// Maximum of a batch's elements (a NaN is passed over: it shows in the sum).
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

// Running maximum m, c = fl(m k), sum of 2^t and sum of 2^t t, t = x k - c.
struct Running {
    float m = -INFINITY, c = -kFar;
    float2 s = make_float2(0.0f, 0.0f), a = make_float2(0.0f, 0.0f);
    __device__ __forceinline__ void raise(float top, float k) {
        if (top > m) {
            m = top;
            const float to = scaled_max(top, k), d = __fadd_rn(c, -to), down = ex2(d);
            a = mul2(fma2(both(d), s, a), both(down));
            s = mul2(s, both(down));
            c = to;
        }
    }
    template <int N>
    __device__ __forceinline__ void add(float (&x)[N], float k) {
        vec_fma(x, k, -c);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 t = make_float2(x[i], x[i + 1]), e = make_float2(ex2(t.x), ex2(t.y));
            s = add2(s, e);
            a = fma2(e, t, a);
        }
    }
    __device__ __forceinline__ void add_one(float x, float k) {
        const float t = __fmaf_rn(x, k, -c), e = ex2(t);
        s.x = __fadd_rn(s.x, e);
        a.x = __fmaf_rn(e, t, a.x);
    }
};

struct Triple {
    float m, s, a;
    __device__ __forceinline__ void to(float top, float k) {
        const float d = __fadd_rn(scaled_max(m, k), -scaled_max(top, k)), down = ex2(d);
        a = __fmul_rn(__fmaf_rn(d, s, a), down);
        s = __fmul_rn(s, down);
        m = top;
    }
    __device__ __forceinline__ void over_warp(float k) {
        to(warp_max(m), k);
        s = warp_sum(s);
        a = warp_sum(a);
    }
};

// An element by value (-0 as +0), then by the lower index, as one number.
__device__ __forceinline__ uint64_t key_of(float v, int index) {
    uint32_t b = __float_as_uint(__fadd_rn(v, 0.0f));
    b = b & 0x80000000u ? ~b : b | 0x80000000u;
    return static_cast<uint64_t>(b) << 32 | static_cast<uint32_t>(~index);
}
__device__ __forceinline__ float key_value(uint64_t key) {
    const uint32_t b = static_cast<uint32_t>(key >> 32);
    return __uint_as_float(b & 0x80000000u ? b & 0x7fffffffu : ~b);
}
__device__ __forceinline__ int key_index(uint64_t key) { return static_cast<int>(~static_cast<uint32_t>(key)); }

// The K-th largest key of a row's elements above -inf (all of them where there
// are fewer), by its digits of 8 bits from the top: a histogram each of the
// elements that share the digits found so far. For rows where too many elements
// are equal; the whole CTA, one row, every reading out of L2.
template <typename T, int NT>
__device__ uint64_t kth_key(const T *z, int V, int K, int *hist) {
    __shared__ uint64_t s_prefix;
    __shared__ int s_left;
    const int tid = threadIdx.x;
    if (tid == 0) s_prefix = 0, s_left = K;
    // value digits 7..4; of the index's 32 bits the upper 8 are the same in all
    for (int digit = 7; digit >= 0; --digit) {
        for (int i = tid; i < 256; i += NT) hist[i] = 0;
        __syncthreads();
        const uint64_t prefix = s_prefix, mask = digit == 7 ? 0 : ~uint64_t{0} << (8 * (digit + 1));
        for (int j = tid; j < V; j += NT) {
            const float v = to_f32(z[j]);
            if (!(v > -INFINITY)) continue;  // a NaN neither
            const uint64_t key = key_of(v, j);
            if ((key & mask) == prefix) atomicAdd(&hist[key >> (8 * digit) & 255], 1);
        }
        __syncthreads();
        if (tid == 0) {
            int left = s_left, b = 255;
            for (; b > 0 && hist[b] < left; --b) left -= hist[b];
            s_left = left;
            s_prefix = prefix | static_cast<uint64_t>(b) << (8 * digit);
        }
        __syncthreads();
    }
    return s_prefix;
}

// The forward pass's shared memory, by name.
template <int NT>
struct __align__(16) Shared {
    float4 triple[2][kMaxCluster * NT / 32];  // the cluster's warps, by row parity
    float bound[2][kMaxCluster];              // lower bounds of the K-th element, likewise
};
template <int NT>
struct __align__(16) TopShared {
    uint64_t key[kCandidates];
    float part[kParts][NT];   // maxima of the threads' parts
    float top[NT];            // of the threads
    int list[NT * kParts];    // parts to read again
    int hist[256];
    int n_list, n_key;
};

template <typename T, int NT, bool TOP>
__global__ void __launch_bounds__(NT, 1024 / NT) logp_rows(const LogpParams p) {
    using View = RowView<T>;
    constexpr int VEC = View::VEC, W = NT / 32, U = 4;
    __shared__ Shared<NT> sh;
    extern __shared__ __align__(16) char smem[];
    TopShared<NT> &ts = *reinterpret_cast<TopShared<NT> *>(smem);
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int size = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
    const uint32_t n_clusters = gridDim.x / size;
    const int n_batches = (p.per + U * NT - 1) / (U * NT);       // of a thread, at most
    const int part_len = (n_batches + kParts - 1) / kParts;      // batches a part
    uint32_t live = 0;  // rows worked on: the exchange's parity
    if (TOP && tid == 0) ts.n_key = 0, ts.n_list = 0;
    if (size > 1) cluster_barrier();  // the other CTAs have started
    else __syncthreads();

    for (uint32_t item = blockIdx.x / size; item < static_cast<uint32_t>(p.T); item += n_clusters) {
        const int64_t row = sched_item(p.sched, item);
        const T *z = static_cast<const T *>(p.z) + row * p.ld;
        const int id = p.ids ? __ldg(p.ids + row) : 0;
        const bool skip = id < 0 || id >= p.V;
        if (skip) {  // not read: zeros, and no alternatives
            if (rank == 0 && tid == 0) {
                if (id >= p.V) record_error(p.hdr, DGR_ERR_INVALID_ARG, kWhereId);
                if (p.logp) p.logp[row] = 0.0f;
                if (p.entropy) p.entropy[row] = 0.0f;
                if (p.lse) p.lse[row] = 0.0f;
                if (p.stats) p.stats[2 * row] = p.stats[2 * row + 1] = 0.0f;
            }
            if (TOP && rank == 0)
                for (int k = tid; k < p.K; k += NT) {
                    if (p.top_ids) p.top_ids[row * p.K + k] = -1;
                    if (p.top_logits) p.top_logits[row * p.K + k] = -INFINITY;
                    if (p.top_logp) p.top_logp[row * p.K + k] = -INFINITY;
                }
            continue;
        }
        const View view(z, p.V, rank, p.per);
        const char *first = reinterpret_cast<const char *>(z + view.head) + static_cast<int64_t>(view.first) * 16;
        float x_id = 0.0f;
        if (p.logp && rank == 0 && w == 0) x_id = to_f32(z[id]);
        float shift = 0.0f, c = 0.0f;
        Triple all{-INFINITY, 0.0f, 0.0f};
        for (bool again = false;; again = true) {
            Running run;
            float part = -INFINITY;
            int in_part = 0, n_part = 0;
            for (int v = tid; v < view.count; v += U * NT) {
                uint4 r[U];
                constexpr uint32_t low = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;  // -inf
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    r[u] = make_uint4(low, low, low, low);
                    load_if<true>(r[u], first + (static_cast<int64_t>(v) + u * NT) * 16, v + u * NT < view.count);
                }
                const float top = max_of<T, U>(r);
                if (TOP && !again) {
                    part = fmaxf(part, top);
                    if (++in_part == part_len) {
                        ts.part[n_part++][tid] = part;
                        part = -INFINITY, in_part = 0;
                    }
                }
                run.raise(__fadd_rn(top, -shift), p.k2);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float x[VEC];
                    if constexpr (sizeof(T) == 2) {
                        if (!again) r[u] = make_uint4(at_least_masked2(r[u].x), at_least_masked2(r[u].y), at_least_masked2(r[u].z), at_least_masked2(r[u].w));
                        unpack<T, VEC>(r[u], x);
                        if (again)
#pragma unroll
                            for (int i = 0; i < VEC; ++i) x[i] = at_least_masked(__fadd_rn(x[i], -shift));
                    } else {
                        unpack<T, VEC>(r[u], x);
#pragma unroll
                        for (int i = 0; i < VEC; ++i) x[i] = at_least_masked(__fadd_rn(x[i], -shift));
                    }
                    run.add(x, p.k2);
                }
            }
            if (TOP && !again)
                for (; n_part < kParts; ++n_part) {
                    ts.part[n_part][tid] = part;
                    part = -INFINITY;
                }
            if (tid < view.n_single) {
                const float x = __fadd_rn(to_f32(z[view.single(tid)]), -shift);
                run.raise(x, p.k2);
                run.add_one(at_least_masked(x), p.k2);
            }
            if (TOP && !again) ts.top[tid] = run.m;
            Triple mine{run.m, across(run.s), across(run.a)};
            mine.over_warp(p.k2);
            if (lane < size) remote_store(remote(&sh.triple[live & 1][rank * W + w], lane), make_float4(mine.m, mine.s, mine.a, 0.0f));
            __syncwarp();
            if (size > 1) cluster_barrier();
            else __syncthreads();
            all = Triple{-INFINITY, 0.0f, 0.0f};
            for (int j = lane; j < size * W; j += 32) all.m = fmaxf(all.m, sh.triple[live & 1][j].x);
            all.m = warp_max(all.m);
            if (again || !(fabsf(all.m) < INFINITY) || fabsf(__fmul_rn(all.m, p.k2)) < kFar) break;
            shift = all.m;  // the same in every warp of the cluster
            if (size > 1) cluster_barrier();  // before the triples are written over
            else __syncthreads();
        }
        // the row's sums and outputs: the first warp of the first CTA
        const float m = shift != 0.0f ? shift : all.m;
        float lns = 0.0f;
        if (rank == 0 && (w == 0 || TOP)) {
            c = scaled_max(all.m, p.k2);
            for (int j = lane; j < size * W; j += 32) {
                const float4 got = sh.triple[live & 1][j];
                Triple t{got.x, got.y, got.z};
                t.to(all.m, p.k2);
                all.s = __fadd_rn(all.s, t.s);
                all.a = __fadd_rn(all.a, t.a);
            }
            all.s = warp_sum(all.s);
            all.a = warp_sum(all.a);
            const bool none = m == -INFINITY;  // nothing is left of the row
            const float ln_s = logf(all.s);
            // ln s for the maximum itself: without the rounding of c
            lns = none ? 0.0f : __fmaf_rn(__fmaf_rn(all.m, p.k2, -c), -kLn2, ln_s);
            if (w == 0 && lane == 0) {
                if (p.logp) p.logp[row] = none ? -INFINITY : __fmaf_rn(__fadd_rn(x_id, -m), p.inv_tau, -lns);
                if (p.entropy) p.entropy[row] = none ? 0.0f : __fmaf_rn(-kLn2, all.a / all.s, ln_s);
                if (p.lse) p.lse[row] = __fmaf_rn(m, p.inv_tau, lns);
                if (p.stats) p.stats[2 * row] = m, p.stats[2 * row + 1] = lns;
            }
        }
        if constexpr (TOP) {
            // the K-th largest of the threads' maxima: the one that K - 1 come before
            const float top = ts.top[tid];
            int before = 0;
            for (int j = 0; j < NT; j += 4) {
                const float4 o = *reinterpret_cast<const float4 *>(&ts.top[j]);
                before += (o.x > top || (o.x == top && j < tid)) + (o.y > top || (o.y == top && j + 1 < tid)) +
                          (o.z > top || (o.z == top && j + 2 < tid)) + (o.w > top || (o.w == top && j + 3 < tid));
            }
            if (before == p.K - 1)
                for (int r = 0; r < size; ++r) remote_store(remote(&sh.bound[live & 1][rank], r), top);
            if (size > 1) cluster_barrier();
            else __syncthreads();
            float bound = sh.bound[live & 1][0];
            for (int r = 1; r < size; ++r) bound = fmaxf(bound, sh.bound[live & 1][r]);
            auto collect = [&](float v, int index) {
                if (v >= bound && v > -INFINITY) {
                    const int at = remote_add(remote(&ts.n_key, 0), 1);
                    if (at < kCandidates) remote_store(remote(&ts.key[at], 0), key_of(v, index));
                }
            };
            if (top >= bound && top > -INFINITY) {
                for (int i = 0; i < kParts; ++i) {
                    const float part = ts.part[i][tid];
                    if (part >= bound && part > -INFINITY) ts.list[atomicAdd(&ts.n_list, 1)] = i * NT + tid;
                }
                if (tid < view.n_single) {
                    const int j = view.single(tid);
                    collect(to_f32(z[j]), j);
                }
            }
            __syncthreads();
            const int per_part = part_len * U;
            for (int i = tid; i < ts.n_list * per_part; i += NT) {
                const int which = ts.list[i / per_part], of = i % per_part;
                const int v = which % NT + (which / NT * per_part + of) * NT;
                if (v >= view.count) continue;
                const uint4 r = __ldg(reinterpret_cast<const uint4 *>(first) + v);
                float x[VEC];
                unpack<T, VEC>(r, x);
#pragma unroll
                for (int j = 0; j < VEC; ++j) collect(x[j], view.head + (view.first + v) * VEC + j);
            }
            if (size > 1) cluster_barrier();
            else __syncthreads();
            if (tid == 0) ts.n_list = 0;
            if (rank == 0) {
                int n = ts.n_key;
                if (n > kCandidates) {
                    const uint64_t least = kth_key<T, NT>(z, p.V, p.K, ts.hist);
                    if (tid == 0) ts.n_key = 0;
                    __syncthreads();
                    for (int j = tid; j < p.V; j += NT) {
                        const float v = to_f32(z[j]);
                        if (!(v > -INFINITY)) continue;
                        const uint64_t key = key_of(v, j);
                        if (key >= least) ts.key[atomicAdd(&ts.n_key, 1)] = key;
                    }
                    __syncthreads();
                    n = ts.n_key;
                }
                for (int i = tid; i < n; i += NT) {
                    const uint64_t key = ts.key[i];
                    int at = 0;
                    for (int j = 0; j < n; ++j) at += ts.key[j] > key;
                    if (at >= p.K) continue;
                    const float v = key_value(key);
                    if (p.top_ids) p.top_ids[row * p.K + at] = key_index(key);
                    if (p.top_logits) p.top_logits[row * p.K + at] = v;
                    if (p.top_logp) p.top_logp[row * p.K + at] = __fmaf_rn(__fadd_rn(v, -m), p.inv_tau, -lns);
                }
                for (int k = n + tid; k < p.K; k += NT) {
                    if (p.top_ids) p.top_ids[row * p.K + k] = -1;
                    if (p.top_logits) p.top_logits[row * p.K + k] = -INFINITY;
                    if (p.top_logp) p.top_logp[row * p.K + k] = -INFINITY;
                }
                __syncthreads();
                if (tid == 0) ts.n_key = 0;  // read by the others behind the next row's barrier
            }
            __syncthreads();
        }
        ++live;
    }
    if (size > 1) cluster_barrier();  // no CTA leaves before its shared memory is read
}

// ---- backward ------------------------------------------------------------------

struct LogpBackParams {
    const void *z;
    int64_t ld, ld_d;
    int32_t T, V;
    const int32_t *ids;
    const float *stats, *entropy, *dlogp, *dentropy;
    float inv_tau, k2;
    void *dz;
    int32_t chunks;  // pieces of a row
    Sched sched;
};

constexpr int kBackThreads = 256;
constexpr int kBackVecs = 4;  // vectors of a thread at a time

// A row's gradient: p = 2^((x - m) k - l), dz = p (A + B log2 p).
struct RowGrad {
    float m, l, k, A, B, at_id;
    bool on;
    __device__ __forceinline__ RowGrad(const LogpBackParams &p, int64_t row, int id) {
        m = __ldg(p.stats + 2 * row);
        l = __fmul_rn(__ldg(p.stats + 2 * row + 1), kLog2e);
        k = p.k2;
        const float a = p.dlogp ? __fmul_rn(__ldg(p.dlogp + row), p.inv_tau) : 0.0f;
        const float b = p.dentropy ? __fmul_rn(__ldg(p.dentropy + row), p.inv_tau) : 0.0f;
        A = -__fmaf_rn(b, p.entropy ? __ldg(p.entropy + row) : 0.0f, a);
        B = __fmul_rn(-kLn2, b);
        at_id = a;
        on = (!p.ids || (id >= 0 && id < p.V)) && m != -INFINITY;
    }
    template <int N>
    __device__ __forceinline__ void of(float (&x)[N]) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float t = at_least(__fmaf_rn(__fadd_rn(x[i], -m), k, -l), -1e4f);  // 2^t is 0 there; 0 * inf would not be
            x[i] = on ? __fmul_rn(ex2(t), __fmaf_rn(B, t, A)) : 0.0f;
        }
    }
};

template <typename T>
__global__ void __launch_bounds__(kBackThreads) logp_back(const LogpBackParams p) {
    constexpr int VEC = 16 / static_cast<int>(sizeof(T));
    constexpr int kStep = kBackThreads * kBackVecs;
    const int tid = threadIdx.x;
    const int64_t items = static_cast<int64_t>(p.T) * p.chunks;
    for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
        const int64_t item = sched_item(p.sched, static_cast<uint32_t>(i));
        const int64_t row = item / p.chunks;
        const int chunk = static_cast<int>(item - row * p.chunks);
        const T *z = static_cast<const T *>(p.z) + row * p.ld;
        T *dz = static_cast<T *>(p.dz) + row * p.ld_d;
        const int id = p.ids ? __ldg(p.ids + row) : -1;
        const RowGrad g(p, row, id);
        // the gradient's vectors; the logits' lie `off` elements before them
        const int out = static_cast<int>(reinterpret_cast<uintptr_t>(dz) & 15) / static_cast<int>(sizeof(T));
        const int head = min(out ? VEC - out : 0, p.V), n_vec = (p.V - head) / VEC;
        const int off = static_cast<int>(reinterpret_cast<uintptr_t>(z + head) & 15) / static_cast<int>(sizeof(T));
        const char *src = reinterpret_cast<const char *>(z + head - off);  // a 16-byte boundary
        // element j, with the given token's part
        auto one = [&](int j) {
            float x[1] = {g.on ? to_f32(z[j]) : 0.0f};
            g.of(x);
            if (j == id && g.on) x[0] = __fadd_rn(x[0], g.at_id);
            *reinterpret_cast<raw_t<T, 1> *>(dz + j) = pack<T, 1>(x);
        };
        for (int v0 = chunk * kStep; v0 < n_vec; v0 += p.chunks * kStep) {
            uint4 r[kBackVecs];
            if (off == 0) {
#pragma unroll
                for (int u = 0; u < kBackVecs; ++u) {
                    const int v = v0 + u * kBackThreads + tid;
                    r[u] = make_uint4(0, 0, 0, 0);
                    load_if<false>(r[u], src + static_cast<int64_t>(v) * 16, v < n_vec && g.on);
                }
            } else {
                // out of the two vectors that it lies across, where both are in the row
                uint4 q[kBackVecs];
#pragma unroll
                for (int u = 0; u < kBackVecs; ++u) {
                    const int v = v0 + u * kBackThreads + tid;
                    const bool whole = v < n_vec && head + v * VEC - off >= 0 && head + v * VEC - off + 2 * VEC <= p.V;
                    r[u] = q[u] = make_uint4(0, 0, 0, 0);
                    load_if<false>(r[u], src + static_cast<int64_t>(v) * 16, whole && g.on);
                    load_if<false>(q[u], src + static_cast<int64_t>(v) * 16 + 16, whole && g.on);
                }
#pragma unroll
                for (int u = 0; u < kBackVecs; ++u) {
                    const int by = off * static_cast<int>(sizeof(T)) * 8;
                    uint32_t b[8] = {r[u].x, r[u].y, r[u].z, r[u].w, q[u].x, q[u].y, q[u].z, q[u].w};
                    if (by & 64)
#pragma unroll
                        for (int i2 = 0; i2 < 6; ++i2) b[i2] = b[i2 + 2];
                    if (by & 32)
#pragma unroll
                        for (int i2 = 0; i2 < 5; ++i2) b[i2] = b[i2 + 1];
                    r[u] = make_uint4(__funnelshift_r(b[0], b[1], by & 31), __funnelshift_r(b[1], b[2], by & 31),
                                      __funnelshift_r(b[2], b[3], by & 31), __funnelshift_r(b[3], b[4], by & 31));
                }
            }
#pragma unroll
            for (int u = 0; u < kBackVecs; ++u) {
                const int v = v0 + u * kBackThreads + tid, j = head + v * VEC;
                if (v >= n_vec) continue;
                if (off != 0 && !(j - off >= 0 && j - off + 2 * VEC <= p.V)) {
                    for (int e = 0; e < VEC; ++e) one(j + e);
                    continue;
                }
                float x[VEC];
                unpack<T, VEC>(r[u], x);
                g.of(x);
                if (static_cast<uint32_t>(id - j) < static_cast<uint32_t>(VEC) && g.on)
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        if (j + e == id) x[e] = __fadd_rn(x[e], g.at_id);
                *reinterpret_cast<uint4 *>(dz + j) = pack<T, VEC>(x);
            }
        }
        // elements around the vectors
        if (chunk == 0 && tid < p.V - n_vec * VEC) one(tid < head ? tid : n_vec * VEC + tid);
    }
}

// ---- host ---------------------------------------------------------------------

template <typename T, int NT, bool TOP>
dgr_status launch_rows(LogpParams &p, int cluster, int sms, cudaStream_t s) {
    auto *k = logp_rows<T, NT, TOP>;
    const int vecs = p.V / (16 / static_cast<int>(sizeof(T)));
    p.per = (vecs + cluster - 1) / cluster;
    if (p.per < 1) p.per = 1;
    const size_t smem = TOP ? sizeof(TopShared<NT>) : 0;
    dgr_status st = allow_smem(k, smem, sizeof(TopShared<NT>));
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
    int clusters = p.T;
    if (static_cast<int64_t>(p.T) * cluster > sms && (cudaOccupancyMaxActiveClusters(&clusters, k, &cfg) != cudaSuccess || clusters < 1)) return DGR_ERR_CUDA;
    const int within = sms * (1024 / NT) / cluster;  // a green context's, or the test's cap
    if (clusters > within) clusters = within > 0 ? within : 1;
    if (clusters > p.T) clusters = p.T;
    const unsigned capped = sched_grid(static_cast<unsigned>(clusters * cluster)) / cluster;
    cfg.gridDim = dim3((capped > 0 ? capped : 1) * cluster);
    return cudaLaunchKernelEx(&cfg, k, p) == cudaSuccess ? DGR_OK : DGR_ERR_CUDA;
}

template <typename T>
dgr_status launch_forward(LogpParams &p, int sms, cudaStream_t s) {
    // few rows: a row over more CTAs, down to 4096 elements each
    int cluster = 1;
    while (cluster < kMaxCluster && static_cast<int64_t>(p.T) * cluster * 2 <= 304 && p.V >= 4096 * cluster * 2) cluster <<= 1;
    return p.K ? launch_rows<T, 256, true>(p, cluster, sms, s) : launch_rows<T, 256, false>(p, cluster, sms, s);
}

size_t extent(int64_t T, int64_t W, int64_t ld, int64_t es) { return T > 0 ? static_cast<size_t>(((T - 1) * ld + W) * es) : 0; }

struct Range {
    const void *q;
    size_t n;
};

dgr_status check_logits(const void *logits, int32_t dtype, int64_t T, int64_t V, int64_t ld, float tau) {
    if (dtype != DGR_DTYPE_BF16 && dtype != DGR_DTYPE_F32) return DGR_ERR_INVALID_ARG;
    if (T < 0 || V < 1 || ld < V || !(tau > 0.0f) || !(tau < INFINITY) || (T > 0 && !logits)) return DGR_ERR_INVALID_ARG;
    if (T > (1 << 26) || V > kMaxVocab || tau < 1e-6f || tau > 1e6f) return DGR_ERR_UNSUPPORTED;
    if (!aligned(logits, dtype == DGR_DTYPE_BF16 ? 2 : 4)) return DGR_ERR_MISALIGNED;
    return DGR_OK;
}

}  // namespace
}  // namespace dgr

using namespace dgr;

extern "C" size_t dgr_token_logprobs_workspace_bytes(int64_t T) { return T < 0 || T > (1 << 26) ? 0 : sizeof(WsHeader); }

extern "C" dgr_status dgr_token_logprobs(const void *logits, int32_t dtype, int64_t T, int64_t V, int64_t ld, const int32_t *ids, float tau,
                                         int32_t K, float *logp, float *entropy, float *lse, float *stats, int32_t *top_ids,
                                         float *top_logits, float *top_logp, void *ws, size_t ws_bytes, void *stream) {
    dgr_status st = check_logits(logits, dtype, T, V, ld, tau);
    if (st != DGR_OK) return st;
    if (K < 0 || !ws || (logp && !ids)) return DGR_ERR_INVALID_ARG;
    const bool top = top_ids || top_logits || top_logp;
    if (T > 0 && (top != (K > 0) || (!logp && !entropy && !lse && !stats && !top))) return DGR_ERR_INVALID_ARG;
    if (K > kMaxTop) return DGR_ERR_UNSUPPORTED;
    for (const void *q : {static_cast<const void *>(ids), static_cast<const void *>(logp), static_cast<const void *>(entropy),
                          static_cast<const void *>(lse), static_cast<const void *>(stats), static_cast<const void *>(top_ids),
                          static_cast<const void *>(top_logits), static_cast<const void *>(top_logp)})
        if (!aligned(q, 4)) return DGR_ERR_MISALIGNED;
    if (ws_bytes < sizeof(WsHeader)) return DGR_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned(ws, kAlign)) return DGR_ERR_MISALIGNED;
    const int es = dtype == DGR_DTYPE_BF16 ? 2 : 4;
    const size_t rows = static_cast<size_t>(T) * 4, lists = rows * static_cast<size_t>(K);
    const Range ins[] = {{logits, extent(T, V, ld, es)}, {ids, rows}};
    const Range outs[] = {{logp, rows}, {entropy, rows}, {lse, rows}, {stats, 2 * rows}, {top_ids, lists}, {top_logits, lists},
                          {top_logp, lists}, {ws, sizeof(WsHeader)}};
    for (const Range &o : outs) {
        for (const Range &i : ins)
            if (ranges_overlap(o.q, o.n, i.q, i.n)) return DGR_ERR_ALIAS;
        for (const Range &b : outs)
            if (&o < &b && ranges_overlap(o.q, o.n, b.q, b.n)) return DGR_ERR_ALIAS;
    }
    if ((st = check_device()) != DGR_OK) return st;
    if (T == 0) return DGR_OK;
    LogpParams p{};
    p.z = logits, p.ld = ld, p.T = static_cast<int32_t>(T), p.V = static_cast<int32_t>(V), p.K = K, p.ids = ids;
    p.inv_tau = static_cast<float>(1.0 / static_cast<double>(tau)), p.k2 = static_cast<float>(1.4426950408889634 / static_cast<double>(tau));
    p.logp = logp, p.entropy = entropy, p.lse = lse, p.stats = stats;
    p.top_ids = top_ids, p.top_logits = top_logits, p.top_logp = top_logp;
    p.hdr = static_cast<WsHeader *>(ws);
    p.sched = sched_for(static_cast<uint32_t>(T));
    int sms = 0;
    if ((st = usable_sms(&sms)) != DGR_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return es == 2 ? launch_forward<bf16>(p, sms, s) : launch_forward<float>(p, sms, s);
}

extern "C" dgr_status dgr_token_logprobs_backward(const void *logits, int32_t dtype, int64_t T, int64_t V, int64_t ld, const int32_t *ids,
                                                  float tau, const float *stats, const float *entropy, const float *dlogp,
                                                  const float *dentropy, void *dlogits, int64_t ld_d, void *stream) {
    dgr_status st = check_logits(logits, dtype, T, V, ld, tau);
    if (st != DGR_OK) return st;
    if (ld_d < V || (T > 0 && (!stats || !dlogits || (!dlogp && !dentropy)))) return DGR_ERR_INVALID_ARG;
    if ((dlogp && !ids) || (dentropy && !entropy)) return DGR_ERR_INVALID_ARG;
    const int es = dtype == DGR_DTYPE_BF16 ? 2 : 4;
    if (!aligned(dlogits, es)) return DGR_ERR_MISALIGNED;
    const size_t rows = static_cast<size_t>(T) * 4, n = extent(T, V, ld_d, es);
    const Range ins[] = {{ids, rows}, {stats, 2 * rows}, {entropy, rows}, {dlogp, rows}, {dentropy, rows}};
    for (const Range &i : ins) {
        if (!aligned(i.q, 4)) return DGR_ERR_MISALIGNED;
        if (ranges_overlap(dlogits, n, i.q, i.n)) return DGR_ERR_ALIAS;
    }
    if (!(dlogits == logits && ld == ld_d) && ranges_overlap(dlogits, n, logits, extent(T, V, ld, es))) return DGR_ERR_ALIAS;
    if ((st = check_device()) != DGR_OK) return st;
    if (T == 0) return DGR_OK;
    LogpBackParams p{};
    p.z = logits, p.ld = ld, p.ld_d = ld_d, p.T = static_cast<int32_t>(T), p.V = static_cast<int32_t>(V), p.ids = ids;
    p.stats = stats, p.entropy = entropy, p.dlogp = dlogp, p.dentropy = dentropy;
    p.inv_tau = static_cast<float>(1.0 / static_cast<double>(tau)), p.k2 = static_cast<float>(1.4426950408889634 / static_cast<double>(tau));
    p.dz = dlogits;
    int sms = 0;
    if ((st = usable_sms(&sms)) != DGR_OK) return st;
    // pieces of a row: enough for every SM's CTAs where rows are few
    const int64_t steps = (V * es / 16 + kBackThreads * kBackVecs - 1) / (kBackThreads * kBackVecs);
    int64_t chunks = (static_cast<int64_t>(sms) * 8 + T - 1) / T;
    if (chunks > steps) chunks = steps;
    p.chunks = static_cast<int32_t>(chunks < 1 ? 1 : chunks);
    const int64_t items = T * p.chunks;
    p.sched = sched_for(static_cast<uint32_t>(items));
    const int64_t most = static_cast<int64_t>(sms) * 8;
    const unsigned grid = sched_grid(static_cast<unsigned>(items < most ? items : most));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (es == 2) logp_back<bf16><<<grid, kBackThreads, 0, s>>>(p);
    else logp_back<float><<<grid, kBackThreads, 0, s>>>(p);
    return launch_status();
}
