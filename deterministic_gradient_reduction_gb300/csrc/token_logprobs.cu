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
// read again (out of L2), their elements above it collected and the lowest K of
// those equal to it; each one's rank among them is counted, by value and then by
// the lower index. A warp that has no share of the rows does this for a row while
// the others read the next one. Where more elements lie above the bound than
// there is space for, that warp finds the K-th by its digits.
// Backward: one pass from the stored m, ln s and H, no sum over the row.
//
// Bound by memory: 4096 x 131072 bf16 forward 155 us (6.9 TB/s, the measured copy
// rate; the exponentials come next, 50 % of the issue slots), backward 326 us (6.6
// TB/s). With lists the next bound is the list warps' latency: 2048 x 50001 fp32, the
// best 64, 85 us (4.8 TB/s). A lone row of 65536: 10 us of latency.
//
// Deterministic: sums go over threads, warps and CTAs in a fixed order set by the
// type, T, V, the alignment and K; the collected elements' order is chance, their
// ranks are not.
#include <cfloat>
#include <climits>
#include <cstddef>

#include "row_common.cuh"

namespace dgr {
namespace {

using namespace row;

constexpr int kMaxTop = 128;
constexpr int kMaxVocab = 1 << 20;
constexpr int kMaxCluster = 8;
constexpr int kCandidates = 512, kCandidatesOfMany = 1536;  // collected elements of a CTA, of a row with several
constexpr int kFew = 256;           // parts, or equal elements, that are taken as they come
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
    __syncwarp();  // .aligned: the warp's lanes together
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(const void *p, uint32_t rank) {
    uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}
__device__ __forceinline__ void remote_store(uint32_t a, float2 v) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(v.x), "f"(v.y) : "memory");
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

// The lowest bf16 that is not below v.
__device__ __forceinline__ uint16_t up_to_bf16(float v) {
    uint32_t b = __float_as_uint(v);
    if (!(b & 0x80000000u) && b << 16) b += 0x10000u;  // (to infinity, at the end); below zero the upper bits are that
    return static_cast<uint16_t>(b >> 16);
}

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
// elements that share the digits found so far. For rows with more candidates than
// there is space for: their large elements lie side by side, in the shares of fewer
// than K threads. One warp reads the row nine times, an element a lane, each reading
// waiting for the one before: a row of 65536 bf16 with 800 tokens raised or left over by
// a mask and K = 128 takes 3.5 to 3.9 ms so (21 us where they are scattered), 1024 rows
// of 131072 26 to 28 ms (0.083).
template <typename T>
__device__ uint64_t kth_key(const T *z, int V, int K, int *hist) {
    const int lane = threadIdx.x & 31;
    uint64_t prefix = 0;
    int left = K;
    for (int digit = 7; digit >= 0; --digit) {
        for (int i = lane; i < 256; i += 32) hist[i] = 0;
        __syncwarp();
        const uint64_t mask = digit == 7 ? 0 : ~uint64_t{0} << (8 * (digit + 1));
        for (int j = lane; j < V; j += 32) {
            const float v = to_f32(z[j]);
            if (!(v > -INFINITY)) continue;  // a NaN neither
            const uint64_t key = key_of(v, j);
            if ((key & mask) == prefix) atomicAdd(&hist[key >> (8 * digit) & 255], 1);
        }
        __syncwarp();
        int b = 255;
        for (; b > 0 && hist[b] < left; --b) left -= hist[b];
        prefix |= static_cast<uint64_t>(b) << (8 * digit);
        __syncwarp();
    }
    return prefix;
}

// The forward pass's shared memory. MT: threads that read rows.
template <int NT>
struct __align__(16) Shared {
    float4 triple[2][kMaxCluster * NT / 32];  // the cluster's warps, by row parity
    float2 bound[2][kMaxCluster];             // lower bounds of the CTAs' K-th element and of their K / CTAs-th, likewise
};
// Kept small: what the four CTAs of an SM leave of it is the cache that loads in
// flight need room in.
template <int MT>
struct __align__(16) TopShared {
    static constexpr bool kFewThreads = MT < kMaxTop;
    static constexpr int kParts = kFewThreads ? 4 : 16;  // parts of a thread's share with a maximum of their own
    static constexpr int kTops = kFewThreads ? kParts * MT : MT;
    uint16_t part[2][kParts][MT];  // maxima of the threads' parts, rounded up to bf16, by row parity
    float top[2][kTops];           // of the threads, or of the parts where threads are few
    uint16_t list[kFew];           // parts to read again
    int same[kFew];                // elements equal to the bound (and a histogram of 256)
    int n_all;
    alignas(16) uint64_t key[];    // this CTA's candidates and two more, then a cluster's; read in twos
};
static_assert(kFew >= 256, "a histogram fits");
template <int MT>
constexpr bool vectors_aligned = offsetof(TopShared<MT>, key) % 16 == 0 && offsetof(TopShared<MT>, part) % 16 == 0 &&
                                 sizeof(uint16_t[TopShared<MT>::kParts][MT]) % 16 == 0 && sizeof(TopShared<MT>) == offsetof(TopShared<MT>, key);
static_assert(vectors_aligned<256> && vectors_aligned<64>, "what is read as vectors of 16 bytes starts at multiples of them");

constexpr int kBatch = 4;  // vectors that a thread reads at a time

// A row's list, by one warp of each CTA of its cluster.
template <typename T, int MT>
struct TopOf {
    using View = RowView<T>;
    enum { VEC = 16 / static_cast<int>(sizeof(T)) };

    const LogpParams &p;
    TopShared<MT> &ts;
    const T *z;
    const View &view;
    const char *first;
    int par, lane, per_part, size;
    int n_key;  // candidates

    // K-th largest of the threads' maxima as a key, two bits at a time; what lies below bit
    // `to` is left out, so that a lower bound comes of it
    __device__ __forceinline__ uint32_t bound(int K, int to) const {
        constexpr int N = TopShared<MT>::kTops / 32;
        uint32_t key[N], at = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) key[i] = static_cast<uint32_t>(key_of(ts.top[par][i * 32 + lane], 0) >> 32);
        for (int bit = 30; bit >= to; bit -= 2) {
            int n[3] = {0, 0, 0};
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (uint32_t d = 1; d < 4; ++d) n[d - 1] += key[i] >= (at | d << bit);
#pragma unroll
            for (int d = 0; d < 3; ++d) n[d] = static_cast<int>(__reduce_add_sync(0xffffffffu, n[d]));
            at |= static_cast<uint32_t>((n[0] >= K) + (n[1] >= K) + (n[2] >= K)) << bit;
        }
        return at;
    }
    // By the upper 16 bits: all that a bf16 value has (its lower ones are 0, or 1 below
    // zero), and near enough else, as long as few parts reach it.
    __device__ __forceinline__ float value_of(uint32_t at) const {
        if (sizeof(T) == 2 && !(at & 0x80000000u)) at |= 0xffffu;
        // (the key of -inf is the least that counts)
        return key_value(static_cast<uint64_t>(max(at, 0x007fffffu)) << 32);
    }
    // by all bits where many more than K threads reach it
    __device__ __forceinline__ float near_bound(int K) const {
        const uint32_t at = bound(K, 16);
        if (sizeof(T) == 4) {
            int n = 0;
            for (int i = lane; i < TopShared<MT>::kTops; i += 32) n += static_cast<uint32_t>(key_of(ts.top[par][i], 0) >> 32) >= at;
            if (static_cast<int>(__reduce_add_sync(0xffffffffu, n)) > K + 32) return value_of(bound(K, 0));
        }
        return value_of(at);
    }
    // to this CTA's candidates: the lanes' elements where `on`
    __device__ __forceinline__ void push(float v, int index, bool on) {
        const uint32_t who = __ballot_sync(0xffffffffu, on);
        const int at = n_key + __popc(who & ((1u << lane) - 1));
        if (on && at < kCandidates) ts.key[at] = key_of(v, index);
        n_key += __popc(who);
    }
    // a cluster's candidates together in the leader, behind its own; too many show in their
    // number, of a CTA as of all: one that had no space for all of its own (a run of large
    // elements side by side) counts as more than a row's space
    __device__ __forceinline__ void gather() {
        __syncwarp();
        int at = 0;
        if (lane == 0) at = remote_add(remote(&ts.n_all, 0), n_key > kCandidates ? kCandidatesOfMany + 1 : n_key);
        at = __shfl_sync(0xffffffffu, at, 0);
        for (int i = lane; i < n_key && i < kCandidates; i += 32)
            if (at + i < kCandidatesOfMany) remote_store(remote(&ts.key[kCandidates + 2 + at + i], 0), ts.key[i]);
        n_key = 0;
    }
    // reads the listed parts: pushes the elements above b and lists those equal to it in
    // `same`; how many these are. A lane has a part, four vectors of it at a time. One
    // warp does this, at four or five cycles an instruction, so they are few: a mask of
    // the elements that reach b, and a word of it by a tree of selections.
    __device__ __forceinline__ int elements(int n_list, float b, bool equal) {
        constexpr int U = kBatch, PER = 4 / static_cast<int>(sizeof(T));  // elements a word
        const float least = b > -INFINITY ? b : -FLT_MAX;           // -inf reaches nothing
        int n_same = 0;
        for (int i0 = 0; i0 < n_list; i0 += 32) {
            const int which = i0 + lane < n_list ? ts.list[i0 + lane] : -1;
            const int v0 = which < 0 ? 0 : which % MT + which / MT * per_part * MT;
            for (int k = 0; k < per_part; k += U) {
                uint4 r[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int v = v0 + (k + u) * MT;
                    constexpr uint32_t low = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;  // -inf
                    r[u] = make_uint4(low, low, low, low);
                    load_if<true>(r[u], first + static_cast<int64_t>(v) * 16, which >= 0 && v < view.count);
                }
                uint32_t reach = 0;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float x[VEC];
                    unpack<T, VEC>(r[u], x);
#pragma unroll
                    for (int j = 0; j < VEC; ++j)
                        if (x[j] >= least) reach |= 1u << (u * VEC + j);
                }
                while (__any_sync(0xffffffffu, reach != 0)) {
                    const int e = __ffs(reach) - 1, word = e / PER;  // (where there is none: of nothing)
                    uint32_t q[4 * U];
#pragma unroll
                    for (int u = 0; u < U; ++u) q[4 * u] = r[u].x, q[4 * u + 1] = r[u].y, q[4 * u + 2] = r[u].z, q[4 * u + 3] = r[u].w;
#pragma unroll
                    for (int half = 2 * U; half > 0; half >>= 1)
#pragma unroll
                        for (int i = 0; i < half; ++i) q[i] = word & half ? q[i + half] : q[i];
                    const float v = sizeof(T) == 4 ? __uint_as_float(q[0]) : __uint_as_float(e & 1 ? q[0] & 0xffff0000u : q[0] << 16);
                    const int index = view.head + (view.first + v0 + (k + e / VEC) * MT) * VEC + e % VEC;
                    const bool on = reach != 0, above = on && v > b;
                    push(v, index, above);
                    if (equal) {
                        const uint32_t who = __ballot_sync(0xffffffffu, on && v == b);
                        const int to = n_same + __popc(who & ((1u << lane) - 1));
                        if (on && v == b && to < kFew) ts.same[to] = index;
                        n_same += __popc(who);
                    }
                    reach &= reach - 1;
                }
            }
        }
        __syncwarp();
        return n_same;
    }
    // lists the parts whose maximum is above `b` (or equal to it), the first kFew; how many
    __device__ __forceinline__ int list_parts(float b, bool equal) const {
        constexpr int n_vec = TopShared<MT>::kParts * MT / 8, per = (n_vec + 31) / 32;
        static_assert(per <= 32, "a bit a vector");
        const uint4 *part = reinterpret_cast<const uint4 *>(&ts.part[par][0][0]);
        auto reaches = [&](float x) { return equal ? x >= b : x > b; };
        // which of a lane's vectors of eight reach it
        uint32_t some = 0;
#pragma unroll
        for (int i = 0; i < per; ++i) {
            const uint4 q = i * 32 + lane < n_vec ? part[i * 32 + lane] : make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
            auto h = [](uint32_t v) { return *reinterpret_cast<const __nv_bfloat162 *>(&v); };
            const __nv_bfloat162 top = __hmax2(__hmax2(h(q.x), h(q.y)), __hmax2(h(q.z), h(q.w)));
            if (reaches(fmaxf(__low2float(top), __high2float(top)))) some |= 1u << i;
        }
        int n = 0;
        while (__any_sync(0xffffffffu, some != 0)) {
            const int i = some ? __ffs(some) - 1 : 0;
            float x[8];
            unpack<bf16, 8>(part[i * 32 + lane < n_vec ? i * 32 + lane : 0], x);
            uint32_t on = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (reaches(x[j]) && x[j] > -INFINITY) on |= 1u << j;
            if (!some) on = 0;
            some &= some - 1;
            while (__any_sync(0xffffffffu, on != 0)) {
                const uint32_t who = __ballot_sync(0xffffffffu, on != 0);
                const int to = n + __popc(who & ((1u << lane) - 1));
                if (on != 0 && to < kFew) ts.list[to] = static_cast<uint16_t>(8 * (i * 32 + lane) + __ffs(on) - 1);
                on &= on - 1;
                n += __popc(who);
            }
        }
        __syncwarp();
        return n;
    }
    // candidates of this CTA's share, each once: all above b, and the lowest K equal to
    // it at least; n: parts that reach it, listed
    __device__ __forceinline__ void collect(float b, int n) {
        if (view.n_single) {
            const int j = lane < view.n_single ? view.single(lane) : 0;
            const float v = lane < view.n_single ? to_f32(z[j]) : -INFINITY;
            push(v, j, v >= b && v > -INFINITY);
        }
        const bool some = b > -INFINITY, many = n > kFew;
        if (some && many) n = list_parts(b, false);
        if (n > kFew) {  // no list of them: all elements
            walk([&](float v) { return v > b; }, INT_MAX);
        } else {
            const int n_same = elements(n, b, some && !many);
            if (some && !many && n_same <= kFew) {
                for (int i0 = 0; i0 < n_same; i0 += 32) push(b, i0 + lane < n_same ? ts.same[i0 + lane] : 0, i0 + lane < n_same);
                __syncwarp();
                return;
            }
        }
        if (some) walk([&](float v) { return v == b; }, p.K);
        __syncwarp();
    }
    // the first `most` elements of this CTA's vectors that are wanted, in order
    template <typename F>
    __device__ __forceinline__ void walk(F wanted, int most) {
        int found = 0;
        for (int v0 = 0; v0 < view.count && found < most; v0 += 32) {
            const int v = v0 + lane;
            uint4 r = make_uint4(0, 0, 0, 0);
            load_if<true>(r, first + static_cast<int64_t>(v) * 16, v < view.count);
            float x[VEC];
            unpack<T, VEC>(r, x);
            int n = 0;
#pragma unroll
            for (int j = 0; j < VEC; ++j) n += v < view.count && wanted(x[j]);
            if (!__any_sync(0xffffffffu, n != 0)) continue;
            int before = n;
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, before, s);
                if (lane >= s) before += o;
            }
            const int all = __shfl_sync(0xffffffffu, before, 31);
            before += found - n;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const bool on = v < view.count && wanted(x[j]);
                push(x[j], view.head + (view.first + v) * VEC + j, on && before < most);
                before += on;
            }
            found += all;
        }
    }
    // ranks and outputs, R keys of a lane at a time
    template <int R>
    __device__ __forceinline__ void ranks(const uint64_t *keys, int n, int64_t row, float m, float lns) const {
        for (int i0 = 0; i0 < n; i0 += 32 * R) {
            uint64_t key[R];
            int at[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                key[r] = i0 + 32 * r + lane < n ? keys[i0 + 32 * r + lane] : 0;
                at[r] = 0;
            }
#pragma unroll 4
            for (int j = 0; j < n; j += 2) {
                const ulonglong2 o = *reinterpret_cast<const ulonglong2 *>(&keys[j]);
#pragma unroll
                for (int r = 0; r < R; ++r) at[r] += (o.x > key[r]) + (o.y > key[r]);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (key[r] == 0 || at[r] >= p.K) continue;
                const float v = key_value(key[r]);
                const int64_t to = row * p.K + at[r];
                if (p.top_ids) p.top_ids[to] = key_index(key[r]);
                if (p.top_logits) p.top_logits[to] = v;
                if (p.top_logp) p.top_logp[to] = __fmaf_rn(__fadd_rn(v, -m), p.inv_tau, -lns);
            }
        }
    }
    // the leader's part: ranks and outputs
    __device__ __forceinline__ void write(int64_t row, float m, float lns) {
        uint64_t *keys = size == 1 ? ts.key : ts.key + kCandidates + 2;
        int n = size == 1 ? n_key : ts.n_all;
        if (n > (size == 1 ? kCandidates : kCandidatesOfMany)) n = by_digits(keys);
        if (n > 128) n = largest(keys, n);
        if (lane == 0 && n % 2) keys[n] = 0;  // below every key; read in twos
        __syncwarp();
        if (n <= 32) ranks<1>(keys, n, row, m, lns);
        else if (n <= 64) ranks<2>(keys, n, row, m, lns);
        else ranks<4>(keys, n, row, m, lns);
        fill(row, n);
        __syncwarp();
        if (lane == 0) ts.n_all = 0;
        n_key = 0;
        __syncwarp();
    }
    // the candidates whose value is at least that of the K-th, in the place of all (ranks
    // take n^2 steps: 500 candidates of a cluster 120,000 cycles); how many
    __device__ __forceinline__ int largest(uint64_t *keys, int n) const {
        const uint32_t *words = reinterpret_cast<const uint32_t *>(keys);
        uint32_t at = 0;
        __syncwarp();
        for (int bit = 30; bit >= 0; bit -= 2) {
            int c[3] = {0, 0, 0};
#pragma unroll 4
            for (int i = lane; i < n; i += 32) {
                const uint32_t v = words[2 * i + 1];
#pragma unroll
                for (uint32_t d = 1; d < 4; ++d) c[d - 1] += v >= (at | d << bit);
            }
#pragma unroll
            for (int d = 0; d < 3; ++d) c[d] = static_cast<int>(__reduce_add_sync(0xffffffffu, c[d]));
            at |= static_cast<uint32_t>((c[0] >= p.K) + (c[1] >= p.K) + (c[2] >= p.K)) << bit;
        }
        int m = 0;
        for (int i0 = 0; i0 < n; i0 += 32) {
            const uint64_t key = i0 + lane < n ? keys[i0 + lane] : 0;
            const bool on = i0 + lane < n && static_cast<uint32_t>(key >> 32) >= at;
            const uint32_t who = __ballot_sync(0xffffffffu, on);  // all have read
            if (on) keys[m + __popc(who & ((1u << lane) - 1))] = key;
            m += __popc(who);
        }
        __syncwarp();
        return m;
    }
    // the row's K largest as the only candidates; how many
    __device__ __forceinline__ int by_digits(uint64_t *keys) const {
        const uint64_t least = kth_key<T>(z, p.V, p.K, ts.same);
        int n = 0;
        for (int j0 = 0; j0 < p.V; j0 += 32) {
            const int j = j0 + lane;
            const float v = j < p.V ? to_f32(z[j]) : -INFINITY;
            const uint64_t key = v > -INFINITY ? key_of(v, j) : 0;
            const bool on = key >= least && key != 0;
            const uint32_t who = __ballot_sync(0xffffffffu, on);
            if (on) keys[n + __popc(who & ((1u << lane) - 1))] = key;
            n += __popc(who);
        }
        __syncwarp();
        return n;
    }
    __device__ __forceinline__ void fill(int64_t row, int from) const {
        for (int k = from + lane; k < p.K; k += 32) {
            if (p.top_ids) p.top_ids[row * p.K + k] = -1;
            if (p.top_logits) p.top_logits[row * p.K + k] = -INFINITY;
            if (p.top_logp) p.top_logp[row * p.K + k] = -INFINITY;
        }
    }
};

// A list takes its warp 10,000 cycles (2,200 of them the bound's, 3,500 to 8,000 what
// is collected and ranked), whatever the row's length: short rows want more such warps
// on an SM, so small CTAs. 8192 rows of 4096 bf16, the best 20: 91 us with 4 CTAs of
// 288 threads on an SM, 46 with 12 of 96.
constexpr int kThreads = 288, kFewThreads = 96;
template <int NT>
constexpr int kCtas = NT == kFewThreads ? 12 : 4;

template <typename T, int NT, bool TOP>
__global__ void __launch_bounds__(NT, kCtas<NT>) logp_rows(const LogpParams p) {
    using View = RowView<T>;
    // warps that read rows; with lists the last one makes those
    constexpr int VEC = View::VEC, W = NT / 32 - (TOP ? 1 : 0), MT = W * 32, U = kBatch;
    __shared__ Shared<NT> sh;
    extern __shared__ __align__(16) char smem[];
    using Top = TopShared<MT>;
    Top &ts = *reinterpret_cast<Top *>(smem);
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int size = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
    const uint32_t n_clusters = gridDim.x / size;
    const int n_batches = (p.per + U * MT - 1) / (U * MT);       // of a thread, at most
    const int part_len = (n_batches + Top::kParts - 1) / Top::kParts;      // batches a part
    uint32_t live = 0;  // rows worked on: the exchange's parity
    if (TOP && tid == 0) ts.n_all = 0;
    if (size > 1) cluster_barrier();  // the other CTAs have started
    else __syncthreads();

    for (uint32_t item = blockIdx.x / size; item < static_cast<uint32_t>(p.T); item += n_clusters) {
        const int64_t row = sched_item(p.sched, item);
        const T *z = static_cast<const T *>(p.z) + row * p.ld;
        const int id = p.ids ? __ldg(p.ids + row) : 0, par = live & 1;
        const View view(z, p.V, rank, p.per);
        const char *first = reinterpret_cast<const char *>(z + view.head) + static_cast<int64_t>(view.first) * 16;
        TopOf<T, MT> top_of{p, ts, z, view, first, par, lane, part_len * U, size, 0};
        if (id < 0 || id >= p.V) {  // not read: zeros, and no alternatives
            if (rank == 0 && tid == 0) {
                if (id >= p.V) record_error(p.hdr, DGR_ERR_INVALID_ARG, kWhereId);
                if (p.logp) p.logp[row] = 0.0f;
                if (p.entropy) p.entropy[row] = 0.0f;
                if (p.lse) p.lse[row] = 0.0f;
                if (p.stats) p.stats[2 * row] = p.stats[2 * row + 1] = 0.0f;
            }
            if (TOP && rank == 0 && w == W) top_of.fill(row, 0);
            continue;
        }
        const bool finisher = rank == 0 && w == (TOP ? W : 0);  // the warp that has the row's outputs
        float x_id = 0.0f;
        if (p.logp && finisher) x_id = to_f32(z[id]);
        float shift = 0.0f;
        Triple all{-INFINITY, 0.0f, 0.0f};
        for (bool again = false;; again = true) {
            if (w < W) {
                Running run;
                float part = -INFINITY;
                int in_part = 0, n_part = 0;
                for (int v = tid; v < view.count; v += U * MT) {
                    uint4 r[U];
                    constexpr uint32_t low = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;  // -inf
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        r[u] = make_uint4(low, low, low, low);
                        load_if<true>(r[u], first + (static_cast<int64_t>(v) + u * MT) * 16, v + u * MT < view.count);
                    }
                    const float top = max_of<T, U>(r);
                    if (TOP && !again) {
                        part = fmaxf(part, top);
                        if (++in_part == part_len) {
                            if (Top::kFewThreads) ts.top[par][n_part * MT + tid] = part;
                            ts.part[par][n_part++][tid] = up_to_bf16(part);
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
                    for (; n_part < Top::kParts; ++n_part) {
                        if (Top::kFewThreads) ts.top[par][n_part * MT + tid] = part;
                        ts.part[par][n_part][tid] = up_to_bf16(part);
                        part = -INFINITY;
                    }
                if (tid < view.n_single) {
                    const float x = __fadd_rn(to_f32(z[view.single(tid)]), -shift);
                    run.raise(x, p.k2);
                    run.add_one(at_least_masked(x), p.k2);
                }
                if (TOP && !Top::kFewThreads && !again) ts.top[par][tid] = run.m;
                Triple mine{run.m, across(run.s), across(run.a)};
                mine.over_warp(p.k2);
                if (lane < size) remote_store(remote(&sh.triple[par][rank * W + w], lane), make_float4(mine.m, mine.s, mine.a, 0.0f));
                __syncwarp();
            }
            if (size > 1) cluster_barrier();
            else __syncthreads();
            all = Triple{-INFINITY, 0.0f, 0.0f};
            for (int j = lane; j < size * W; j += 32) all.m = fmaxf(all.m, sh.triple[par][j].x);
            all.m = warp_max(all.m);
            if (again || !(fabsf(all.m) < INFINITY) || fabsf(__fmul_rn(all.m, p.k2)) < kFar) break;
            shift = all.m;  // the same in every warp of the cluster
            if (size > 1) cluster_barrier();  // before the triples are written over
            else __syncthreads();
        }
        const float m = shift != 0.0f ? shift : all.m;
        float lns = 0.0f;
        if (finisher) {
            const float c = scaled_max(all.m, p.k2);
            for (int j = lane; j < size * W; j += 32) {
                const float4 got = sh.triple[par][j];
                Triple t{got.x, got.y, got.z};
                t.to(all.m, p.k2);
                all.s = __fadd_rn(all.s, t.s);
                all.a = __fadd_rn(all.a, t.a);
            }
            all.s = warp_sum(all.s);
            all.a = warp_sum(all.a);
            const bool none = m == -INFINITY && all.s == 0.0f;  // nothing is left of the row (a sum of NaN: it holds NaN)
            const float ln_s = logf(all.s);
            // ln s for the maximum itself: without the rounding of c
            lns = none ? 0.0f : __fmaf_rn(__fmaf_rn(all.m, p.k2, -c), -kLn2, ln_s);
            if (lane == 0) {
                if (p.logp) p.logp[row] = none ? -INFINITY : __fmaf_rn(__fadd_rn(x_id, -m), p.inv_tau, -lns);
                if (p.entropy) p.entropy[row] = none ? 0.0f : __fmaf_rn(-kLn2, all.a / all.s, ln_s);
                if (p.lse) p.lse[row] = __fmaf_rn(m, p.inv_tau, lns);
                if (p.stats) p.stats[2 * row] = m, p.stats[2 * row + 1] = lns;
            }
        }
        if constexpr (TOP) {
            // the last warp makes the list while the others go on to the next row
            // (where a row has several CTAs, they meet at the barriers)
            float bound = 0.0f;
            int reach = 0;
            if (w == W && size == 1) {
                bound = top_of.value_of(top_of.bound(p.K, 16));
                reach = top_of.list_parts(bound, true);
                if (sizeof(T) == 4 && reach > kFew) {
                    bound = top_of.value_of(top_of.bound(p.K, 0));
                    reach = top_of.list_parts(bound, true);
                }
            }
            if (size > 1) {
                // the row has K elements from any CTA's K-th on, and from the least of
                // their K / CTAs-th on, which is nearer where the large ones are spread
                if (w == W) {
                    const float2 mine = make_float2(top_of.near_bound(p.K), top_of.near_bound((p.K + size - 1) / size));
                    if (lane < size) remote_store(remote(&sh.bound[par][rank], lane), mine);
                }
                cluster_barrier();
                float one = -INFINITY, each = INFINITY;
                for (int r = 0; r < size; ++r) one = fmaxf(one, sh.bound[par][r].x), each = fminf(each, sh.bound[par][r].y);
                bound = fmaxf(one, each);
                if (w == W) reach = top_of.list_parts(bound, true);
            }
            if (w == W) {
                top_of.collect(bound, reach);
                if (size > 1) top_of.gather();
            }
            if (size > 1) cluster_barrier();
            if (w == W && rank == 0) top_of.write(row, m, lns);
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
        // (no maximum and a logarithm of the sum that is a number: a row of nothing but -inf)
        on = (!p.ids || (id >= 0 && id < p.V)) && !(m == -INFINITY && l == l);
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
    constexpr size_t kTop = sizeof(TopShared<NT - 32>);
    const size_t smem = TOP ? kTop + static_cast<size_t>(kCandidates + 2 + (cluster == 1 ? 0 : kCandidatesOfMany + 2)) * 8 : 0;
    dgr_status st = allow_smem(k, smem, kTop + (kCandidates + 2 + kCandidatesOfMany + 2) * 8);
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
    cfg.numAttrs = NT != kFewThreads;  // (an SM has 8 CTAs of clusters at most, of one CTA too)
    int clusters = p.T;
    if (cluster > 1 && static_cast<int64_t>(p.T) * cluster > sms && (cudaOccupancyMaxActiveClusters(&clusters, k, &cfg) != cudaSuccess || clusters < 1)) return DGR_ERR_CUDA;
    const int within = sms * kCtas<NT> / cluster;  // a green context's, or the test's cap
    if (clusters > within) clusters = within > 0 ? within : 1;
    if (clusters > p.T) clusters = p.T;
    const unsigned capped = sched_grid(static_cast<unsigned>(clusters * cluster)) / cluster;
    cfg.gridDim = dim3((capped > 0 ? capped : 1) * cluster);
    return cudaLaunchKernelEx(&cfg, k, p) == cudaSuccess ? DGR_OK : DGR_ERR_CUDA;
}

// Rows for the small CTAs: short, as two warps have too few loads in flight for long
// ones (2048 vectors, the best 20 of 8192 fp32 rows: 71 us, with large CTAs 93; 4096
// vectors: 126 and 116); with maxima of parts enough for a bound that leaves few (2 K);
// and so many that the large CTAs' list warps would be behind (300 rows of 8192 bf16,
// the best 20: 15.5 us with the small ones, 14.5 with the large; 700, the best 64: 19.5
// and 24.7). The device's SMs
// have no say: a row's sums are in the same order on a part of it.
constexpr int kShort = 2048, kMany = 608;

template <typename T>
dgr_status launch_forward(LogpParams &p, int sms, cudaStream_t s) {
    // few rows: a row over more CTAs, down to 4096 elements each
    int cluster = 1;
    while (cluster < kMaxCluster && static_cast<int64_t>(p.T) * cluster * 2 <= 304 && p.V >= 4096 * cluster * 2) cluster <<= 1;
    if (!p.K) return launch_rows<T, 256, false>(p, cluster, sms, s);
    constexpr int kReaders = kFewThreads - 32, kRound = kReaders * kBatch;
    const int64_t vecs = p.V / (16 / static_cast<int>(sizeof(T))), last = vecs % kRound;
    const int64_t maxima = vecs / kRound * kReaders + (last < kReaders ? last : kReaders);
    const bool small = vecs <= kShort && maxima >= 2 * p.K && p.T > kMany;
    return small ? launch_rows<T, kFewThreads, true>(p, 1, sms, s) : launch_rows<T, kThreads, true>(p, cluster, sms, s);
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
    if (!(dlogits == logits && ld == ld_d) && runs_overlap({dlogits, ld_d * es, T, 0, 1, V * es}, {logits, ld * es, T, 0, 1, V * es})) return DGR_ERR_ALIAS;
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
