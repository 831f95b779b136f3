// Router balance loss with per-expert counts, and its gradient.
//
//   p_t = softmax(l_t), or the sigmoids of l_t divided by their sum;
//   c[g][e] = slots (t, k) of group g's valid tokens with ids[t][k] = e,
//   n_g = valid tokens of group g;
//   loss = sum_g a_g sum_e c[g][e] sum_{t in g} p_t[e],  a_g = coeff E / (G K n_g^2);
//   dl_t[e] = dloss a_g p_t[e] (c[g][e] - sum_j c[g][j] p_t[j])  [(1 - sigmoid(l_t[e]))].
//
// Megatron-LM PR #7441, Source 5, reduces the loss with a cross-block float
// atomicAdd; here every sum has one writer and a fixed order.
//
// Forward, one launch: a CTA per tile of consecutive tokens of one group. A row
// is held by the fewest lanes that cover it with 16 logits each, so a softmax's
// maximum and sum cost log2(E / 16) shuffles for several rows at a time; the
// next rows' logits are loaded before the present ones are worked on. A lane
// keeps the running sums of its own experts' probabilities over the tile, which
// lanes, then warps, then tiles add in ascending order. The counts are integer
// sums (shared-memory integer atomics: any order, the same value). The CTA that
// finishes a group last folds the group's tiles, and the one that finishes the
// last group adds the groups.
#include "row_common.cuh"

namespace dgr {
namespace {

using namespace row;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBackThreads = 256;
constexpr int kBackTile = 128;  // tokens a backward tile
constexpr int kMaxExperts = 1024;
constexpr int kMaxGroups = 1024;
constexpr int kMaxTile = 16384;  // tokens: a lane's running sums stay short

enum { kWhereOffsets = 301, kWhereExpertId = 302 };

struct BalParams {
    const void *logits;
    int64_t ld;
    const int32_t *ids;
    int64_t ld_ids;
    const uint8_t *mask;
    const int64_t *offs;  // null: one group of all N tokens
    int32_t N, E, K, G;
    int32_t sigmoid;
    int32_t tile;         // tokens a tile
    int32_t lanes;        // lanes a row
    uint64_t k_magic;     // ceil(2^40 / K): i / K for i < 2^24
    float coef;           // coeff E / (G K)
    int32_t *counts, *tokens;
    float *loss;
    // forward's workspace
    WsHeader *hdr;        // pad[0]: groups done
    int32_t *done;        // [G] tiles done
    float *group_loss;    // [G]
    float *mass;          // [tiles][E]
    int32_t *part;        // [tiles][E]: counts
    int32_t *live;        // [tiles]: valid tokens
    // backward
    const float *dloss;
    void *dlogits;
    int64_t ld_d;
    int32_t accumulate;
    Sched sched;
};

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
    for (int s = 1; s < lanes; s <<= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, s));
    return v;
}

__device__ __forceinline__ float lanes_max(float v, int lanes) {
    for (int s = 1; s < lanes; s <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, s));
    return v;
}

// The row's probabilities in place of its logits (lanes without an expert
// hold -inf and get 0; a row of -inf only gets 0 everywhere). A NaN or +inf
// logit makes the row NaN, as the formula does.
template <int E>
__device__ __forceinline__ void scores(float (&x)[E], int lanes, int sigmoid) {
    float m = x[0];
#pragma unroll
    for (int e = 1; e < E; ++e) m = fmaxf(m, x[e]);
    m = lanes_max(m, lanes);
    const bool empty = m == -INFINITY;
    float s = 0.0f;
    if (!sigmoid) {
        const float c = empty ? 0.0f : m;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            x[e] = ex2(__fmul_rn(__fadd_rn(x[e], -c), kLog2e));
            s = __fadd_rn(s, x[e]);
        }
    } else {
        // all logits below 0: each sigmoid divided by exp(m), so that rows far
        // below 0 keep their shares
        const bool low = m < 0.0f && !empty;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float a = low ? ex2(__fmul_rn(__fadd_rn(x[e], -m), kLog2e)) : 1.0f;
            x[e] = __fdividef(a, __fadd_rn(1.0f, ex2(__fmul_rn(low ? x[e] : -x[e], kLog2e))));
            s = __fadd_rn(s, x[e]);
        }
    }
    s = lanes_sum(s, lanes);
    const float inv = s == 0.0f ? 0.0f : 1.0f / s;
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = __fmul_rn(x[e], inv);
}

// A lane's experts: vector i of NV starts at expert (i * lanes + sub) * VEC.
template <typename T, int VEC, int NV>
struct Logits {
    raw_t<T, VEC> v[NV];
    uint32_t there;  // vectors with experts

    __device__ __forceinline__ void load(const T *row, int sub, int lanes, int E, bool live) {
        there = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (i * lanes + sub) * VEC;
            if (live && e < E) {
                v[i] = *reinterpret_cast<const raw_t<T, VEC> *>(row + e);
                there |= 1u << i;
            }
        }
    }
    __device__ __forceinline__ void get(float *x) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            unpack<T, VEC>(v[i], x + i * VEC);
            if (!(there >> i & 1))
#pragma unroll
                for (int j = 0; j < VEC; ++j) x[i * VEC + j] = -INFINITY;
        }
    }
};

// tbase[g] = first tile of group g, offsets into so[]; false when the offsets
// break their contract. Every block computes the same.
__device__ bool group_tiles(const BalParams &p, int32_t *tbase, int64_t *so, int32_t *wsum, int32_t *bad) {
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    if (!p.offs) {
        if (tid == 0) {
            so[0] = 0, so[1] = p.N;
            tbase[0] = 0, tbase[1] = (p.N + p.tile - 1) / p.tile;
        }
        __syncthreads();
        return true;
    }
    if (tid == 0) *bad = 0;
    __syncthreads();
    int32_t run = 0;
    for (int g0 = 0; g0 < p.G; g0 += kThreads) {
        const int g = g0 + tid;
        int32_t c = 0;
        if (g < p.G) {
            const int64_t a = p.offs[g], b = p.offs[g + 1];
            so[g] = a;
            if (g == p.G - 1) so[p.G] = b;
            if (b < a || a < 0 || b > p.N || (g == 0 && a != 0) || (g == p.G - 1 && b != p.N)) *bad = 1;
            else c = static_cast<int32_t>((b - a + p.tile - 1) / p.tile);
        }
        int32_t incl = c;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const int32_t o = __shfl_up_sync(0xffffffffu, incl, s);
            if (lane >= s) incl += o;
        }
        if (lane == 31) wsum[w] = incl;
        __syncthreads();
        int32_t before = run;
        for (int v = 0; v < w; ++v) before += wsum[v];
        if (g < p.G) tbase[g] = before + incl - c;
        for (int v = 0; v < kWarps; ++v) run += wsum[v];
        __syncthreads();
    }
    if (tid == 0) tbase[p.G] = run;
    __syncthreads();
    return *bad == 0;
}

// The last g with table[g] <= v (table ascending, table[0] <= v < table[n]):
// a group with something in it, as empty ones share their start with the next.
template <typename I>
__device__ __forceinline__ int group_of(const I *table, int n, I v) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (table[mid] <= v) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Adds a group's tiles, CV experts a thread: `ways` threads share an expert's
// tiles (way w takes w, w + ways, ...), their sums are added in ascending
// order. Writes the group's counts; returns this thread's part of their dot
// product with the probabilities.
template <int CV>
__device__ float fold_tiles(const BalParams &p, int first, int n, int g, float *buf) {
    const int tid = threadIdx.x, n_col = p.E / CV;
    int span = 1;
    while (span < n_col && span < kThreads) span <<= 1;
    const int ways = kThreads / span, way = tid / span;
    float dot = 0.0f;
    int32_t *ibuf = reinterpret_cast<int32_t *>(buf) + CV * kThreads;
    for (int c0 = 0; c0 < n_col; c0 += span) {
        const int col = c0 + (tid & (span - 1));
        float m[CV];
        int32_t c[CV];
#pragma unroll
        for (int j = 0; j < CV; ++j) m[j] = 0.0f, c[j] = 0;
        if (col < n_col)
#pragma unroll 8
            for (int t = way; t < n; t += ways) {
                const int64_t at = static_cast<int64_t>(first + t) * p.E + col * CV;
                if constexpr (CV == 4) {
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(p.mass + at));
                    const int4 k = __ldcg(reinterpret_cast<const int4 *>(p.part + at));
                    m[0] = __fadd_rn(m[0], v.x), m[1] = __fadd_rn(m[1], v.y), m[2] = __fadd_rn(m[2], v.z), m[3] = __fadd_rn(m[3], v.w);
                    c[0] += k.x, c[1] += k.y, c[2] += k.z, c[3] += k.w;
                } else {
                    m[0] = __fadd_rn(m[0], __ldcg(p.mass + at));
                    c[0] += __ldcg(p.part + at);
                }
            }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < CV; ++j) buf[j * kThreads + tid] = m[j], ibuf[j * kThreads + tid] = c[j];
        __syncthreads();
        // one thread an expert
        for (int e = tid; e < span * CV; e += kThreads) {
            const int j = e & (CV - 1), k0 = e / CV;
            if (c0 + k0 >= n_col) continue;
            float v = buf[j * kThreads + k0];
            int32_t k = ibuf[j * kThreads + k0];
            for (int q = 1; q < ways; ++q) {
                v = __fadd_rn(v, buf[j * kThreads + q * span + k0]);
                k += ibuf[j * kThreads + q * span + k0];
            }
            p.counts[static_cast<int64_t>(g) * p.E + (c0 + k0) * CV + j] = k;
            dot = __fmaf_rn(static_cast<float>(k), v, dot);
        }
    }
    return dot;
}

template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(kThreads) balance_forward(const BalParams p) {
    extern __shared__ char smem[];
    int64_t *so = reinterpret_cast<int64_t *>(smem);                        // [G + 1]
    int32_t *tbase = reinterpret_cast<int32_t *>(so + p.G + 1);             // [G + 1]
    int32_t *hist = tbase + p.G + 1;                                        // [E]
    float *cols = reinterpret_cast<float *>(hist + p.E);                    // [kWarps][E], later [kThreads]
    __shared__ int32_t wsum[kWarps], bad, valid, last, n_groups;
    __shared__ float red[32];
    constexpr int EL = NV * VEC;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    if (!group_tiles(p, tbase, so, wsum, &bad)) {
        if (blockIdx.x == 0 && tid == 0) record_error(p.hdr, DGR_ERR_INVALID_ARG, kWhereOffsets);
        return;
    }
    const int n_tiles = tbase[p.G];
    // groups without tokens: nothing counts
    for (int g = blockIdx.x; g < p.G; g += gridDim.x)
        if (tbase[g + 1] == tbase[g]) {
            for (int e = tid; e < p.E; e += kThreads) p.counts[static_cast<int64_t>(g) * p.E + e] = 0;
            if (tid == 0) p.tokens[g] = 0;
        }
    if (n_tiles == 0) {
        if (blockIdx.x == 0 && tid == 0) *p.loss = 0.0f;
        return;
    }
    if (tid == 0) n_groups = 0;
    __syncthreads();
    for (int g = tid; g < p.G; g += kThreads)
        if (tbase[g + 1] > tbase[g]) atomicAdd(&n_groups, 1);
    const int sub = lane & (p.lanes - 1), rows_warp = 32 / p.lanes, my_row = lane / p.lanes;
    const Sched sched = sched_over(p.sched, static_cast<uint32_t>(n_tiles));
    for (int it = blockIdx.x; it < n_tiles; it += gridDim.x) {
        const int tile = static_cast<int>(sched_item(sched, static_cast<uint32_t>(it)));
        const int g = p.G == 1 ? 0 : group_of(tbase, p.G, tile);
        const int64_t t0 = so[g] + static_cast<int64_t>(tile - tbase[g]) * p.tile;
        const int count = static_cast<int>(min(static_cast<int64_t>(p.tile), so[g + 1] - t0));
        for (int e = tid; e < p.E; e += kThreads) hist[e] = 0;
        if (tid == 0) valid = 0;
        __syncthreads();
        // the first rows' logits are on their way while the counts are made
        const T *base = static_cast<const T *>(p.logits) + t0 * p.ld;
        auto is_live = [&](int r) { return r < count && (!p.mask || p.mask[t0 + r]); };
        Logits<T, VEC, NV> cur, nxt;
        bool live = is_live(w * rows_warp + my_row), live_next = false;
        cur.load(base + static_cast<int64_t>(w * rows_warp + my_row) * p.ld, sub, p.lanes, p.E, live);
        const int n_ids = count * p.K;
        for (int i0 = tid; i0 < n_ids; i0 += 4 * kThreads) {
            int32_t id[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = i0 + j * kThreads;
                id[j] = -1;
                if (i < n_ids) {
                    const int r = static_cast<int>((static_cast<uint64_t>(i) * p.k_magic) >> 40);
                    if (!p.mask || p.mask[t0 + r]) id[j] = __ldg(p.ids + (t0 + r) * p.ld_ids + (i - r * p.K));
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (id[j] < 0) continue;
                if (id[j] >= p.E) record_error(p.hdr, DGR_ERR_INVALID_ARG, kWhereExpertId);
                else atomicAdd(&hist[id[j]], 1);
            }
        }
        if (p.mask) {
            int mine = 0;
            for (int r = tid; r < count; r += kThreads) mine += p.mask[t0 + r] != 0;
            mine = __reduce_add_sync(0xffffffffu, mine);
            if (lane == 0 && mine) atomicAdd(&valid, mine);
        } else if (tid == 0) {
            valid = count;
        }
        // the experts' probabilities over the tile's tokens
        float acc[EL];
#pragma unroll
        for (int e = 0; e < EL; ++e) acc[e] = 0.0f;
        for (int b = w * rows_warp; b < count; b += kWarps * rows_warp) {
            const int r = b + kWarps * rows_warp + my_row;
            live_next = is_live(r);
            nxt.load(base + static_cast<int64_t>(r) * p.ld, sub, p.lanes, p.E, live_next);
            float x[EL];
            cur.get(x);
            scores(x, p.lanes, p.sigmoid);
#pragma unroll
            for (int e = 0; e < EL; ++e) acc[e] = __fadd_rn(acc[e], live ? x[e] : 0.0f);
            cur = nxt;
            live = live_next;
        }
#pragma unroll
        for (int e = 0; e < EL; ++e)
            for (int s = p.lanes; s < 32; s <<= 1) acc[e] = __fadd_rn(acc[e], __shfl_xor_sync(0xffffffffu, acc[e], s));
        if (lane < p.lanes) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const int e = (i * p.lanes + sub) * VEC + j;
                    if (e < p.E) cols[w * p.E + e] = acc[i * VEC + j];
                }
        }
        __syncthreads();
        float *mass = p.mass + static_cast<int64_t>(tile) * p.E;
        int32_t *part = p.part + static_cast<int64_t>(tile) * p.E;
        for (int e = tid; e < p.E; e += kThreads) {
            float v = cols[e];
#pragma unroll
            for (int k = 1; k < kWarps; ++k) v = __fadd_rn(v, cols[k * p.E + e]);
            mass[e] = v;
            part[e] = hist[e];
        }
        if (tid == 0) p.live[tile] = valid;
        __threadfence();
        __syncthreads();
        if (tid == 0) last = atomicAdd(&p.done[g], 1) == tbase[g + 1] - tbase[g] - 1;
        __syncthreads();
        if (!last) continue;
        // this group's tiles are all in: fold them
        __threadfence();
        const int first = tbase[g], n = tbase[g + 1] - first;
        int32_t tokens = 0;
        for (int j = tid; j < n; j += kThreads) tokens += __ldcg(p.live + first + j);
        if (tid == 0) valid = 0;
        __syncthreads();
        tokens = __reduce_add_sync(0xffffffffu, tokens);
        if (lane == 0 && tokens) atomicAdd(&valid, tokens);
        const float dot = p.E % 4 == 0 ? fold_tiles<4>(p, first, n, g, cols) : fold_tiles<1>(p, first, n, g, cols);
        float s[1] = {dot};
        block_sum<1>(s, red, kWarps);
        if (tid == 0) {
            const float nt = static_cast<float>(max(valid, 1));
            p.tokens[g] = valid;
            p.group_loss[g] = p.coef * s[0] / (nt * nt);
            p.done[g] = 0;  // ready for the next call
            __threadfence();
            last = atomicAdd(&p.hdr->pad[0], 1) == n_groups - 1;
        }
        __syncthreads();
        if (!last) continue;
        __threadfence();
        float t[1] = {0.0f};
        for (int k = tid; k < p.G; k += kThreads)
            if (tbase[k + 1] > tbase[k]) t[0] = __fadd_rn(t[0], __ldcg(p.group_loss + k));
        block_sum<1>(t, red, kWarps);
        if (tid == 0) {
            *p.loss = t[0];
            p.hdr->pad[0] = 0;
        }
        return;
    }
}

template <typename T, int VEC, int NV, bool SIGMOID>
__global__ void __launch_bounds__(kBackThreads) balance_backward(const BalParams p) {
    extern __shared__ char smem[];
    int64_t *so = reinterpret_cast<int64_t *>(smem);  // [G + 1] when there are offsets
    constexpr int EL = NV * VEC, kBackWarps = kBackThreads / 32;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    if (p.offs) {
        for (int g = tid; g <= p.G; g += kBackThreads) so[g] = p.offs[g];
        __syncthreads();
    }
    const int sub = lane & (p.lanes - 1), rows_warp = 32 / p.lanes, my_row = lane / p.lanes;
    const int step = kBackWarps * rows_warp;
    const float up = p.dloss ? __fmul_rn(__ldg(p.dloss), p.coef) : p.coef;
    const int n_tiles = (p.N + kBackTile - 1) / kBackTile;
    for (int it = blockIdx.x; it < n_tiles; it += gridDim.x) {
        const int64_t t0 = static_cast<int64_t>(sched_item(p.sched, static_cast<uint32_t>(it))) * kBackTile;
        const int count = static_cast<int>(min(static_cast<int64_t>(kBackTile), p.N - t0));
        const T *base = static_cast<const T *>(p.logits) + t0 * p.ld;
        // offsets outside their contract leave tokens without a group: no gradient
        auto is_live = [&](int r) {
            return r < count && (!p.mask || p.mask[t0 + r]) && (!p.offs || (t0 + r >= so[0] && t0 + r < so[p.G]));
        };
        int have = -1;
        float a[EL];  // the group's counts times its factor
#pragma unroll
        for (int e = 0; e < EL; ++e) a[e] = 0.0f;
        Logits<T, VEC, NV> cur, nxt;
        bool live = is_live(w * rows_warp + my_row), live_next = false;
        cur.load(base + static_cast<int64_t>(w * rows_warp + my_row) * p.ld, sub, p.lanes, p.E, live);
        for (int b = w * rows_warp; b < count; b += step) {
            const int r = b + my_row;
            live_next = is_live(r + step);
            nxt.load(base + static_cast<int64_t>(r + step) * p.ld, sub, p.lanes, p.E, live_next);
            const int g = live && p.offs ? group_of(so, p.G, t0 + r) : 0;
            if (live && g != have) {
                have = g;
                const float nt = static_cast<float>(max(__ldg(p.tokens + g), 1));
                const float f = up / (nt * nt);
                const int32_t *counts = p.counts + static_cast<int64_t>(g) * p.E;
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const int e = (i * p.lanes + sub) * VEC + j;
                        a[i * VEC + j] = e < p.E ? __fmul_rn(f, static_cast<float>(__ldg(counts + e))) : 0.0f;
                    }
            }
            float q[EL];
            cur.get(q);
            scores(q, p.lanes, SIGMOID);
            float inner = 0.0f;
#pragma unroll
            for (int e = 0; e < EL; ++e) inner = __fmaf_rn(a[e], live ? q[e] : 0.0f, inner);
            inner = lanes_sum(inner, p.lanes);
            if (r < count) {
                T *dst = static_cast<T *>(p.dlogits) + (t0 + r) * p.ld_d;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int e = (i * p.lanes + sub) * VEC;
                    if (e >= p.E) continue;
                    float d[VEC], x[VEC];
                    if (SIGMOID) unpack<T, VEC>(cur.v[i], x);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const int k = i * VEC + j;
                        d[j] = __fmul_rn(q[k], __fadd_rn(a[k], -inner));
                        if (SIGMOID) d[j] = __fdividef(d[j], __fadd_rn(1.0f, ex2(__fmul_rn(x[j], kLog2e))));
                        if (!live) d[j] = 0.0f;
                    }
                    raw_t<T, VEC> *to = reinterpret_cast<raw_t<T, VEC> *>(dst + e);
                    if (p.accumulate) {
                        float old[VEC];
                        unpack<T, VEC>(*to, old);
#pragma unroll
                        for (int j = 0; j < VEC; ++j) d[j] = live ? __fadd_rn(old[j], d[j]) : old[j];
                    }
                    *to = pack<T, VEC>(d);
                }
            }
            cur = nxt;
            live = live_next;
        }
    }
}

// Host side -------------------------------------------------------------------

// Tokens a tile: about one tile an SM of the 152, at least 8192 logits (below
// that a tile's fold costs more than its rows).
int32_t balance_tile(int64_t N, int64_t E) {
    const int64_t per = (N + 151) / 152, least = (8192 + E - 1) / E;
    const int64_t t = ((per > least ? per : least) + 31) / 32 * 32;
    return static_cast<int32_t>(t < kMaxTile ? t : kMaxTile);
}

struct BalLayout {
    int64_t tiles;
    size_t done, group_loss, mass, part, live, total;
};

BalLayout balance_layout(int64_t N, int64_t E, int64_t G) {
    BalLayout L{};
    const int64_t tile = balance_tile(N, E);
    L.tiles = (N + tile - 1) / tile + (G > 1 ? G : 0);
    L.done = sizeof(WsHeader);
    L.group_loss = L.done + align_up(static_cast<size_t>(G) * 4);
    L.mass = L.group_loss + align_up(static_cast<size_t>(G) * 4);
    L.part = L.mass + align_up(static_cast<size_t>(L.tiles) * E * 4);
    L.live = L.part + align_up(static_cast<size_t>(L.tiles) * E * 4);
    L.total = L.live + align_up(static_cast<size_t>(L.tiles) * 4);
    return L;
}

template <typename T, int VEC, int NV>
dgr_status launch_nv(bool backward, const BalParams &p, unsigned grid, cudaStream_t s) {
    if (backward) {
        const size_t smem = p.offs ? (p.G + 1) * 8 : 0;
        if (p.sigmoid) balance_backward<T, VEC, NV, true><<<grid, kBackThreads, smem, s>>>(p);
        else balance_backward<T, VEC, NV, false><<<grid, kBackThreads, smem, s>>>(p);
    } else {
        const size_t cols = static_cast<size_t>(kWarps) * p.E * 4, fold = kThreads * (p.E % 4 == 0 ? 32 : 8);  // the fold reuses the columns' place
        const size_t smem = (p.G + 1) * 12 + p.E * 4 + (cols > fold ? cols : fold);
        if (smem > 47 * 1024 && cudaFuncSetAttribute(balance_forward<T, VEC, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
            return DGR_ERR_CUDA;
        balance_forward<T, VEC, NV><<<grid, kThreads, smem, s>>>(p);
    }
    return launch_status();
}

template <typename T, int VEC>
dgr_status launch_vec(bool backward, BalParams &p, unsigned grid, cudaStream_t s) {
    // 16 logits a lane (fewer lanes, fewer shuffles) until a row takes the whole warp
    const int n_vec = (p.E + VEC - 1) / VEC;
    p.lanes = 1;
    while (p.lanes < 32 && p.lanes * 16 < n_vec * VEC) p.lanes <<= 1;
    const int nv = (n_vec + p.lanes - 1) / p.lanes;
    if constexpr (VEC == 4) {
        if (nv <= 2) return launch_nv<T, VEC, 2>(backward, p, grid, s);
        if (nv <= 4) return launch_nv<T, VEC, 4>(backward, p, grid, s);
        return launch_nv<T, VEC, 8>(backward, p, grid, s);
    } else {
        if (nv <= 8) return launch_nv<T, VEC, 8>(backward, p, grid, s);
        if (nv <= 16) return launch_nv<T, VEC, 16>(backward, p, grid, s);
        return launch_nv<T, VEC, 32>(backward, p, grid, s);
    }
}

// Vectors of 4 experts where every row starts at a multiple of them.
template <typename T>
dgr_status launch_type(bool backward, BalParams &p, unsigned grid, cudaStream_t s) {
    const bool vec = p.E % 4 == 0 && p.ld % 4 == 0 && aligned(p.logits, 4 * sizeof(T)) &&
                     (!backward || (p.ld_d % 4 == 0 && aligned(p.dlogits, 4 * sizeof(T))));
    return vec ? launch_vec<T, 4>(backward, p, grid, s) : launch_vec<T, 1>(backward, p, grid, s);
}

size_t extent(int64_t N, int64_t W, int64_t ld, int64_t es) { return N > 0 ? static_cast<size_t>(((N - 1) * ld + W) * es) : 0; }

}  // namespace
}  // namespace dgr

using namespace dgr;

extern "C" size_t dgr_router_balance_workspace_bytes(int64_t N, int32_t E, int32_t G) {
    if (N < 0 || N > INT32_MAX || E < 1 || E > kMaxExperts || G < 1 || G > kMaxGroups) return 0;
    return balance_layout(N, E, G).total;
}

extern "C" dgr_status dgr_router_balance(const void *logits, int32_t dtype, int64_t N, int32_t E, int64_t ld,
                                         const int32_t *ids, int32_t K, int64_t ld_ids, const uint8_t *mask,
                                         const int64_t *d_offs, int32_t G, int32_t score, float coeff, int32_t *counts,
                                         int32_t *tokens, float *loss, void *ws, size_t ws_bytes, void *stream) {
    if ((dtype != DGR_DTYPE_BF16 && dtype != DGR_DTYPE_F32) || score < 0 || score > 1) return DGR_ERR_INVALID_ARG;
    if (N < 0 || E < 1 || K < 1 || G < 1 || ld < E || ld_ids < K || (!d_offs && G != 1)) return DGR_ERR_INVALID_ARG;
    if (!counts || !tokens || !loss || !ws || (N > 0 && (!logits || !ids))) return DGR_ERR_INVALID_ARG;
    if (N > INT32_MAX || E > kMaxExperts || K > kMaxExperts || G > kMaxGroups) return DGR_ERR_UNSUPPORTED;
    const int es = dtype == DGR_DTYPE_BF16 ? 2 : 4;
    if (!aligned(logits, es) || !aligned(ids, 4) || !aligned(d_offs, 8) || !aligned(counts, 4) || !aligned(tokens, 4) || !aligned(loss, 4))
        return DGR_ERR_MISALIGNED;
    const BalLayout L = balance_layout(N, E, G);
    if (ws_bytes < L.total) return DGR_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned(ws, kAlign)) return DGR_ERR_MISALIGNED;
    struct Range { const void *q; size_t n; };
    const Range ins[] = {{logits, extent(N, E, ld, es)}, {ids, extent(N, K, ld_ids, 4)}, {mask, static_cast<size_t>(N)},
                         {d_offs, static_cast<size_t>(G + 1) * 8}};
    const Range outs[] = {{counts, static_cast<size_t>(G) * E * 4}, {tokens, static_cast<size_t>(G) * 4}, {loss, 4}, {ws, L.total}};
    for (const Range &o : outs) {
        for (const Range &i : ins)
            if (ranges_overlap(o.q, o.n, i.q, i.n)) return DGR_ERR_ALIAS;
        for (const Range &b : outs)
            if (&o < &b && ranges_overlap(o.q, o.n, b.q, b.n)) return DGR_ERR_ALIAS;
    }
    dgr_status st = check_device();
    if (st != DGR_OK) return st;
    BalParams p{};
    p.logits = logits, p.ld = ld, p.ids = ids, p.ld_ids = ld_ids, p.mask = mask, p.offs = d_offs;
    p.N = static_cast<int32_t>(N), p.E = E, p.K = K, p.G = G, p.sigmoid = score;
    p.tile = balance_tile(N, E);
    p.coef = static_cast<float>(static_cast<double>(coeff) * E / (static_cast<double>(G) * K));
    p.counts = counts, p.tokens = tokens, p.loss = loss;
    char *b = static_cast<char *>(ws);
    p.hdr = reinterpret_cast<WsHeader *>(b);
    p.done = reinterpret_cast<int32_t *>(b + L.done);
    p.group_loss = reinterpret_cast<float *>(b + L.group_loss);
    p.mass = reinterpret_cast<float *>(b + L.mass);
    p.part = reinterpret_cast<int32_t *>(b + L.part);
    p.live = reinterpret_cast<int32_t *>(b + L.live);
    p.k_magic = ((1ull << 40) + K - 1) / K;
    p.sched = sched_setting();
    const unsigned grid = sched_grid(static_cast<unsigned>(L.tiles > 0 ? L.tiles : 1));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return es == 2 ? launch_type<bf16>(false, p, grid, s) : launch_type<float>(false, p, grid, s);
}

extern "C" dgr_status dgr_router_balance_backward(const void *logits, int32_t dtype, int64_t N, int32_t E, int64_t ld,
                                                  const uint8_t *mask, const int64_t *d_offs, int32_t G, int32_t score,
                                                  int32_t K, float coeff, const int32_t *counts, const int32_t *tokens,
                                                  const float *dloss, void *dlogits, int64_t ld_d, int32_t accumulate,
                                                  void *stream) {
    if ((dtype != DGR_DTYPE_BF16 && dtype != DGR_DTYPE_F32) || score < 0 || score > 1) return DGR_ERR_INVALID_ARG;
    if (N < 0 || E < 1 || K < 1 || G < 1 || ld < E || ld_d < E || (!d_offs && G != 1)) return DGR_ERR_INVALID_ARG;
    if (!counts || !tokens || (N > 0 && (!logits || !dlogits))) return DGR_ERR_INVALID_ARG;
    if (N > INT32_MAX || E > kMaxExperts || K > kMaxExperts || G > kMaxGroups) return DGR_ERR_UNSUPPORTED;
    const int es = dtype == DGR_DTYPE_BF16 ? 2 : 4;
    if (!aligned(logits, es) || !aligned(dlogits, es) || !aligned(d_offs, 8) || !aligned(counts, 4) || !aligned(tokens, 4) || !aligned(dloss, 4))
        return DGR_ERR_MISALIGNED;
    const size_t bl = extent(N, E, ld, es), bd = extent(N, E, ld_d, es);
    if (ranges_overlap(dlogits, bd, logits, bl) || ranges_overlap(dlogits, bd, mask, N) || ranges_overlap(dlogits, bd, d_offs, (G + 1) * 8) ||
        ranges_overlap(dlogits, bd, counts, static_cast<size_t>(G) * E * 4) || ranges_overlap(dlogits, bd, tokens, G * 4) ||
        ranges_overlap(dlogits, bd, dloss, 4))
        return DGR_ERR_ALIAS;
    dgr_status st = check_device();
    if (st != DGR_OK || N == 0) return st;
    BalParams p{};
    p.logits = logits, p.ld = ld, p.mask = mask, p.offs = d_offs;
    p.N = static_cast<int32_t>(N), p.E = E, p.K = K, p.G = G, p.sigmoid = score;
    p.coef = static_cast<float>(static_cast<double>(coeff) * E / (static_cast<double>(G) * K));
    p.counts = const_cast<int32_t *>(counts), p.tokens = const_cast<int32_t *>(tokens), p.dloss = dloss;
    p.dlogits = dlogits, p.ld_d = ld_d, p.accumulate = accumulate ? 1 : 0;
    const uint32_t tiles = static_cast<uint32_t>((N + kBackTile - 1) / kBackTile);
    p.sched = sched_for(tiles);
    const unsigned most = 152 * 16;
    const unsigned grid = sched_grid(tiles < most ? tiles : most);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return es == 2 ? launch_type<bf16>(true, p, grid, s) : launch_type<float>(true, p, grid, s);
}
