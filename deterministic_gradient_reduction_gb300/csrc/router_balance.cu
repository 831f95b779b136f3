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
// maximum and sum cost log2(E / 16) shuffles for several rows at a time. A lane
// keeps the running sums of its own experts' probabilities over the tile, which
// lanes, then warps, then tiles add in ascending order. The counts are integer
// sums (shared-memory integer atomics: any order, the same value). The CTA that
// finishes a group last folds the group's tiles, and the one that finishes the
// last group adds the groups.
//
// Measured on one GB300: forward 65536 x 128 fp32 (35.7 MB) 15.2 us, of which
// the last CTA's ticket and fold are about a third; backward 65536 x 128 bf16
// (33.6 MB) 10.2 us, bound by latency (issue 46 to 54 %, DRAM 17 to 21 %, 36 % of
// the warps resident).
#include "row_common.cuh"

namespace dgr {
namespace {

using namespace row;

// Forward threads: 1024 while a lane holds up to 16 logits (64 registers a thread), 512 beyond.
template <int EL>
constexpr int kThreadsFor = EL <= 16 ? 1024 : 512;
constexpr int kBackThreads = 256;
constexpr int kMaxExperts = 1024;
constexpr int kMaxGroups = 1024;
constexpr int kMaxTile = 16384;  // tokens: a lane's running sums stay short

// x log2(e) - fl(m log2(e)) carries the rounding of the product, up to half a
// unit of its size: 1/4 below this maximum, where it cancels between an
// exponential and its row's sum; at 1e10 it is in the hundreds, and ex2 would
// give infinity or 0. Beyond, the maximum is subtracted before scaling.
constexpr float kFarLogit = 4194304.0f;

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

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v, int lanes) {
    if constexpr (LANES > 0) {
#pragma unroll
        for (int s = 1; s < LANES; s <<= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, s));
    } else {
        for (int s = 1; s < lanes; s <<= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, s));
    }
    return v;
}

template <int LANES>
__device__ __forceinline__ float lanes_max(float v, int lanes) {
    if constexpr (LANES > 0) {
#pragma unroll
        for (int s = 1; s < LANES; s <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, s));
    } else {
        for (int s = 1; s < lanes; s <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, s));
    }
    return v;
}

// The row's probabilities in place of its logits (-inf where a lane has no
// expert); 0 for a row that is not live, whose logits must be finite, and for
// a row of -inf only. A NaN logit makes the row NaN, and so does a +inf in the
// softmax, as the formula does; a +inf's sigmoid is 1.
template <int E, int LANES, bool SIGMOID>
__device__ __forceinline__ void scores(float (&x)[E], int lanes, bool live) {
    float m = x[0];
#pragma unroll
    for (int e = 1; e < E; ++e) m = fmaxf(m, x[e]);
    m = lanes_max<LANES>(m, lanes);
    const bool empty = m == -INFINITY;
    if constexpr (!SIGMOID) {
        if (fabsf(m) > kFarLogit && !empty) {
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = __fadd_rn(x[e], -m);
            m = 0.0f;
        }
        vec_fma(x, kLog2e, empty ? 0.0f : -__fmul_rn(m, kLog2e));
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = ex2(x[e]);
    } else {
        // all logits below 0: each sigmoid divided by exp(m), so that rows far
        // below 0 keep their shares
        const bool low = m < 0.0f && !empty;
        const float c = low ? m : 0.0f, k = low ? kLog2e : -kLog2e;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float a = low ? ex2(__fmul_rn(__fadd_rn(x[e], -c), kLog2e)) : 1.0f;
            x[e] = __fdividef(a, __fadd_rn(1.0f, ex2(__fmul_rn(x[e], k))));
        }
    }
    const float s = lanes_sum<LANES>(vec_sum(x), lanes);
    vec_scale(x, live && s != 0.0f ? 1.0f / s : 0.0f);
}

// A lane's experts: vector i of NV starts at expert (i * lanes + sub) * VEC.
// LANES > 0: that many lanes a row, and their vectors cover exactly the E
// experts; LANES = 0: as many as the launch says, which may hold more. Rows
// that are not live are not read (zeros).
template <typename T, int VEC, int NV, int LANES>
__device__ __forceinline__ void load_raw(raw_t<T, VEC> (&v)[NV], const T *row, int sub, int lanes, int E, bool live) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = (i * lanes + sub) * VEC;
        v[i] = raw_t<T, VEC>{};
        load_if<true>(v[i], row + e, live && (LANES > 0 || e < E));
    }
}

template <typename T, int VEC, int NV, int LANES>
__device__ __forceinline__ void to_logits(float (&x)[NV * VEC], const raw_t<T, VEC> (&v)[NV], int sub, int lanes, int E) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        unpack<T, VEC>(v[i], x + i * VEC);
        if (LANES == 0 && (i * lanes + sub) * VEC >= E)
#pragma unroll
            for (int j = 0; j < VEC; ++j) x[i * VEC + j] = -INFINITY;
    }
}

// tbase[g] = first tile of group g, offsets into so[], the groups with tiles;
// false when the offsets break their contract. Every block computes the same.
template <int kThreads>
__device__ bool group_tiles(const BalParams &p, int32_t *tbase, int64_t *so, int32_t *wsum, int32_t *n_groups) {
    constexpr int kWarps = kThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    if (!p.offs) {
        if (tid == 0) {
            so[0] = 0, so[1] = p.N;
            tbase[0] = 0, tbase[1] = (p.N + p.tile - 1) / p.tile;
            *n_groups = 1;
        }
        __syncthreads();
        return true;
    }
    bool broken = false;
    int32_t run = 0, filled = 0;
    for (int g0 = 0; g0 < p.G; g0 += kThreads) {
        const int g = g0 + tid;
        int32_t c = 0;
        if (g < p.G) {
            const int64_t a = p.offs[g], b = p.offs[g + 1];
            so[g] = a;
            if (g == p.G - 1) so[p.G] = b;
            if (b < a || a < 0 || b > p.N || (g == 0 && a != 0) || (g == p.G - 1 && b != p.N)) broken = true;
            else c = static_cast<int32_t>((b - a + p.tile - 1) / p.tile);
        }
        int32_t incl = c;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const int32_t o = __shfl_up_sync(0xffffffffu, incl, s);
            if (lane >= s) incl += o;
        }
        if (lane == 31) wsum[w] = incl;
        filled += __syncthreads_count(c > 0);
        const int32_t v = lane < kWarps ? wsum[lane] : 0;
        if (g < p.G) tbase[g] = run + incl - c;
        const int32_t before = __reduce_add_sync(0xffffffffu, lane < w ? v : 0);
        if (g < p.G) tbase[g] += before;
        run += __reduce_add_sync(0xffffffffu, v);
        if (g0 + kThreads < p.G) __syncthreads();  // all have read wsum before the next round writes it
    }
    if (tid == 0) tbase[p.G] = run, *n_groups = filled;
    return !__syncthreads_or(broken);
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

// The fold's shape: threads that add one expert's ways, and a way's distance in
// shared memory, such that neighbouring helpers meet different banks.
struct FoldShape {
    int ways, helpers, stride;
};
template <int CV>
__host__ __device__ inline FoldShape fold_shape(int E, int threads) {
    int span = 1;
    while (span < E / CV && span < threads) span <<= 1;
    FoldShape f{threads / span, threads / span / CV, 0};
    f.helpers = f.helpers < 1 ? 1 : f.helpers > 32 ? 32 : f.helpers;
    f.stride = span + 32 / f.helpers;
    return f;
}

// Adds a group's tiles, CV experts a thread: `ways` threads share an expert's
// tiles (way w takes w, w + ways, ... in ascending order, up to 8 of them in
// flight), then neighbouring threads add the ways in a fixed order. Writes the
// group's counts; returns this thread's part of their dot product with the
// probabilities.
template <int CV, int kThreads>
__device__ float fold_tiles(const BalParams &p, int first, int n, int g, float *buf) {
    constexpr int kFlight = CV == 4 ? 4 : 8;
    const int tid = threadIdx.x, n_col = p.E / CV;
    int span = 1;
    while (span < n_col && span < kThreads) span <<= 1;
    const int ways = kThreads / span, way = tid / span;
    const FoldShape f = fold_shape<CV>(p.E, kThreads);
    const int log_span = __ffs(span) - 1, log_help = __ffs(f.helpers) - 1, plane = ways * f.stride;
    float dot = 0.0f;
    int32_t *ibuf = reinterpret_cast<int32_t *>(buf) + CV * plane;
    for (int c0 = 0; c0 < n_col; c0 += span) {
        const int col = c0 + (tid & (span - 1));
        float m[CV];
        int32_t c[CV];
#pragma unroll
        for (int j = 0; j < CV; ++j) m[j] = 0.0f, c[j] = 0;
        for (int t0 = way; t0 < n; t0 += kFlight * ways) {
            uint4 v[kFlight], k[kFlight];
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                const int t = t0 + i * ways;
                v[i] = k[i] = make_uint4(0, 0, 0, 0);
                const bool on = t < n && col < n_col;
                const int64_t at = static_cast<int64_t>(first + t) * p.E + col * CV;
                if constexpr (CV == 4) {  // written by other CTAs of this launch, never read before: no stale line in L1
                    load_if<false>(v[i], p.mass + at, on);
                    load_if<false>(k[i], p.part + at, on);
                } else {
                    load_if<false>(v[i].x, p.mass + at, on);
                    load_if<false>(k[i].x, p.part + at, on);
                }
            }
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                const uint32_t vw[4] = {v[i].x, v[i].y, v[i].z, v[i].w}, kw[4] = {k[i].x, k[i].y, k[i].z, k[i].w};
#pragma unroll
                for (int j = 0; j < CV; ++j) m[j] = __fadd_rn(m[j], __uint_as_float(vw[j])), c[j] += kw[j];
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < CV; ++j) {
            buf[j * plane + way * f.stride + (tid & (span - 1))] = m[j];
            ibuf[j * plane + way * f.stride + (tid & (span - 1))] = c[j];
        }
        __syncthreads();
        // `helpers` neighbouring threads an expert (whole warps go round together)
        const int n_out = span * CV * f.helpers;
        for (int i = tid; i < ((n_out + 31) & ~31); i += kThreads) {
            const int h = i & (f.helpers - 1), e = i >> log_help, j = e >> log_span, k0 = e & (span - 1);
            float v = 0.0f;
            int32_t k = 0;
            if (i < n_out)
#pragma unroll 4
                for (int q = h; q < ways; q += f.helpers) {
                    v = __fadd_rn(v, buf[j * plane + q * f.stride + k0]);
                    k += ibuf[j * plane + q * f.stride + k0];
                }
            for (int s = 1; s < f.helpers; s <<= 1) {
                v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, s));
                k += __shfl_xor_sync(0xffffffffu, k, s);
            }
            if (h == 0 && i < n_out && c0 + k0 < n_col) {
                p.counts[static_cast<int64_t>(g) * p.E + (c0 + k0) * CV + j] = k;
                dot = __fmaf_rn(static_cast<float>(k), v, dot);
            }
        }
    }
    return dot;
}

// Adds EL columns over the row groups of a warp (LANES lanes a row): at each
// step a lane hands half of its columns to its partner and adds the other half,
// then put(column, sum) for those that it is left with.
template <int EL, int LANES, int VEC, int S = 16, typename Put>
__device__ __forceinline__ void scatter_columns(const float (&acc)[EL], int lane, Put put, int first = 0) {
    if constexpr (S < LANES) {
#pragma unroll
        for (int e = 0; e < EL; ++e) put(first + e, acc[e]);
    } else if constexpr (EL == 1) {
        const float v[1] = {__fadd_rn(acc[0], __shfl_xor_sync(0xffffffffu, acc[0], S))};
        scatter_columns<1, LANES, VEC, S / 2>(v, lane, put, first);  // both lanes hold it
    } else {
        const bool up = (lane & S) != 0;
        float half[EL / 2];
#pragma unroll
        for (int e = 0; e < EL / 2; ++e) {
            const float give = up ? acc[e] : acc[e + EL / 2], keep = up ? acc[e + EL / 2] : acc[e];
            half[e] = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, give, S));
        }
        scatter_columns<EL / 2, LANES, VEC, S / 2>(half, lane, put, first + (up ? EL / 2 : 0));
    }
}

template <typename T, int VEC, int NV, int LANES, bool SIGMOID>
__global__ void __launch_bounds__(kThreadsFor<NV * VEC>) balance_forward(const BalParams p) {
    constexpr int kThreads = kThreadsFor<NV * VEC>, kWarps = kThreads / 32;
    extern __shared__ char smem[];
    int64_t *so = reinterpret_cast<int64_t *>(smem);                        // [G + 1]
    int32_t *tbase = reinterpret_cast<int32_t *>(so + p.G + 1);             // [G + 1]
    int32_t *hist = tbase + p.G + 1;                                        // [E]
    float *cols = reinterpret_cast<float *>(hist + p.E);                    // [kWarps][stride], later the fold's
    __shared__ int32_t wsum[kWarps], valid, last, n_groups;
    __shared__ float red[32];
    constexpr int EL = NV * VEC;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    if (!group_tiles<kThreads>(p, tbase, so, wsum, &n_groups)) {
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
    const int lanes = LANES > 0 ? LANES : p.lanes;
    const int sub = lane & (lanes - 1), rows_warp = 32 / lanes, my_row = lane / lanes;
    int helpers = 32;
    while (helpers > 1 && p.E * helpers > kThreads) helpers >>= 1;
    const int log_help = __ffs(helpers) - 1;
    const int stride = p.E + (32 >> log_help);  // of a warp's columns: its helpers meet different banks
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
        raw_t<T, VEC> v[NV];
        bool live = is_live(w * rows_warp + my_row);
        load_raw<T, VEC, NV, LANES>(v, base + static_cast<int64_t>(w * rows_warp + my_row) * p.ld, sub, lanes, p.E, live);
        const int n_ids = count * p.K;
        for (int i0 = tid; i0 < n_ids; i0 += 4 * kThreads) {
            int32_t id[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = i0 + j * kThreads;
                const int r = static_cast<int>((static_cast<uint64_t>(i) * p.k_magic) >> 40);
                uint32_t got = 0xffffffffu;
                load_if<true>(got, p.ids + (t0 + r) * p.ld_ids + (i - r * p.K), i < n_ids && (!p.mask || p.mask[t0 + r]));
                id[j] = static_cast<int32_t>(got);
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
            float x[EL];
            to_logits<T, VEC, NV, LANES>(x, v, sub, lanes, p.E);
            const bool was = live;
            const int r = b + kWarps * rows_warp + my_row;
            live = is_live(r);
            load_raw<T, VEC, NV, LANES>(v, base + static_cast<int64_t>(r) * p.ld, sub, lanes, p.E, live);
            scores<EL, LANES, SIGMOID>(x, lanes, was);
            vec_add(acc, x);
        }
        // rows side by side in the warp: halves of the columns are exchanged, so
        // that each lane ends with its share of them; without known lanes every
        // lane adds all
        float *mine = cols + w * stride;
        if constexpr (LANES > 0) {
            scatter_columns<EL, LANES, VEC>(acc, lane, [&](int k, float v) {
                mine[((k / VEC) * LANES + sub) * VEC + k % VEC] = v;
            });
        } else {
            for (int s = lanes; s < 32; s <<= 1)
#pragma unroll
                for (int e = 0; e < EL; ++e) acc[e] = __fadd_rn(acc[e], __shfl_xor_sync(0xffffffffu, acc[e], s));
            if (lane < lanes) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const int e = (i * lanes + sub) * VEC + j;
                        if (e < p.E) mine[e] = acc[i * VEC + j];
                    }
            }
        }
        __syncthreads();
        const int first = tbase[g], n = tbase[g + 1] - first;
        float dot = 0.0f;
        // `helpers` neighbouring threads add a column's warps
        for (int i = tid; i < ((p.E * helpers + 31) & ~31); i += kThreads) {
            const int e = i >> log_help, h = i & (helpers - 1);
            float v = 0.0f;
            if (e < p.E)
#pragma unroll 4
                for (int k = h; k < kWarps; k += helpers) v = __fadd_rn(v, cols[k * stride + e]);
            for (int s = 1; s < helpers; s <<= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, s));
            if (h != 0 || e >= p.E) continue;
            if (n == 1) {  // the group's only tile
                p.counts[static_cast<int64_t>(g) * p.E + e] = hist[e];
                dot = __fmaf_rn(static_cast<float>(hist[e]), v, dot);
            } else {
                p.mass[static_cast<int64_t>(tile) * p.E + e] = v;
                p.part[static_cast<int64_t>(tile) * p.E + e] = hist[e];
            }
        }
        if (n > 1) {
            if (tid == 0) p.live[tile] = valid;
            __syncthreads();
            if (tid == 0) {  // the block's writes before the ticket, the others' before what is read after it
                __threadfence();
                last = atomicAdd(&p.done[g], 1) == n - 1;
                __threadfence();
                valid = 0;
            }
            __syncthreads();
            if (!last) continue;
            // this group's tiles are all in: fold them
            int32_t tokens = 0;
            for (int j = tid; j < n; j += kThreads) tokens += __ldcg(p.live + first + j);
            dot = p.E % 4 == 0 ? fold_tiles<4, kThreads>(p, first, n, g, cols) : fold_tiles<1, kThreads>(p, first, n, g, cols);
            tokens = __reduce_add_sync(0xffffffffu, tokens);
            if (lane == 0 && tokens) atomicAdd(&valid, tokens);
        }
        float s[1] = {dot};
        block_sum<1>(s, red, kWarps);
        if (tid == 0) {
            const float nt = static_cast<float>(max(valid, 1));
            const float loss = p.coef * s[0] / (nt * nt);
            p.tokens[g] = valid;
            if (n > 1) p.done[g] = 0;  // ready for the next call
            if (n_groups == 1) {
                *p.loss = loss;
                last = 0;
            } else {
                p.group_loss[g] = loss;
                __threadfence();
                last = atomicAdd(&p.hdr->pad[0], 1) == n_groups - 1;
                __threadfence();
            }
        }
        __syncthreads();
        if (!last) continue;
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

// A warp takes rows_warp consecutive rows at a time; the next ones are on
// their way while it works. Rows are independent: no order to keep.
template <typename T, int VEC, int NV, int LANES, bool SIGMOID>
__global__ void __launch_bounds__(kBackThreads) balance_backward(const BalParams p) {
    extern __shared__ char smem[];
    int64_t *so = reinterpret_cast<int64_t *>(smem);  // [G + 1] when there are offsets
    constexpr int EL = NV * VEC, kBackWarps = kBackThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31;
    if (p.offs) {
        for (int g = tid; g <= p.G; g += kBackThreads) so[g] = p.offs[g];
        __syncthreads();
    }
    const int lanes = LANES > 0 ? LANES : p.lanes;
    const int sub = lane & (lanes - 1), rows_warp = 32 / lanes, my_row = lane / lanes;
    const float up = p.dloss ? __fmul_rn(__ldg(p.dloss), p.coef) : p.coef;
    // offsets outside their contract leave tokens without a group: no gradient
    auto is_live = [&](int64_t t) {
        return t < p.N && (!p.mask || p.mask[t]) && (!p.offs || (t >= so[0] && t < so[p.G]));
    };
    const T *logits = static_cast<const T *>(p.logits);
    uint32_t item = blockIdx.x * kBackWarps + (tid >> 5);
    const uint32_t n_items = p.sched.n, step = gridDim.x * kBackWarps;
    if (item >= n_items) return;
    auto row_of = [&](uint32_t i) { return static_cast<int64_t>(sched_item(p.sched, i)) * rows_warp + my_row; };
    int have = -1;
    float a[EL];  // the group's counts times its factor
#pragma unroll
    for (int e = 0; e < EL; ++e) a[e] = 0.0f;
    raw_t<T, VEC> v[NV], next[NV];
    int64_t t = row_of(item);
    bool live = is_live(t);
    load_raw<T, VEC, NV, LANES>(v, logits + t * p.ld, sub, lanes, p.E, live);
    for (;;) {
        const bool more = item + step < n_items;
        int64_t t_next = 0;
        bool live_next = false;
        if (more) {
            t_next = row_of(item + step);
            live_next = is_live(t_next);
            load_raw<T, VEC, NV, LANES>(next, logits + t_next * p.ld, sub, lanes, p.E, live_next);
        }
        const int g = live && p.offs ? group_of(so, p.G, t) : 0;
        if (live && g != have) {
            have = g;
            const float nt = static_cast<float>(max(__ldg(p.tokens + g), 1));
            const float f = up / (nt * nt);
            const int32_t *counts = p.counts + static_cast<int64_t>(g) * p.E;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const int e = (i * lanes + sub) * VEC + j;
                    a[i * VEC + j] = LANES > 0 || e < p.E ? __fmul_rn(f, static_cast<float>(__ldg(counts + e))) : 0.0f;
                }
        }
        float q[EL];
        to_logits<T, VEC, NV, LANES>(q, v, sub, lanes, p.E);
        scores<EL, LANES, SIGMOID>(q, lanes, live);
        const float inner = lanes_sum<LANES>(vec_dot(a, q), lanes);
        if (t < p.N) {
            T *dst = static_cast<T *>(p.dlogits) + t * p.ld_d;
            auto gradient = [&](int i, float *d) {
                float x[VEC];
                if (SIGMOID) unpack<T, VEC>(v[i], x);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    d[j] = __fmul_rn(q[i * VEC + j], __fadd_rn(a[i * VEC + j], -inner));  // 0 where not live: q is
                    if (SIGMOID) d[j] = __fdividef(d[j], __fadd_rn(1.0f, ex2(__fmul_rn(x[j], kLog2e))));
                }
            };
            if (!p.accumulate) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int e = (i * lanes + sub) * VEC;
                    if (LANES == 0 && e >= p.E) continue;
                    float d[VEC];
                    gradient(i, d);
                    *reinterpret_cast<raw_t<T, VEC> *>(dst + e) = pack<T, VEC>(d);
                }
            } else if (live) {  // a loop of its own, so that the common one is not slowed by it
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int e = (i * lanes + sub) * VEC;
                    if (LANES == 0 && e >= p.E) continue;
                    float d[VEC], old[VEC];
                    gradient(i, d);
                    raw_t<T, VEC> *to = reinterpret_cast<raw_t<T, VEC> *>(dst + e);
                    unpack<T, VEC>(*to, old);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) d[j] = __fadd_rn(old[j], d[j]);
                    *to = pack<T, VEC>(d);
                }
            }
        }
        if (!more) break;
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = next[i];
        t = t_next;
        live = live_next;
        item += step;
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

// The counters come first and have room for the most groups, so that they lie
// at the same place whatever the sizes: what one call leaves in its sums is never
// another's counter, and a workspace serves calls of any sizes that fit it.
BalLayout balance_layout(int64_t N, int64_t E, int64_t G) {
    BalLayout L{};
    const int64_t tile = balance_tile(N, E);
    L.tiles = (N + tile - 1) / tile + (G > 1 ? G : 0);
    L.done = sizeof(WsHeader);
    L.group_loss = L.done + align_up(static_cast<size_t>(kMaxGroups) * 4);
    L.mass = L.group_loss + align_up(static_cast<size_t>(G) * 4);
    L.part = L.mass + align_up(static_cast<size_t>(L.tiles) * E * 4);
    L.live = L.part + align_up(static_cast<size_t>(L.tiles) * E * 4);
    L.total = L.live + align_up(static_cast<size_t>(L.tiles) * 4);
    return L;
}

// The forward kernel asks for at most 83,980 bytes (1024 experts and 1024
// groups, of which the warps' columns are 67,584).
constexpr size_t kMostSmem = 84 * 1024;

size_t fold_bytes(int E, int threads) {
    const FoldShape f = E % 4 == 0 ? fold_shape<4>(E, threads) : fold_shape<1>(E, threads);
    return static_cast<size_t>(E % 4 == 0 ? 4 : 1) * f.ways * f.stride * 8;
}

template <typename T, int VEC, int NV, int LANES, bool SIGMOID>
dgr_status launch_one(bool backward, BalParams &p, unsigned grid, cudaStream_t s) {
    if (backward) {
        const int64_t rows_warp = 32 / p.lanes;
        p.sched = sched_for(static_cast<uint32_t>((p.N + rows_warp - 1) / rows_warp));
        // one wave: what a warp sets up (the counts) serves all its rows
        const unsigned want = (p.sched.n + kBackThreads / 32 - 1) / (kBackThreads / 32), most = 152 * 3;
        balance_backward<T, VEC, NV, LANES, SIGMOID><<<sched_grid(want < most ? want : most), kBackThreads, p.offs ? (p.G + 1) * 8 : 0, s>>>(p);
    } else {
        constexpr int threads = kThreadsFor<NV * VEC>;
        const size_t cols = static_cast<size_t>(threads / 32) * (p.E + 32) * 4, fold = fold_bytes(p.E, threads);  // the fold takes the columns' place
        const size_t smem = (p.G + 1) * 12 + p.E * 4 + (cols > fold ? cols : fold);
        auto *k = balance_forward<T, VEC, NV, LANES, SIGMOID>;
        const dgr_status st = allow_smem(k, smem, kMostSmem);
        if (st != DGR_OK) return st;
        k<<<grid, threads, smem, s>>>(p);
    }
    return launch_status();
}

template <typename T, int VEC, int NV, int LANES>
dgr_status launch_score(bool backward, BalParams &p, unsigned grid, cudaStream_t s) {
    return p.sigmoid ? launch_one<T, VEC, NV, LANES, true>(backward, p, grid, s) : launch_one<T, VEC, NV, LANES, false>(backward, p, grid, s);
}

// 16 logits a lane (fewer lanes, fewer shuffles) until a row takes the whole
// warp. Expert counts that fill their lanes have kernels of their own: with the
// lanes known the 65536 x 128 backward runs 7.1 million warp instructions
// instead of 8.1 million.
template <typename T, int VEC>
dgr_status launch_vec(bool backward, BalParams &p, unsigned grid, cudaStream_t s) {
    const int n_vec = (p.E + VEC - 1) / VEC;
    p.lanes = 1;
    while (p.lanes < 32 && p.lanes * 16 < n_vec * VEC) p.lanes <<= 1;
    const int nv = (n_vec + p.lanes - 1) / p.lanes;
    if constexpr (VEC == 4) {
        switch (p.E) {
            case 8: return launch_score<T, VEC, 2, 1>(backward, p, grid, s);
            case 16: return launch_score<T, VEC, 4, 1>(backward, p, grid, s);
            case 32: return launch_score<T, VEC, 4, 2>(backward, p, grid, s);
            case 64: return launch_score<T, VEC, 4, 4>(backward, p, grid, s);
            case 128: return launch_score<T, VEC, 4, 8>(backward, p, grid, s);
            case 256: return launch_score<T, VEC, 4, 16>(backward, p, grid, s);
            case 512: return launch_score<T, VEC, 4, 32>(backward, p, grid, s);
            default: break;
        }
        if (nv <= 4) return launch_score<T, VEC, 4, 0>(backward, p, grid, s);
        return launch_score<T, VEC, 8, 0>(backward, p, grid, s);
    } else {
        if (nv <= 16) return launch_score<T, VEC, 16, 0>(backward, p, grid, s);
        return launch_score<T, VEC, 32, 0>(backward, p, grid, s);
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
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return es == 2 ? launch_type<bf16>(true, p, 0, s) : launch_type<float>(true, p, 0, s);
}
