// Norm of queries and keys a head, and their rotation by position, in one pass,
// forward and backward.
//
// For every head v [D] of a token at position t:
//   r = (mean(v^2) + eps)^(-1/2),  n = v r w,
//   (y_lo, y_hi) = (n_lo c - n_hi s, n_hi c + n_lo s) for each of the R / 2 pairs,
// c and s the table's cosine and sine of the pair's angle at t; the elements
// behind R stay. Pairs are (i, i + R/2) or, interleaved, (2i, 2i + 1).
// Backwards, from dy: g = dy turned back (s -> -s),
//   dw = sum over tokens and heads of g v r,
//   dv = r (g w) - (v r) (r (r (g w . v) / D)): no factor is larger than what comes
//        of it, so that heads close to 0, whose r^2 or r^3 is out of range, have theirs.
// All in binary32 from the stored heads; every output rounded once.
//
// A team of lanes has a head: lane l of it V pairs (the same places of the lower
// and the upper half, so a rotation stays in the lane) and NV such groups; a
// warp has several teams, which share a token, so that its cosines and sines are
// read once for all of the token's heads.
//
// Bound by memory, each head read and written once: 16384 tokens of 32 + 8 heads of
// 128 bf16 forward 58 us (5.9 TB/s, 0.87 of the measured copy rate), backward 91 us
// (5.6 TB/s, 0.83; 344 instructions a warp and group of heads, half of the issue
// slots, and 128 registers, so 16 warps on an SM). Few tokens: the launches, 3 us
// forward and, with the fold, 7 backward; 3001 x (12 + 4) x 80 fp32 backward 26 us
// in a graph too: the device's, not the host's.
//
// Deterministic: a head's sums go over its team in a fixed order; dw goes through
// a number of slots set by the sizes alone: a slot's warps take their units in
// ascending order, its warps and teams are added in order, and a second launch
// adds the slots in a fixed tree.
#include "row_common.cuh"

namespace dgr {
namespace {

using namespace row;

constexpr int kWarps = 8;
constexpr int kMaxDim = 512;
constexpr int kMaxHeads = 1024;
constexpr int kSlots = 304;     // CTAs of the backward pass at most, two an SM
constexpr int kFoldCols = 8, kFoldWays = 32;
constexpr int kWherePos = 420;

// Heads of one kind (queries or keys): element (t, head, d) at t * st + head * sh + d.
struct Heads {
    const void *v, *dy;
    void *out;  // forward: y; backward: dv
    int64_t st, sh, st_dy, sh_dy, st_out, sh_out;
    int32_t n;
    const void *w;
    float *dw;
};

struct QkParams {
    Heads kind[2];
    int32_t T, D, R, w_bf16, P;
    const float *cos, *sin;    // [P, R/2]
    const int32_t *pos;
    float eps;
    int32_t team, chunks;      // lanes a head; warps a token
    // slots of dw_q and of dw_k; turns: what CTAs take, one slot of each, or (split) one
    int32_t count[2], turns, split, accumulate;
    float *slots;              // [count[0] + count[1], D]
    WsHeader *hdr;
    Sched sched;
};

// Where this lane's pairs lie: group i of it starts at pair b = (i * team + tl) * V.
template <int V, int NV, bool INTER>
struct Pairs {
    int lo[NV], hi[NV];  // element offsets of the first of V; interleaved: of 2 V neighbours, in two vectors
    int at[NV];          // pair
    bool has[NV];
    __device__ __forceinline__ Pairs(const QkParams &p, int tl) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int b = (i * p.team + tl) * V;
            has[i] = b < p.D / 2;
            at[i] = b;
            if (INTER) {
                lo[i] = 2 * b, hi[i] = 2 * b + V;
            } else if (b < p.R / 2) {
                lo[i] = b, hi[i] = b + p.R / 2;
            } else {
                lo[i] = p.R / 2 + b, hi[i] = p.D / 2 + b;
            }
        }
    }
};

// The first and second elements of V pairs out of their two vectors, and back.
template <typename T, int V, bool INTER>
__device__ __forceinline__ void split(const raw_t<T, V> &x, const raw_t<T, V> &y, float (&a)[V], float (&b)[V]) {
    if constexpr (!INTER) {
        unpack<T, V>(x, a);
        unpack<T, V>(y, b);
    } else {
        float f[2 * V];
        unpack<T, V>(x, f);
        unpack<T, V>(y, f + V);
#pragma unroll
        for (int j = 0; j < V; ++j) a[j] = f[2 * j], b[j] = f[2 * j + 1];
    }
}
template <typename T, int V, bool INTER>
__device__ __forceinline__ void join(const float (&a)[V], const float (&b)[V], raw_t<T, V> &x, raw_t<T, V> &y) {
    if constexpr (!INTER) {
        x = pack<T, V>(a);
        y = pack<T, V>(b);
    } else {
        float f[2 * V];
#pragma unroll
        for (int j = 0; j < V; ++j) f[2 * j] = a[j], f[2 * j + 1] = b[j];
        x = pack<T, V>(f);
        y = pack<T, V>(f + V);
    }
}

__device__ __forceinline__ float team_sum(float v, int team) {
    for (int s = team >> 1; s > 0; s >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, s));
    return v;
}

// Cosines and sines of the lane's pairs at a position (1 and 0 behind R).
template <int V, int NV, bool INTER>
__device__ __forceinline__ void angles(const QkParams &p, const Pairs<V, NV, INTER> &m, int32_t pos, float (&c)[NV][V], float (&s)[NV][V]) {
    const int64_t row = static_cast<int64_t>(pos) * (p.R / 2);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const bool on = m.has[i] && m.at[i] < p.R / 2;
#pragma unroll
        for (int j = 0; j < V; ++j) c[i][j] = 1.0f, s[i][j] = 0.0f;
        if (!on) continue;
        if constexpr (V % 4 == 0) {
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                unpack<float, 4>(__ldg(reinterpret_cast<const uint4 *>(p.cos + row + m.at[i] + j)), &c[i][j]);
                unpack<float, 4>(__ldg(reinterpret_cast<const uint4 *>(p.sin + row + m.at[i] + j)), &s[i][j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) c[i][j] = __ldg(p.cos + row + m.at[i] + j), s[i][j] = __ldg(p.sin + row + m.at[i] + j);
        }
    }
}

// Both weights as binary32 into shared memory (1 where there is none), in the
// order of the pairs: first elements, then second ones.
template <bool INTER>
__device__ __forceinline__ void load_weights(const QkParams &p, float (*w)[kMaxDim]) {
    for (int i = threadIdx.x; i < 2 * p.D; i += kWarps * 32) {
        const int kind = i >= p.D, e = i - kind * p.D;
        const void *from = p.kind[kind].w;
        int pair, second;
        if (INTER) pair = e >> 1, second = e & 1;
        else if (e < p.R) second = e >= p.R / 2, pair = e - second * (p.R / 2);
        else second = e - p.R >= (p.D - p.R) / 2, pair = p.R / 2 + (e - p.R) - second * ((p.D - p.R) / 2);
        w[kind][second * (kMaxDim / 2) + pair] = from ? param(from, p.w_bf16, e) : 1.0f;
    }
    __syncthreads();
}

// V floats from a multiple of 4 on, out of shared memory.
template <int V>
__device__ __forceinline__ void four_by_four(const float *w, float *f) {
#pragma unroll
    for (int j = 0; j < V; j += 4) unpack<float, 4>(*reinterpret_cast<const uint4 *>(w + j), f + j);
}

template <int V, int NV, bool INTER>
__device__ __forceinline__ void lane_weights(const QkParams &p, const Pairs<V, NV, INTER> &m, const float *w, float (&a)[NV][V], float (&b)[NV][V]) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            a[i][j] = m.has[i] ? w[m.at[i] + j] : 0.0f;
            b[i][j] = m.has[i] ? w[kMaxDim / 2 + m.at[i] + j] : 0.0f;
        }
}

// The position of a token; outside the table it is recorded and false is returned.
__device__ __forceinline__ bool position(const QkParams &p, int64_t t, int32_t &pos) {
    pos = __ldg(p.pos + t);
    if (pos >= 0 && pos < p.P) return true;
    if ((threadIdx.x & 31) == 0) record_error(p.hdr, DGR_ERR_INVALID_ARG, kWherePos);
    return false;
}

template <typename T, int V, int NV, bool INTER, int U>
__global__ void __launch_bounds__(kWarps * 32) qk_forward(const QkParams p) {
    using raw = raw_t<T, V>;
    __shared__ __align__(16) float s_w[2][kMaxDim];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tl = lane & (p.team - 1), mine = lane / p.team, teams = 32 / p.team;
    const Pairs<V, NV, INTER> m(p, tl);
    load_weights<INTER>(p, s_w);
    const int64_t units = static_cast<int64_t>(p.T) * p.chunks;
    const float inv_d = 1.0f / static_cast<float>(p.D);
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + warp; u < units; u += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t i = sched_item(p.sched, static_cast<uint32_t>(u));
        const int64_t t = i / p.chunks;
        const int chunk = static_cast<int>(i - t * p.chunks);
        int32_t pos;
        const bool good = position(p, t, pos);
        float c[NV][V], s[NV][V];
        angles<V, NV, INTER>(p, m, good ? pos : 0, c, s);
        int first = chunk;  // this warp's first group of heads among the kind's
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
            const Heads &h = p.kind[kind];
            const int groups = (h.n + teams - 1) / teams;
            const T *v = static_cast<const T *>(h.v) + t * h.st;
            T *out = static_cast<T *>(h.out) + t * h.st_out;
            float wa[NV][V], wb[NV][V];
            if (first < groups) lane_weights<V, NV, INTER>(p, m, s_w[kind], wa, wb);
            for (int g0 = first; g0 < groups; g0 += U * p.chunks) {
                raw lo[U][NV] = {}, hi[U][NV] = {};
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int head = (g0 + k * p.chunks) * teams + mine;
#pragma unroll
                    for (int n = 0; n < NV; ++n) {
                        const bool on = head < h.n && m.has[n];
                        load_if<false>(lo[k][n], v + head * h.sh + m.lo[n], on);
                        load_if<false>(hi[k][n], v + head * h.sh + m.hi[n], on);
                    }
                }
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int head = (g0 + k * p.chunks) * teams + mine;
                    float a[NV][V], b[NV][V], ss = 0.0f;
#pragma unroll
                    for (int n = 0; n < NV; ++n) {
                        split<T, V, INTER>(lo[k][n], hi[k][n], a[n], b[n]);
                        ss = __fadd_rn(ss, __fadd_rn(vec_dot(a[n], a[n]), vec_dot(b[n], b[n])));
                    }
                    const float r = rsqrtf(__fmaf_rn(team_sum(ss, p.team), inv_d, p.eps));
#pragma unroll
                    for (int n = 0; n < NV; ++n) {
                        float x[V], y[V];
#pragma unroll
                        for (int j = 0; j < V; ++j) {
                            const float na = __fmul_rn(__fmul_rn(a[n][j], r), wa[n][j]), nb = __fmul_rn(__fmul_rn(b[n][j], r), wb[n][j]);
                            x[j] = good ? __fmaf_rn(na, c[n][j], -__fmul_rn(nb, s[n][j])) : 0.0f;
                            y[j] = good ? __fmaf_rn(nb, c[n][j], __fmul_rn(na, s[n][j])) : 0.0f;
                        }
                        raw rx, ry;
                        join<T, V, INTER>(x, y, rx, ry);
                        if (head < h.n && m.has[n]) {
                            *reinterpret_cast<raw *>(out + head * h.sh_out + m.lo[n]) = rx;
                            *reinterpret_cast<raw *>(out + head * h.sh_out + m.hi[n]) = ry;
                        }
                    }
                }
            }
            first = (first - groups % p.chunks + p.chunks) % p.chunks;  // groups go round the chunks, over both kinds
        }
    }
}

// The sums of a warp's lanes for dw: its teams, then the slot's warps, into the slot.
template <int V, int NV, bool INTER>
__device__ __forceinline__ void slot_sums(const QkParams &p, const Pairs<V, NV, INTER> &m, float (&acc_a)[NV][V], float (&acc_b)[NV][V], float *s_dw,
                                          int slot, int warp, int mine) {
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            for (int sh = p.team; sh < 32; sh <<= 1) {
                acc_a[n][j] = __fadd_rn(acc_a[n][j], __shfl_xor_sync(0xffffffffu, acc_a[n][j], sh));
                acc_b[n][j] = __fadd_rn(acc_b[n][j], __shfl_xor_sync(0xffffffffu, acc_b[n][j], sh));
            }
            if (mine == 0 && m.has[n]) {
                const int first = INTER ? 2 * (m.at[n] + j) : m.lo[n] + j, second = INTER ? first + 1 : m.hi[n] + j;
                s_dw[warp * p.D + first] = acc_a[n][j];
                s_dw[warp * p.D + second] = acc_b[n][j];
            }
        }
    __syncthreads();
    for (int d = threadIdx.x; d < p.D; d += kWarps * 32) {
        float v = s_dw[d];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) v = __fadd_rn(v, s_dw[w * p.D + d]);
        p.slots[static_cast<int64_t>(slot) * p.D + d] = v;
    }
    __syncthreads();
}

template <typename T, int V, int NV, bool INTER, int U>
__global__ void __launch_bounds__(kWarps * 32, 2) qk_backward(const QkParams p) {
    using raw = raw_t<T, V>;
    __shared__ __align__(16) float s_w[2][kMaxDim];
    __shared__ float s_dw[kWarps * kMaxDim];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tl = lane & (p.team - 1), mine = lane / p.team, teams = 32 / p.team;
    const Pairs<V, NV, INTER> m(p, tl);
    load_weights<INTER>(p, s_w);
    const int64_t units = static_cast<int64_t>(p.T) * p.chunks;
    const float inv_d = 1.0f / static_cast<float>(p.D);
    for (int i = blockIdx.x; i < p.turns; i += gridDim.x) {
        const int turn = static_cast<int>(sched_item(p.sched, static_cast<uint32_t>(i)));
#pragma unroll 1
        for (int kind = 0; kind < 2; ++kind) {
            const int mine_of = p.split && kind ? turn - p.count[0] : turn;  // which of the kind's slots
            if (mine_of < 0 || mine_of >= p.count[kind]) continue;
            const int slot_out = mine_of + (kind ? p.count[0] : 0);
            const Heads &h = p.kind[kind];
            const int groups = (h.n + teams - 1) / teams;
            float acc_a[NV][V] = {}, acc_b[NV][V] = {}, wa[NV][V], wb[NV][V];
            lane_weights<V, NV, INTER>(p, m, s_w[kind], wa, wb);
            for (int64_t u = static_cast<int64_t>(mine_of) * kWarps + warp; u < units; u += static_cast<int64_t>(p.count[kind]) * kWarps) {
                const int64_t t = u / p.chunks;
                const int first = static_cast<int>(u - t * p.chunks);
                if (first >= groups) continue;
                int32_t pos;
                const bool good = position(p, t, pos);
                float c[NV][V], s[NV][V];
                angles<V, NV, INTER>(p, m, good ? pos : 0, c, s);
                const T *v = static_cast<const T *>(h.v) + t * h.st;
                const T *dy = static_cast<const T *>(h.dy) + t * h.st_dy;
                T *out = static_cast<T *>(h.out) + t * h.st_out;
                for (int g0 = first; g0 < groups; g0 += U * p.chunks) {
                    raw lo[U][NV] = {}, hi[U][NV] = {}, dlo[U][NV] = {}, dhi[U][NV] = {};
#pragma unroll
                    for (int k = 0; k < U; ++k) {
                        const int head = (g0 + k * p.chunks) * teams + mine;
#pragma unroll
                        for (int n = 0; n < NV; ++n) {
                            const bool on = head < h.n && m.has[n] && good;
                            load_if<false>(lo[k][n], v + head * h.sh + m.lo[n], on);
                            load_if<false>(hi[k][n], v + head * h.sh + m.hi[n], on);
                            load_if<false>(dlo[k][n], dy + head * h.sh_dy + m.lo[n], on);
                            load_if<false>(dhi[k][n], dy + head * h.sh_dy + m.hi[n], on);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < U; ++k) {
                        const int head = (g0 + k * p.chunks) * teams + mine;
                        float a[NV][V], b[NV][V], ga[NV][V], gb[NV][V], ss = 0.0f, dot = 0.0f;
#pragma unroll
                        for (int n = 0; n < NV; ++n) {
                            float x[V], y[V];
                            split<T, V, INTER>(lo[k][n], hi[k][n], a[n], b[n]);
                            split<T, V, INTER>(dlo[k][n], dhi[k][n], x, y);
                            ss = __fadd_rn(ss, __fadd_rn(vec_dot(a[n], a[n]), vec_dot(b[n], b[n])));
#pragma unroll
                            for (int j = 0; j < V; ++j) {
                                ga[n][j] = __fmaf_rn(x[j], c[n][j], __fmul_rn(y[j], s[n][j]));
                                gb[n][j] = __fmaf_rn(y[j], c[n][j], -__fmul_rn(x[j], s[n][j]));
                                dot = __fmaf_rn(__fmul_rn(ga[n][j], wa[n][j]), a[n][j], dot);
                                dot = __fmaf_rn(__fmul_rn(gb[n][j], wb[n][j]), b[n][j], dot);
                            }
                        }
                        for (int sh = p.team >> 1; sh > 0; sh >>= 1) {
                            ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, sh));
                            dot = __fadd_rn(dot, __shfl_xor_sync(0xffffffffu, dot, sh));
                        }
                        // a place without a head, or a token without a position: nothing for dw
                        const bool on = head < h.n && good;
                        const float r = on ? rsqrtf(__fmaf_rn(ss, inv_d, p.eps)) : 0.0f;
                        const float back = on ? __fmul_rn(r, __fmul_rn(r, __fmul_rn(dot, inv_d))) : 0.0f;  // (times v r)
#pragma unroll
                        for (int n = 0; n < NV; ++n) {
                            float x[V], y[V];
#pragma unroll
                            for (int j = 0; j < V; ++j) {
                                const float na = __fmul_rn(a[n][j], r), nb = __fmul_rn(b[n][j], r);
                                acc_a[n][j] = __fmaf_rn(na, ga[n][j], acc_a[n][j]);
                                acc_b[n][j] = __fmaf_rn(nb, gb[n][j], acc_b[n][j]);
                                x[j] = __fmaf_rn(__fmul_rn(ga[n][j], wa[n][j]), r, -__fmul_rn(na, back));
                                y[j] = __fmaf_rn(__fmul_rn(gb[n][j], wb[n][j]), r, -__fmul_rn(nb, back));
                            }
                            raw rx, ry;
                            join<T, V, INTER>(x, y, rx, ry);
                            if (head < h.n && m.has[n]) {
                                *reinterpret_cast<raw *>(out + head * h.sh_out + m.lo[n]) = rx;
                                *reinterpret_cast<raw *>(out + head * h.sh_out + m.hi[n]) = ry;
                            }
                        }
                    }
                }
            }
            if (!h.dw) continue;
            slot_sums<V, NV, INTER>(p, m, acc_a, acc_b, s_dw, slot_out, warp, mine);
        }
    }
}

// ---- heads on their way in shared memory ----------------------------------------
//
// For heads in vectors of 16 bytes: each lane has the next DEPTH groups of heads of
// its warp on their way in shared memory (it reads what it fetched itself, so
// nothing has to meet for it), a unit's cosines and sines with its first group,
// the position one unit earlier still.

// The groups of heads that a warp takes, one after another: of its units (a token,
// or a part of a token's groups) those of the queries, then of the keys; or, with
// only >= 0, those of one kind. N addresses of the lane's head go along: of p's
// inputs, or of its output (one a group: the step from a group to the next is an
// addition each).
enum Along { kInputs, kInputAndGradient, kOutput };
template <typename T, Along WHAT>
struct Walk {
    static constexpr int N = WHAT == kInputAndGradient ? 2 : 1;
    const QkParams &p;
    int teams, mine, only;
    bool scheduled;
    int32_t u, stride, units, G0;
    int32_t t = 0;  // the unit's token
    int chunk = 0, kind = 0;
    int head = 0;   // the group's first
    int n = 0;      // heads of the kind
    T *at[N];
    int64_t step[N];
    __device__ __forceinline__ Walk(const QkParams &p_, int teams_, int mine_, int only_, bool scheduled_, int32_t u_, int32_t stride_)
        : p(p_), teams(teams_), mine(mine_), only(only_), scheduled(scheduled_), u(u_), stride(stride_), units(p_.T * p_.chunks) {
        G0 = (p.kind[0].n + teams - 1) / teams;
        enter();
    }
    __device__ __forceinline__ bool done() const { return u >= units; }
    __device__ __forceinline__ int32_t token(int32_t unit, int &part) const {
        const int32_t i = scheduled ? static_cast<int32_t>(sched_item(p.sched, static_cast<uint32_t>(unit))) : unit;
        part = 0;
        if (p.chunks == 1) return i;
        const int32_t to = i / p.chunks;
        part = i - to * p.chunks;
        return to;
    }
    // to the unit's first group of a kind, if it has one; a token's groups go round its units, over both kinds
    __device__ __forceinline__ bool begin(int k) {
        const Heads &h = p.kind[k];
        kind = k, n = h.n;
        head = (k == 0 || only >= 0 || p.chunks == 1 ? chunk : (chunk - G0 % p.chunks + p.chunks) % p.chunks) * teams;
        if (head >= n) return false;
        auto set = [&](int i, const void *base, int64_t st, int64_t sh) {
            at[i] = const_cast<T *>(static_cast<const T *>(base)) + t * st + (head + mine) * sh;
            step[i] = static_cast<int64_t>(p.chunks * teams) * sh;
        };
        if (WHAT == kOutput) set(0, h.out, h.st_out, h.sh_out);
        else set(0, h.v, h.st, h.sh);
        if (WHAT == kInputAndGradient) set(N - 1, h.dy, h.st_dy, h.sh_dy);
        return true;
    }
    __device__ __forceinline__ void enter() {
        for (; u < units; u += stride) {
            t = token(u, chunk);
            if (only <= 0 && begin(0)) return;
            if (only != 0 && begin(1)) return;
        }
    }
    __device__ __forceinline__ void next() {
        head += p.chunks * teams;
#pragma unroll
        for (int i = 0; i < N; ++i) at[i] += step[i];
        if (head < n) return;
        if (only < 0 && kind == 0 && begin(1)) return;
        u += stride;
        enter();
    }
    __device__ __forceinline__ bool has_head() const { return head + mine < n; }
};

// Shared memory by its 32-bit addresses.
__device__ __forceinline__ uint32_t shared_address(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ uint4 load_shared(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void copy_to(uint32_t a, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(a), "l"(src) : "memory");
}

// A warp's ring. Of a slot: PARTS vectors of each lane's group of heads and, with
// a unit's first group, its cosines and sines, fetched by one team for all, and
// whether its position lies in the table.
template <int V, int NV, bool INTER, int DEPTH, int PARTS>
struct Ring {
    static constexpr int kTurns = 2 * NV * V / 4;  // vectors of a lane's cosines and sines
    const QkParams &p;
    const Pairs<V, NV, INTER> &m;
    int tl, mine;
    uint32_t heads, turns;  // addresses
    int32_t *good_;
    float c[NV][V], s[NV][V];  // of the unit that is worked on
    bool good = false;
    int32_t in = -1, out = -1, pos_next = 0;  // units
    // bytes of all warps, behind `teams` lanes' worth of cosines and sines
    static size_t bytes(int team) { return static_cast<size_t>(kWarps) * DEPTH * (PARTS * 32 * 16 + kTurns * team * 16 + 16); }
    __device__ __forceinline__ Ring(const QkParams &p_, const Pairs<V, NV, INTER> &m_, uint4 *smem, int warp, int lane, int tl_, int mine_)
        : p(p_), m(m_), tl(tl_), mine(mine_) {
        heads = shared_address(smem + warp * DEPTH * PARTS * 32 + lane);
        smem += kWarps * DEPTH * PARTS * 32;
        turns = shared_address(smem + warp * DEPTH * kTurns * p.team + tl);
        smem += kWarps * DEPTH * kTurns * p.team;
        good_ = reinterpret_cast<int32_t *>(smem + warp * DEPTH);
    }
    __device__ __forceinline__ uint32_t at(int slot, int i) const { return heads + static_cast<uint32_t>(slot * PARTS + i) * 512u; }
    __device__ __forceinline__ uint32_t turn(int slot, int i) const { return turns + static_cast<uint32_t>((slot * kTurns + i) * p.team) * 16u; }
    // with a unit's first group
    template <typename W>
    __device__ __forceinline__ void put_angles(const W &w, int slot) {
        if (w.u == in) return;
        int part;
        const int32_t pos = in >= 0 && w.u - in == w.stride ? pos_next : __ldg(p.pos + w.t);
        in = w.u;
        pos_next = w.units - w.u > w.stride ? __ldg(p.pos + w.token(w.u + w.stride, part)) : 0;
        const bool ok = pos >= 0 && pos < p.P;
        if (mine == 0) {
            const int64_t row = static_cast<int64_t>(ok ? pos : 0) * (p.R / 2);
#pragma unroll
            for (int n = 0; n < NV; ++n)
                if (m.has[n] && m.at[n] < p.R / 2)
#pragma unroll
                    for (int j = 0; j < V; j += 4) {
                        copy_to(turn(slot, (n * V + j) / 2), p.cos + row + m.at[n] + j);
                        copy_to(turn(slot, (n * V + j) / 2 + 1), p.sin + row + m.at[n] + j);
                    }
            if (tl == 0) {
                good_[slot * 4] = ok;
                if (!ok) record_error(p.hdr, DGR_ERR_INVALID_ARG, kWherePos);
            }
        }
    }
    // when the slot's copies have come
    template <typename W>
    __device__ __forceinline__ void take_angles(const W &w, int slot) {
        if (w.u == out) return;
        out = w.u;
        __syncwarp();
        good = good_[slot * 4] != 0;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const bool turned = m.has[n] && m.at[n] < p.R / 2;
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                float x[4], y[4];
                unpack<float, 4>(load_shared(turn(slot, (n * V + j) / 2)), x);
                unpack<float, 4>(load_shared(turn(slot, (n * V + j) / 2 + 1)), y);
#pragma unroll
                for (int i = 0; i < 4; ++i) c[n][j + i] = turned ? x[i] : 1.0f, s[n][j + i] = turned ? y[i] : 0.0f;
            }
        }
        __syncwarp();  // before the next copies into this slot
    }
};

template <int N>
__device__ __forceinline__ void copy_wait_newest() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

constexpr int kDepthForward = 4;
template <typename T>
constexpr int kDepthBackward = sizeof(T) == 2 ? 4 : 2;

template <typename T, int NV, bool INTER>
__global__ void __launch_bounds__(kWarps * 32, 2) qk_forward_ring(const QkParams p) {
    constexpr int V = 16 / static_cast<int>(sizeof(T)), DEPTH = kDepthForward, PARTS = 2 * NV;
    extern __shared__ __align__(16) uint4 smem[];
    __shared__ __align__(16) float s_w[2][kMaxDim];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tl = lane & (p.team - 1), mine = lane / p.team, teams = 32 / p.team;
    const Pairs<V, NV, INTER> m(p, tl);
    Ring<V, NV, INTER, DEPTH, PARTS> ring(p, m, smem, warp, lane, tl, mine);
    const int32_t u0 = static_cast<int32_t>(blockIdx.x) * kWarps + warp, stride = static_cast<int32_t>(gridDim.x) * kWarps;
    Walk<T, kInputs> put(p, teams, mine, -1, true, u0, stride);
    Walk<T, kOutput> get(p, teams, mine, -1, true, u0, stride);
    auto issue = [&](int slot) {
        if (!put.done()) {
            ring.put_angles(put, slot);
            if (put.has_head())
#pragma unroll
                for (int n = 0; n < NV; ++n)
                    if (m.has[n]) {
                        copy_to(ring.at(slot, 2 * n), put.at[0] + m.lo[n]);
                        copy_to(ring.at(slot, 2 * n + 1), put.at[0] + m.hi[n]);
                    }
            put.next();
        }
        copy_commit();
    };
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) issue(d);
    load_weights<INTER>(p, s_w);
    const float inv_d = 1.0f / static_cast<float>(p.D);
    for (int slot = 0; !get.done(); slot = slot + 1 == DEPTH ? 0 : slot + 1, get.next()) {
        copy_wait_newest<DEPTH - 1>();
        ring.take_angles(get, slot);
        const bool on = get.has_head(), whole = __all_sync(0xffffffffu, on && m.has[NV - 1]);  // every lane has all its places
        float a[NV][V], b[NV][V], ss = 0.0f;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            split<T, V, INTER>(load_shared(ring.at(slot, 2 * n)), load_shared(ring.at(slot, 2 * n + 1)), a[n], b[n]);
            if (!whole && !(on && m.has[n]))  // never fetched
#pragma unroll
                for (int j = 0; j < V; ++j) a[n][j] = b[n][j] = 0.0f;
            ss = __fadd_rn(ss, __fadd_rn(vec_dot(a[n], a[n]), vec_dot(b[n], b[n])));
        }
        issue(slot);
        const float r = rsqrtf(__fmaf_rn(team_sum(ss, p.team), inv_d, p.eps));
        const float *w = s_w[get.kind];
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            if (!m.has[n]) continue;
            float x[V], y[V], wa[V], wb[V];
            four_by_four<V>(w + m.at[n], wa);
            four_by_four<V>(w + kMaxDim / 2 + m.at[n], wb);
#pragma unroll
            for (int j = 0; j < V; j += 2) {
                const float2 na = mul2(mul2(make_float2(a[n][j], a[n][j + 1]), both(r)), make_float2(wa[j], wa[j + 1]));
                const float2 nb = mul2(mul2(make_float2(b[n][j], b[n][j + 1]), both(r)), make_float2(wb[j], wb[j + 1]));
                const float2 c = make_float2(ring.c[n][j], ring.c[n][j + 1]), s = make_float2(ring.s[n][j], ring.s[n][j + 1]);
                const float2 xx = fma2(mul2(nb, both(-1.0f)), s, mul2(na, c)), yy = fma2(na, s, mul2(nb, c));
                x[j] = xx.x, x[j + 1] = xx.y, y[j] = yy.x, y[j + 1] = yy.y;
            }
            if (!ring.good)
#pragma unroll
                for (int j = 0; j < V; ++j) x[j] = y[j] = 0.0f;
            uint4 rx, ry;
            join<T, V, INTER>(x, y, rx, ry);
            if (on) {
                *reinterpret_cast<uint4 *>(get.at[0] + m.lo[n]) = rx;
                *reinterpret_cast<uint4 *>(get.at[0] + m.hi[n]) = ry;
            }
        }
    }
    copy_wait();
}

template <typename T, int NV, bool INTER>
__global__ void __launch_bounds__(kWarps * 32, 2) qk_backward_ring(const QkParams p) {
    constexpr int V = 16 / static_cast<int>(sizeof(T)), DEPTH = kDepthBackward<T>, PARTS = 4 * NV;
    extern __shared__ __align__(16) uint4 smem[];
    __shared__ __align__(16) float s_w[2][kMaxDim];
    float *s_dw = reinterpret_cast<float *>(smem);  // [kWarps][D]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tl = lane & (p.team - 1), mine = lane / p.team, teams = 32 / p.team;
    const Pairs<V, NV, INTER> m(p, tl);
    load_weights<INTER>(p, s_w);
    const float inv_d = 1.0f / static_cast<float>(p.D);
    for (int i = blockIdx.x; i < p.turns; i += gridDim.x) {
        const int turn = static_cast<int>(sched_item(p.sched, static_cast<uint32_t>(i)));
#pragma unroll 1
        for (int kind = 0; kind < 2; ++kind) {
            const int mine_of = p.split && kind ? turn - p.count[0] : turn;  // which of the kind's slots
            if (mine_of < 0 || mine_of >= p.count[kind]) continue;
            const int slot_out = mine_of + (kind ? p.count[0] : 0);
            const Heads &h = p.kind[kind];
            const int32_t u0 = mine_of * kWarps + warp, stride = p.count[kind] * kWarps;
            Walk<T, kInputAndGradient> put(p, teams, mine, kind, false, u0, stride);
            Walk<T, kOutput> get(p, teams, mine, kind, false, u0, stride);
            Ring<V, NV, INTER, DEPTH, PARTS> ring(p, m, smem + kWarps * p.D / 4, warp, lane, tl, mine);
            auto issue = [&](int slot) {
                if (!put.done()) {
                    ring.put_angles(put, slot);
                    if (put.has_head())
#pragma unroll
                        for (int n = 0; n < NV; ++n)
                            if (m.has[n]) {
                                copy_to(ring.at(slot, 4 * n), put.at[0] + m.lo[n]);
                                copy_to(ring.at(slot, 4 * n + 1), put.at[0] + m.hi[n]);
                                copy_to(ring.at(slot, 4 * n + 2), put.at[1] + m.lo[n]);
                                copy_to(ring.at(slot, 4 * n + 3), put.at[1] + m.hi[n]);
                            }
                    put.next();
                }
                copy_commit();
            };
#pragma unroll
            for (int d = 0; d < DEPTH; ++d) issue(d);
            float acc_a[NV][V] = {}, acc_b[NV][V] = {};
            const float *w = s_w[kind];
#pragma unroll 1
            for (int slot = 0; !get.done(); slot = slot + 1 == DEPTH ? 0 : slot + 1, get.next()) {
                copy_wait_newest<DEPTH - 1>();
                ring.take_angles(get, slot);
                const bool here = get.has_head(), on = here && ring.good, whole = __all_sync(0xffffffffu, on && m.has[NV - 1]);
                float2 a[NV][V / 2], b[NV][V / 2], ga[NV][V / 2], gb[NV][V / 2], wa[NV][V / 2], wb[NV][V / 2], ss = both(0.0f), dot = both(0.0f);
#pragma unroll
                for (int n = 0; n < NV; ++n) {
                    float fa[V], fb[V], x[V], y[V];
                    split<T, V, INTER>(load_shared(ring.at(slot, 4 * n)), load_shared(ring.at(slot, 4 * n + 1)), fa, fb);
                    split<T, V, INTER>(load_shared(ring.at(slot, 4 * n + 2)), load_shared(ring.at(slot, 4 * n + 3)), x, y);
                    if (!whole && !(on && m.has[n]))  // never fetched, or without a position
#pragma unroll
                        for (int j = 0; j < V; ++j) fa[j] = fb[j] = x[j] = y[j] = 0.0f;
                    // places that the lane does not have read a weight of another (of no weight)
                    const int at = m.has[n] ? m.at[n] : 0;
                    float fw[V], gw[V];
                    four_by_four<V>(w + at, fw);
                    four_by_four<V>(w + kMaxDim / 2 + at, gw);
#pragma unroll
                    for (int j = 0; j < V; j += 2) {
                        const float2 c = make_float2(ring.c[n][j], ring.c[n][j + 1]), s = make_float2(ring.s[n][j], ring.s[n][j + 1]);
                        const float2 dx = make_float2(x[j], x[j + 1]), dy = make_float2(y[j], y[j + 1]);
                        const int i = j / 2;
                        a[n][i] = make_float2(fa[j], fa[j + 1]), b[n][i] = make_float2(fb[j], fb[j + 1]);
                        ga[n][i] = fma2(dx, c, mul2(dy, s));
                        gb[n][i] = fma2(mul2(dx, both(-1.0f)), s, mul2(dy, c));
                        ss = fma2(a[n][i], a[n][i], ss);
                        ss = fma2(b[n][i], b[n][i], ss);
                        // g w is all that is needed of the weights later on too
                        wa[n][i] = mul2(ga[n][i], make_float2(fw[j], fw[j + 1])), wb[n][i] = mul2(gb[n][i], make_float2(gw[j], gw[j + 1]));
                        dot = fma2(wa[n][i], a[n][i], dot);
                        dot = fma2(wb[n][i], b[n][i], dot);
                    }
                }
                issue(slot);
                float sum = across(ss), inner = across(dot);
                for (int sh = p.team >> 1; sh > 0; sh >>= 1) {
                    sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, sh));
                    inner = __fadd_rn(inner, __shfl_xor_sync(0xffffffffu, inner, sh));
                }
                // a place without a head, or a token without a position: nothing for dw
                const float r = on ? rsqrtf(__fmaf_rn(sum, inv_d, p.eps)) : 0.0f;
                const float back = on ? -__fmul_rn(r, __fmul_rn(r, __fmul_rn(inner, inv_d))) : 0.0f;  // (times v r)
#pragma unroll
                for (int n = 0; n < NV; ++n) {
                    float x[V], y[V];
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        const float2 na = mul2(a[n][i], both(r)), nb = mul2(b[n][i], both(r));
                        const float2 sa = fma2(na, ga[n][i], make_float2(acc_a[n][2 * i], acc_a[n][2 * i + 1]));
                        const float2 sb = fma2(nb, gb[n][i], make_float2(acc_b[n][2 * i], acc_b[n][2 * i + 1]));
                        acc_a[n][2 * i] = sa.x, acc_a[n][2 * i + 1] = sa.y, acc_b[n][2 * i] = sb.x, acc_b[n][2 * i + 1] = sb.y;
                        const float2 da = fma2(wa[n][i], both(r), mul2(na, both(back))), db = fma2(wb[n][i], both(r), mul2(nb, both(back)));
                        x[2 * i] = da.x, x[2 * i + 1] = da.y, y[2 * i] = db.x, y[2 * i + 1] = db.y;
                    }
                    uint4 rx, ry;
                    join<T, V, INTER>(x, y, rx, ry);
                    if (here && m.has[n]) {
                        *reinterpret_cast<uint4 *>(get.at[0] + m.lo[n]) = rx;
                        *reinterpret_cast<uint4 *>(get.at[0] + m.hi[n]) = ry;
                    }
                }
            }
            copy_wait();
            if (h.dw) slot_sums<V, NV, INTER>(p, m, acc_a, acc_b, s_dw, slot_out, warp, mine);
        }
    }
}

// dw from the slots: kFoldWays threads a column, then a tree.
__global__ void __launch_bounds__(kFoldCols *kFoldWays) qk_fold(const QkParams p) {
    __shared__ float part[kFoldWays][kFoldCols + 1];
    const int col = threadIdx.x % kFoldCols, way = threadIdx.x / kFoldCols;
    const int i = blockIdx.x * kFoldCols + col, kind = i >= p.D;
    const bool on = i < 2 * p.D && p.kind[kind].dw;
    // all of a way's slots on their way at once
    constexpr int kMost = (kSlots + kFoldWays - 1) / kFoldWays;
    float x[kMost], v = 0.0f;
    const int first = kind ? p.count[0] : 0, n = p.count[kind];
    const float *from = p.slots + static_cast<int64_t>(first) * p.D + (i - kind * p.D);
#pragma unroll
    for (int k = 0; k < kMost; ++k) x[k] = on && way + k * kFoldWays < n ? __ldcg(from + static_cast<int64_t>(way + k * kFoldWays) * p.D) : 0.0f;
#pragma unroll
    for (int k = 0; k < kMost; ++k) v = __fadd_rn(v, x[k]);
    part[way][col] = v;
    for (int half = kFoldWays / 2; half > 0; half >>= 1) {
        __syncthreads();
        if (way < half) part[way][col] = __fadd_rn(part[way][col], part[way + half][col]);
    }
    if (on && way == 0) {
        float *to = p.kind[kind].dw + i - kind * p.D;
        *to = p.accumulate ? __fadd_rn(*to, part[0][col]) : part[0][col];
    }
}

// ---- host ---------------------------------------------------------------------

// A [T, n, D] view with contiguous heads.
struct View {
    const void *p;
    int64_t st, sh, n;
};

struct Layout {
    int64_t T, D, es;
    // its heads, token by token or (where these lie further apart) head by head
    Runs runs(const View &v) const {
        const bool heads_outside = v.n > 1 && T > 1 && v.sh >= (T - 1) * v.st + D;
        if (heads_outside) return {v.p, v.sh * es, v.n, v.st * es, T, D * es};
        return {v.p, v.st * es, T, v.sh * es, v.n, D * es};
    }
    size_t extent(const View &v) const { return runs(v).extent(); }
    bool overlap(const View &a, const View &b) const { return runs_overlap(runs(a), runs(b)); }
    // heads apart from each other: tokens outside heads, or heads outside tokens
    bool valid(const View &v) const {
        if (v.n == 0 || T == 0) return true;
        if ((v.n > 1 && v.sh < D) || (T > 1 && v.st < D)) return false;
        return T == 1 || v.n == 1 || v.st >= (v.n - 1) * v.sh + D || v.sh >= (T - 1) * v.st + D;
    }
};

struct Call {
    Layout lay;
    View in[2], dy[2], out[2];
    const void *w[2];
    float *dw[2];
    int32_t dtype, w_dtype, R, P, interleaved, accumulate;
    const float *cos, *sin;
    const int32_t *pos;
    float eps;
    void *ws;
    size_t ws_bytes;
    bool backward;
};

// Slots for the queries and for the keys. Few units: a CTA has one of either, as
// many of each as its heads are (every CTA starts its copies once; 4096 x 32+8 x 64
// bf16 29 -> 23 us). Many: each CTA has one of both, so that all have the same to do
// (16384 x 32+8 x 128 bf16 102 us, 112 with the split).
void slots_of(QkParams &p, int64_t units) {
    const int64_t heads = p.kind[0].n + p.kind[1].n, most = (units + kWarps - 1) / kWarps;
    p.split = units < static_cast<int64_t>(kSlots) * kWarps * 3;
    for (int k = 0; k < 2; ++k) {
        const int64_t n = p.kind[k].n;
        int64_t s = !p.split ? kSlots : (kSlots - 1) * n / heads;  // together at most kSlots - 1, and one for who has none
        if (s < 1) s = 1;
        p.count[k] = static_cast<int32_t>(n == 0 ? 0 : s < most ? s : most);
    }
    p.turns = p.split ? p.count[0] + p.count[1] : p.count[0] > p.count[1] ? p.count[0] : p.count[1];
}

dgr_status check(const Call &c) {
    const Layout &l = c.lay;
    if ((c.dtype != DGR_DTYPE_BF16 && c.dtype != DGR_DTYPE_F32) || (c.w_dtype != DGR_DTYPE_BF16 && c.w_dtype != DGR_DTYPE_F32)) return DGR_ERR_INVALID_ARG;
    if (l.T < 0 || l.D < 2 || l.D % 2 || c.R < 2 || c.R % 2 || c.R > l.D || c.P < 1 || !(c.eps >= 0.0f) || c.in[0].n < 0 || c.in[1].n < 0 ||
        c.in[0].n + c.in[1].n < 1)
        return DGR_ERR_INVALID_ARG;
    if (!c.ws) return DGR_ERR_INVALID_ARG;
    if (l.T > (1 << 26) || l.D > kMaxDim || c.in[0].n > kMaxHeads || c.in[1].n > kMaxHeads) return DGR_ERR_UNSUPPORTED;
    if (l.T > 0 && (!c.cos || !c.sin || !c.pos)) return DGR_ERR_INVALID_ARG;
    const size_t es = static_cast<size_t>(l.es), wes = c.w_dtype == DGR_DTYPE_BF16 ? 2 : 4;
    for (int k = 0; k < 2; ++k) {
        if (c.in[k].n == 0) {
            if (c.dw[k]) return DGR_ERR_INVALID_ARG;
            continue;
        }
        if (l.T > 0 && (!c.in[k].p || !c.out[k].p || (c.backward && !c.dy[k].p))) return DGR_ERR_INVALID_ARG;
        if (c.backward && c.dw[k] && !c.w[k]) return DGR_ERR_INVALID_ARG;
        for (const View *v : {&c.in[k], &c.out[k], &c.dy[k]}) {
            if (v->p && !l.valid(*v)) return DGR_ERR_INVALID_ARG;
            if (!aligned(v->p, es)) return DGR_ERR_MISALIGNED;
        }
        if (!aligned(c.w[k], wes) || !aligned(c.dw[k], 4)) return DGR_ERR_MISALIGNED;
    }
    if (!aligned(c.cos, 4) || !aligned(c.sin, 4) || !aligned(c.pos, 4) || !aligned(c.ws, kAlign)) return DGR_ERR_MISALIGNED;
    const size_t need = c.backward ? dgr_qk_norm_rope_workspace_bytes(l.T, static_cast<int32_t>(c.in[0].n), static_cast<int32_t>(c.in[1].n),
                                                                      static_cast<int32_t>(l.D))
                                   : sizeof(WsHeader);
    if (c.ws_bytes < need) return DGR_ERR_WORKSPACE_TOO_SMALL;
    struct Range { const void *p; size_t n; };
    const size_t table = static_cast<size_t>(c.P) * (c.R / 2) * 4, d = static_cast<size_t>(l.D);
    const Range flat[] = {{c.cos, table}, {c.sin, table}, {c.pos, static_cast<size_t>(l.T) * 4}, {c.w[0], d * wes}, {c.w[1], d * wes}};
    const Range flat_out[] = {{c.ws, need}, {c.dw[0], d * 4}, {c.dw[1], d * 4}};
    for (int k = 0; k < 2; ++k) {
        const View &o = c.out[k];
        const size_t n = l.extent(o);
        for (const Range &r : flat)
            if (ranges_overlap(o.p, n, r.p, r.n)) return DGR_ERR_ALIAS;
        for (const Range &r : flat_out)
            if (ranges_overlap(o.p, n, r.p, r.n)) return DGR_ERR_ALIAS;
        for (int j = 0; j < 2; ++j) {
            // in place: each head is read by the lanes that write it (forward over v, backward over dy)
            const View &home = c.backward ? c.dy[j] : c.in[j];
            const bool same = j == k && home.p == o.p && home.st == o.st && home.sh == o.sh;
            if (!same && l.overlap(o, home)) return DGR_ERR_ALIAS;
            if (c.backward && l.overlap(o, c.in[j])) return DGR_ERR_ALIAS;
        }
    }
    if (l.overlap(c.out[0], c.out[1])) return DGR_ERR_ALIAS;
    for (const Range &o : flat_out) {
        for (const Range &r : flat)
            if (ranges_overlap(o.p, o.n, r.p, r.n)) return DGR_ERR_ALIAS;
        for (int j = 0; j < 2; ++j)
            if (ranges_overlap(o.p, o.n, c.in[j].p, l.extent(c.in[j])) || ranges_overlap(o.p, o.n, c.dy[j].p, l.extent(c.dy[j]))) return DGR_ERR_ALIAS;
        for (const Range &r : flat_out)
            if (&r < &o && ranges_overlap(o.p, o.n, r.p, r.n)) return DGR_ERR_ALIAS;
    }
    return DGR_OK;
}

// RING: heads in vectors of 16 bytes.
template <typename T, int V, int NV, bool INTER, bool RING>
dgr_status launch(QkParams p, bool backward, int sms, cudaStream_t s) {
    const int vecs = (p.D / 2 + V - 1) / V;  // groups of pairs a head
    int team = 1;
    while (team * NV < vecs) team <<= 1;
    p.team = team;
    const int teams = 32 / team;
    const int groups = (p.kind[0].n + teams - 1) / teams + (p.kind[1].n + teams - 1) / teams;
    // few tokens: a token over several warps, down to one group of heads each
    int64_t chunks = p.T > 0 ? (kSlots * kWarps + p.T - 1) / p.T : 1;
    if (chunks > groups) chunks = groups;
    p.chunks = static_cast<int32_t>(chunks);
    const int64_t units = static_cast<int64_t>(p.T) * p.chunks;
    if (units > (1 << 30)) return DGR_ERR_UNSUPPORTED;
    if (!backward) {
        p.sched = sched_for(static_cast<uint32_t>(units));
        const int64_t ctas = (units + kWarps - 1) / kWarps, most = static_cast<int64_t>(sms) * 2;
        const unsigned grid = sched_grid(static_cast<unsigned>(ctas < most ? ctas : most));
        if constexpr (RING) {
            using R = Ring<V, NV, INTER, kDepthForward, 2 * NV>;
            const size_t smem = R::bytes(team);
            const dgr_status st = allow_smem(qk_forward_ring<T, NV, INTER>, smem, R::bytes(32));
            if (st != DGR_OK) return st;
            qk_forward_ring<T, NV, INTER><<<grid, kWarps * 32, smem, s>>>(p);
        } else {
            qk_forward<T, V, NV, INTER, 2><<<grid, kWarps * 32, 0, s>>>(p);
        }
        return launch_status();
    }
    slots_of(p, units);
    p.sched = sched_for(static_cast<uint32_t>(p.turns));
    const int most = sms * 2;
    const unsigned grid = sched_grid(static_cast<unsigned>(p.turns < most ? p.turns : most));
    dgr_status st = DGR_OK;
    if (p.turns == 0) {  // no tokens: dw is 0
    } else if constexpr (RING) {
        using R = Ring<V, NV, INTER, kDepthBackward<T>, 4 * NV>;
        const size_t smem = R::bytes(team) + sizeof(float) * kWarps * p.D;
        if ((st = allow_smem(qk_backward_ring<T, NV, INTER>, smem, R::bytes(32) + sizeof(float) * kWarps * kMaxDim)) != DGR_OK) return st;
        qk_backward_ring<T, NV, INTER><<<grid, kWarps * 32, smem, s>>>(p);
    } else {
        qk_backward<T, V, NV, INTER, 1><<<grid, kWarps * 32, 0, s>>>(p);
    }
    st = launch_status();
    if (st != DGR_OK || (!p.kind[0].dw && !p.kind[1].dw)) return st;
    qk_fold<<<static_cast<unsigned>((2 * p.D + kFoldCols - 1) / kFoldCols), kFoldCols * kFoldWays, 0, s>>>(p);
    return launch_status();
}

template <typename T, bool INTER>
dgr_status launch_width(const QkParams &p, int vec, bool backward, int sms, cudaStream_t s) {
    constexpr int W = 16 / static_cast<int>(sizeof(T));
    if (vec == W) return launch<T, W, 8 / W, INTER, true>(p, backward, sms, s);
    if (vec == 2) return launch<T, 2, 4, INTER, false>(p, backward, sms, s);
    return launch<T, 1, 8, INTER, false>(p, backward, sms, s);
}

dgr_status run(const Call &c, void *stream) {
    dgr_status st = check(c);
    if (st != DGR_OK) return st;
    if ((st = check_device()) != DGR_OK) return st;
    const Layout &l = c.lay;
    if (l.T == 0 && (!c.backward || (!c.dw[0] && !c.dw[1]))) return DGR_OK;
    QkParams p{};
    // pairs in a vector: of 16 bytes, 2 or 1, as far as heads, halves and tables start at multiples of it
    const int es = static_cast<int>(l.es);
    int vec = 16 / es;
    auto fits = [&](int v) {
        if (c.R / 2 % v || l.D / 2 % v) return false;
        if (v % 4 == 0 && (!aligned(c.cos, 16) || !aligned(c.sin, 16))) return false;
        for (int k = 0; k < 2; ++k)
            for (const View *w : {&c.in[k], &c.out[k], &c.dy[k]})
                if (w->p && w->n > 0 &&
                    (!aligned(w->p, static_cast<size_t>(v * es)) || (l.T > 1 && w->st % v) || (w->n > 1 && w->sh % v)))
                    return false;
        return true;
    };
    if (!fits(vec)) vec = fits(2) ? 2 : 1;
    for (int k = 0; k < 2; ++k) {
        Heads &h = p.kind[k];
        h.n = static_cast<int32_t>(c.in[k].n);
        h.v = c.in[k].p, h.st = c.in[k].st, h.sh = c.in[k].sh;
        h.dy = c.dy[k].p, h.st_dy = c.dy[k].st, h.sh_dy = c.dy[k].sh;
        h.out = const_cast<void *>(c.out[k].p), h.st_out = c.out[k].st, h.sh_out = c.out[k].sh;
        h.w = c.w[k], h.dw = c.dw[k];
    }
    p.T = static_cast<int32_t>(l.T), p.D = static_cast<int32_t>(l.D), p.R = c.R, p.P = c.P;
    p.w_bf16 = c.w_dtype == DGR_DTYPE_BF16;
    p.cos = c.cos, p.sin = c.sin, p.pos = c.pos, p.eps = c.eps;
    p.accumulate = c.accumulate ? 1 : 0;
    p.hdr = static_cast<WsHeader *>(c.ws);
    p.slots = reinterpret_cast<float *>(static_cast<char *>(c.ws) + sizeof(WsHeader));
    int sms = 0;
    if ((st = usable_sms(&sms)) != DGR_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (es == 2) return c.interleaved ? launch_width<bf16, true>(p, vec, c.backward, sms, s) : launch_width<bf16, false>(p, vec, c.backward, sms, s);
    return c.interleaved ? launch_width<float, true>(p, vec, c.backward, sms, s) : launch_width<float, false>(p, vec, c.backward, sms, s);
}

}  // namespace
}  // namespace dgr

using namespace dgr;

extern "C" size_t dgr_qk_norm_rope_workspace_bytes(int64_t T, int32_t n_q, int32_t n_k, int32_t D) {
    if (T < 0 || T > (1 << 26) || n_q < 0 || n_k < 0 || n_q + n_k < 1 || n_q > kMaxHeads || n_k > kMaxHeads || D < 2 || D > kMaxDim) return 0;
    return sizeof(WsHeader) + static_cast<size_t>(kSlots) * 2 * static_cast<size_t>(D) * 4;
}

extern "C" dgr_status dgr_qk_norm_rope(const void *q, int64_t q_token, int64_t q_head, int32_t n_q, const void *k, int64_t k_token,
                                       int64_t k_head, int32_t n_k, int32_t dtype, int64_t T, int32_t D, const void *w_q,
                                       const void *w_k, int32_t w_dtype, const float *cos, const float *sin, int32_t P, int32_t R,
                                       int32_t interleaved, const int32_t *positions, float eps, void *q_out, int64_t qo_token,
                                       int64_t qo_head, void *k_out, int64_t ko_token, int64_t ko_head, void *ws, size_t ws_bytes,
                                       void *stream) {
    Call c{};
    c.lay = {T, D, dtype == DGR_DTYPE_BF16 ? 2 : 4};
    c.in[0] = {q, q_token, q_head, n_q}, c.in[1] = {k, k_token, k_head, n_k};
    c.out[0] = {q_out, qo_token, qo_head, n_q}, c.out[1] = {k_out, ko_token, ko_head, n_k};
    c.w[0] = w_q, c.w[1] = w_k;
    c.dtype = dtype, c.w_dtype = w_dtype, c.R = R, c.P = P, c.interleaved = interleaved;
    c.cos = cos, c.sin = sin, c.pos = positions, c.eps = eps;
    c.ws = ws, c.ws_bytes = ws_bytes;
    return run(c, stream);
}

extern "C" dgr_status dgr_qk_norm_rope_backward(const void *dq_out, int64_t dqo_token, int64_t dqo_head, const void *dk_out,
                                                int64_t dko_token, int64_t dko_head, const void *q, int64_t q_token, int64_t q_head,
                                                int32_t n_q, const void *k, int64_t k_token, int64_t k_head, int32_t n_k,
                                                int32_t dtype, int64_t T, int32_t D, const void *w_q, const void *w_k,
                                                int32_t w_dtype, const float *cos, const float *sin, int32_t P, int32_t R,
                                                int32_t interleaved, const int32_t *positions, float eps, void *dq, int64_t dq_token,
                                                int64_t dq_head, void *dk, int64_t dk_token, int64_t dk_head, float *dw_q, float *dw_k,
                                                int32_t accumulate, void *ws, size_t ws_bytes, void *stream) {
    Call c{};
    c.lay = {T, D, dtype == DGR_DTYPE_BF16 ? 2 : 4};
    c.in[0] = {q, q_token, q_head, n_q}, c.in[1] = {k, k_token, k_head, n_k};
    c.dy[0] = {dq_out, dqo_token, dqo_head, n_q}, c.dy[1] = {dk_out, dko_token, dko_head, n_k};
    c.out[0] = {dq, dq_token, dq_head, n_q}, c.out[1] = {dk, dk_token, dk_head, n_k};
    c.w[0] = w_q, c.w[1] = w_k, c.dw[0] = dw_q, c.dw[1] = dw_k;
    c.dtype = dtype, c.w_dtype = w_dtype, c.R = R, c.P = P, c.interleaved = interleaved, c.accumulate = accumulate;
    c.cos = cos, c.sin = sin, c.pos = positions, c.eps = eps;
    c.ws = ws, c.ws_bytes = ws_bytes;
    c.backward = true;
    return run(c, stream);
}
