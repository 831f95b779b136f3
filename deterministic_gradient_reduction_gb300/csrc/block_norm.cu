// Norms before and after a block, fused with its gate and residual scale.
//
// For every token (row) of the residual stream x and the block's output y:
//   r1 = (mean(y^2) + eps)^(-1/2),  n = y r1 w_post          (norm after the block)
//   h  = a x + g n                                            (gate g, residual scale a)
//   r2 = (mean(h^2) + eps)^(-1/2),  u = h r2 w_pre           (norm before the next block)
// and backwards, from dh and du (gradients of h and u):
//   v  = du w_pre,  D = dh + r2 v - (r2^3 / H) (v . h) h,  dx = a D
//   q  = g w_post D,  dy = r1 q - (r1^3 / H) (q . y) y
//   dw_pre = sum_t du h r2,  C = sum_t [g_t] D y r1,
//   dw_post = [g] C,  dgate = w_post C (a gate a channel) or D . n (a gate a token).
// All in binary32 from the stored rows; h and u are rounded once, u from the
// unrounded h (a second rounding in between would add its error to u's).
//
// Deterministic: a row's sums are made by one team of threads in a fixed
// order; the sums over tokens go through a fixed number of slots (set by T and
// H alone): slot s takes the rows s, s + P, s + 2P, ... in ascending order,
// and a second launch adds the slots in a fixed tree.
#include "row_common.cuh"

namespace dgr {
namespace {

using namespace row;

constexpr int kWarpTeams = 8;     // rows side by side in a CTA where a warp takes a row
constexpr int kFoldCols = 16;     // columns of a fold CTA (64 bytes of a slot)
constexpr int kFoldWays = 32;     // threads that share a column's slots
constexpr int64_t kMaxWidth = 16384;

enum { kGateNone = 0, kGateChannel = 1, kGateToken = 2 };

struct NormParams {
    const void *x, *y;          // forward
    const void *h, *dh, *du;    // backward (h: the forward's output)
    int64_t ld_x, ld_y, ld_h, ld_dh, ld_du;
    void *out_h, *out_u;        // forward: h, u; backward: dx, dy
    int64_t ld_oh, ld_ou;
    const void *w_post, *gate, *w_pre;
    int32_t w_bf16, gate_mode;
    int32_t w_vec;              // the weights start at multiples of 16 bytes
    int32_t T, H;
    float alpha, eps;
    float *dw_post, *dgate, *dw_pre;
    float *slots;               // [n_slots, 2H]: C, then dw_pre
    int32_t n_slots, accumulate;
    int32_t depth;              // rows in shared memory
    Sched sched;
};

// The row's elements of this thread: vector i of its NV is number i * team + tl.
// They are worked on in pairs (two at a time by the packed instructions): unit
// u is vector u, or vectors 2 u and 2 u + 1 where a vector is one element.
template <int VEC>
struct Cols {
    static constexpr int kPer = VEC == 1 ? 2 : 1;     // vectors a unit
    static constexpr int kPairs = VEC * kPer / 2;     // pairs a unit
    int team, tl, n_vec;
    __device__ __forceinline__ bool has(int i) const { return i * team + tl < n_vec; }
    __device__ __forceinline__ int at(int i) const { return (i * team + tl) * VEC; }
    // element j of unit u: its vector and its column
    __device__ __forceinline__ int vec(int u, int j) const { return VEC == 1 ? 2 * u + j : u; }
    __device__ __forceinline__ int col(int u, int j) const { return VEC == 1 ? at(2 * u + j) : at(u) + j; }
};

// gw = w_post times the channel gate (1 where there is none), w2 = w_pre; 0
// where the thread has no element.
template <int VEC, int NU>
__device__ __forceinline__ void load_weights(float2 *gw, float2 *w2, const NormParams &p, const Cols<VEC> &c) {
    constexpr int P = Cols<VEC>::kPairs;
    const void *gate = p.gate_mode == kGateChannel ? p.gate : nullptr;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
        float a[2 * P], g[2 * P], b[2 * P];
        auto unit = [&](const void *w, float *f, float without) {
#pragma unroll
            for (int j = 0; j < 2 * P; ++j) f[j] = c.has(c.vec(u, j)) ? without : 0.0f;
            if (!w) return;
            if constexpr (VEC >= 4) {
                if (p.w_vec && c.has(u)) {  // VEC columns from a multiple of VEC on
                    if (p.w_bf16) {
                        unpack<bf16, VEC>(__ldg(reinterpret_cast<const raw_t<bf16, VEC> *>(static_cast<const bf16 *>(w) + c.at(u))), f);
                    } else {
#pragma unroll
                        for (int j = 0; j < VEC; j += 4) unpack<float, 4>(__ldg(reinterpret_cast<const uint4 *>(static_cast<const float *>(w) + c.at(u) + j)), f + j);
                    }
                    return;
                }
            }
#pragma unroll
            for (int j = 0; j < 2 * P; ++j)
                if (c.has(c.vec(u, j))) f[j] = param(w, p.w_bf16, c.col(u, j));
        };
        unit(p.w_post, a, 1.0f);
        unit(gate, g, 1.0f);
        unit(p.w_pre, b, 0.0f);
#pragma unroll
        for (int j = 0; j < P; ++j) {
            gw[u * P + j] = mul2(make_float2(a[2 * j], a[2 * j + 1]), make_float2(g[2 * j], g[2 * j + 1]));
            w2[u * P + j] = make_float2(b[2 * j], b[2 * j + 1]);
        }
    }
}

// The rows' elements on their way: `depth` rows of S streams in shared memory,
// every element fetched and read by the same thread, so no barrier is needed
// for it. Elements of 2 bytes (rows that start at odd ones) are too small for
// such copies, and rows too wide for shared memory (depth 0) do not fit: they
// are loaded where they are used.
// Places that a thread never fetches are zeroed once and stay so.
template <typename T, int VEC, int NV, int S, int MAXT>
struct Feed {
    using raw = raw_t<T, VEC>;
    static constexpr bool kRing = sizeof(raw) >= 4;
    static constexpr int kStage = S * NV * MAXT;
    raw *mine;
    const T *rows[S];
    int64_t ld[S];
    const Cols<VEC> &c;
    int in = 0, out = 0, end, depth;  // offsets of stages

    __device__ __forceinline__ Feed(char *smem, const void *const (&src)[S], const int64_t (&strides)[S], const Cols<VEC> &cols, int d)
        : mine(reinterpret_cast<raw *>(smem) + threadIdx.x), c(cols), end(d * kStage), depth(d) {
#pragma unroll
        for (int s = 0; s < S; ++s) rows[s] = static_cast<const T *>(src[s]), ld[s] = strides[s];
        clear();
    }
    __device__ __forceinline__ void clear() {
        if constexpr (kRing)
            for (int k = 0; k < depth; ++k)
#pragma unroll
                for (int s = 0; s < S; ++s)
#pragma unroll
                    for (int i = 0; i < NV; ++i)
                        if (!rows[s] || !c.has(i)) mine[k * kStage + (s * NV + i) * MAXT] = raw{};
    }
    __device__ __forceinline__ void fetch(int64_t row, bool on) {
        if constexpr (kRing) {
            if (on && depth)
#pragma unroll
                for (int s = 0; s < S; ++s)
                    if (rows[s]) {
                        const T *src = rows[s] + row * ld[s] + c.tl * VEC;
#pragma unroll
                        for (int i = 0; i < NV; ++i)
                            if (c.has(i)) copy_async<sizeof(raw)>(mine + in + (s * NV + i) * MAXT, src + i * c.team * VEC);
                    }
            copy_commit();
            in = in + kStage >= end ? 0 : in + kStage;
        }
    }
    __device__ __forceinline__ raw vector(int64_t row, int s, int i) const {
        raw v{};
        if (kRing && depth) v = mine[out + (s * NV + i) * MAXT];
        else if (rows[s] && c.has(i)) v = *reinterpret_cast<const raw *>(rows[s] + row * ld[s] + c.at(i));
        return v;
    }
    // unit u of stream s of the row in use (zeros where the thread has none)
    __device__ __forceinline__ void get(float2 *f, int64_t row, int s, int u) const {
        float e[VEC * Cols<VEC>::kPer];
#pragma unroll
        for (int k = 0; k < Cols<VEC>::kPer; ++k) unpack<T, VEC>(vector(row, s, u * Cols<VEC>::kPer + k), e + k * VEC);
#pragma unroll
        for (int j = 0; j < Cols<VEC>::kPairs; ++j) f[j] = make_float2(e[2 * j], e[2 * j + 1]);
    }
    __device__ __forceinline__ void next() {
        if constexpr (kRing) out = out + kStage >= end ? 0 : out + kStage;
    }
    __device__ __forceinline__ void restart() { in = out = 0; }
};

template <typename T, int VEC>
__device__ __forceinline__ void put(const float2 *f, void *base, int64_t row_at, const Cols<VEC> &c, int u) {
    float e[VEC * Cols<VEC>::kPer];
#pragma unroll
    for (int j = 0; j < Cols<VEC>::kPairs; ++j) e[2 * j] = f[j].x, e[2 * j + 1] = f[j].y;
#pragma unroll
    for (int k = 0; k < Cols<VEC>::kPer; ++k) {
        const int i = u * Cols<VEC>::kPer + k;
        if (c.has(i)) *reinterpret_cast<raw_t<T, VEC> *>(static_cast<T *>(base) + row_at + c.at(i)) = pack<T, VEC>(e + k * VEC);
    }
}

// The sum of v over the team that has a row: a warp, or the whole block (two
// buffers in turn, so that one barrier a sum is enough).
template <bool WARP>
__device__ __forceinline__ float team_sum(float v, float *buf, int &turn) {
    v = warp_sum(v);
    if constexpr (!WARP) {
        float *b = buf + turn * 32;
        turn ^= 1;
        if ((threadIdx.x & 31) == 0) b[threadIdx.x >> 5] = v;
        __syncthreads();
        const int n = blockDim.x >> 5;
        v = (threadIdx.x & 31) < n ? b[threadIdx.x & 31] : 0.0f;
        for (int s = 1; s < n; s <<= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, s));
        v = __shfl_sync(0xffffffffu, v, 0);
    }
    return v;
}

template <typename T, int VEC, int NV, int MAXT, int MINB, bool WARP>
__global__ void __launch_bounds__(MAXT, MINB) norm_forward(const NormParams p) {
    extern __shared__ __align__(16) char smem[];
    __shared__ float buf[2 * 32];
    constexpr int P = Cols<VEC>::kPairs, NU = NV / Cols<VEC>::kPer;
    const int teams = WARP ? kWarpTeams : 1;
    const Cols<VEC> c{WARP ? 32 : static_cast<int>(blockDim.x), static_cast<int>(WARP ? threadIdx.x & 31 : threadIdx.x), p.H / VEC};
    Feed<T, VEC, NV, 2, MAXT> feed(smem, {p.x, p.y}, {p.ld_x, p.ld_y}, c, p.depth);
    const int64_t step = static_cast<int64_t>(gridDim.x) * teams;
    int64_t it = static_cast<int64_t>(blockIdx.x) * teams + (WARP ? threadIdx.x >> 5 : 0);
    auto row_of = [&](int64_t i) { return static_cast<int64_t>(sched_item(p.sched, static_cast<uint32_t>(i < p.T ? i : 0))); };
    for (int d = 0; d + 1 < p.depth; ++d) feed.fetch(row_of(it + d * step), it + d * step < p.T);
    float2 gw[NU * P], w2[NU * P];
    load_weights<VEC, NU>(gw, w2, p, c);
    const float inv_h = 1.0f / static_cast<float>(p.H);
    int turn = 0;
    for (; it < p.T; it += step) {
        const int64_t row = row_of(it), ahead = it + (p.depth > 0 ? p.depth - 1 : 0) * step;
        feed.fetch(row_of(ahead), ahead < p.T);
        float f = p.gate_mode == kGateToken ? param(p.gate, p.w_bf16, row) : 1.0f;
        copy_wait_for(p.depth);
        float2 h[NU * P];
        if (p.y) {
            if (p.w_post) {
                float2 s = both(0.0f);
#pragma unroll
                for (int i = 0; i < NU; ++i) {
                    float2 y[P];
                    feed.get(y, row, 1, i);
#pragma unroll
                    for (int j = 0; j < P; ++j) s = fma2(y[j], y[j], s);
                }
                f = __fmul_rn(f, rsqrtf(__fmaf_rn(team_sum<WARP>(across(s), buf, turn), inv_h, p.eps)));
            }
#pragma unroll
            for (int i = 0; i < NU; ++i) {
                float2 x[P], y[P];
                feed.get(x, row, 0, i);
                feed.get(y, row, 1, i);
#pragma unroll
                for (int j = 0; j < P; ++j) h[i * P + j] = fma2(both(p.alpha), x[j], mul2(mul2(y[j], both(f)), gw[i * P + j]));
                put<T, VEC>(h + i * P, p.out_h, row * p.ld_oh, c, i);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NU; ++i) feed.get(h + i * P, row, 0, i);
        }
        if (p.out_u) {
            float2 s = both(0.0f);
#pragma unroll
            for (int e = 0; e < NU * P; ++e) s = fma2(h[e], h[e], s);
            const float r = rsqrtf(__fmaf_rn(team_sum<WARP>(across(s), buf, turn), inv_h, p.eps));
#pragma unroll
            for (int i = 0; i < NU; ++i) {
#pragma unroll
                for (int j = 0; j < P; ++j) h[i * P + j] = mul2(mul2(h[i * P + j], both(r)), w2[i * P + j]);
                put<T, VEC>(h + i * P, p.out_u, row * p.ld_ou, c, i);
            }
        }
        feed.next();
    }
    copy_wait();
}

// The sum of column e of [C, dw_pre] to where it goes.
__device__ __forceinline__ void put_column(const NormParams &p, int e, float v) {
    auto put = [&](float *dst, int i, float g) {
        if (dst) dst[i] = p.accumulate ? __fadd_rn(dst[i], g) : g;
    };
    if (e >= p.H) {
        put(p.dw_pre, e - p.H, v);
    } else {
        const bool channel = p.gate_mode == kGateChannel;
        put(p.dw_post, e, channel ? __fmul_rn(param(p.gate, p.w_bf16, e), v) : v);
        if (channel) put(p.dgate, e, p.w_post ? __fmul_rn(param(p.w_post, p.w_bf16, e), v) : v);
    }
}

// One round of sums a row: with gy = gw y,
//   q . y = dh . gy + r2 v . gy - (r2^3 / H) (v . h) h . gy,
// so D need not be known before the second norm's sum is made.
template <typename T, int VEC, int NV, int MAXT, int MINB, bool WARP>
__global__ void __launch_bounds__(MAXT, MINB) norm_backward(const NormParams p) {
    extern __shared__ __align__(16) char smem[];  // the rows on their way; at the end WARP: the teams' columns [kWarpTeams][2H]
    __shared__ float buf[2][32][8];
    constexpr int P = Cols<VEC>::kPairs, NU = NV / Cols<VEC>::kPer;
    enum { kH, kDh, kDu, kY };
    const int teams = WARP ? kWarpTeams : 1, lane = threadIdx.x & 31;
    const int team = WARP ? threadIdx.x >> 5 : 0;
    const Cols<VEC> c{WARP ? 32 : static_cast<int>(blockDim.x), static_cast<int>(WARP ? threadIdx.x & 31 : threadIdx.x), p.H / VEC};
    Feed<T, VEC, NV, 4, MAXT> feed(smem, {p.h, p.dh, p.du, p.y}, {p.ld_h, p.ld_dh, p.ld_du, p.ld_y}, c, p.depth);
    const int64_t step = static_cast<int64_t>(p.n_slots) * teams;
    float2 gw[NU * P], w2[NU * P];
    const float inv_h = 1.0f / static_cast<float>(p.H);
    int turn = 0;
    bool first = true;
    for (int32_t is = blockIdx.x; is < p.n_slots; is += gridDim.x) {
        const int32_t slot = static_cast<int32_t>(sched_item(p.sched, static_cast<uint32_t>(is)));
        const int64_t row0 = static_cast<int64_t>(slot) * teams + team;
        for (int d = 0; d + 1 < p.depth; ++d) feed.fetch(row0 + d * step, row0 + d * step < p.T);
        if (first) load_weights<VEC, NU>(gw, w2, p, c);
        first = false;
        float2 accC[NU * P], accW[NU * P];
#pragma unroll
        for (int e = 0; e < NU * P; ++e) accC[e] = accW[e] = both(0.0f);
        for (int64_t row = row0; row < p.T; row += step) {
            const int64_t ahead = row + (p.depth > 0 ? p.depth - 1 : 0) * step;
            feed.fetch(ahead, ahead < p.T);
            const float gt = p.gate_mode == kGateToken ? param(p.gate, p.w_bf16, row) : 1.0f;
            copy_wait_for(p.depth);
            float2 q[6];  // h.h, v.h, y.y, dh.gy, v.gy, h.gy
#pragma unroll
            for (int k = 0; k < 6; ++k) q[k] = both(0.0f);
#pragma unroll
            for (int i = 0; i < NU; ++i) {
                float2 h[P], dh[P], du[P], y[P];
                feed.get(h, row, kH, i);
                feed.get(dh, row, kDh, i);
                feed.get(du, row, kDu, i);
                feed.get(y, row, kY, i);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const float2 v = mul2(du[j], w2[i * P + j]), gy = mul2(gw[i * P + j], y[j]);
                    q[0] = fma2(h[j], h[j], q[0]);
                    q[1] = fma2(v, h[j], q[1]);
                    q[2] = fma2(y[j], y[j], q[2]);
                    q[3] = fma2(dh[j], gy, q[3]);
                    q[4] = fma2(v, gy, q[4]);
                    q[5] = fma2(h[j], gy, q[5]);
                }
            }
            float s[8] = {across(q[0]), across(q[1]), across(q[2]), across(q[3]), across(q[4]), across(q[5]), 0.0f, 0.0f};
            float t = warp_sum8(s, lane);  // of sum lane / 4
            if constexpr (!WARP) {
                if ((lane & 3) == 0) buf[turn][threadIdx.x >> 5][lane >> 2] = t;
                __syncthreads();
                // lane: sum lane % 8 of the warps lane / 8, lane / 8 + 4, ...
                const int n = blockDim.x >> 5;
                t = 0.0f;
                for (int w = lane >> 3; w < n; w += 4) t = __fadd_rn(t, buf[turn][w][lane & 7]);
                t = __fadd_rn(t, __shfl_xor_sync(0xffffffffu, t, 8));
                t = __fadd_rn(t, __shfl_xor_sync(0xffffffffu, t, 16));
                turn ^= 1;
            }
#pragma unroll
            for (int k = 0; k < 6; ++k) s[k] = __shfl_sync(0xffffffffu, t, WARP ? 4 * k : k);
            float r2 = 0.0f, k2 = 0.0f;  // D = dh + r2 v - k2 h
            if (p.w_pre) {
                r2 = rsqrtf(__fmaf_rn(s[0], inv_h, p.eps));
                k2 = __fmul_rn(__fmul_rn(__fmul_rn(__fmul_rn(s[1], inv_h), r2), r2), r2);  // r2^3 alone may underflow
            }
            const float dot = __fmaf_rn(-k2, s[5], __fmaf_rn(r2, s[4], s[3]));  // D . gy
            float r1 = 1.0f, k1 = 0.0f;  // dy = gt (r1 gw D - k1 y)
            if (p.w_post) {
                r1 = rsqrtf(__fmaf_rn(s[2], inv_h, p.eps));
                k1 = __fmul_rn(__fmul_rn(__fmul_rn(__fmul_rn(dot, inv_h), r1), r1), r1);
            }
            if (p.gate_mode == kGateToken && p.dgate && c.tl == 0) {
                const float g = __fmul_rn(r1, dot);
                p.dgate[row] = p.accumulate ? __fadd_rn(p.dgate[row], g) : g;
            }
            const float yr = __fmul_rn(r1, gt), kg = __fmul_rn(k1, gt);
#pragma unroll
            for (int i = 0; i < NU; ++i) {
                float2 h[P], dh[P], du[P], y[P];
                feed.get(h, row, kH, i);
                feed.get(dh, row, kDh, i);
                feed.get(du, row, kDu, i);
                feed.get(y, row, kY, i);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const int e = i * P + j;
                    const float2 D = fma2(both(-k2), h[j], fma2(both(r2), mul2(du[j], w2[e]), dh[j]));
                    accW[e] = fma2(du[j], mul2(h[j], both(r2)), accW[e]);
                    accC[e] = fma2(D, mul2(y[j], both(yr)), accC[e]);
                    y[j] = fma2(both(-kg), y[j], mul2(mul2(gw[e], both(yr)), D));
                    h[j] = mul2(both(p.alpha), D);
                }
                put<T, VEC>(h, p.out_h, row * p.ld_oh, c, i);
                if (p.y) put<T, VEC>(y, p.out_u, row * p.ld_ou, c, i);
            }
            feed.next();
        }
        copy_wait();  // (nothing but empty groups)
        feed.restart();
        // the fold's CTAs may come as this kernel's leave; they wait for all of them
        if (is + gridDim.x >= p.n_slots) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        float *dst = p.slots + static_cast<int64_t>(slot) * 2 * p.H;
        if constexpr (WARP) {  // the warps' sums, in ascending order
            float *team_cols = reinterpret_cast<float *>(smem);
            float *mine = team_cols + static_cast<int64_t>(team) * 2 * p.H;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NU; ++i)
#pragma unroll
                for (int j = 0; j < 2 * P; ++j)
                    if (c.has(c.vec(i, j))) {
                        mine[c.col(i, j)] = j & 1 ? accC[i * P + j / 2].y : accC[i * P + j / 2].x;
                        mine[p.H + c.col(i, j)] = j & 1 ? accW[i * P + j / 2].y : accW[i * P + j / 2].x;
                    }
            __syncthreads();
            for (int e = threadIdx.x; e < 2 * p.H; e += blockDim.x) {
                float v = team_cols[e];
                for (int k = 1; k < kWarpTeams; ++k) v = __fadd_rn(v, team_cols[k * 2 * p.H + e]);
                if (p.n_slots == 1) put_column(p, e, v);
                else dst[e] = v;
            }
            __syncthreads();
            feed.clear();  // the columns lay where the rows go
        } else if (p.n_slots == 1) {  // nothing to fold
#pragma unroll
            for (int i = 0; i < NU; ++i)
#pragma unroll
                for (int j = 0; j < 2 * P; ++j)
                    if (c.has(c.vec(i, j))) {
                        put_column(p, c.col(i, j), j & 1 ? accC[i * P + j / 2].y : accC[i * P + j / 2].x);
                        put_column(p, p.H + c.col(i, j), j & 1 ? accW[i * P + j / 2].y : accW[i * P + j / 2].x);
                    }
        } else {
#pragma unroll
            for (int i = 0; i < NU; ++i) {
                if constexpr (VEC >= 4) {  // H is a multiple of 4
                    if (!c.has(i)) continue;
#pragma unroll
                    for (int j = 0; j < P; j += 2) {
                        *reinterpret_cast<float4 *>(dst + c.at(i) + 2 * j) = make_float4(accC[i * P + j].x, accC[i * P + j].y, accC[i * P + j + 1].x, accC[i * P + j + 1].y);
                        *reinterpret_cast<float4 *>(dst + p.H + c.at(i) + 2 * j) = make_float4(accW[i * P + j].x, accW[i * P + j].y, accW[i * P + j + 1].x, accW[i * P + j + 1].y);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 2 * P; ++j)
                        if (c.has(c.vec(i, j))) {
                            dst[c.col(i, j)] = j & 1 ? accC[i * P + j / 2].y : accC[i * P + j / 2].x;
                            dst[p.H + c.col(i, j)] = j & 1 ? accW[i * P + j / 2].y : accW[i * P + j / 2].x;
                        }
                }
            }
        }
    }
}

// The slots of a column: way w of 32 takes the slots w, w + 32, ... in order (8
// of them in flight), the ways meet in a fixed pairwise tree.
__global__ void __launch_bounds__(kFoldCols *kFoldWays) norm_fold(const NormParams p) {
    __shared__ float part[kFoldWays][kFoldCols + 1];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int w = threadIdx.y;
    const int e = blockIdx.x * kFoldCols + threadIdx.x, n = 2 * p.H;
    float v = 0.0f;
    for (int s = w; s < p.n_slots; s += 8 * kFoldWays) {
        uint32_t r[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            r[k] = 0;
            load_if<false>(r[k], p.slots + static_cast<int64_t>(s + k * kFoldWays) * n + e, e < n && s + k * kFoldWays < p.n_slots);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) v = __fadd_rn(v, __uint_as_float(r[k]));
    }
    part[w][threadIdx.x] = v;
    __syncthreads();
#pragma unroll
    for (int s = 1; s < kFoldWays; s <<= 1) {
        if ((w & (2 * s - 1)) == 0) part[w][threadIdx.x] = __fadd_rn(part[w][threadIdx.x], part[w + s][threadIdx.x]);
        __syncthreads();
    }
    if (w != 0 || e >= n) return;
    put_column(p, e, part[0][threadIdx.x]);
}

// Host side -------------------------------------------------------------------

// Elements a thread: 16 from 2048 columns on (or where a warp takes the row),
// 8 below.
struct NormPlan {
    bool warp;
    int ept, threads;
    int slots;
};

NormPlan norm_plan(int64_t T, int64_t H) {
    NormPlan pl{};
    pl.warp = H <= 512;
    pl.ept = (pl.warp ? H > 256 : H > 1024) ? 16 : 8;
    pl.threads = pl.warp ? 32 * kWarpTeams : static_cast<int>(((H + pl.ept - 1) / pl.ept + 31) / 32 * 32);
    const int64_t teams = pl.warp ? kWarpTeams : 1;
    const int64_t most = (!pl.warp && pl.threads <= 128) ? 608 : 304;
    const int64_t want = (T + teams - 1) / teams;
    // up to 2 rows a team: one CTA, whose sums need no second launch (2 x 816 fp32
    // 14.0 us instead of about 16.5; 3 rows of 4096 one after another 19.2)
    pl.slots = static_cast<int>(want <= 2 ? 1 : want < most ? want : most);
    return pl;
}

// FB, BB: CTAs that an SM is to hold, forward and backward (registers and, by
// the ring's depth, shared memory). Few rows streamed at a time suit the memory:
// 16384 x 4096 bf16 forward 89.4 us with 2 CTAs an SM, 100.5 with 3, 125.8 with
// 1; 32768 x 2048 88.5 us with 3, 98.9 with 4, 118.5 with 2; 65536 x 1024 90.2 us
// with 6, 97.4 with 5, 102 with 12. Backward 65536 x 1024 140 us with room for
// 6, 151 with 4; 16384 x 4096 134 us with 2, 176 with 1.
template <typename T, int VEC, int EPT, int MAXT, int FB, int BB, bool WARP>
dgr_status launch_norm(bool backward, NormParams &p, const NormPlan &pl, int sms, cudaStream_t s) {
    constexpr int NV = EPT / VEC;
    constexpr bool ring = VEC * sizeof(T) >= 4;
    const size_t row = ring ? static_cast<size_t>(MAXT) * EPT * sizeof(T) * (backward ? 4 : 2) : 0;
    const size_t room = (224 * 1024) / (backward ? BB : FB);
    p.depth = 0;
    if (ring) p.depth = static_cast<int>(room / (row + 1 - ring) < 3 ? room / (row + 1 - ring) : 3);  // 0 where one does not fit
    // no more than the rows that a CTA has
    const int64_t teams = WARP ? kWarpTeams : 1, ctas = backward ? pl.slots : static_cast<int64_t>(sms) * FB;
    const int64_t rows = (p.T + teams * ctas - 1) / (teams * ctas);
    if (rows < p.depth) p.depth = static_cast<int>(rows);
    size_t smem = row * p.depth;
    if (!backward) {
        auto *k = norm_forward<T, VEC, NV, MAXT, FB, WARP>;
        const dgr_status st = allow_smem(k, smem, room);
        if (st != DGR_OK) return st;
        const int64_t want = (p.T + teams - 1) / teams, most = static_cast<int64_t>(sms) * FB;
        k<<<sched_grid(static_cast<unsigned>(want < most ? want : most)), pl.threads, smem, s>>>(p);
        return launch_status();
    }
    const size_t cols = WARP ? static_cast<size_t>(kWarpTeams) * 2 * p.H * 4 : 0;  // at most 32 KB
    if (smem < cols) smem = cols;
    auto *k = norm_backward<T, VEC, NV, MAXT, BB, WARP>;
    const dgr_status st = allow_smem(k, smem, room);
    if (st != DGR_OK) return st;
    k<<<sched_grid(static_cast<unsigned>(pl.slots)), pl.threads, smem, s>>>(p);
    return launch_status();
}

template <typename T, int VEC>
dgr_status launch_width(bool backward, NormParams &p, const NormPlan &pl, int sms, cudaStream_t s) {
    if (pl.warp)
        return pl.ept == 8 ? launch_norm<T, VEC, 8, 256, 4, 2, true>(backward, p, pl, sms, s)
                           : launch_norm<T, VEC, 16, 256, 2, 2, true>(backward, p, pl, sms, s);
    if (pl.ept == 8) return launch_norm<T, VEC, 8, 128, 6, 6, false>(backward, p, pl, sms, s);
    if (pl.threads <= 128) return launch_norm<T, VEC, 16, 128, 3, 4, false>(backward, p, pl, sms, s);
    if (pl.threads <= 256) return launch_norm<T, VEC, 16, 256, 2, 2, false>(backward, p, pl, sms, s);
    if (pl.threads <= 512) return launch_norm<T, VEC, 16, 512, 1, 1, false>(backward, p, pl, sms, s);
    return launch_norm<T, VEC, 16, 1024, 1, 1, false>(backward, p, pl, sms, s);
}

// The widest vector that every row's start allows: 16 bytes, 4, or one bf16.
template <typename T>
dgr_status launch_type(bool backward, NormParams &p, const NormPlan &pl, int sms, cudaStream_t s, size_t align) {
    constexpr int full = 16 / static_cast<int>(sizeof(T)), word = 4 / static_cast<int>(sizeof(T));
    if (align >= 16 && p.H % full == 0) return launch_width<T, full>(backward, p, pl, sms, s);
    if constexpr (sizeof(T) == 2) {
        if (align < 4 || p.H % word != 0) return launch_width<T, 1>(backward, p, pl, sms, s);
    }
    return launch_width<T, word>(backward, p, pl, sms, s);
}

// The power of two (at most 16) that divides every row's address.
size_t row_align(size_t a, const void *base, int64_t ld, int es) {
    if (!base) return a;
    const uintptr_t v = reinterpret_cast<uintptr_t>(base) | static_cast<uintptr_t>(ld * es);
    while (a > 1 && v % a) a >>= 1;
    return a;
}

size_t extent(int64_t T, int64_t H, int64_t ld, int es) { return T > 0 && H > 0 ? static_cast<size_t>(((T - 1) * ld + H) * es) : 0; }

}  // namespace
}  // namespace dgr

using namespace dgr;

extern "C" size_t dgr_block_norm_workspace_bytes(int64_t T, int64_t H) {
    if (T < 0 || T > INT32_MAX || H < 1 || H > kMaxWidth) return 0;
    return sizeof(WsHeader) + align_up(static_cast<size_t>(norm_plan(T, H).slots) * 2 * H * 4);
}

extern "C" dgr_status dgr_block_norm(const void *x, int64_t ld_x, const void *y, int64_t ld_y, int32_t dtype, int64_t T,
                                     int64_t H, const void *w_post, const void *gate, int32_t gate_mode,
                                     const void *w_pre, int32_t w_dtype, float res_scale, float eps, void *h,
                                     int64_t ld_h, void *u, int64_t ld_u, void *stream) {
    if ((dtype != DGR_DTYPE_BF16 && dtype != DGR_DTYPE_F32) || (w_dtype != DGR_DTYPE_BF16 && w_dtype != DGR_DTYPE_F32))
        return DGR_ERR_INVALID_ARG;
    if (T < 0 || H < 1 || !(eps >= 0.0f) || gate_mode < kGateNone || gate_mode > kGateToken) return DGR_ERR_INVALID_ARG;
    if (T == 0) return check_device();  // no rows: row pointers may be null
    if ((gate_mode != kGateNone) != (gate != nullptr) || (w_pre != nullptr) != (u != nullptr)) return DGR_ERR_INVALID_ARG;
    if (!y && (w_post || gate || h || res_scale != 1.0f || !w_pre)) return DGR_ERR_INVALID_ARG;
    if (y && !h) return DGR_ERR_INVALID_ARG;
    if (ld_x < H || (y && (ld_y < H || ld_h < H)) || (u && ld_u < H)) return DGR_ERR_INVALID_ARG;
    if (T > INT32_MAX || H > kMaxWidth) return DGR_ERR_UNSUPPORTED;
    if (!x) return DGR_ERR_INVALID_ARG;
    const int es = dtype == DGR_DTYPE_BF16 ? 2 : 4, ws = w_dtype == DGR_DTYPE_BF16 ? 2 : 4;
    for (const void *q : {x, y, static_cast<const void *>(h), static_cast<const void *>(u)})
        if (!aligned(q, es)) return DGR_ERR_MISALIGNED;
    for (const void *q : {w_post, gate, w_pre})
        if (!aligned(q, ws)) return DGR_ERR_MISALIGNED;
    const size_t bx = extent(T, H, ld_x, es), by = extent(T, H, ld_y, es), bh = extent(T, H, ld_h, es), bu = extent(T, H, ld_u, es);
    const size_t bg = static_cast<size_t>(gate_mode == kGateToken ? T : H) * ws;
    if (ranges_overlap(h, bh, x, bx) && !(h == x && ld_h == ld_x)) return DGR_ERR_ALIAS;
    if (ranges_overlap(h, bh, y, by) || ranges_overlap(h, bh, u, bu) || ranges_overlap(u, bu, x, bx) || ranges_overlap(u, bu, y, by))
        return DGR_ERR_ALIAS;
    const struct { const void *q; size_t n; } params[3] = {{w_post, H * static_cast<size_t>(ws)}, {gate, bg}, {w_pre, H * static_cast<size_t>(ws)}};
    for (const auto &a : params)
        if (ranges_overlap(h, bh, a.q, a.n) || ranges_overlap(u, bu, a.q, a.n)) return DGR_ERR_ALIAS;
    dgr_status st = check_device();
    if (st != DGR_OK) return st;
    NormParams p{};
    p.x = x, p.y = y, p.ld_x = ld_x, p.ld_y = ld_y;
    p.out_h = h, p.out_u = u, p.ld_oh = ld_h, p.ld_ou = ld_u;
    p.w_post = w_post, p.gate = gate, p.w_pre = w_pre, p.w_bf16 = ws == 2, p.gate_mode = gate_mode;
    p.w_vec = aligned(w_post, 16) && aligned(gate, 16) && aligned(w_pre, 16);
    p.T = static_cast<int32_t>(T), p.H = static_cast<int32_t>(H), p.alpha = res_scale, p.eps = eps;
    p.sched = sched_for(static_cast<uint32_t>(T));
    size_t al = row_align(16, x, ld_x, es);
    al = row_align(al, y, ld_y, es);
    al = row_align(al, h, ld_h, es);
    al = row_align(al, u, ld_u, es);
    int sms = 0;
    if ((st = usable_sms(&sms)) != DGR_OK) return st;
    const NormPlan pl = norm_plan(T, H);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return es == 2 ? launch_type<bf16>(false, p, pl, sms, s, al) : launch_type<float>(false, p, pl, sms, s, al);
}

extern "C" dgr_status dgr_block_norm_backward(const void *h, int64_t ld_h, const void *y, int64_t ld_y, const void *dh,
                                              int64_t ld_dh, const void *du, int64_t ld_du, int32_t dtype, int64_t T,
                                              int64_t H, const void *w_post, const void *gate, int32_t gate_mode,
                                              const void *w_pre, int32_t w_dtype, float res_scale, float eps, void *dx,
                                              int64_t ld_dx, void *dy, int64_t ld_dy, float *dw_post, float *dgate,
                                              float *dw_pre, int32_t accumulate, void *ws, size_t ws_bytes, void *stream) {
    if ((dtype != DGR_DTYPE_BF16 && dtype != DGR_DTYPE_F32) || (w_dtype != DGR_DTYPE_BF16 && w_dtype != DGR_DTYPE_F32))
        return DGR_ERR_INVALID_ARG;
    if (T < 0 || H < 1 || !(eps >= 0.0f) || gate_mode < kGateNone || gate_mode > kGateToken) return DGR_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) {  // no rows (their pointers may be null): sums of nothing are +0.0 on overwrite, untouched on accumulate
        const dgr_status st = check_device();
        if (st != DGR_OK || accumulate) return st;
        for (float *w : {dw_post, gate_mode == kGateChannel ? dgate : nullptr, dw_pre})
            if (w && cudaMemsetAsync(w, 0, static_cast<size_t>(H) * 4, s) != cudaSuccess) return DGR_ERR_CUDA;
        return DGR_OK;
    }
    if ((gate_mode != kGateNone) != (gate != nullptr)) return DGR_ERR_INVALID_ARG;
    if ((w_pre != nullptr) != (du != nullptr) || (w_pre && !h) || (!w_pre && !dh) || (!w_pre && dw_pre)) return DGR_ERR_INVALID_ARG;
    if (!y && (w_post || gate || dy || res_scale != 1.0f || !w_pre)) return DGR_ERR_INVALID_ARG;
    if ((y && !dy) || !dx || (dw_post && !w_post) || (dgate && !gate)) return DGR_ERR_INVALID_ARG;
    if ((w_pre && (ld_h < H || ld_du < H)) || (y && (ld_y < H || ld_dy < H)) || (dh && ld_dh < H) || ld_dx < H)
        return DGR_ERR_INVALID_ARG;
    if (T > INT32_MAX || H > kMaxWidth) return DGR_ERR_UNSUPPORTED;
    const int es = dtype == DGR_DTYPE_BF16 ? 2 : 4, wes = w_dtype == DGR_DTYPE_BF16 ? 2 : 4;
    for (const void *q : {w_pre ? h : nullptr, y, dh, du, static_cast<const void *>(dx), static_cast<const void *>(dy)})
        if (!aligned(q, es)) return DGR_ERR_MISALIGNED;
    for (const void *q : {w_post, gate, w_pre})
        if (!aligned(q, wes)) return DGR_ERR_MISALIGNED;
    for (const void *q : {dw_post, dgate, dw_pre})
        if (!aligned(q, 4)) return DGR_ERR_MISALIGNED;
    const size_t need = dgr_block_norm_workspace_bytes(T, H);
    if (!ws) return DGR_ERR_INVALID_ARG;
    if (ws_bytes < need) return DGR_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned(ws, kAlign)) return DGR_ERR_MISALIGNED;
    struct Range { const void *q; size_t n; };
    const size_t hb = static_cast<size_t>(H);
    const size_t gn = gate_mode == kGateToken ? static_cast<size_t>(T) : hb;
    const Range ins[] = {{w_pre ? h : nullptr, extent(T, H, ld_h, es)}, {y, extent(T, H, ld_y, es)}, {dh, extent(T, H, ld_dh, es)},
                         {du, extent(T, H, ld_du, es)}, {w_post, hb * wes}, {gate, gn * wes}, {w_pre, hb * wes}};
    const Range outs[] = {{dx, extent(T, H, ld_dx, es)}, {dy, extent(T, H, ld_dy, es)}, {dw_post, hb * 4}, {dgate, gn * 4},
                          {dw_pre, hb * 4}, {ws, need}};
    for (const Range &o : outs) {
        for (const Range &i : ins)
            if (ranges_overlap(o.q, o.n, i.q, i.n) && !(o.q == dx && i.q == dh && dx == dh && ld_dx == ld_dh)) return DGR_ERR_ALIAS;
        for (const Range &b : outs)
            if (&o < &b && ranges_overlap(o.q, o.n, b.q, b.n)) return DGR_ERR_ALIAS;
    }
    dgr_status st = check_device();
    if (st != DGR_OK) return st;
    NormParams p{};
    p.h = w_pre ? h : nullptr, p.y = y, p.dh = dh, p.du = du;
    p.ld_h = ld_h, p.ld_y = ld_y, p.ld_dh = ld_dh, p.ld_du = ld_du;
    p.out_h = dx, p.out_u = dy, p.ld_oh = ld_dx, p.ld_ou = ld_dy;
    p.w_post = w_post, p.gate = gate, p.w_pre = w_pre, p.w_bf16 = wes == 2, p.gate_mode = gate_mode;
    p.w_vec = aligned(w_post, 16) && aligned(gate, 16) && aligned(w_pre, 16);
    p.T = static_cast<int32_t>(T), p.H = static_cast<int32_t>(H), p.alpha = res_scale, p.eps = eps;
    p.dw_post = dw_post, p.dgate = dgate, p.dw_pre = dw_pre, p.accumulate = accumulate ? 1 : 0;
    const NormPlan pl = norm_plan(T, H);
    p.n_slots = pl.slots;
    p.slots = reinterpret_cast<float *>(static_cast<char *>(ws) + sizeof(WsHeader));
    p.sched = sched_for(static_cast<uint32_t>(pl.slots));
    size_t al = 16;
    if (w_pre) al = row_align(al, h, ld_h, es);
    al = row_align(al, y, ld_y, es);
    al = row_align(al, dh, ld_dh, es);
    al = row_align(al, du, ld_du, es);
    al = row_align(al, dx, ld_dx, es);
    al = row_align(al, dy, ld_dy, es);
    st = es == 2 ? launch_type<bf16>(true, p, pl, 0, s, al) : launch_type<float>(true, p, pl, 0, s, al);
    if (st != DGR_OK || pl.slots == 1 || (!dw_post && !dw_pre && !(dgate && gate_mode == kGateChannel))) return st;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>((2 * H + kFoldCols - 1) / kFoldCols));
    cfg.blockDim = dim3(kFoldCols, kFoldWays);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_fold, p) == cudaSuccess ? DGR_OK : DGR_ERR_CUDA;
}
