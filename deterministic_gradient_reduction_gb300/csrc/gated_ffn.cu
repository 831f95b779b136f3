// Gated feed-forward of grouped experts, forward and backward.
//
// The rows d_offs[e] .. d_offs[e+1]-1 of x belong to expert e:
//   a = x Wg_e^T,  b = x Wu_e^T,  h = act(a) b            (a, b in binary32, h rounded once);
//   da = dh b act'(a),  db = dh act(a),  dx = da Wg_e + db Wu_e.
// Both activations are v sigmoid(s(v)): silu with s(v) = v, the tanh form of
// gelu with s(v) = 2 sqrt(2 / pi) (v + 0.044715 v^3), as (1 + tanh u) / 2 =
// sigmoid(2 u); written so, nothing cancels for small v.
//
// Forward, one launch: a persistent kernel, 12 warps a CTA, one CTA per SM. A tile
// is, for calls with many rows, 256 rows of one expert (counted from its first row)
// by 256 columns of the product, shared by a pair of CTAs (cta_group::2: each loads
// half of either operand); for few rows 128 rows and a single CTA, as many columns as
// waste least of the last wave (choose). The columns are half rows of Wg_e, half rows
// of Wu_e, one after another in shared memory, so a and b of an element end in the
// same lane of TMEM, and the epilogue has both. Warp 0 loads 64-deep stages by TMA (x
// and the weights K-major as they lie, 128-byte swizzle; what is past a matrix's end
// comes as zeros), warp 1 issues tcgen05.mma into one of two accumulators, warps
// 4-11 (lane quarter q, column half) read one while the other fills.
// Backward: da and db element by element (memory bound), and dx by the same
// kernel with the two parts of its sum, da Wg_e and db Wu_e, one after another
// along K in one accumulator (weights N-major as they lie). Where dx is bound by
// its products, warps of that kernel with nothing else to do make da and db, the
// loads of a tile wait for its rows' counters, and the elements' traffic goes on
// under the products; else two launches. The gradients of the weights are
// dgr_grouped_wgrad_accumulate's.
//
// Bound by the tensor cores, and over seconds by the power that these take: 32768 rows,
// 2048 x 4096, 8 experts, forward 587 us in a burst (1.87 PFLOP/s, 0.97 of the measured
// rate), with a and b kept and over seconds 710 (1.55, 0.89 of the sustained rate).
// Backward 720 in a burst, 823 over seconds; as two launches 884. Few rows are bound by
// reading the weights: 1 x 4096 x 8192 in 28 us (4.8 TB/s), 38 with cold caches; a
// kernel that only reads them takes 23, and 28 with cold caches.
//
// da and db are rounded to bf16 before they are multiplied, as they are stored: beside
// bf16 weights a tensor-core operand has no wider form, and two bf16 terms for each
// would be twice the products. dx is 0.0023 of its size off 64 bits for it; with da and
// db in 32 bits its own rounding alone would leave 0.0017.
//
// Rows of a tile past the expert's end are another expert's (or zeros): a row of
// the product depends on its own row of x alone, and they are not written.
// Deterministic: K in ascending order into one accumulator, one writer an element.
// Every wait is bounded; a timeout aborts the CTA, which then waits (bounded
// again) for its copies in flight and for its MMAs before it frees its TMEM.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "row_common.cuh"
#include "tc_common.cuh"

namespace dgr {
namespace {

using namespace tc;

constexpr int BM = 128;  // rows of a tile (TMEM lanes)
constexpr int BK = 64;   // k per stage: one 128-byte row of a swizzle atom
constexpr int kEpiWarps = 8;
constexpr int kThreads = (4 + kEpiWarps) * 32;
constexpr int kPreWarps = 6;  // of a CTA that makes da and db too: warps 2, 3 and four behind the epilogue's
constexpr int kReadyRows = 32;  // rows of da and db that one counter stands for
constexpr uint64_t kStageNs = 390;  // of a pair's tile, as measured (choose)
constexpr int kMaxExperts = 1024;
constexpr uint32_t kStageA = BM * 128;
constexpr uint32_t kRing = 192 * 1024;  // stages, beside 4 KB of offsets and the barriers
constexpr uint32_t kSBO = 1024;         // between 8-row groups of an atom
constexpr uint32_t kLboK = 16;          // K-major: one atom spans the K16 step
constexpr uint32_t kLboN = 64 * 128;    // N-major: between 64-wide atoms along n

enum { kSilu = 0, kGelu = 1 };

// CG CTAs share a tile of CG * 128 rows. Pairs have 256 columns of the product;
// a single CTA's width goes by the call (Tiles, below).
constexpr int kMaxStages = 24;
constexpr int kMaxN = 256;  // columns of the product a tile: half of TMEM
// tcgen05 instruction descriptor: fp32 D, bf16 A and B, A K-major, B K-major or (bit 16) N-major
__host__ __device__ constexpr uint32_t idesc(int m, int n, bool n_major) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (n_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

// How a call is cut into tiles and stages.
struct Tiles {
    int32_t cols;    // columns of the output a tile
    int32_t nbs;     // column blocks
    int32_t box;     // rows of x (or da, db) in one copy: 8, 32 or 128
    int32_t room;    // rows of x that a stage has room for
    int32_t stages;  // slots of the ring
};

struct Ctl {
    uint64_t full[kMaxStages];
    uint64_t empty[kMaxStages];
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint32_t tmem_base;
    int abort;
};

constexpr uint32_t kBox = 32 * 64;  // an epilogue warp's block of 32 x 32 bf16
constexpr size_t kSmem = 1024 + kRing + kEpiWarps * kBox + sizeof(Ctl);

// Maps over the outputs, for whole blocks of 32 rows by 32 columns (h, a, b; or dx).
struct Outputs {
    CUtensorMap out, gate, up;
};

struct FfnParams {
    const int64_t *offs;  // or null: one expert with all rows
    int32_t E, T;
    int32_t K;            // of one part (forward: H, backward: F)
    int32_t N;            // columns of the output (forward: F, backward: H)
    Tiles cut;
    uint16_t *out, *gate, *up;  // forward: h and, or null, a and b; backward: dx
    int64_t ld_out, ld_gate, ld_up;
    WsHeader *hdr;
    Sched sched;  // the setting; bound to the tile count on the device
};

// mb_base[e] = first row block of expert e (mb_base[E] = all row blocks), by the
// whole block; false when the offsets break the contract.
__device__ bool row_blocks(const FfnParams &p, int rows, int32_t *mb_base, int32_t *wsum, int32_t *bad) {
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, nt = blockDim.x, nw = nt >> 5;
    if (!p.offs) {
        if (tid == 0) mb_base[0] = 0, mb_base[1] = (p.T + rows - 1) / rows;
        __syncthreads();
        return true;
    }
    if (tid == 0) *bad = 0;
    __syncthreads();
    int32_t run = 0;
    for (int e0 = 0; e0 < p.E; e0 += nt) {
        const int e = e0 + tid;
        int32_t c = 0;
        if (e < p.E) {
            const int64_t a = p.offs[e], b = p.offs[e + 1];
            if (a < 0 || b < a || b > p.T || (e == 0 && a != 0) || (e == p.E - 1 && b != p.T)) *bad = 1;
            else c = static_cast<int32_t>((b - a + rows - 1) / rows);
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
        if (e < p.E) mb_base[e] = before + incl - c;
        for (int v = 0; v < nw; ++v) run += wsum[v];
        __syncthreads();
    }
    if (tid == 0) mb_base[p.E] = run;
    __syncthreads();
    return *bad == 0;
}

struct Tile {
    int e, nb;
    int32_t row, end;  // first row; the expert's end
};

// tile tau: row blocks expert by expert, the column blocks of one after another
__device__ __forceinline__ Tile tile_of(const FfnParams &p, int rows, const int32_t *mb_base, uint32_t tau) {
    const int32_t gmb = static_cast<int32_t>(tau / static_cast<uint32_t>(p.cut.nbs));
    Tile t;
    t.nb = static_cast<int>(tau - static_cast<uint32_t>(gmb) * static_cast<uint32_t>(p.cut.nbs));
    int lo = 0, hi = p.E - 1;
    while (lo < hi) {  // the last expert that starts at or before gmb (empty ones start where the next does)
        const int mid = (lo + hi + 1) >> 1;
        if (mb_base[mid] <= gmb) lo = mid;
        else hi = mid - 1;
    }
    t.e = lo;
    t.row = (p.offs ? static_cast<int32_t>(p.offs[lo]) : 0) + (gmb - mb_base[lo]) * rows;
    t.end = p.offs ? static_cast<int32_t>(p.offs[lo + 1]) : p.T;
    return t;
}

__device__ __forceinline__ float rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// sigmoid(s(v)) = 1 / (1 + 2^(-s log2 e)), two at a time; an exponential beyond
// the range gives 0. Approximations of 2^x and 1 / x are good to a unit or two.
template <int ACT>
__device__ __forceinline__ float2 gate_sigmoid(float2 v) {
    constexpr float kTwice = 1.5957691216057308f;  // 2 sqrt(2 / pi)
    float2 t;
    if (ACT == kSilu) t = mul2(v, row::both(-row::kLog2e));
    else t = mul2(v, row::fma2(mul2(v, v), row::both(-kTwice * 0.044715f * row::kLog2e), row::both(-kTwice * row::kLog2e)));
    const float2 d = row::fma2(make_float2(row::ex2(t.x), row::ex2(t.y)), row::both(1.0f), row::both(1.0f));
    return make_float2(rcp(d.x), rcp(d.y));
}

// 16 bf16 values to columns c .. c + 15 of a row, those below n (a multiple of 8).
__device__ __forceinline__ void store16(uint16_t *to, int c, int n, const float (&v)[16]) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = row::pack2(v[2 * i], v[2 * i + 1]);
    to += c;
    if (c + 16 <= n && (reinterpret_cast<uintptr_t>(to) & 31) == 0) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        if (c + 8 <= n) *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
        if (c + 16 <= n) *reinterpret_cast<uint4 *>(to + 8) = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// A lane's row of 16 values as 16-byte chunks i and i + 1 of its 64 bytes in a 32 x
// 32 block, in the 64-byte swizzle of its map (chunk ^ row / 2 % 4): the lanes of
// a store spread over the banks.
__device__ __forceinline__ void block_row(uint32_t box, int lane, int i, const float (&v)[16]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t to = box + lane * 64 + 16 * ((i + j) ^ (lane >> 1 & 3));
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(row::pack2(v[8 * j], v[8 * j + 1])), "r"(row::pack2(v[8 * j + 2], v[8 * j + 3])),
                     "r"(row::pack2(v[8 * j + 4], v[8 * j + 5])), "r"(row::pack2(v[8 * j + 6], v[8 * j + 7]))
                     : "memory");
    }
}
__device__ __forceinline__ void store_2d(const CUtensorMap *map, uint32_t src, int32_t x, int32_t y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(reinterpret_cast<uint64_t>(map)), "r"(src),
                 "r"(x), "r"(y)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// The thread's committed copies have read their shared memory; are complete.
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// The wait for a load, with its registers taken through (tmem_wait_ld says why).
__device__ __forceinline__ void tmem_wait16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}

// ---- pairs of CTAs (clusters of two: the even one leads) -----------------------

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The leader's copy of a barrier.
__device__ __forceinline__ uint32_t of_leader(const uint64_t *bar) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(bar)));
    return r;
}
__device__ __forceinline__ void arrive_at(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// A copy into this CTA; a pair's reports to the leader's barrier.
template <int CG>
__device__ __forceinline__ void load_3d(uint32_t to, const CUtensorMap *map, uint32_t bar, int32_t x, int32_t y, int32_t z) {
    if constexpr (CG == 1) {
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(to),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
            : "memory");
    } else {
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
            " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(to),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
            : "memory");
    }
}

template <int CG>
__device__ __forceinline__ void mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    if constexpr (CG == 1) {
        mma_bf16(d_tmem, a_desc, b_desc, idesc, accumulate);
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
    }
}
// Arrive on `bar`, of both CTAs of a pair, once every MMA issued so far by this thread is done.
template <int CG>
__device__ __forceinline__ void commit(uint64_t *bar) {
    if constexpr (CG == 1) {
        mma_commit(bar);
    } else {
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
                     "h"(static_cast<uint16_t>(3))
                     : "memory");
    }
}
template <int CG>
__device__ __forceinline__ void alloc_tmem(uint32_t *dst, uint32_t cols) {
    if constexpr (CG == 1) {
        tmem_alloc(dst, cols);
        tmem_relinquish();
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}
template <int CG>
__device__ __forceinline__ void free_tmem(uint32_t taddr, uint32_t cols) {
    if constexpr (CG == 1) tmem_dealloc(taddr, cols);
    else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}
// All threads of the CTA, or of both.
template <int CG>
__device__ __forceinline__ void tile_sync() {
    if constexpr (CG == 1) __syncthreads();
    else cluster_barrier();
}

// ---- da and db ----------------------------------------------------------------

struct PreParams {
    const uint16_t *dh, *gate, *up;
    uint16_t *dgate, *dup;
    int64_t ld_dh, ld_gate, ld_up, ld_dgate, ld_dup;
    int32_t T, vecs;    // 8-element vectors a row
    int32_t rows_item;  // of pre_rows
    int32_t *ready;     // rows written, of each kReadyRows
    int32_t *begun;     // tiles begun
    int32_t *taken;     // shares of pre_rows taken
    int32_t nbs, lead;  // tiles a row block; rows of da and db ahead of the tiles (0: any)
    uint64_t lead_ns;   // that they wait for the tiles at most
};

// da = dh b act'(a), db = dh act(a); act'(v) = g + v g (1 - g) s'(v), g = sigmoid(s(v)).
// g (1 - g) is 0 long before s'(v) leaves the range, so their product counts as 0 then.
template <int ACT>
__device__ __forceinline__ void pre_grad(float2 dh, float2 a, float2 b, float2 &da, float2 &db) {
    const float2 g = gate_sigmoid<ACT>(a), down = mul2(g, row::fma2(g, row::both(-1.0f), row::both(1.0f)));
    float2 turn = down;
    if (ACT == kGelu) {
        constexpr double kTwice = 1.5957691216057308;  // s'(a) = 2 sqrt(2 / pi) (1 + 3 0.044715 a^2)
        const float2 s = row::fma2(mul2(row::both(static_cast<float>(kTwice * 3 * 0.044715)), a), a, row::both(static_cast<float>(kTwice)));
        turn = make_float2(down.x > 0.0f ? __fmul_rn(down.x, s.x) : down.x, down.y > 0.0f ? __fmul_rn(down.y, s.y) : down.y);
    }
    db = mul2(dh, mul2(a, g));
    da = mul2(mul2(dh, b), row::fma2(a, turn, g));
}

// Eight elements of da and db from vector c of row t.
template <int ACT>
struct PreVec {
    uint4 d, a, b;
    __device__ __forceinline__ void load(const PreParams &p, int64_t t, int c, bool on) {
        d = a = b = make_uint4(0, 0, 0, 0);
        row::load_if<false>(d, p.dh + t * p.ld_dh + c, on);
        row::load_if<false>(a, p.gate + t * p.ld_gate + c, on);
        row::load_if<false>(b, p.up + t * p.ld_up + c, on);
    }
    __device__ __forceinline__ void store(const PreParams &p, int64_t t, int c) const {
        float x[8], y[8], z[8], da[8], db[8];
        row::unpack<row::bf16, 8>(d, x);
        row::unpack<row::bf16, 8>(a, y);
        row::unpack<row::bf16, 8>(b, z);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            float2 u, v;
            pre_grad<ACT>(make_float2(x[j], x[j + 1]), make_float2(y[j], y[j + 1]), make_float2(z[j], z[j + 1]), u, v);
            da[j] = u.x, da[j + 1] = u.y, db[j] = v.x, db[j + 1] = v.y;
        }
        *reinterpret_cast<uint4 *>(p.dgate + t * p.ld_dgate + c) = row::pack<row::bf16, 8>(da);
        *reinterpret_cast<uint4 *>(p.dup + t * p.ld_dup + c) = row::pack<row::bf16, 8>(db);
    }
};

// da and db by the spare warps of the kernel that multiplies them: rows in
// ascending order, a few of them (rows_item, a divisor of kReadyRows) a warp at a
// time, over all CTAs; each adds its rows to their counter when they are written. A
// share of the rows belongs to the warp that takes it, and who is done takes another:
// no tile waits for a CTA that has no SM yet (another call's CTAs may have the other
// SMs, and wait for theirs).
__device__ __forceinline__ int take(int32_t *from, int lane) {
    const int n = lane == 0 ? atomicAdd(from, 1) : 0;
    return __shfl_sync(0xffffffffu, n, 0);
}
template <int ACT>
__device__ __forceinline__ void pre_rows(const PreParams &p, int lane) {
    constexpr int U = 4;
    const int items = (p.T + p.rows_item - 1) / p.rows_item;
    int64_t limit = p.lead ? p.lead : INT64_MAX;  // rows that may be made by now
    const int shares = kPreWarps * static_cast<int>(gridDim.x);
    for (int share = take(p.taken, lane); share < shares; share = take(p.taken, lane)) {
        for (int i = share; i < items; i += shares) {
            const int64_t t0 = static_cast<int64_t>(i) * p.rows_item;
            // no further ahead of the tiles than L2 holds. All pairs begin their tiles a tile's
            // time apart at most; CTAs without an SM (another stream's kernel has it) begin none,
            // so the wait ends, and then there is none again: to be early is no error (on 120 of
            // 152 SMs 32768 rows of 2048 x 4096 took 5.1 ms with a limit of 5 ms)
            if (t0 >= limit) {
                const int64_t blocks = (t0 - p.lead) / (2 * BM) + 1;
                int there = 1;
                const int32_t tiles = static_cast<int32_t>(blocks * p.nbs < INT32_MAX ? blocks * p.nbs : INT32_MAX);
                if (lane == 0) there = wait_counter_geq(p.begun, tiles, p.lead_ns);
                there = __shfl_sync(0xffffffffu, there, 0);
                limit = there ? blocks * (2 * BM) + p.lead : INT64_MAX;
            }
            const int rows = min(p.rows_item, static_cast<int>(p.T - t0)), n = rows * p.vecs;
            for (int v = lane; v < n; v += 32 * U) {
                PreVec<ACT> x[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int w = v + 32 * u, r = w / p.vecs;
                    x[u].load(p, t0 + r, (w - r * p.vecs) * 8, w < n);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int w = v + 32 * u, r = w / p.vecs;
                    if (w < n) x[u].store(p, t0 + r, (w - r * p.vecs) * 8);
                }
            }
            // seen by the copy engines of all SMs before the count is
            asm volatile("fence.proxy.async;" ::: "memory");
            __threadfence();
            __syncwarp();
            if (lane == 0) asm volatile("red.release.gpu.global.add.s32 [%0], %1;" ::"l"(p.ready + t0 / kReadyRows), "r"(rows) : "memory");
        }
    }
}

// Until the rows [first, end) of da and db are written (bounded); by a whole warp.
__device__ __forceinline__ bool wait_rows(const PreParams &p, int32_t first, int32_t end, int lane, volatile int *abort_flag, WsHeader *hdr) {
    bool ok = true;
    for (int g = first / kReadyRows + lane; g * kReadyRows < end && ok; g += 32) {
        const int32_t want = min(kReadyRows, p.T - g * kReadyRows);
        if (!wait_counter_geq(p.ready + g, want)) {
            record_error(hdr, DGR_ERR_TIMEOUT, 405);
            *abort_flag = 1;
            ok = false;
        }
    }
    ok = __all_sync(0xffffffffu, ok);
    // the lanes' readings of the counters come before lane 0's copies: the warp's barrier
    // orders memory between lanes (a vote does not), the fence behind it the copy engine
    __syncwarp();
    asm volatile("fence.proxy.async;" ::: "memory");
    return ok;
}

template <int ACT>
__global__ void __launch_bounds__(256) ffn_pre_grad(const PreParams p) {
    const int64_t n = static_cast<int64_t>(p.T) * p.vecs;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t t = i / p.vecs;
        const int c = static_cast<int>(i - t * p.vecs) * 8;
        PreVec<ACT> x;
        x.load(p, t, c, true);
        x.store(p, t, c);
    }
}

// FWD: a, b and h; else dx. Maps: A (and A2, the second part's), B and B2
// (forward Wg and Wu, FT rows a box; backward the same, 64 x 64 atoms).
// PRE: da and db are made here too.
template <int CG, bool FWD, int ACT, bool PRE>
__global__ void __launch_bounds__(kThreads + (PRE ? (kPreWarps - 2) * 32 : 0), 1)
    ffn_gemm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA2,
             const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmB2,
             const __grid_constant__ Outputs outs, const FfnParams p, const PreParams pre) {
    constexpr int kRows = CG * BM;
    const int cols = CG == 2 ? (FWD ? kMaxN / 2 : kMaxN) : p.cut.cols;  // columns of the output a tile
    const int width = FWD ? 2 * cols : cols;                            // of the product
    const uint32_t stage_b = static_cast<uint32_t>(width / CG) * 128u;
    // a call of few rows: a stage has room for those, so there are more stages (1 x 4096 x
    // 8192 cold 40 -> 38 us); what the MMAs read as the others are bytes of the ring behind
    // them, and those rows' products are not written
    const uint32_t stage_a = CG == 2 ? kStageA : static_cast<uint32_t>(p.cut.room) * 128u, stage_bytes = stage_a + stage_b;
    const uint32_t stages = CG == 2 ? kRing / (kStageA + kMaxN / 2 * 128) : static_cast<uint32_t>(p.cut.stages);
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Ctl *ctl = reinterpret_cast<Ctl *>(smem + kRing + kEpiWarps * kBox);
    __shared__ int32_t mb_base[kMaxExperts + 1];
    __shared__ int32_t wsum[kThreads / 32 + 4];
    __shared__ int32_t bad;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = CG == 1 ? 0 : static_cast<int>(cluster_rank());
    const uint32_t first = blockIdx.x / CG, step = gridDim.x / CG;  // tiles of this CTA or pair
    volatile int *abort_flag = &ctl->abort;

    if (!row_blocks(p, kRows, mb_base, wsum, &bad)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) record_error(p.hdr, DGR_ERR_INVALID_ARG, 400);
        return;
    }
    const uint32_t n_tiles = static_cast<uint32_t>(mb_base[p.E]) * static_cast<uint32_t>(p.cut.nbs);
    const Sched sched = sched_over(p.sched, n_tiles);
    const int part_k = (p.K + BK - 1) / BK;  // stages of one part
    const int n_k = FWD ? part_k : 2 * part_k;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxStages; ++s) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ctl->tfull[b], 1);
            mbar_init(&ctl->tempty[b], CG * kEpiWarps);
        }
        ctl->abort = 0;
        fence_mbar_init();
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
        prefetch_tmap(&tmB2);
        if (!FWD) prefetch_tmap(&tmA2);
    }
    if (warp == 1) {
        alloc_tmem<CG>(&ctl->tmem_base, 2 * kMaxN);
    }
    tc_fence_before();
    tile_sync<CG>();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;

    if (warp == 0) {
        // ---------------- TMA producer ----------------
        // one lane; where rows have to be waited for, the others help to watch them
        if (PRE || lane == 0) {
            uint32_t stage = 0, phase = 0, issued = 0;
            uint32_t at = smem_u32(smem);  // the stage's
            bool ok = true;
            for (uint32_t tau = first; ok && tau < n_tiles; tau += step) {
                const Tile t = tile_of(p, kRows, mb_base, sched_item(sched, tau));
                // few rows: only the copies that hold some of the tile's
                const int boxes = p.cut.box == BM ? 1 : (min(t.end - t.row, BM) + p.cut.box - 1) / p.cut.box;
                const uint32_t bytes = CG * (static_cast<uint32_t>(boxes * p.cut.box) * 128u + stage_b);
                const int32_t row0 = t.row + rank * BM, col0 = t.nb * cols + (FWD ? 0 : rank * (cols / CG));
                if (PRE) {
                    if (rank == 0 && lane == 0) atomicAdd(pre.begun, 1);
                    ok = wait_rows(pre, row0, min(row0 + BM, t.end), lane, abort_flag, p.hdr);
                }
                for (int kb = 0; ok && lane == 0 && kb < n_k; ++kb) {
                    if (!mbar_wait(&ctl->empty[stage], phase ^ 1, abort_flag, p.hdr, 401)) {
                        ok = false;
                        break;
                    }
                    uint64_t *full = &ctl->full[stage];
                    if (rank == 0) mbar_arrive_expect_tx(full, bytes);
                    ++issued;
                    const uint32_t bar = CG == 1 ? smem_u32(full) : of_leader(full), sB = at + stage_a;
                    auto load = [&](uint32_t to, const CUtensorMap *map, int32_t x, int32_t y, int32_t z) { load_3d<CG>(to, map, bar, x, y, z); };
                    // a pair's CTAs have 128 of its rows each and half of its columns
                    if (FWD) {
                        load(at, &tmA, kb * BK, row0, 0);
                        for (int b = 1; b < boxes; ++b) load(at + b * p.cut.box * 128, &tmA, kb * BK, row0 + b * p.cut.box, 0);
                        if (CG == 1) {
                            load(sB, &tmB, kb * BK, col0, t.e);
                            load(sB + cols * 128, &tmB2, kb * BK, col0, t.e);
                        } else {
                            load(sB, rank ? &tmB2 : &tmB, kb * BK, col0, t.e);
                        }
                    } else {
                        const bool second = kb >= part_k;
                        const int k0 = (second ? kb - part_k : kb) * BK;
                        load(at, second ? &tmA2 : &tmA, k0, row0, 0);
                        for (int b = 1; b < boxes; ++b) load(at + b * p.cut.box * 128, second ? &tmA2 : &tmA, k0, row0 + b * p.cut.box, 0);
                        for (int j = 0; j < cols / CG / 64; ++j) load(sB + j * kLboN, second ? &tmB2 : &tmB, col0 + 64 * j, k0, t.e);
                    }
                    at += stage_bytes;
                    if (++stage == stages) {
                        stage = 0;
                        at = smem_u32(smem);
                        phase ^= 1;
                    }
                }
                if (PRE) ok = __shfl_sync(0xffffffffu, ok, 0);  // the lanes leave together
            }
            if (!ok && rank == 0 && lane == 0) {  // aborted: let the copies in flight land (bounded) before the CTA, or the pair, exits
                int dummy = 0;
                for (uint32_t i = 0; i < stages && i < issued; ++i) {  // the latest use of each stage, backwards
                    phase ^= stage == 0;
                    stage = (stage == 0 ? stages : stage) - 1;
                    mbar_wait(&ctl->full[stage], phase, &dummy, nullptr, kWaitLimitNs);
                }
            }
        }
    } else if (warp == 1 && rank == 0) {
        // ---------------- MMA issuer ----------------
        // one lane, descriptors by addition: a stage's instructions, at four or five cycles
        // each, were near to what its MMAs take (32768 rows of 2048 x 4096 598 us, so 587)
        if (lane == 0) {
            const uint32_t desc = idesc(kRows, width, !FWD);
            const uint64_t a_desc = smem_desc_sw128(smem_u32(smem), kLboK, kSBO);
            const uint64_t b_desc = smem_desc_sw128(smem_u32(smem) + stage_a, FWD ? kLboK : kLboN, kSBO);
            constexpr uint32_t kStepA = 32 >> 4, kStepB = (FWD ? 32 : 2048) >> 4;  // a K16 step in a descriptor's address
            uint32_t stage = 0, phase = 0, g = 0, at = 0;  // at: the stage's, likewise
            uint32_t last_stage = 0, last_phase = 0;       // the latest stage-release commit
            bool committed = false, ok = true;
            for (uint32_t tau = first; ok && tau < n_tiles; tau += step, ++g) {
                const uint32_t buf = g & 1, tph = (g >> 1) & 1;
                if (!mbar_wait(&ctl->tempty[buf], tph ^ 1, abort_flag, p.hdr, 402)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem + buf * kMaxN;
                for (int kb = 0; kb < n_k; ++kb) {
                    if (!mbar_wait(&ctl->full[stage], phase, abort_flag, p.hdr, 403)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = a_desc + at, bd = b_desc + at;
                    mma<CG>(d_tmem, ad, bd, desc, kb > 0 ? 1u : 0u);
                    mma<CG>(d_tmem, ad + kStepA, bd + kStepB, desc, 1u);
                    mma<CG>(d_tmem, ad + 2 * kStepA, bd + 2 * kStepB, desc, 1u);
                    mma<CG>(d_tmem, ad + 3 * kStepA, bd + 3 * kStepB, desc, 1u);
                    commit<CG>(&ctl->empty[stage]);
                    committed = true;
                    last_stage = stage;
                    last_phase = phase;
                    at += stage_bytes >> 4;
                    if (++stage == stages) {
                        stage = at = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
                commit<CG>(&ctl->tfull[buf]);
            }
            if (!ok && committed) {
                // aborted: wait (bounded) until the MMAs issued here are done, as
                // their latest commit says, before the CTA frees its TMEM and exits
                int dummy = 0;
                mbar_wait(&ctl->empty[last_stage], last_phase, &dummy, nullptr, kWaitLimitNs);
            }
        }
    } else if (PRE && (warp == 2 || warp == 3 || warp >= 4 + kEpiWarps)) {
        // ---------------- da and db ----------------
        pre_rows<ACT>(pre, lane);
    } else if (warp >= 4) {
        // ---------------- epilogue ----------------
        const int q = warp & 3;         // TMEM lane quarter this warp may access
        const int half = (warp - 4) >> 2;
        const uint32_t box = smem_u32(smem + kRing) + (warp - 4) * kBox;
        uint32_t g = 0;
        for (uint32_t tau = first; tau < n_tiles; tau += step, ++g) {
            const Tile t = tile_of(p, kRows, mb_base, sched_item(sched, tau));
            const int32_t row = t.row + rank * BM + 32 * q + lane;
            const bool mine = row < t.end;
            const uint32_t buf = g & 1, tph = (g >> 1) & 1;
            if (!mbar_wait(&ctl->tfull[buf], tph, abort_flag, p.hdr, 404)) break;
            tc_fence_after();
            const uint32_t base = tmem + (static_cast<uint32_t>(32 * q) << 16) + buf * kMaxN;
            const int c_tile = t.nb * cols, c_end = min(c_tile + cols, p.N);
            // products to outputs, 16 columns from c on
            auto finish = [&](const uint32_t (&ra)[16], const uint32_t (&rb)[16], float (&h)[16]) {
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float2 a = make_float2(__uint_as_float(ra[i]), __uint_as_float(ra[i + 1]));
                    const float2 b = make_float2(__uint_as_float(rb[i]), __uint_as_float(rb[i + 1]));
                    const float2 v = mul2(mul2(a, gate_sigmoid<ACT>(a)), b);
                    h[i] = v.x, h[i + 1] = v.y;
                }
            };
            auto floats = [](const uint32_t (&r)[16], float (&f)[16]) {
#pragma unroll
                for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(r[i]);
            };
            if (CG == 2 && t.row + rank * BM + 32 * q + 32 <= t.end) {
                // a whole block of rows: 32 x 32 values through shared memory and the copy
                // engine. Stores from the lanes (32 bytes a row each) are many more requests
                // beside the loads: 32768 rows of 2048 x 4096 741 us, so 725
                auto send = [&](const CUtensorMap *map, const float (&v0)[16], const float (&v1)[16], int c) {
                    if (lane == 0) bulk_wait_read();
                    __syncwarp();
                    block_row(box, lane, 0, v0);
                    block_row(box, lane, 2, v1);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        store_2d(map, box, c_tile + c, row - lane);
                        bulk_commit();
                    }
                };
#pragma unroll 1
                for (int c = 32 * half; c < cols && c_tile + c < p.N; c += 64) {
                    uint32_t a0[16], a1[16];
                    float v0[16], v1[16];
                    tmem_ld16(base + c, a0);
                    tmem_ld16(base + c + 16, a1);
                    if constexpr (FWD) {
                        uint32_t b0[16], b1[16];
                        tmem_ld16(base + cols + c, b0);
                        tmem_ld16(base + cols + c + 16, b1);
                        tmem_wait16(a0), tmem_wait16(a1), tmem_wait16(b0), tmem_wait16(b1);
                        if (p.gate) {
                            floats(a0, v0), floats(a1, v1);
                            send(&outs.gate, v0, v1, c);
                        }
                        if (p.up) {
                            floats(b0, v0), floats(b1, v1);
                            send(&outs.up, v0, v1, c);
                        }
                        finish(a0, b0, v0), finish(a1, b1, v1);
                    } else {
                        tmem_wait16(a0), tmem_wait16(a1);
                        floats(a0, v0), floats(a1, v1);
                    }
                    send(&outs.out, v0, v1, c);
                }
            } else {
                // 16 columns at a time, of a tile's last ones those that are its own
#pragma unroll 1
                for (int c = 16 * half; c < cols; c += 32) {
                    uint32_t ra[16], rb[16];
                    tmem_ld16(base + c, ra);
                    if (FWD) tmem_ld16(base + cols + c, rb);
                    tmem_wait16(ra);
                    if (FWD) tmem_wait16(rb);
                    if (mine) {
                        float v[16];
                        if constexpr (FWD) {
                            if (p.gate) {
                                floats(ra, v);
                                store16(p.gate + row * p.ld_gate, c_tile + c, c_end, v);
                            }
                            if (p.up) {
                                floats(rb, v);
                                store16(p.up + row * p.ld_up, c_tile + c, c_end, v);
                            }
                            finish(ra, rb, v);
                        } else {
                            floats(ra, v);
                        }
                        store16(p.out + row * p.ld_out, c_tile + c, c_end, v);
                    }
                    __syncwarp();
                }
            }
            // the accumulator is read: the MMA may refill it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (CG == 1) mbar_arrive(&ctl->tempty[buf]);
                else arrive_at(of_leader(&ctl->tempty[buf]));
            }
        }
        if (CG == 2 && lane == 0) bulk_wait();  // this warp's last blocks are written
    }
    tc_fence_before();
    tile_sync<CG>();  // no CTA of a pair leaves while the other reads its memory
    if (warp == 1) {
        tc_fence_after();
        free_tmem<CG>(tmem, 2 * kMaxN);
    }
}

// ---- host ---------------------------------------------------------------------

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

dgr_status encode_fn(PFN_cuTensorMapEncodeTiled_v12000 *fn) {
    std::call_once(g_encode_once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    if (!g_encode) return DGR_ERR_CUDA;
    *fn = g_encode;
    return DGR_OK;
}

// Map over `count` row-major bf16 matrices [rows, cols], one behind the other
// (row stride ld): boxes of 64 columns by box_rows rows of one matrix, 128-byte
// swizzle, zeros past its last row and column.
dgr_status make_map(CUtensorMap *m, const void *base, int64_t cols, int64_t rows, int64_t ld, int64_t count, uint32_t box_rows) {
    PFN_cuTensorMapEncodeTiled_v12000 enc;
    const dgr_status st = encode_fn(&enc);
    if (st != DGR_OK) return st;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(count)};
    // (of a single matrix the distance to the next one says nothing, and might be out of a map's range)
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld * 2), static_cast<cuuint64_t>((count > 1 ? rows : 1) * ld * 2)};
    const cuuint32_t box[3] = {64, box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? DGR_OK : DGR_ERR_CUDA;
}

// Map over the rows of an output, in blocks of 32 x 32, 64-byte swizzle.
dgr_status make_block_map(CUtensorMap *m, void *base, int64_t cols, int64_t rows, int64_t ld) {
    PFN_cuTensorMapEncodeTiled_v12000 enc;
    const dgr_status st = encode_fn(&enc);
    if (st != DGR_OK) return st;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld * 2)};
    const cuuint32_t box[2] = {32, 32};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? DGR_OK : DGR_ERR_CUDA;
}

// The counters of rows, one of tiles and one of shares.
size_t ready_bytes(int64_t T) { return static_cast<size_t>((T + kReadyRows - 1) / kReadyRows + 2) * 4; }
constexpr int kLeadBlocks = 4;
constexpr uint64_t kTileLeastNs = 10000;  // a tile of few stages takes its epilogue's time

struct Operand {
    const void *a, *a2;
    int64_t ld_a, ld_a2;
    const void *b, *b2;
};

// Row blocks of `rows` rows at most: every expert may end in a ragged one.
int64_t row_blocks_most(const FfnParams &p, int rows) {
    const int64_t whole = (static_cast<int64_t>(p.T) + rows - 1) / rows;
    return p.offs ? whole + (p.E < p.T ? p.E : p.T) : whole;
}

template <int CG, bool FWD, int ACT, bool PRE>
dgr_status launch_tiles(FfnParams p, const PreParams &pre, const Operand &o, int sms, cudaStream_t s) {
    constexpr int kRows = CG * BM;
    CUtensorMap mA, mA2, mB, mB2;
    dgr_status st;
    if ((st = make_map(&mA, o.a, p.K, p.T, o.ld_a, 1, p.cut.box)) != DGR_OK) return st;
    mA2 = mA;
    if (!FWD && (st = make_map(&mA2, o.a2, p.K, p.T, o.ld_a2, 1, p.cut.box)) != DGR_OK) return st;
    // the weights are [E, F, H]: forward N = F by K = H, backward K = F by N = H
    const int64_t F = FWD ? p.N : p.K, H = FWD ? p.K : p.N;
    const uint32_t box = FWD ? p.cut.cols : 64;
    if ((st = make_map(&mB, o.b, H, F, H, p.E, box)) != DGR_OK || (st = make_map(&mB2, o.b2, H, F, H, p.E, box)) != DGR_OK) return st;
    Outputs outs{};
    if (CG == 2) {
        if ((st = make_block_map(&outs.out, p.out, p.N, p.T, p.ld_out)) != DGR_OK) return st;
        if (p.gate && (st = make_block_map(&outs.gate, p.gate, p.N, p.T, p.ld_gate)) != DGR_OK) return st;
        if (p.up && (st = make_block_map(&outs.up, p.up, p.N, p.T, p.ld_up)) != DGR_OK) return st;
    }
    p.cut.nbs = (p.N + p.cut.cols - 1) / p.cut.cols;
    // as many stages as fit, the last one's A read as 128 rows too
    p.cut.room = p.T < BM ? (p.T + p.cut.box - 1) / p.cut.box * p.cut.box : BM;
    const uint32_t stage_a = static_cast<uint32_t>(p.cut.room) * 128u, stage = stage_a + static_cast<uint32_t>(FWD ? 2 * p.cut.cols : p.cut.cols) * 128u;
    const uint32_t by_end = kRing / stage, by_last = 1 + (kRing - kStageA) / stage;
    p.cut.stages = static_cast<int32_t>(by_end < by_last ? by_end : by_last);
    if (p.cut.stages > kMaxStages) p.cut.stages = kMaxStages;
    const int64_t tiles = row_blocks_most(p, kRows) * p.cut.nbs, most = sms / CG > 0 ? sms / CG : 1;
    if (tiles > INT32_MAX) return DGR_ERR_UNSUPPORTED;
    auto *k = ffn_gemm<CG, FWD, ACT, PRE>;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem)) != cudaSuccess) return DGR_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    const unsigned groups = sched_grid(static_cast<unsigned>((tiles < most ? tiles : most) * CG)) / CG;
    cfg.gridDim = dim3((groups > 0 ? groups : 1) * CG);
    cfg.blockDim = dim3(kThreads + (PRE ? (kPreWarps - 2) * 32 : 0));
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = CG;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, mA, mA2, mB, mB2, outs, p, pre) == cudaSuccess ? DGR_OK : DGR_ERR_CUDA;
}

// How a call is cut: in pairs of CTAs (cut.cols 0), or in single ones whose tiles
// are so many columns wide. The cost of a cut is that of the SM with the most to
// do, waves of tiles times a stage of one: 0.39 us of a pair (256 x 256); of a
// single CTA 0.10 us and 0.37 us for 256 columns of the product (0.47 us at 128 x
// 256, 0.2 us at 64, as measured: what a stage costs however narrow, its weights'
// reading and its MMAs). So large batches come in pairs, few rows in as many
// narrow tiles as there are SMs, and batches in between as their last wave and
// their experts' ragged ends make it.
template <bool FWD>
Tiles choose(const FfnParams &p, int sms) {
    constexpr int kStep = FWD ? 8 : 64, kMost = FWD ? kMaxN / 2 : kMaxN, kPerCol = FWD ? 2 : 1;
    // row blocks as they are likely to be: a ragged one for most experts
    const int64_t some = p.E < p.T ? p.E : p.T;
    auto blocks = [&](int rows) {
        const int64_t half = (static_cast<int64_t>(p.T) + rows - 1) / rows + (some > 1 ? some / 2 : 0);
        return some > half ? some : half;
    };
    auto waves = [&](int rows, int cols, int64_t at_once) { return (blocks(rows) * ((p.N + cols - 1) / cols) + at_once - 1) / at_once; };
    Tiles best{};
    double least = static_cast<double>(waves(2 * BM, kMost, sms / 2 > 0 ? sms / 2 : 1)) * 0.39;
    for (int cols = kMost; cols >= kStep; cols -= kStep) {
        const double cost = static_cast<double>(waves(BM, cols, sms)) * (0.10 + 0.37 / kMaxN * kPerCol * cols);
        if (cost < least) least = cost, best.cols = cols;
    }
    best.box = p.T >= 128 * static_cast<int64_t>(p.E) ? BM : p.T <= 8 ? 8 : 32;
    return best;
}

template <bool FWD, int ACT, bool PRE>
dgr_status launch_pairs(FfnParams p, const PreParams &pre, const Operand &o, int sms, cudaStream_t s) {
    p.cut.cols = FWD ? kMaxN / 2 : kMaxN, p.cut.box = BM;
    return launch_tiles<2, FWD, ACT, PRE>(p, pre, o, sms, s);
}

template <int ACT>
dgr_status launch_forward(FfnParams p, const Operand &o, int sms, cudaStream_t s) {
    p.cut = choose<true>(p, sms);
    return p.cut.cols ? launch_tiles<1, true, ACT, false>(p, PreParams{}, o, sms, s) : launch_pairs<true, ACT, false>(p, PreParams{}, o, sms, s);
}

// da and db element by element, then dx; in one kernel where its products take far
// longer than the elements' 10 bytes, so that the one's memory traffic goes on
// under the other: back to back, one kernel and two, 16384 rows of 2048 x 4096 in 8
// experts 401 and 453 us, 8192 218 and 229, 4096 147 and 148, 8192 of 1024 x 4096
// 160 and 144, 5723 of 1024 x 2048 in 16 experts 85 and 72.
constexpr int kFusedWidth = 1536, kFusedWaves = 3;

template <int ACT>
dgr_status launch_backward(FfnParams p, PreParams &g, const Operand &o, int sms, cudaStream_t s) {
    if (p.out) p.cut = choose<false>(p, sms);
    const int64_t pairs = sms / 2 > 0 ? sms / 2 : 1, pair_tiles = row_blocks_most(p, 2 * BM) * ((p.N + kMaxN - 1) / kMaxN);
    if (p.out && p.cut.cols == 0 && p.N >= kFusedWidth && pair_tiles >= kFusedWaves * pairs) {
        g.rows_item = g.vecs >= 256 ? 1 : g.vecs >= 128 ? 2 : g.vecs >= 64 ? 4 : 8;
        g.taken = g.ready + ready_bytes(p.T) / 4 - 1, g.begun = g.taken - 1;
        g.nbs = (p.N + kMaxN - 1) / kMaxN;
        // the row blocks that all pairs are at, and a few; in another order than the
        // rows' the tiles may want any
        g.lead = p.sched.order == 0 ? (sms / 2 / g.nbs + 1 + kLeadBlocks) * 2 * BM : 0;
        // twice the time of a tile's stages (0.1 ms at F = 4096): clocks may be down by a quarter
        const uint64_t tile_ns = 2 * static_cast<uint64_t>((p.K + BK - 1) / BK) * kStageNs;
        g.lead_ns = 2 * (tile_ns > kTileLeastNs ? tile_ns : kTileLeastNs);
        if (cudaMemsetAsync(g.ready, 0, ready_bytes(p.T), s) != cudaSuccess) return DGR_ERR_CUDA;
        return launch_pairs<false, ACT, true>(p, g, o, sms, s);
    }
    const int64_t n = static_cast<int64_t>(p.T) * g.vecs, ctas = (n + 255) / 256, most = static_cast<int64_t>(sms) * 8;
    ffn_pre_grad<ACT><<<static_cast<unsigned>(ctas < most ? ctas : most), 256, 0, s>>>(g);
    const dgr_status st = launch_status();
    if (st != DGR_OK || !p.out) return st;
    // (no activation in these)
    return p.cut.cols ? launch_tiles<1, false, kSilu, false>(p, PreParams{}, o, sms, s) : launch_pairs<false, kSilu, false>(p, PreParams{}, o, sms, s);
}

// What both entries check of the rows, sizes, offsets and workspace.
dgr_status check_sizes(int64_t T, int64_t H, int64_t F, int32_t E, int32_t act, const int64_t *offs) {
    if (T < 0 || H < 1 || F < 1 || E < 1 || (act != kSilu && act != kGelu) || (!offs && E != 1)) return DGR_ERR_INVALID_ARG;
    if (T > INT32_MAX - 256 || H > (1 << 20) || F > (1 << 20) || E > kMaxExperts) return DGR_ERR_UNSUPPORTED;
    if (H * F >= (int64_t{1} << 39)) return DGR_ERR_UNSUPPORTED;  // bytes from one expert's weights to the next
    if (H % 8 != 0 || F % 8 != 0) return DGR_ERR_MISALIGNED;
    return DGR_OK;
}

struct Rows {
    const void *p;
    int64_t ld, cols;
};
Runs runs(int64_t T, const Rows &r) { return {r.p, r.ld * 2, T, 0, 1, r.cols * 2}; }
size_t extent(int64_t T, const Rows &r) { return runs(T, r).extent(); }
bool overlap(int64_t T, const Rows &a, const Rows &b) { return runs_overlap(runs(T, a), runs(T, b)); }  // parts of one row do not

}  // namespace
}  // namespace dgr

using namespace dgr;

extern "C" size_t dgr_gated_ffn_workspace_bytes(int64_t T, int64_t H, int64_t F, int32_t E) {
    if (T < 0 || H < 1 || F < 1 || E < 1 || E > kMaxExperts || T > INT32_MAX - 256 || H > (1 << 20) || F > (1 << 20)) return 0;
    return sizeof(WsHeader) + align_up(ready_bytes(T));
}

extern "C" dgr_status dgr_gated_ffn(const void *x, int64_t ld_x, const void *w_gate, const void *w_up, const int64_t *d_offs,
                                    int32_t E, int64_t T, int64_t H, int64_t F, int32_t act, void *h, int64_t ld_h, void *gate,
                                    int64_t ld_gate, void *up, int64_t ld_up, void *ws, size_t ws_bytes, void *stream) {
    dgr_status st = check_sizes(T, H, F, E, act, d_offs);
    if (st != DGR_OK) return st;
    const Rows in = {x, ld_x, H}, outs[] = {{h, ld_h, F}, {gate, ld_gate, F}, {up, ld_up, F}};
    if (!ws || (T > 0 && (!x || !w_gate || !w_up || !h))) return DGR_ERR_INVALID_ARG;
    if (ld_x < H) return DGR_ERR_INVALID_ARG;
    for (const Rows &o : outs)
        if (o.p && o.ld < F) return DGR_ERR_INVALID_ARG;
    if (!aligned(x, 16) || ld_x % 8 || !aligned(w_gate, 16) || !aligned(w_up, 16) || !aligned(d_offs, 8) || !aligned(ws, kAlign))
        return DGR_ERR_MISALIGNED;
    for (const Rows &o : outs)
        if (o.p && (!aligned(o.p, 16) || o.ld % 8)) return DGR_ERR_MISALIGNED;
    if (ws_bytes < sizeof(WsHeader)) return DGR_ERR_WORKSPACE_TOO_SMALL;
    const size_t weights = static_cast<size_t>(E) * F * H * 2;
    for (const Rows &o : outs) {
        const size_t n = extent(T, o);
        if (overlap(T, o, in) || ranges_overlap(o.p, n, w_gate, weights) || ranges_overlap(o.p, n, w_up, weights) ||
            ranges_overlap(o.p, n, d_offs, (static_cast<size_t>(E) + 1) * 8) || ranges_overlap(o.p, n, ws, sizeof(WsHeader)))
            return DGR_ERR_ALIAS;
        for (const Rows &q : outs)
            if (&q < &o && overlap(T, o, q)) return DGR_ERR_ALIAS;
    }
    for (const Rows &i : {in, Rows{w_gate, 0, 0}, Rows{w_up, 0, 0}})
        if (ranges_overlap(ws, sizeof(WsHeader), i.p, i.cols ? extent(T, i) : weights)) return DGR_ERR_ALIAS;
    if ((st = check_device()) != DGR_OK) return st;
    if (T == 0) return DGR_OK;
    FfnParams p{};
    p.offs = d_offs, p.E = E, p.T = static_cast<int32_t>(T);
    p.K = static_cast<int32_t>(H), p.N = static_cast<int32_t>(F);
    p.out = static_cast<uint16_t *>(h), p.gate = static_cast<uint16_t *>(gate), p.up = static_cast<uint16_t *>(up);
    p.ld_out = ld_h, p.ld_gate = ld_gate, p.ld_up = ld_up;
    p.hdr = static_cast<WsHeader *>(ws);
    p.sched = sched_setting();
    int sms = 0;
    if ((st = usable_sms(&sms)) != DGR_OK) return st;
    const Operand o{x, nullptr, ld_x, 0, w_gate, w_up};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return act == kSilu ? launch_forward<kSilu>(p, o, sms, s) : launch_forward<kGelu>(p, o, sms, s);
}

extern "C" dgr_status dgr_gated_ffn_backward(const void *dh, int64_t ld_dh, const void *gate, int64_t ld_gate, const void *up,
                                             int64_t ld_up, const void *w_gate, const void *w_up, const int64_t *d_offs, int32_t E,
                                             int64_t T, int64_t H, int64_t F, int32_t act, void *dgate, int64_t ld_dgate,
                                             void *dup, int64_t ld_dup, void *dx, int64_t ld_dx, void *ws, size_t ws_bytes,
                                             void *stream) {
    dgr_status st = check_sizes(T, H, F, E, act, d_offs);
    if (st != DGR_OK) return st;
    const Rows ins[] = {{dh, ld_dh, F}, {gate, ld_gate, F}, {up, ld_up, F}}, outs[] = {{dgate, ld_dgate, F}, {dup, ld_dup, F}, {dx, ld_dx, H}};
    if (!ws || (T > 0 && (!dh || !gate || !up || !dgate || !dup || (dx && (!w_gate || !w_up))))) return DGR_ERR_INVALID_ARG;
    for (const Rows &r : ins)
        if (r.ld < F) return DGR_ERR_INVALID_ARG;
    for (const Rows &r : outs)
        if (r.p && r.ld < r.cols) return DGR_ERR_INVALID_ARG;
    for (const Rows &r : ins)
        if (!aligned(r.p, 16) || r.ld % 8) return DGR_ERR_MISALIGNED;
    for (const Rows &r : outs)
        if (r.p && (!aligned(r.p, 16) || r.ld % 8)) return DGR_ERR_MISALIGNED;
    if (!aligned(w_gate, 16) || !aligned(w_up, 16) || !aligned(d_offs, 8) || !aligned(ws, kAlign)) return DGR_ERR_MISALIGNED;
    const size_t need = dgr_gated_ffn_workspace_bytes(T, H, F, E);
    if (ws_bytes < need) return DGR_ERR_WORKSPACE_TOO_SMALL;
    const size_t weights = static_cast<size_t>(E) * F * H * 2;
    for (const Rows &o : outs) {
        const size_t n = extent(T, o);
        for (const Rows &i : ins) {
            // dgate in gate's place, dup in up's: the same pointer and stride
            const bool in_place = ((o.p == dgate && i.p == gate) || (o.p == dup && i.p == up)) && o.p == i.p && o.ld == i.ld;
            if (!in_place && overlap(T, o, i)) return DGR_ERR_ALIAS;
        }
        if (ranges_overlap(o.p, n, w_gate, weights) || ranges_overlap(o.p, n, w_up, weights) ||
            ranges_overlap(o.p, n, d_offs, (static_cast<size_t>(E) + 1) * 8) || ranges_overlap(o.p, n, ws, need))
            return DGR_ERR_ALIAS;
        for (const Rows &q : outs)
            if (&q < &o && overlap(T, o, q)) return DGR_ERR_ALIAS;
    }
    for (const Rows &i : ins)
        if (ranges_overlap(ws, need, i.p, extent(T, i))) return DGR_ERR_ALIAS;
    if (ranges_overlap(ws, need, w_gate, weights) || ranges_overlap(ws, need, w_up, weights)) return DGR_ERR_ALIAS;
    if ((st = check_device()) != DGR_OK) return st;
    if (T == 0) return DGR_OK;
    int sms = 0;
    if ((st = usable_sms(&sms)) != DGR_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    PreParams g{};
    g.dh = static_cast<const uint16_t *>(dh), g.gate = static_cast<const uint16_t *>(gate), g.up = static_cast<const uint16_t *>(up);
    g.dgate = static_cast<uint16_t *>(dgate), g.dup = static_cast<uint16_t *>(dup);
    g.ld_dh = ld_dh, g.ld_gate = ld_gate, g.ld_up = ld_up, g.ld_dgate = ld_dgate, g.ld_dup = ld_dup;
    g.T = static_cast<int32_t>(T), g.vecs = static_cast<int32_t>(F / 8);
    g.ready = reinterpret_cast<int32_t *>(static_cast<char *>(ws) + sizeof(WsHeader));
    FfnParams p{};
    p.offs = d_offs, p.E = E, p.T = static_cast<int32_t>(T);
    p.K = static_cast<int32_t>(F), p.N = static_cast<int32_t>(H);
    p.out = static_cast<uint16_t *>(dx), p.ld_out = ld_dx;
    p.hdr = static_cast<WsHeader *>(ws);
    p.sched = sched_setting();
    const Operand o{dgate, dup, ld_dgate, ld_dup, w_gate, w_up};
    return act == kSilu ? launch_backward<kSilu>(p, g, o, sms, s) : launch_backward<kGelu>(p, g, o, sms, s);
}
