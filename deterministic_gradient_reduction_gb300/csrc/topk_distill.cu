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
// A row of weight 0, and one whose list is empty, is not read and has loss 0
// and gradient 0.
//
// The softmax's maximum and sum are carried along in one pass. With q_r the
// list's tokens are left out of that pass (a bit a token in shared memory) and
// added back afterwards, so that p_r is a sum of its own and not a difference
// from 1; the gradient outside is then
//   exp(z_j / tau - m) (S exp(m - lse) - q_r / s),  m, s: maximum and sum outside,
// which stays finite however small p_r is. Exponentials are taken to base 2
// (k = log2(e) / tau): every one of a row is ex2(z k - fl(m k)) with the same
// rounded product fl(m k), so its rounding cancels between numerator and sum.
//
// Deterministic: a row's sums go over threads, warps and the block in a fixed
// order, the rows' losses over one CTA in a fixed order.
#include "row_common.cuh"

namespace dgr {
namespace {

using namespace row;

constexpr int kMaxList = 1024;
constexpr int kMaxVocab = 1 << 20;
constexpr int kWhereId = 311;
constexpr float kLn2 = 0.69314718055994531f;

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
    int32_t same_align;  // z's and dz's rows start at the same place of a 16-byte vector
    WsHeader *hdr;       // pad[0]: CTAs done
    Sched sched;
};

// A row as whole 16-byte vectors between a few single elements.
template <typename T>
struct RowView {
    static constexpr int VEC = 16 / static_cast<int>(sizeof(T));
    int head, n_vec, n_single;
    __device__ __forceinline__ RowView(const T *z, int V) {
        const int off = static_cast<int>(reinterpret_cast<uintptr_t>(z) & 15) / static_cast<int>(sizeof(T));
        head = min(V, off ? VEC - off : 0);
        n_vec = (V - head) / VEC;
        n_single = V - n_vec * VEC;
    }
    // element of single i: before the vectors, then behind them
    __device__ __forceinline__ int single(int i) const { return i < head ? i : n_vec * VEC + i; }
    // the bit of element j in the list's mask: a vector's bits lie together
    __device__ __forceinline__ int bit(int j) const { return j - head + VEC; }
};

__device__ __forceinline__ float block_max(float v, float *buf, int n_warps) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, s));
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    v = buf[0];
    for (int k = 1; k < n_warps; ++k) v = fmaxf(v, buf[k]);
    return v;
}

// Running maximum and sum of exp2(x k - m k).
struct Running {
    float m = -INFINITY, c = 0.0f, s = 0.0f;  // c = fl(m k), 0 while m is -inf
    template <int N>
    __device__ __forceinline__ void add(const float (&x)[N], float k) {
        float top = x[0];
#pragma unroll
        for (int i = 1; i < N; ++i) top = fmaxf(top, x[i]);
        if (top > m) {
            const float to = __fmul_rn(top, k);
            s = m == -INFINITY ? s : __fmul_rn(s, ex2(__fadd_rn(c, -to)));
            m = top;
            c = to;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) s = __fadd_rn(s, ex2(__fmaf_rn(x[i], k, -c)));
    }
};

template <typename T, int NT, bool TAIL>
__global__ void __launch_bounds__(NT) distill_rows(const DistillParams p) {
    constexpr int VEC = RowView<T>::VEC, W = NT / 32;
    extern __shared__ char smem[];
    int32_t *s_id = reinterpret_cast<int32_t *>(smem);        // [K], -1: none
    float *s_q = reinterpret_cast<float *>(s_id + p.K);       // [K]
    uint32_t *s_mask = reinterpret_cast<uint32_t *>(s_q + p.K);  // TAIL: a bit a token
    __shared__ float buf[6][32 * 4];
    __shared__ int last;
    const int tid = threadIdx.x;
    if constexpr (TAIL) {
        for (int i = tid; i < (p.V + 2 * VEC) / 32 + 1; i += NT) s_mask[i] = 0;
        __syncthreads();
    }
    for (int32_t it = blockIdx.x; it < p.T; it += gridDim.x) {
        const int32_t row = static_cast<int32_t>(sched_item(p.sched, static_cast<uint32_t>(it)));
        const float weight = p.weights ? __ldg(p.weights + row) : 1.0f;
        const T *z = static_cast<const T *>(p.z) + row * p.ld;
        T *dz = static_cast<T *>(p.dz) + row * p.ld_dz;
        const RowView<T> view(z, p.V);
        const float lse_t = TAIL ? __ldg(p.teacher_lse + row) : 0.0f;
        // the list: each thread keeps entries tid, tid + NT, ...
        float top = -INFINITY;
        int any = 0;
        if (weight != 0.0f)
            for (int i = tid; i < p.K; i += NT) {
                int id = p.ids[row * p.ld_ids + i];
                if (id >= p.V) {
                    if (p.hdr) record_error(p.hdr, DGR_ERR_INVALID_ARG, kWhereId);
                    id = -1;
                }
                const float t = id < 0 ? -INFINITY : __fmul_rn(p.teacher[row * p.ld_t + i], p.inv_tau);
                s_id[i] = id < 0 ? -1 : id;
                s_q[i] = t;
                top = fmaxf(top, t);
                any |= id >= 0 && (TAIL || !(t == -INFINITY));
                if (TAIL && id >= 0) atomicOr(&s_mask[view.bit(id) >> 5], 1u << (view.bit(id) & 31));
            }
        if (!__syncthreads_or(any)) {  // nothing taught here
            if (p.row_loss && tid == 0) p.row_loss[row] = 0.0f;
            if (p.dz) {
                T zero{};
                for (int j = tid; j < p.V; j += NT) dz[j] = zero;
            }
            __syncthreads();
            continue;
        }
        top = block_max(top, buf[0], W);
        float part[2] = {0.0f, 0.0f};  // sum of q, sum of q ln q
        // student logits at the list's entries; an id that comes twice counts once in the student's sum
        float m_list = -INFINITY;
        {
            float sum[1] = {0.0f};
            for (int i = tid; i < p.K; i += NT)
                if (!TAIL) sum[0] = __fadd_rn(sum[0], expf(__fadd_rn(s_q[i], -top)));
            if (!TAIL) block_sum<1>(sum, buf[1], W);
            const float base = TAIL ? lse_t : __fadd_rn(top, logf(sum[0]));
            for (int i = tid; i < p.K; i += NT) {
                const float lq = TAIL ? __fadd_rn(s_q[i], -base) : __fadd_rn(__fadd_rn(s_q[i], -top), -logf(sum[0]));
                const float q = s_id[i] < 0 ? 0.0f : expf(lq);
                part[0] = __fadd_rn(part[0], q);
                if (q != 0.0f) part[1] = __fmaf_rn(q, lq, part[1]);
                s_q[i] = q;
                if (s_id[i] >= 0) m_list = fmaxf(m_list, to_f32(z[s_id[i]]));
            }
        }
        // the row, once
        Running run;
        for (int v = tid; v < view.n_vec; v += NT) {
            float x[VEC];
            unpack<T, VEC>(*reinterpret_cast<const raw_t<T, VEC> *>(z + view.head + v * VEC), x);
            if constexpr (TAIL) {
                const int b = (v + 1) * VEC;
                const uint32_t bits = (s_mask[b >> 5] >> (b & 31)) & ((1u << VEC) - 1);
                if (bits)
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        if (bits >> i & 1) x[i] = -INFINITY;
            }
            run.add(x, p.k2);
        }
        if (tid < view.n_single) {
            const int j = view.single(tid);
            float x[1] = {to_f32(z[j])};
            if (TAIL && (s_mask[view.bit(j) >> 5] >> (view.bit(j) & 31) & 1)) x[0] = -INFINITY;
            run.add(x, p.k2);
        }
        const float m = block_max(run.m, buf[2], W);          // outside the list (TAIL), else of all
        const float c = m == -INFINITY ? 0.0f : __fmul_rn(m, p.k2);
        float m_all = m, c_all = c;
        if (TAIL) {
            m_all = fmaxf(m, block_max(m_list, buf[3], W));
            c_all = m_all == -INFINITY ? 0.0f : __fmul_rn(m_all, p.k2);
        }
        // sums: outside, in the list, q, q ln q
        float sums[4] = {run.m == -INFINITY ? run.s : __fmul_rn(run.s, ex2(__fadd_rn(run.c, -c))), 0.0f, part[0], part[1]};
        if (TAIL)
            for (int i = tid; i < p.K; i += NT) {
                const int id = s_id[i];
                bool first = id >= 0;
                for (int j = 0; j < i && first; ++j) first = s_id[j] != id;
                if (first) sums[1] = __fadd_rn(sums[1], ex2(__fmaf_rn(to_f32(z[id]), p.k2, -c_all)));
            }
        block_sum<4>(sums, buf[4], W);
        const float rest = sums[0];
        const float shift = m == -INFINITY ? 0.0f : ex2(__fadd_rn(c, -c_all));
        const float total = TAIL ? __fmaf_rn(rest, shift, sums[1]) : rest;
        const float inv = 1.0f / total, ln_total = logf(total);
        const float q_rest = TAIL && m != -INFINITY ? fmaxf(__fadd_rn(1.0f, -sums[2]), 0.0f) : 0.0f;
        const float mass = !TAIL || q_rest > 0.0f ? 1.0f : sums[2];
        // loss: sum of q ln q less sum of q ln p, entry by entry
        float lp[1] = {0.0f};
        if (p.row_loss)
            for (int i = tid; i < p.K; i += NT)
                if (s_q[i] != 0.0f)
                    lp[0] = __fmaf_rn(s_q[i], __fmaf_rn(__fmaf_rn(to_f32(z[s_id[i]]), p.k2, -c_all), kLn2, -ln_total), lp[0]);
        // what the gradient writes into: the list's student logits have to be read before
        const float inv_mass = __fmul_rn(inv, mass);
        const float f = __fmul_rn(__fmul_rn(__fmul_rn(p.scale, weight), p.inv_tau), p.dloss ? __ldg(p.dloss) : 1.0f);
        float fix[(kMaxList + NT - 1) / NT];
        if (p.dz) {
#pragma unroll
            for (int n = 0; n < (kMaxList + NT - 1) / NT; ++n) {
                const int i = tid + n * NT;
                fix[n] = 0.0f;
                if (i < p.K && s_id[i] >= 0) {
                    const int id = s_id[i];
                    float q = 0.0f;
                    for (int j = 0; j < p.K; ++j)
                        if (s_id[j] == id) q = __fadd_rn(q, s_q[j]);
                    fix[n] = __fmul_rn(__fadd_rn(__fmul_rn(ex2(__fmaf_rn(to_f32(z[id]), p.k2, -c_all)), inv_mass), -q), f);
                }
            }
        }
        block_sum<1>(lp, buf[5], W);
        if (p.row_loss && tid == 0) {
            float L = __fadd_rn(sums[3], -lp[0]);
            if (q_rest > 0.0f)
                L = __fadd_rn(L, __fmul_rn(q_rest, __fadd_rn(logf(q_rest), -__fadd_rn(__fmaf_rn(__fadd_rn(c, -c_all), kLn2, logf(rest)), -ln_total))));
            p.row_loss[row] = L;
        }
        if (p.dz) {
            const float a = __fmul_rn(TAIL ? __fadd_rn(__fmul_rn(shift, inv_mass), q_rest > 0.0f ? -q_rest / rest : 0.0f) : inv, f);
            for (int v = tid; v < view.n_vec; v += NT) {
                const int j = view.head + v * VEC;
                float x[VEC];
                unpack<T, VEC>(*reinterpret_cast<const raw_t<T, VEC> *>(z + j), x);
#pragma unroll
                for (int i = 0; i < VEC; ++i) x[i] = __fmul_rn(ex2(__fmaf_rn(x[i], p.k2, -c)), a);
                if (p.same_align) {
                    *reinterpret_cast<raw_t<T, VEC> *>(dz + j) = pack<T, VEC>(x);
                } else {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) *reinterpret_cast<raw_t<T, 1> *>(dz + j + i) = pack<T, 1>(x + i);
                }
            }
            if (tid < view.n_single) {
                const int j = view.single(tid);
                const float x = __fmul_rn(ex2(__fmaf_rn(to_f32(z[j]), p.k2, -c)), a);
                *reinterpret_cast<raw_t<T, 1> *>(dz + j) = pack<T, 1>(&x);
            }
            __syncthreads();  // the list's tokens are written over
#pragma unroll
            for (int n = 0; n < (kMaxList + NT - 1) / NT; ++n) {
                const int i = tid + n * NT;
                if (i < p.K && s_id[i] >= 0) *reinterpret_cast<raw_t<T, 1> *>(dz + s_id[i]) = pack<T, 1>(&fix[n]);
            }
        }
        __syncthreads();
        if constexpr (TAIL) {
            for (int i = tid; i < p.K; i += NT)
                if (s_id[i] >= 0) s_mask[view.bit(s_id[i]) >> 5] = 0;
            __syncthreads();
        }
    }
    if (!p.loss) return;
    // the CTA that ends last adds the rows' losses
    __threadfence();
    __syncthreads();
    if (tid == 0) last = atomicAdd(&p.hdr->pad[0], 1) == static_cast<int>(gridDim.x) - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    float s[1] = {0.0f};
    for (int t = tid; t < p.T; t += NT) {
        const float w = p.weights ? __ldg(p.weights + t) : 1.0f;
        if (w != 0.0f) s[0] = __fmaf_rn(w, __ldcg(p.row_loss + t), s[0]);
    }
    block_sum<1>(s, buf[0], W);
    if (tid == 0) {
        *p.loss = __fmul_rn(p.scale, s[0]);
        p.hdr->pad[0] = 0;  // ready for the next call
    }
}

// Host side -------------------------------------------------------------------

template <typename T, int NT, bool TAIL>
dgr_status launch_rows(const DistillParams &p, int sms, cudaStream_t s) {
    constexpr int VEC = RowView<T>::VEC;
    size_t smem = static_cast<size_t>(p.K) * 8;
    if (TAIL) smem += (static_cast<size_t>(p.V + 2 * VEC) / 32 + 1) * 4;
    if (smem > 40 * 1024 && cudaFuncSetAttribute(distill_rows<T, NT, TAIL>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
        return DGR_ERR_CUDA;
    const int64_t most = static_cast<int64_t>(sms) * (1536 / NT), want = p.T > 0 ? p.T : 1;
    distill_rows<T, NT, TAIL><<<sched_grid(static_cast<unsigned>(want < most ? want : most)), NT, smem, s>>>(p);
    return launch_status();
}

template <typename T>
dgr_status launch_type(const DistillParams &p, int sms, cudaStream_t s) {
    if (p.teacher_lse) return p.V >= 16384 ? launch_rows<T, 512, true>(p, sms, s) : launch_rows<T, 128, true>(p, sms, s);
    return p.V >= 16384 ? launch_rows<T, 512, false>(p, sms, s) : launch_rows<T, 128, false>(p, sms, s);
}

size_t extent(int64_t T, int64_t W, int64_t ld, int64_t es) { return T > 0 ? static_cast<size_t>(((T - 1) * ld + W) * es) : 0; }

}  // namespace
}  // namespace dgr

using namespace dgr;

extern "C" size_t dgr_topk_distill_workspace_bytes(int64_t T) { return T < 0 || T > INT32_MAX ? 0 : sizeof(WsHeader); }

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
    const intptr_t apart = reinterpret_cast<intptr_t>(dlogits) - reinterpret_cast<intptr_t>(logits);
    p.same_align = dlogits && apart % 16 == 0 && ((ld_d - ld) * es) % 16 == 0;
    p.hdr = static_cast<WsHeader *>(ws);
    p.sched = sched_for(static_cast<uint32_t>(T));
    int sms = 0;
    if ((st = usable_sms(&sms)) != DGR_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return es == 2 ? launch_type<bf16>(p, sms, s) : launch_type<float>(p, sms, s);
}
