// Helpers of the row-wise kernels (norms, softmaxes): vectors of bf16 or fp32
// elements, fixed-order sums over a warp and a block.
#pragma once

#include <cuda_bf16.h>

#include "dgr_common.cuh"

namespace dgr {
namespace row {

using bf16 = __nv_bfloat16;

// VEC elements of T as one load or store (2, 4, 8 or 16 bytes).
template <int BYTES>
struct Raw;
template <>
struct Raw<2> {
    using type = uint16_t;
};
template <>
struct Raw<4> {
    using type = uint32_t;
};
template <>
struct Raw<8> {
    using type = uint2;
};
template <>
struct Raw<16> {
    using type = uint4;
};
template <typename T, int VEC>
using raw_t = typename Raw<static_cast<int>(sizeof(T)) * VEC>::type;

template <typename T, int VEC>
__device__ __forceinline__ void unpack(const raw_t<T, VEC> &v, float *f) {
    if constexpr (sizeof(T) == 4) {
        if constexpr (VEC == 1) {
            f[0] = __uint_as_float(v);
        } else if constexpr (VEC == 2) {
            f[0] = __uint_as_float(v.x);
            f[1] = __uint_as_float(v.y);
        } else {
            f[0] = __uint_as_float(v.x);
            f[1] = __uint_as_float(v.y);
            f[2] = __uint_as_float(v.z);
            f[3] = __uint_as_float(v.w);
        }
    } else {
        auto two = [](uint32_t w, float *g) {
            g[0] = __uint_as_float(w << 16);
            g[1] = __uint_as_float(w & 0xffff0000u);
        };
        if constexpr (VEC == 1) {
            f[0] = bf16_bits_to_f32(v);
        } else if constexpr (VEC == 2) {
            two(v, f);
        } else if constexpr (VEC == 4) {
            two(v.x, f);
            two(v.y, f + 2);
        } else {
            two(v.x, f);
            two(v.y, f + 2);
            two(v.z, f + 4);
            two(v.w, f + 6);
        }
    }
}

// Loads under a predicate: the destination keeps its value where it is off.
// NC: data that nothing writes during the launch; otherwise a plain load.
template <bool NC>
__device__ __forceinline__ void load_if(uint16_t &v, const void *p, bool on) {
    if constexpr (NC) asm volatile("{ .reg .pred q; setp.ne.b32 q, %2, 0; @q ld.global.nc.b16 %0, [%1]; }" : "+h"(v) : "l"(p), "r"(static_cast<int>(on)));
    else asm volatile("{ .reg .pred q; setp.ne.b32 q, %2, 0; @q ld.global.b16 %0, [%1]; }" : "+h"(v) : "l"(p), "r"(static_cast<int>(on)) : "memory");
}

template <bool NC>
__device__ __forceinline__ void load_if(uint32_t &v, const void *p, bool on) {
    if constexpr (NC) asm volatile("{ .reg .pred q; setp.ne.b32 q, %2, 0; @q ld.global.nc.b32 %0, [%1]; }" : "+r"(v) : "l"(p), "r"(static_cast<int>(on)));
    else asm volatile("{ .reg .pred q; setp.ne.b32 q, %2, 0; @q ld.global.b32 %0, [%1]; }" : "+r"(v) : "l"(p), "r"(static_cast<int>(on)) : "memory");
}

template <bool NC>
__device__ __forceinline__ void load_if(uint2 &v, const void *p, bool on) {
    if constexpr (NC)
        asm volatile("{ .reg .pred q; setp.ne.b32 q, %3, 0; @q ld.global.nc.v2.b32 {%0, %1}, [%2]; }" : "+r"(v.x), "+r"(v.y) : "l"(p), "r"(static_cast<int>(on)));
    else
        asm volatile("{ .reg .pred q; setp.ne.b32 q, %3, 0; @q ld.global.v2.b32 {%0, %1}, [%2]; }" : "+r"(v.x), "+r"(v.y) : "l"(p), "r"(static_cast<int>(on)) : "memory");
}

template <bool NC>
__device__ __forceinline__ void load_if(uint4 &v, const void *p, bool on) {
    if constexpr (NC)
        asm volatile("{ .reg .pred q; setp.ne.b32 q, %5, 0; @q ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4]; }"
                     : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w) : "l"(p), "r"(static_cast<int>(on)));
    else
        asm volatile("{ .reg .pred q; setp.ne.b32 q, %5, 0; @q ld.global.v4.b32 {%0, %1, %2, %3}, [%4]; }"
                     : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w) : "l"(p), "r"(static_cast<int>(on)) : "memory");
}

// Rounded to nearest even, once.
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <typename T, int VEC>
__device__ __forceinline__ raw_t<T, VEC> pack(const float *f) {
    if constexpr (sizeof(T) == 4) {
        if constexpr (VEC == 1) return __float_as_uint(f[0]);
        else if constexpr (VEC == 2) return make_uint2(__float_as_uint(f[0]), __float_as_uint(f[1]));
        else return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    } else {
        if constexpr (VEC == 1) return __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
        else if constexpr (VEC == 2) return pack2(f[0], f[1]);
        else if constexpr (VEC == 4) return make_uint2(pack2(f[0], f[1]), pack2(f[2], f[3]));
        else return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
    }
}

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
    if constexpr (sizeof(T) == 4) return v;
    else return __bfloat162float(v);
}

// A 32-bit or bf16 parameter read as binary32.
__device__ __forceinline__ float param(const void *p, int bf, int64_t i) {
    return bf ? bf16_bits_to_f32(__ldg(static_cast<const uint16_t *>(p) + i)) : __ldg(static_cast<const float *>(p) + i);
}

// Sum over the warp, the same bits in every lane (each step adds the same
// pair in both lanes of it).
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, s));
    return v;
}

// N sums over the block, the same bits in every thread; `buf` holds
// N * 32 floats and must not be reused before the next barrier of the caller.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float *buf, int n_warps) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = warp_sum(v[i]);
        if (lane == 0) buf[i * 32 + w] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float s = buf[i * 32];
        for (int k = 1; k < n_warps; ++k) s = __fadd_rn(s, buf[i * 32 + k]);
        v[i] = s;
    }
}

// Eight sums over the warp at once: lanes 4 j .. 4 j + 3 end with the sum of
// v[j] (halves of the values are exchanged at each step: 9 shuffles, not 40).
__device__ __forceinline__ float warp_sum8(const float (&v)[8], int lane) {
    float a[4], b[2];
    const bool up16 = (lane & 16) != 0, up8 = (lane & 8) != 0, up4 = (lane & 4) != 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        a[i] = __fadd_rn(up16 ? v[i + 4] : v[i], __shfl_xor_sync(0xffffffffu, up16 ? v[i] : v[i + 4], 16));
#pragma unroll
    for (int i = 0; i < 2; ++i)
        b[i] = __fadd_rn(up8 ? a[i + 2] : a[i], __shfl_xor_sync(0xffffffffu, up8 ? a[i] : a[i + 2], 8));
    float c = __fadd_rn(up4 ? b[1] : b[0], __shfl_xor_sync(0xffffffffu, up4 ? b[0] : b[1], 4));
    c = __fadd_rn(c, __shfl_xor_sync(0xffffffffu, c, 2));
    return __fadd_rn(c, __shfl_xor_sync(0xffffffffu, c, 1));
}

// Copies of 4 or 16 bytes from global to shared memory, in groups.
template <int BYTES>
__device__ __forceinline__ void copy_async(void *dst, const void *src) {
    const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }
// Until all but the newest `depth` - 1 groups have come (depth 1 to 3).
__device__ __forceinline__ void copy_wait_for(int depth) {
    if (depth == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (depth == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else copy_wait();
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// a b + c, two at a time, each rounded once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// v[e] = v[e] * k + c, v[e] = v[e] * k, r[e] = a[e] * b[e] + r[e], in pairs (N even, or 1).
template <int N>
__device__ __forceinline__ void vec_fma(float (&v)[N], float k, float c) {
    if constexpr (N == 1) v[0] = __fmaf_rn(v[0], k, c);
#pragma unroll
    for (int e = 0; e + 1 < N; e += 2) {
        const float2 r = fma2(make_float2(v[e], v[e + 1]), make_float2(k, k), make_float2(c, c));
        v[e] = r.x, v[e + 1] = r.y;
    }
}

template <int N>
__device__ __forceinline__ void vec_scale(float (&v)[N], float k) {
    if constexpr (N == 1) v[0] = __fmul_rn(v[0], k);
#pragma unroll
    for (int e = 0; e + 1 < N; e += 2) {
        const float2 r = mul2(make_float2(v[e], v[e + 1]), make_float2(k, k));
        v[e] = r.x, v[e + 1] = r.y;
    }
}

template <int N>
__device__ __forceinline__ void vec_add(float (&r)[N], const float (&a)[N]) {
    if constexpr (N == 1) r[0] = __fadd_rn(r[0], a[0]);
#pragma unroll
    for (int e = 0; e + 1 < N; e += 2) {
        const float2 s = add2(make_float2(r[e], r[e + 1]), make_float2(a[e], a[e + 1]));
        r[e] = s.x, r[e + 1] = s.y;
    }
}

// Sum of v and dot product of a and b: even and odd elements apart, then together.
template <int N>
__device__ __forceinline__ float vec_sum(const float (&v)[N]) {
    if constexpr (N == 1) return v[0];
    float2 s = make_float2(v[0], v[1]);
#pragma unroll
    for (int e = 2; e + 1 < N; e += 2) s = add2(s, make_float2(v[e], v[e + 1]));
    return __fadd_rn(s.x, s.y);
}

template <int N>
__device__ __forceinline__ float vec_dot(const float (&a)[N], const float (&b)[N]) {
    if constexpr (N == 1) return __fmul_rn(a[0], b[0]);
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int e = 0; e + 1 < N; e += 2) s = fma2(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]), s);
    return __fadd_rn(s.x, s.y);
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float across(float2 v) { return __fadd_rn(v.x, v.y); }

constexpr float kLog2e = 1.4426950408889634f;

}  // namespace row
}  // namespace dgr
