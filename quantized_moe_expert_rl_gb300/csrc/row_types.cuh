// row_types.cuh - element types of the row operators (rl_add_rmsnorm, rl_q4_matvec, rl_logprobs):
// 16-byte loads and stores of 8 values as f32, whatever the type in memory.
#pragma once
#include <cuda_fp8.h>

#include <type_traits>

#include "rl_common.cuh"

namespace rl {

__host__ __device__ inline size_t dtype_bytes(int dt) { return dt == RL_F32 ? 4 : dt == RL_F8_E4M3 ? 1 : 2; }

__device__ __forceinline__ float2 unpack2(uint32_t w, __half) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
__device__ __forceinline__ float2 unpack2(uint32_t w, __nv_bfloat16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// 8 consecutive values at p (aligned to 8 values, at most 16 bytes)
template <typename E>
__device__ __forceinline__ void load8(const E *p, float (&v)[8]) {
    const uint4 q = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2(w[i], E());
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
template <>
__device__ __forceinline__ void load8<float>(const float *p, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
template <typename E>
__device__ __forceinline__ void store8(E *p, const float (&v)[8]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack2(v[0], v[1], E()), pack2(v[2], v[3], E()), pack2(v[4], v[5], E()),
                                               pack2(v[6], v[7], E()));
}
template <>
__device__ __forceinline__ void store8<float>(float *p, const float (&v)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
// v = a + b rounded to the element type.  A 16-bit add rounds the exact sum once, which is what adding in
// f32 and rounding gives: rounding first to p >= 2 q + 2 bits changes no sum's rounding to q bits (24
// against 11 for half, 8 for bf16).
template <typename E>
__device__ __forceinline__ void add8(const E *a, const E *b, float (&v)[8]) {
    const uint4 p = *reinterpret_cast<const uint4 *>(a), q = *reinterpret_cast<const uint4 *>(b);
    const uint32_t x[4] = {p.x, p.y, p.z, p.w}, y[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t s;
        if constexpr (sizeof(E) == 2) {
            using E2 = typename std::conditional<std::is_same<E, __half>::value, __half2, __nv_bfloat162>::type;
            const E2 t = __hadd2_rn(*reinterpret_cast<const E2 *>(&x[i]), *reinterpret_cast<const E2 *>(&y[i]));
            s = *reinterpret_cast<const uint32_t *>(&t);
        }
        const float2 f = unpack2(s, E());
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
template <>
__device__ __forceinline__ void add8<float>(const float *a, const float *b, float (&v)[8]) {
    float w[8];
    load8(a, v);
    load8(b, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += w[j];
}
// larger magnitude; a NaN wins
__device__ __forceinline__ float max_abs_nan(float m, float v) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename E>
__device__ __forceinline__ E from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// four f32 -> four e4m3 bytes, round to nearest even, beyond 448 to 448
__device__ __forceinline__ uint32_t pack4_e4m3(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// ---- 16-byte asynchronous copies into shared memory (the rest of `bytes` < 16 reads as zero) ----
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
template <int B>
__device__ __forceinline__ void cp_async_ca(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(B), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait_all_but() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace rl
