// add_norm.cu - rl_add_rmsnorm: residual addition, RMSNorm and an e4m3 copy with group scales, one
// pass over the row.
//
//   s = x + res (rounded to the row type: the residual stream as it is kept)
//   v = s / sqrt(mean(s^2) + eps) * gain,  xn = round(v)
//   scale_g = max_{h in g} |v_h| / 448,  q_h = e4m3(v_h * (448 / max_g))
//
// A row is read once and stays in registers: a thread owns NC runs of 8 consecutive values (one
// 16-byte load of a 16-bit row), so that a group of 32 / 64 / 128 values is 4 / 8 / 16 neighbouring
// lanes and its maximum takes 2 to 4 shuffles; the sum of squares takes one CTA barrier.  Rows of
// fewer than 256 threads share a CTA of about 256 threads.
//
// Bound: memory for many rows, the launch and two memory round trips for few.  Measured back to back in a
// graph: 8192 rows of 2048 bf16 values with residual, gain and the 8-bit copy (151 MB) 29.7 us, 5.1 TB/s; 2048
// rows 10.5 to 10.9 us, 3.5 TB/s; one row 2.8 us; 8192 and 2048 f32 rows 44.3 us, 6.4 TB/s, and 14.3 us.  Two and four runs per thread, which leave fewer warps to meet
// per row, were the same to 15% slower from 2048 rows on.
#include "qdot.cuh"
#include "row_types.cuh"

using namespace rl;

namespace {

constexpr int kNormMaxH = 16384;

struct NormArgs {
    const void *x, *res;
    const float *gain;
    void *x_out, *xn;
    uint8_t *q;
    float *scale;
    float eps;
    int T, H, tpr, rows, group;  // threads per row (a multiple of 32), rows per CTA
};

// sum (or maximum) of v over the threads of a row: warps of the row through shared memory
template <bool MAX>
__device__ __forceinline__ float row_reduce(float v, float *part, int warp0, int nwarps) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float w = __shfl_xor_sync(kFull, v, o);
        v = MAX ? fmaxf(v, w) : v + w;
    }
    if (nwarps == 1) return v;
    __syncthreads();  // an earlier reduction's values have been read
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    float r = part[warp0];
#pragma unroll 8
    for (int i = 1; i < nwarps; ++i) r = MAX ? fmaxf(r, part[warp0 + i]) : r + part[warp0 + i];
    return r;
}

// GL: lanes per group of the 8-bit copy (0: no copy)
template <typename E, int NC, int GL>
__global__ void __launch_bounds__(1024) add_norm_kernel(const NormArgs a) {
    __shared__ float part[32];
    const int rowi = threadIdx.x / a.tpr, tr = threadIdx.x - rowi * a.tpr;
    const int row = blockIdx.x * a.rows + rowi, nw = a.tpr >> 5, w0 = rowi * nw;
    const int lane = threadIdx.x & 31;
    const size_t base = (size_t)row * a.H;
    const bool live = row < a.T;
    pdl_wait();
    pdl_trigger();
    float s[NC][8];
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int h = 8 * (c * a.tpr + tr);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[c][j] = 0.f;
        if (live && h < a.H) {
            if (a.res) add8(static_cast<const E *>(a.x) + base + h, static_cast<const E *>(a.res) + base + h, s[c]);
            else load8(static_cast<const E *>(a.x) + base + h, s[c]);
        }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int h = 8 * (c * a.tpr + tr);
        if (a.x_out && live && h < a.H) store8(static_cast<E *>(a.x_out) + base + h, s[c]);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(s[c][j], s[c][j], ss);
    }
    ss = row_reduce<false>(ss, part, w0, nw);
    float r = 1.0f / sqrtf(ss / (float)a.H + a.eps);
    // Squares outside the f32 range (values beyond about 1e18, or all below about 1e-15): the sum is
    // taken again over values scaled by a power of two.  The vote makes the branch uniform.
    const bool odd = live && !(ss < 1e37f && ss > 1e-30f * (float)a.H);
    if (a.rows == 1 ? odd : __syncthreads_or(odd)) {
        float m = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(s[c][j]));
        m = row_reduce<true>(m, part, w0, nw);
        int ex = 0;
        const bool fin = m > 0.f && m < __int_as_float(0x7f800000);
        if (fin) frexpf(m, &ex);
        float s2 = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float v = ldexpf(s[c][j], -ex);
                s2 = fmaf(v, v, s2);
            }
        s2 = row_reduce<false>(s2, part, w0, nw);
        if (odd && fin && s2 == s2) {
            double rd = 1.0 / sqrt(ldexp((double)s2 / a.H, 2 * ex) + (double)a.eps);
            if (rd > 1e38) {  // beyond f32: 2^64 of it go to the values, which are below 2e-36 (rd is at most 2^156)
                rd *= 1.0 / 18446744073709551616.0;
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int j = 0; j < 8; ++j) s[c][j] *= 18446744073709551616.0f;
            }
            r = (float)rd;
        }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int h = 8 * (c * a.tpr + tr);
        const bool in = live && h < a.H;
        float v[8];
        if (a.gain && in) {
            load8(a.gain + h, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= s[c][j] * r;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = s[c][j] * r;
        }
        if (a.xn && in) store8(static_cast<E *>(a.xn) + base + h, v);
        if (GL == 0) continue;
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max_abs_nan(m, v[j]);
#pragma unroll
        for (int o = 1; o < GL; o <<= 1) m = max_nan(m, __shfl_xor_sync(kFull, m, o));
        if (!in) continue;
        // One correctly rounded reciprocal for the group.  Over 100.7M values 58 round to the other neighbour of what
        // 64 bits give; with an approximate reciprocal 66 to 70, with a division per value 57 to 61, which
        // takes 11.7 us for 2048 rows of 2048 bf16 values instead of 10.5.
        float sc = m * (1.0f / 448.0f), inv = __fdiv_rn(448.0f, m);
        if (!(m >= 1e-30f && m < __int_as_float(0x7f800000))) {  // zeros, far below f32's range, infinity or NaN
            inv = 0.f;
            if (!(m < __int_as_float(0x7f800000))) {
                sc = __int_as_float(0x7fffffff);
            } else if (m > 0.f) {  // 448 / m must stay finite: scale both by 2^64
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] *= 18446744073709551616.0f;
                inv = 448.0f / (m * 18446744073709551616.0f);
            }
        }
        uint2 o8 = make_uint2(0u, 0u);
        if (inv > 0.f) {
            o8.x = pack4_e4m3(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
            o8.y = pack4_e4m3(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
        }
        *reinterpret_cast<uint2 *>(a.q + base + h) = o8;
        if ((lane & (GL - 1)) == 0) a.scale[(size_t)row * (a.H / (8 * (GL ? GL : 1))) + h / (8 * (GL ? GL : 1))] = sc;
    }
}

template <typename E>
rl_status launch_norm(NormArgs &a, cudaStream_t s) {
    // a thread per 8 values up to rows of 8192, two runs per thread beyond
    const int oct = a.H / 8, nc = oct > 1024 ? 2 : 1;
    a.tpr = (int)align_up((size_t)(oct + nc - 1) / nc, 32);
    a.rows = a.tpr >= 256 ? 1 : 256 / a.tpr;
    if (a.rows > a.T) a.rows = a.T;
    const dim3 grid((a.T + a.rows - 1) / a.rows), block(a.tpr * a.rows);
#define RL_NORM(NC)                                                                                             \
    (a.group == 0    ? launch_pdl(add_norm_kernel<E, NC, 0>, grid, block, 0, s, "rl_add_rmsnorm", a)              \
     : a.group == 32 ? launch_pdl(add_norm_kernel<E, NC, 4>, grid, block, 0, s, "rl_add_rmsnorm", a)              \
     : a.group == 64 ? launch_pdl(add_norm_kernel<E, NC, 8>, grid, block, 0, s, "rl_add_rmsnorm", a)              \
                     : launch_pdl(add_norm_kernel<E, NC, 16>, grid, block, 0, s, "rl_add_rmsnorm", a))
    return nc == 2 ? RL_NORM(2) : RL_NORM(1);
#undef RL_NORM
}

}  // namespace

extern "C" rl_status rl_add_rmsnorm(const void *x, const void *res, const float *gain, int32_t dtype, int32_t T,
                                    int32_t H, float eps, void *x_out, void *xn, uint8_t *q, float *scale,
                                    int32_t group, void *stream) {
    if (dtype != RL_F32 && dtype != RL_F16 && dtype != RL_BF16)
        return fail(RL_ERR_INVALID, "rl_add_rmsnorm: dtype %d is none of RL_F32, RL_F16, RL_BF16", dtype);
    if (T < 0 || H <= 0 || !(eps >= 0.f)) return fail(RL_ERR_INVALID, "rl_add_rmsnorm: T=%d H=%d eps=%g", T, H, eps);
    if (H % 8 != 0 || H > kNormMaxH)
        return fail(RL_ERR_UNSUPPORTED, "rl_add_rmsnorm: H=%d is not a multiple of 8 up to %d", H, kNormMaxH);
    if (q && !(group == 32 || group == 64 || group == 128))
        return fail(RL_ERR_UNSUPPORTED, "rl_add_rmsnorm: group=%d: supported 32, 64, 128", group);
    if (q && H % group != 0)
        return fail(RL_ERR_INVALID, "rl_add_rmsnorm: H=%d is not a multiple of group=%d", H, group);
    if (T == 0) return RL_OK;
    if (!x) return fail(RL_ERR_INVALID, "rl_add_rmsnorm: NULL x");
    if ((q == nullptr) != (scale == nullptr))
        return fail(RL_ERR_INVALID, "rl_add_rmsnorm: q and scale come together");
    if (!x_out && !xn && !q) return fail(RL_ERR_INVALID, "rl_add_rmsnorm: no output");
    if (x_out && x_out == xn) return fail(RL_ERR_INVALID, "rl_add_rmsnorm: x_out and xn are the same buffer");
    if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(res) | reinterpret_cast<uintptr_t>(gain) |
         reinterpret_cast<uintptr_t>(x_out) | reinterpret_cast<uintptr_t>(xn) | reinterpret_cast<uintptr_t>(q)) & 15)
        return fail(RL_ERR_INVALID, "rl_add_rmsnorm: x, res, gain, x_out, xn and q must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(scale) & 3)
        return fail(RL_ERR_INVALID, "rl_add_rmsnorm: scale must be 4-byte aligned");
    NormArgs a = {x, res, gain, x_out, xn, q, scale, eps, T, H, 0, 0, q ? group : 0};
    cudaStream_t s = as_stream(stream);
    if (dtype == RL_F32) return launch_norm<float>(a, s);
    if (dtype == RL_F16) return launch_norm<__half>(a, s);
    return launch_norm<__nv_bfloat16>(a, s);
}
