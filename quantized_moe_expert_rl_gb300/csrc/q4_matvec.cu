// q4_matvec.cu - rl_q4_matvec: products of a matrix of 4-bit weights with group scales and a few
// activation rows.
//
//   y[t][n] (+)= sum_g ws[n][g] * xs[t][g] * sum_{k in g} (q[n][k] - 8) * x[t][k]
//
// For a few rows the product is bound by the weights' bytes, so the work per weight has to stay
// below about 2.8 lane instructions (128 lanes per clock and SM against 45 weights per clock and SM
// at the measured HBM rate):
//
// - Two nibbles 16 bits apart become a pair of MMA operands in two instructions.  One AND-OR puts
//   them under the exponent of 1024, where a half's last bit is 1: bits 0-3 give 1024 + q, bits 4-7
//   give 1024 + 16 q; one packed add (-1032) or multiply-add (/16 - 72) gives q - 8, exactly.  (Read
//   as subnormal halves the nibbles would need no second instruction, but the tensor core aligns its
//   products by exponent, and subnormals leave the upper bits of its window empty: with f32
//   activations the error was 3.3e-6 instead of 1e-7.)
// - mma.m16n8k16 takes 16 weight rows as A and 8 activation columns as B, f32 accumulation.
// - The order of k inside a group is free as long as A and B agree, so the words go to the MMA as
//   they lie in memory (ldmatrix hands lane (g, t) word t of row g), 8 values of k per word.
// - Activations are laid out as B fragments once per CTA.  e4m3 values are exact in half precision and
//   keep their group scales; f16 and bf16 rows are scaled by one power of two (the row's largest
//   magnitude to 2^14, so that a half resolves 2^-38 of it), f32 rows the same way and split into two
//   halves (22 bits) in two columns.
//
// Weights stream through per-warp rings of 16-byte asynchronous copies (16 rows x 256 values per
// stage), swizzled so that ldmatrix meets no bank conflict.  W warps share a 16-row tile and add
// their partial sums in a fixed order; results do not depend on timing.
//
// Measured back to back in a graph: 131072 x 2048, groups of 128, one e4m3 row 29.4 us (138.9 MB, 4.7 TB/s,
// 70% of the measured copy rate); 100003 x 2048, groups of 32, 16 bf16 rows 38.4 us (47%); 512 x 2048, one
// row 4.2 us (latency).  The large ones are bound by instruction issue (60% of the slots used, 37
// instructions per 512 weights and column tile, 18 of them the conversion); DRAM reads are the weights once.
#include "qdot.cuh"
#include "row_types.cuh"

using namespace rl;

namespace {

constexpr int kQ4Threads = 512, kQ4Warps = kQ4Threads / 32;
constexpr int kQ4Stage = 16 * 128 + 16 * 16;  // 16 rows x 256 nibbles, then 16 bytes of scales per row
constexpr int kQ4MaxK = 8192;

// activations: e4m3 with group scales; f16 or bf16; f32 in two columns per token
enum { kQ4F8 = 0, kQ4Half = 1, kQ4Split = 2 };

struct Q4Args {
    const uint8_t *w;
    const __half *ws;
    const void *x;
    const float *xs;
    void *y;
    int N, K, T, group, xdt, ydt, acc;
    uint32_t inv;  // 2^32 / (octets of a padded row), rounded up: i / KO = umulhi(i, inv) for the i that occur
    int KC, W, stages, wide;  // stages of 256 values per row, warps per tile, ring depth, scales by wide copies
};

struct Q4Layout {
    size_t o_sc, o_ring, o_red, total;
    Q4Layout(int KC, int NT, int kind, int group, int W, int stages) {
        const bool split = kind == kQ4Split;
        o_sc = (size_t)KC * 8 * NT * 512;
        // e4m3: a scale per (group, token); else one per token, and its largest magnitude
        o_ring = o_sc + align_up(kind == kQ4F8 ? (size_t)KC * (256 / group) * NT * 8 * sizeof(float) : (size_t)NT * 8 * 2 * sizeof(float), 128);
        o_red = o_ring + (size_t)kQ4Warps * stages * kQ4Stage;
        total = o_red + (W > 1 ? (size_t)2 * kQ4Warps * NT * (split ? 256 : 512) : 0);
    }
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// d = (ADD ? d : 0) + a (16 x 16, half) * b (16 x 8, half), f32 accumulation
template <bool ADD>
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(ADD ? d[0] : 0.f), "f"(ADD ? d[1] : 0.f),
          "f"(ADD ? d[2] : 0.f), "f"(ADD ? d[3] : 0.f));
}

// 8 activations k = 8 o .. 8 o + 7 of token `tok` as f32; zero outside the matrix
__device__ __forceinline__ void q4_load_x(const Q4Args &a, int tok, int o, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
    if (tok >= a.T || 8 * o >= a.K) return;
    const size_t at = (size_t)tok * a.K + 8 * o;
    if (a.xdt == RL_F32) {
        load8(static_cast<const float *>(a.x) + at, v);
    } else if (a.xdt == RL_F16) {
        load8(static_cast<const __half *>(a.x) + at, v);
    } else if (a.xdt == RL_BF16) {
        load8(static_cast<const __nv_bfloat16 *>(a.x) + at, v);
    } else {
        const uint2 q = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(a.x) + at);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t two = ((j < 2 ? q.x : q.y) >> (16 * (j & 1))) & 0xffffu;
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            v[2 * j] = f.x;
            v[2 * j + 1] = f.y;
        }
    }
}

__device__ __forceinline__ uint4 q4_fragment(const float (&v)[8]) {
    return make_uint4(pack2(v[0], v[4], __half()), pack2(v[1], v[5], __half()), pack2(v[2], v[6], __half()),
                      pack2(v[3], v[7], __half()));
}

// Lay the activations out as B fragments: the 16 bytes of (32-value chunk c, column n, quarter t)
// at 16 * ((c * 8 NT + n) * 4 + t), so that the lanes of a warp read 512 consecutive bytes; and their
// scales: sc[group][token] for e4m3, else sc[token].
template <int NT, int KIND>
__device__ __forceinline__ void q4_stage_x(const Q4Args &a, uint8_t *bs, float *sc) {
    constexpr int TOK = NT * (KIND == kQ4Split ? 4 : 8);
    const int KO = a.KC * 32, lane = threadIdx.x & 31;
    uint32_t *top = reinterpret_cast<uint32_t *>(sc + TOK);  // [TOK]
    if (KIND != kQ4F8) {  // the largest magnitude of every row, as an integer (a NaN or infinity ranks highest)
        if (threadIdx.x < TOK) top[threadIdx.x] = 0u;
        __syncthreads();
#pragma unroll 1
        for (int i0 = threadIdx.x; i0 < a.T * KO; i0 += 4 * kQ4Threads) {  // four loads in flight
            float v[4][8];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = i0 + u * kQ4Threads, tok = (int)__umulhi((uint32_t)i, a.inv);
                q4_load_x(a, tok, i - tok * KO, v[u]);  // (zeros past the last token)
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int tok = (int)__umulhi((uint32_t)(i0 + u * kQ4Threads), a.inv);  // KO is a multiple of 32: one per warp
                uint32_t mb = 0u;
#pragma unroll
                for (int j = 0; j < 8; ++j) mb = max(mb, __float_as_uint(v[u][j]) & 0x7fffffffu);
                mb = __reduce_max_sync(kFull, mb);
                if (lane == 0 && tok < a.T) atomicMax(top + tok, mb);
            }
            __syncwarp();
        }
        __syncthreads();
        if (threadIdx.x < TOK) {
            const uint32_t mb = top[threadIdx.x];
            // 2^14 over the power of two at or below the largest magnitude (at most 2^127)
            sc[threadIdx.x] = 1.0f / __uint_as_float((uint32_t)min(268 - (int)(mb >> 23), 254) << 23);
        }
        __syncthreads();
    }
#pragma unroll 1
    for (int i0 = threadIdx.x; i0 < TOK * KO; i0 += 4 * kQ4Threads) {
        float x[4][8];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * kQ4Threads, tok = (int)__umulhi((uint32_t)i, a.inv);
            q4_load_x(a, tok, i - tok * KO, x[u]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * kQ4Threads, tok = (int)__umulhi((uint32_t)i, a.inv), o = i - tok * KO;
            if (tok >= TOK) break;
            float (&v)[8] = x[u];
            uint8_t *at = bs + ((size_t)(o >> 2) * NT * 8 + (KIND == kQ4Split ? 2 * tok : tok)) * 64 + (o & 3) * 16;
            if (KIND != kQ4F8) {
                const float mult = 1.0f / sc[tok];  // a power of two: exact
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] *= mult;
            } else if ((8 * o) % a.group == 0) {
                sc[(8 * o / a.group) * TOK + tok] = tok < a.T && 8 * o < a.K ? a.xs[(size_t)tok * (a.K / a.group) + 8 * o / a.group] : 0.f;
            }
            if (KIND == kQ4Split) {
                float lo[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float hi = __half2float(__float2half_rn(v[j]));
                    lo[j] = v[j] - hi;
                    v[j] = hi;
                }
                *reinterpret_cast<uint4 *>(at) = q4_fragment(v);
                *reinterpret_cast<uint4 *>(at + 64) = q4_fragment(lo);
            } else {
                *reinterpret_cast<uint4 *>(at) = q4_fragment(v);
            }
        }
    }
}

// The masks and constants of the conversion, held in registers: with immediates the AND-OR would take
// two instructions.
struct Q4Const {
    uint32_t lo, hi, bias;
};
__device__ __forceinline__ Q4Const q4_const() {
    Q4Const c;
    asm volatile("mov.b32 %0, 0x000f000f;\n\tmov.b32 %1, 0x00f000f0;\n\tmov.b32 %2, 0x64006400;"
                 : "=r"(c.lo), "=r"(c.hi), "=r"(c.bias));
    return c;
}
// q - 8 for the nibbles at bits 0-3 (LO) or 4-7 of both 16-bit halves of w, as a pair of halves
template <bool LO>
__device__ __forceinline__ uint32_t q4_pair(uint32_t w, const Q4Const &c) {
    uint32_t biased;  // (w & mask) | bias
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(biased) : "r"(w), "r"(LO ? c.lo : c.hi), "r"(c.bias));
    const __half2 h = *reinterpret_cast<const __half2 *>(&biased);
    const __half2 r = LO ? __hadd2(h, __floats2half2_rn(-1032.f, -1032.f))
                         : __hfma2(h, __floats2half2_rn(0.0625f, 0.0625f), __floats2half2_rn(-72.f, -72.f));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// The copies of one warp: 16 rows x 256 values per stage, every W-th stage of its tiles.
struct Q4Feed {
    const uint8_t *p;   // this lane's 16 bytes of rows (lane / 8) + 4 i, i = 0..3, at the present stage
    const __half *q;    // lanes 0..15: the scales of row `lane` at the present stage
    int tile, st;
    bool full;          // all 16 rows are in the matrix
};
__device__ __forceinline__ void q4_seek(const Q4Args &a, Q4Feed &f, int tile, int st) {
    const int lane = threadIdx.x & 31;
    f.tile = tile;
    f.st = st;
    f.full = tile * 16 + 16 <= a.N;
    f.p = a.w + (size_t)(tile * 16 + (lane >> 3)) * (a.K >> 1) + st * 128 + (lane & 7) * 16;
    f.q = a.ws + (size_t)(tile * 16 + (lane & 15)) * (a.K / a.group) + st * (256 / a.group);
}
// Copy the present stage into a ring slot (row r's piece j of 16 bytes at 128 r + 16 (j ^ (r & 7)), then 16
// bytes of scales per row); rows and values outside read as zero.
template <int GL>
__device__ __forceinline__ void q4_issue(const Q4Args &a, const Q4Feed &f, uint8_t *slot) {
    constexpr int gs = 8 / GL;  // groups per stage
    const int lane = threadIdx.x & 31, r0 = lane >> 3, j = lane & 7;
    const uint32_t base = smem_addr(slot), d0 = base + r0 * 128 + ((j ^ r0) << 4), d1 = (d0 ^ 64) + 512;
    const size_t step = (size_t)a.K * 2;  // four rows
    if (a.wide && f.full) {
        cp_async16(d0, f.p, 16);
        cp_async16(d1, f.p + step, 16);
        cp_async16(d0 + 1024, f.p + 2 * step, 16);
        cp_async16(d1 + 1024, f.p + 3 * step, 16);
        if (lane < 16) {
            const uint32_t dst = base + 2048 + lane * 16;
            if (gs == 8) cp_async16(dst, f.q, 16);
            else cp_async_ca<gs * 2>(dst, f.q, gs * 2);
        }
    } else {
        const bool kin = (f.st * 8 + j) * 32 < a.K;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool in = kin && f.tile * 16 + r0 + 4 * i < a.N;
            cp_async16((i & 1 ? d1 : d0) + (i >> 1) * 1024, in ? f.p + i * step : a.w, in ? 16 : 0);
        }
        const int G = a.K / a.group;
        __half *d = reinterpret_cast<__half *>(slot + 2048);
        for (int i = lane; i < 16 * gs; i += 32) {
            const int r = i / gs, g = f.st * gs + i % gs, row = f.tile * 16 + r;
            d[r * 8 + i % gs] = row < a.N && g < G ? a.ws[(size_t)row * G + g] : __half();
        }
    }
}

__device__ __forceinline__ void q4_store(const Q4Args &a, int tok, int row, float v) {
    if (tok >= a.T || row >= a.N) return;
    const size_t at = (size_t)tok * a.N + row;
    if (a.ydt == RL_F32) {
        float *y = static_cast<float *>(a.y) + at;
        *y = a.acc ? *y + v : v;
    } else if (a.ydt == RL_F16) {
        __half *y = static_cast<__half *>(a.y) + at;
        *y = __float2half_rn(a.acc ? __half2float(*y) + v : v);
    } else {
        __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(a.y) + at;
        *y = __float2bfloat16_rn(a.acc ? __bfloat162float(*y) + v : v);
    }
}

// NT: column tiles of 8; GL: 32-value chunks per group
template <int NT, int KIND, int GL>
__global__ void __launch_bounds__(kQ4Threads, 1) q4_kernel(const Q4Args call, const Q4Layout lay) {
    constexpr bool SPLIT = KIND == kQ4Split;
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int TOK = NT * (SPLIT ? 4 : 8);
    // CTA row blockIdx.y takes TOK tokens of its own
    Q4Args a = call;
    if (blockIdx.y) {
        const int t0 = blockIdx.y * TOK;
        a.x = static_cast<const uint8_t *>(call.x) + (size_t)t0 * call.K * dtype_bytes(call.xdt);
        if (KIND == kQ4F8) a.xs = call.xs + (size_t)t0 * (call.K / call.group);
        a.y = static_cast<uint8_t *>(call.y) + (size_t)t0 * call.N * dtype_bytes(call.ydt);
        a.T -= t0;
    }
    if (a.T > TOK) a.T = TOK;
    constexpr int GS = 8 / GL;         // groups per stage: 8, 4, 2
    constexpr int YV = SPLIT ? 2 : 4;  // outputs per lane and column tile
    float *sc = reinterpret_cast<float *>(smem + lay.o_sc);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int grp = warp / a.W, sub = warp - grp * a.W, ngrp = kQ4Warps / a.W;
    const int tiles = (a.N + 15) / 16, first = grp * gridDim.x + blockIdx.x, step = ngrp * gridDim.x;
    uint8_t *ring = smem + lay.o_ring + (size_t)warp * a.stages * kQ4Stage;
    pdl_wait();
    pdl_trigger();
    // fill the ring; a commit per stage keeps the group count fixed
    Q4Feed feed;
    q4_seek(a, feed, first, sub);
    int pslot = 0;
    auto issue_next = [&]() {
        if (feed.tile < tiles) {
            q4_issue<GL>(a, feed, ring + pslot * kQ4Stage);
            feed.st += a.W;
            if (feed.st >= a.KC) {
                q4_seek(a, feed, feed.tile + step, sub);
            } else {
                feed.p += a.W * 128;
                feed.q += a.W * (8 / GL);
            }
        }
        cp_async_commit();
        if (++pslot == a.stages) pslot = 0;
    };
    for (int s = 0; s < a.stages - 1; ++s) issue_next();
    q4_stage_x<NT, KIND>(a, smem, sc);
    __syncthreads();
    const uint4 *bs = reinterpret_cast<const uint4 *>(smem) + lane;
    // ldmatrix: lane l addresses row (l & 7) + 8 (bit 3 of l) of 16-byte piece 2 jj + (l >> 4)
    const int lr = (lane & 7) + ((lane >> 3) & 1) * 8, lp = lane >> 4;
    const uint32_t lrow = smem_addr(ring) + lr * 128, x0 = (lp ^ (lr & 7)) << 4, x1 = x0 ^ 32, x2 = x0 ^ 64, x3 = x0 ^ 96;
    const Q4Const kc = q4_const();
    int slot = 0, parity = 0;
    for (int tile = first; tile < tiles; tile += step) {
        float y[NT][YV];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < YV; ++i) y[n][i] = 0.f;
        for (int st = sub; st < a.KC; st += a.W) {
            if (a.stages == 4) cp_async_wait_all_but<2>();
            else cp_async_wait_all_but<0>();
            __syncwarp();  // every lane's copies of this stage; the stage before has been read
            issue_next();
            const uint32_t sb = lrow + slot * kQ4Stage;
            const uint4 *bst = bs + st * (8 * NT * 32);
            const uint8_t *wsp = ring + slot * kQ4Stage + 2048 + g * 16;
            uint32_t sw[2][GS / 2 + (GS & 1)];  // the stage's scales of rows g and g + 8
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (GS == 8) {
                    const uint4 q = *reinterpret_cast<const uint4 *>(wsp + 128 * h);
                    sw[h][0] = q.x, sw[h][GS / 8] = q.y, sw[h][GS / 4] = q.z, sw[h][GS / 2 - 1] = q.w;
                } else if (GS == 4) {
                    const uint2 q = *reinterpret_cast<const uint2 *>(wsp + 128 * h);
                    sw[h][0] = q.x, sw[h][GS / 2 - 1] = q.y;
                } else {
                    sw[h][0] = *reinterpret_cast<const uint32_t *>(wsp + 128 * h);
                }
            }
            float acc[NT][4];
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
                uint32_t r[4];
                ldmatrix4(r, sb + (jj == 0 ? x0 : jj == 1 ? x1 : jj == 2 ? x2 : x3));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int c = 2 * jj + h;
                    const uint32_t w0 = r[2 * h], w1 = r[2 * h + 1], v0 = w0 >> 8, v1 = w1 >> 8;
                    const uint32_t a0 = q4_pair<true>(w0, kc), a1 = q4_pair<true>(w1, kc), a2 = q4_pair<false>(w0, kc),
                                   a3 = q4_pair<false>(w1, kc), a4 = q4_pair<true>(v0, kc), a5 = q4_pair<true>(v1, kc),
                                   a6 = q4_pair<false>(v0, kc), a7 = q4_pair<false>(v1, kc);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint4 b = bst[(c * NT + n) * 32];
                        if (c % GL == 0) mma_f16<false>(acc[n], a0, a1, a2, a3, b.x, b.y);
                        else mma_f16<true>(acc[n], a0, a1, a2, a3, b.x, b.y);
                        mma_f16<true>(acc[n], a4, a5, a6, a7, b.z, b.w);
                    }
                    if (c % GL == GL - 1) {
                        const int gi = c / GL;
                        const float2 f0 = unpack2(sw[0][gi >> 1], __half()), f1 = unpack2(sw[1][gi >> 1], __half());
                        const float s0 = gi & 1 ? f0.y : f0.x, s1 = gi & 1 ? f1.y : f1.x;
                        const float *p = sc + (st * (8 / GL) + gi) * TOK;
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            if (KIND == kQ4Split) {
                                y[n][0] = fmaf(s0, acc[n][0] + acc[n][1], y[n][0]);
                                y[n][1] = fmaf(s1, acc[n][2] + acc[n][3], y[n][1]);
                            } else {
                                float2 q = make_float2(1.f, 1.f);
                                if (KIND == kQ4F8) q = *reinterpret_cast<const float2 *>(p + n * 8 + 2 * t);
                                y[n][0] = fmaf(KIND == kQ4F8 ? s0 * q.x : s0, acc[n][0], y[n][0]);
                                y[n][1] = fmaf(KIND == kQ4F8 ? s0 * q.y : s0, acc[n][1], y[n][1]);
                                y[n][YV - 2] = fmaf(KIND == kQ4F8 ? s1 * q.x : s1, acc[n][2], y[n][YV - 2]);
                                y[n][YV - 1] = fmaf(KIND == kQ4F8 ? s1 * q.y : s1, acc[n][3], y[n][YV - 1]);
                            }
                        }
                    }
                }
            }
            if (++slot == a.stages) slot = 0;
        }
        // output i of column tile n: row g (+ 8 in the second half), token
        auto put = [&](int n, int i, int ln, float v) {
            const int row = tile * 16 + (ln >> 2) + (i >= YV / 2 ? 8 : 0);
            const int tok = SPLIT ? n * 4 + (ln & 3) : n * 8 + 2 * (ln & 3) + (i & 1);
            q4_store(a, tok, row, KIND == kQ4F8 ? v : v * sc[tok]);
        };
        if (a.W == 1) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < YV; ++i) put(n, i, lane, y[n][i]);
            continue;
        }
        // the W warps of the tile: partial sums through shared memory, two buffers in turn (a warp
        // that writes buffer p again has passed the barrier after everybody read it)
        constexpr int RV = NT * YV * 32;
        float *red = reinterpret_cast<float *>(smem + lay.o_red) + parity * kQ4Warps * RV + grp * a.W * RV;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < YV; ++i) red[sub * RV + (n * YV + i) * 32 + lane] = y[n][i];
        asm volatile("bar.sync %0, %1;" ::"r"(grp + 1), "r"(a.W * 32) : "memory");
        for (int e = sub; e < NT * YV; e += a.W) {
            float v = 0.f;
            for (int k = 0; k < a.W; ++k) v += red[k * RV + e * 32 + lane];
            put(e / YV, e % YV, lane, v);
        }
        parity ^= 1;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

struct Q4Plan {
    int NT, W, stages;
};

// NT column tiles: as few as hold the tokens of the launch.  W warps share a tile where the tiles alone do not
// fill every warp of the GPU (512 rows of 2048: 8 warps per tile); where they do, one warp per tile
// takes 29.6 us on the 131072-row head, two 31.5 and four 32.9 (no partial sums to exchange).  Four
// column tiles leave no room for the partial sums, so they need tiles for every warp.
bool q4_plan(int N, int K, int cols, int group, int kind, Q4Plan &p) {
    const int KC = (K + 255) / 256, tiles = (N + 15) / 16;
    const size_t room = 227 * 1024;
    p.NT = cols > 16 && tiles >= 152 * kQ4Warps ? 4 : cols > 8 ? 2 : 1;
    for (; p.NT >= 1; p.NT >>= 1) {
        p.W = 1;
        if (p.NT < 4)
            while (p.W < 8 && 2 * p.W <= KC && tiles * p.W < 152 * kQ4Warps) p.W *= 2;
        for (; p.W >= 1; p.W >>= 1)
            for (p.stages = 4; p.stages >= 2; p.stages -= 2)
                if (Q4Layout(KC, p.NT, kind, group, p.W, p.stages).total <= room) return true;
    }
    return false;
}

template <int NT, int KIND>
rl_status launch_q4(const Q4Args &a, const Q4Layout &lay, cudaStream_t s) {
    const int tiles = (a.N + 15) / 16, sms = sm_count();
    const int tok = NT * (KIND == kQ4Split ? 4 : 8);
    const dim3 grid(tiles < sms ? tiles : sms, (a.T + tok - 1) / tok), block(kQ4Threads);
    if (a.group == 32) return launch_pdl(q4_kernel<NT, KIND, 1>, grid, block, lay.total, s, "rl_q4_matvec", a, lay);
    if (a.group == 64) return launch_pdl(q4_kernel<NT, KIND, 2>, grid, block, lay.total, s, "rl_q4_matvec", a, lay);
    return launch_pdl(q4_kernel<NT, KIND, 4>, grid, block, lay.total, s, "rl_q4_matvec", a, lay);
}

template <int KIND>
rl_status launch_q4_kind(const Q4Args &a, const Q4Layout &lay, int NT, cudaStream_t s) {
    return NT == 4 ? launch_q4<4, KIND>(a, lay, s) : NT == 2 ? launch_q4<2, KIND>(a, lay, s) : launch_q4<1, KIND>(a, lay, s);
}

}  // namespace

extern "C" rl_status rl_q4_matvec(const uint8_t *w, const void *w_scale, int32_t N, int32_t K, int32_t group,
                                  const void *x, int32_t x_dtype, const float *x_scale, int32_t T, void *y,
                                  int32_t y_dtype, int32_t accumulate, void *stream) {
    if (x_dtype != RL_F32 && x_dtype != RL_F16 && x_dtype != RL_BF16 && x_dtype != RL_F8_E4M3)
        return fail(RL_ERR_INVALID, "rl_q4_matvec: unknown x_dtype %d", x_dtype);
    if (y_dtype != RL_F32 && y_dtype != RL_F16 && y_dtype != RL_BF16)
        return fail(RL_ERR_INVALID, "rl_q4_matvec: y_dtype %d is none of RL_F32, RL_F16, RL_BF16", y_dtype);
    if (N <= 0 || K <= 0 || T < 0) return fail(RL_ERR_INVALID, "rl_q4_matvec: N=%d K=%d T=%d", N, K, T);
    if (!(group == 32 || group == 64 || group == 128))
        return fail(RL_ERR_UNSUPPORTED, "rl_q4_matvec: group=%d: supported 32, 64, 128", group);
    if (K % group != 0) return fail(RL_ERR_INVALID, "rl_q4_matvec: K=%d is not a multiple of group=%d", K, group);
    if (K > kQ4MaxK) return fail(RL_ERR_UNSUPPORTED, "rl_q4_matvec: K=%d > %d", K, kQ4MaxK);
    if (N > (1 << 26)) return fail(RL_ERR_UNSUPPORTED, "rl_q4_matvec: N=%d > 2^26", N);
    if (T == 0) return RL_OK;
    if (!w || !w_scale || !x || !y) return fail(RL_ERR_INVALID, "rl_q4_matvec: NULL buffer");
    if ((x_dtype == RL_F8_E4M3) != (x_scale != nullptr))
        return fail(RL_ERR_INVALID, "rl_q4_matvec: x_scale comes with RL_F8_E4M3 activations");
    if ((reinterpret_cast<uintptr_t>(w) | reinterpret_cast<uintptr_t>(w_scale) | reinterpret_cast<uintptr_t>(x)) & 15)
        return fail(RL_ERR_INVALID, "rl_q4_matvec: w, w_scale and x must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(x_scale) & 3 || reinterpret_cast<uintptr_t>(y) % dtype_bytes(y_dtype))
        return fail(RL_ERR_INVALID, "rl_q4_matvec: x_scale or y misaligned");
    const int kind = x_dtype == RL_F32 ? kQ4Split : x_dtype == RL_F8_E4M3 ? kQ4F8 : kQ4Half;
    const int per = kind == kQ4Split ? 2 : 1;  // columns per token
    cudaStream_t s = as_stream(stream);
    for (int t0 = 0; t0 < T;) {
        Q4Plan p;
        if (!q4_plan(N, K, (T - t0) * per < 32 ? (T - t0) * per : 32, group, kind, p))
            return fail(RL_ERR_UNSUPPORTED, "rl_q4_matvec: K=%d does not fit", K);
        const int most = 8 * p.NT / per;
        Q4Args a = {};
        a.w = w;
        a.ws = static_cast<const __half *>(w_scale);
        a.x = static_cast<const uint8_t *>(x) + (size_t)t0 * K * dtype_bytes(x_dtype);
        a.xs = x_scale ? x_scale + (size_t)t0 * (K / group) : nullptr;
        a.y = static_cast<uint8_t *>(y) + (size_t)t0 * N * dtype_bytes(y_dtype);
        a.N = N;
        a.K = K;
        // All full column groups in one launch (64 f32 rows: 512 x 2048 takes 11.7 us, with a launch per group
        // 44.4; 20000 x 2048 78.5 and 94.7).  The rest joins it where the tiles leave SMs idle; a larger
        // matrix takes the rest with fewer columns (100003 x 2048, 40 bf16 rows: 85.8 us, joined 109).
        const int rest = T - t0, full = rest / most * most;
        a.T = rest < most || (N + 15) / 16 < sm_count() ? rest : full;
        if (a.T > most * 65535) a.T = most * 65535;
        a.group = group;
        a.xdt = x_dtype;
        a.ydt = y_dtype;
        a.acc = accumulate != 0;
        a.KC = (K + 255) / 256;
        a.inv = (uint32_t)(((1ull << 32) + a.KC * 32 - 1) / (a.KC * 32));
        a.W = p.W;
        a.stages = p.stages;
        a.wide = K % 256 == 0;
        const Q4Layout lay(a.KC, p.NT, kind, group, p.W, p.stages);
        const rl_status st = kind == kQ4Split ? launch_q4_kind<kQ4Split>(a, lay, p.NT, s)
                             : kind == kQ4F8  ? launch_q4_kind<kQ4F8>(a, lay, p.NT, s)
                                              : launch_q4_kind<kQ4Half>(a, lay, p.NT, s);
        if (st != RL_OK) return st;
        t0 += a.T;
    }
    return RL_OK;
}
