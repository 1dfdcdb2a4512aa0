// f8_matmul.cu - rl_f8_matmul and rl_f8_gated: products of 8-bit activations (e4m3, an f32 scale per 128
// values of a row) and 8-bit weights (e4m3, an f32 scale per block of 128 x 128).
//
//   acc[t][n] = sum_b xs[t][b] ws[n / 128][b] sum_{k in block b} x[t][k] w[n][k]
//   rl_f8_matmul: y = acc (+ res);  rl_f8_gated: h = silu(acc of gate) * (acc of up), as it is or in 8 bits
//
// The sum over a block of 128 runs on the tensor cores (tcgen05, kind::f8f6f4, f32 accumulators in tensor
// memory); the two scales multiply it when it is read back, in f32 registers ("promotion"), while the tensor
// cores work on the next block in another accumulator.  Two kernels:
//
//   rows  up to 128 rows per pass.  A operand: 128 weight rows, B operand: the activation rows (16, 32, 64
//         or 128 of them), so that few rows waste no tensor work.  Lane = weight row, column = token.
//   wide  many rows.  A operand: 256 activation rows over a pair of CTAs, B operand: 256 weight rows.  Lane =
//         token, so that a lane's scale is one number per block.
//
// Up to 128 rows (64 in the gated form) take the first kernel.  Both sides of that, rows / wide, in us:
//   8192 x 8192: 128 rows 23 / 42, 129 37 / 41, 384 72 / 42      10007 x 1040: 65 rows 9.5 / 10.1, 128 11.1 / 11.1, 129 14.7 / 11.0
//   32768 x 2048: 64 rows 24 / 25, 128 29 / 26, 129 45 / 27      2048 x 512: 128 rows 6.8 / 8.0, 256 7.2 / 8.1, 384 8.4 / 8.1
//   gated 8192 x 4096: 64 rows 19 / 30, 128 26 / 30, 129 47 / 31        gated 512 x 2048: 64 rows 7.7 / 18, 128 8.0 / 18, 256 15 / 15
// A pass over the rows in the first kernel reads all weights, so the limit is where a second pass would begin; matrices with
// fewer tiles than SMs would bear two or three (512 x 2048 and 65 gated rows: 18 where 8 would do).
// Small matrices are split over clusters of up to 8 CTAs along the shared dimension, so that one row of 512 x 2048 does not run
// through four CTAs alone.
//
// Measured back to back in a graph (us; the copy rate allows, where bytes bound): 1 row of 2048 x 512 4.6; 8 rows of 131072 x
// 2048 47 to 50 (41: 82 to 87% of the copy rate); 77 rows of 10007 x 1040 9.5 to 10 (1.8; the latency of nine blocks, start and
// stores); 4096 rows of 8192 x 8192 253, 2.17 PFLOP/s, 1.13 times what the cuBLAS bf16 product reaches; gated 512 x 2048: 1 row
// 5.3, 2048 rows 14.6; gated 8192 x 4096, 4096 rows 281, 1.96 PFLOP/s.  The large products are bound by the way of a block from the end of its
// MMAs over the waiting warp, the reads of tensor memory and the other CTA's arrival back to the issuing thread: two
// accumulators of 256 columns fill tensor memory, so only one other block hides it (the tensor pipe is 45% busy).
//
// Both: the first 8 or 16 warps promote (warp w reads the lanes of quadrant w % 4, a share of the columns
// each), one warp loads (tensor copies with the 128-byte swizzle, 4-byte asynchronous copies for the
// scales), one thread of another issues the MMAs (wide: a thread each of two others, every other block), one warp waits for the
// promoting ones.
#include "qdot.cuh"
#include "row_types.cuh"
#include "tc_desc.cuh"

using namespace rl;

namespace {

constexpr int kG = 128;                       // values per scale
constexpr int kTileBytes = 128 * kG;          // 128 rows of one block
constexpr int kThreads = 352, kLoadW = 8, kMmaW = 9, kPollW = 10;
constexpr int kMaxCluster = 8;

struct F8Args {
    CUtensorMap wmap[2];   // weights (gate, up), boxes of 128 rows x 128 values
    CUtensorMap xmap;      // activations, boxes of the kernel's row tile x 128 values
    const float *ws[2];    // [ceil(N / 128)][KB]
    const float *xs;       // [T][KB]
    void *y;               // [T][N] of dtype (gated: h, may be NULL)
    const void *res;       // [T][N] of dtype or NULL
    uint8_t *q;            // gated: e4m3 [T][N]
    float *scale;          // gated: [T][ceil(N / 128)]
    int32_t *ctrl;
    int layer;
    int T, N, K, KB, dtype;
    int tiles_n, tiles;    // weight tiles, all tiles
};

__device__ __forceinline__ float load1(const void *p, size_t i, int dt) {
    if (dt == RL_F32) return static_cast<const float *>(p)[i];
    if (dt == RL_F16) return __half2float(static_cast<const __half *>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}
__device__ __forceinline__ void store1(void *p, size_t i, float v, int dt) {
    if (dt == RL_F32) static_cast<float *>(p)[i] = v;
    else if (dt == RL_F16) static_cast<__half *>(p)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ unsigned long long dup2(float v) { return pack2(__float_as_uint(v), __float_as_uint(v)); }
__device__ __forceinline__ unsigned long long fmul2(unsigned long long a, unsigned long long b) {
    unsigned long long d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float lo2(unsigned long long v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi2(unsigned long long v) { return __uint_as_float((uint32_t)(v >> 32)); }

// arrives on `bar` (which counts every lane) when this thread's cp.async copies so far have landed
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t a, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 ld_peer4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
    return v;
}
// The sum over the cluster's S CTAs, in rank order, of the four values at this shared-memory address in each; all loads are
// on their way before the first is used (one after the other they cost 700 cycles each).
__device__ __forceinline__ float4 sum_peers(uint32_t at, int S) {
    float4 v[kMaxCluster];
#pragma unroll
    for (int p = 0; p < kMaxCluster; ++p) v[p] = p < S ? ld_peer4(peer_addr(at, p)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int p = 1; p < kMaxCluster; ++p)
        if (p < S) v[0].x += v[p].x, v[0].y += v[p].y, v[0].z += v[p].z, v[0].w += v[p].w;
    return v[0];
}
__device__ __forceinline__ float4 lds_f4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ void epi_sync() {  // the 256 promoting threads
    asm volatile("bar.sync 1, 256;" ::: "memory");
    __syncwarp();
}

// The outputs of the gated form for 128 values of one row, lane L holding values 4 L .. 4 L + 3 of group g:
// stored in the row type, or as e4m3 with the group's scale max|h| / 448 (a group that holds an infinity or
// a NaN: scale NaN, zeros).  Whole warp.
__device__ __forceinline__ void gated_store(const F8Args &a, int t, int g, float (&h)[4]) {
    const int lane = threadIdx.x & 31, i = g * kG + 4 * lane;
    const size_t at = (size_t)t * a.N + i;
    if (a.y) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j < a.N) store1(a.y, at + j, h[j], a.dtype);
    }
    if (!a.q) return;
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max_abs_nan(m, i + j < a.N ? h[j] : 0.f);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(kFull, m, o));
    const bool bad = !(m < INFINITY);
    const float f = m > 0.f && !bad ? 448.f / m : 0.f;
    if (lane == 0) a.scale[(size_t)t * a.tiles_n + g] = bad ? __int_as_float(0x7fffffff) : m / 448.f;
    uint32_t w = 0u;
    if (f > 0.f) {
        // a quotient beyond f32 (m below 448 / the largest f32) goes in two steps
        if (f < INFINITY) w = pack4_e4m3(h[0] * f, h[1] * f, h[2] * f, h[3] * f);
        else {
            const float s = 18446744073709551616.f, f2 = 448.f / (m * s);
            w = pack4_e4m3(h[0] * s * f2, h[1] * s * f2, h[2] * s * f2, h[3] * s * f2);
        }
    }
    if (i + 4 <= a.N && (a.N & 3) == 0) {
        *reinterpret_cast<uint32_t *>(a.q + at) = w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j < a.N) a.q[at + j] = (uint8_t)(w >> (8 * j));
    }
}

// After a wait that ran out: NaN as the outputs of rows t0 .. t0 + rows - 1 and columns n0 .. n0 + cols - 1 (gated: a group; its scale
// NaN and q 0).  By the first `threads` threads.
template <bool GATED>
__device__ __noinline__ void spoil(const F8Args &a, int threads, int t0, int rows, int n0, int cols) {
    for (int e = threadIdx.x; e < rows * cols && threadIdx.x < threads; e += threads) {
        const int t = t0 + e / cols, n = n0 + e % cols;
        if (t >= a.T || n >= a.N) continue;
        const size_t at = (size_t)t * a.N + n;
        if (a.y) store1(a.y, at, __int_as_float(0x7fffffff), a.dtype);
        if (GATED && a.q) {
            a.q[at] = 0;
            if (n == n0) a.scale[(size_t)t * a.tiles_n + n0 / kG] = __int_as_float(0x7fffffff);
        }
    }
    __syncwarp();
}

// ---- rows: 128 weight rows x TT tokens per tile -----------------------------------------------
template <int TT, bool GATED>
struct Rows {
    static constexpr int NA = GATED ? 2 : 1;
    static constexpr int kStage = NA * kTileBytes + TT * kG;
    static constexpr int kStages = GATED ? 3 : TT >= 128 ? 4 : 5;
    static constexpr int kBufs = NA * TT >= 128 ? 2 : 4;              // accumulators in tensor memory
    static constexpr int kCols = kBufs * NA * TT < 32 ? 32 : kBufs * NA * TT;
    static constexpr int kScales = TT + 4;                             // floats per block: xs of the tokens, ws
    // A slot's (and its barrier's) last block was released when the MMAs of the block kStages before are done, for they
    // followed the release of the one kBufs before those.  A barrier per stage would not do: MMAs do not wait for
    // scales, so a lane's arrival for the stage's next block could count for a block whose copies are still on their way.
    static constexpr int kSlots = 16;
    static_assert(kSlots >= kStages + kBufs, "scales are not overwritten before their block is released");
    static constexpr int o_sc = 1024;
    static constexpr int o_ring = (o_sc + kSlots * kScales * 4 + 1023) / 1024 * 1024;
    static constexpr int o_part = o_ring + kStages * kStage;           // f32 [NA][TT][128] (see below)
    // A tile's sums go through shared memory, and a short loop makes the outputs: straight code that a CTA runs once costs
    // 17 cycles an instruction (64 outputs, or 32 activations, per thread unrolled: 5 to 9 us).
    static constexpr bool kStaged = GATED || TT >= 64;
    static constexpr size_t bytes(bool split) {
        return o_part + (split || kStaged ? NA * TT * 512 : 0);
    }
    static_assert(o_part + NA * TT * 512 <= 232448, "shared memory of one CTA");
};

// Tiles of 128 weight rows (of each matrix) x TT tokens.  With a cluster of S > 1 CTAs every CTA takes a
// share of the blocks of one tile, the partial sums are left in shared memory and added in rank order by
// the cluster, each CTA a share of the outputs; with S = 1 the CTAs walk over the tiles.
template <int TT, bool GATED>
__global__ void __launch_bounds__(kThreads, 1) f8_rows_kernel(const __grid_constant__ F8Args a, int S) {
    using R = Rows<TT, GATED>;
    constexpr int NA = R::NA, CW = TT / 2;  // columns per promoting warp
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *full = reinterpret_cast<uint64_t *>(smem), *empty = full + 8, *sc_full = full + 16;
    uint64_t *d_full = full + 32, *d_empty = full + 36, *fin = full + 40;
    uint32_t *tmem_s = reinterpret_cast<uint32_t *>(smem + 512);
    int *abort_s = reinterpret_cast<int *>(smem + 516), *leave_s = reinterpret_cast<int *>(smem + 520);
    int *left_s = reinterpret_cast<int *>(smem + 524);  // the first tile without sums
    float *sc = reinterpret_cast<float *>(smem + R::o_sc);
    float *part = reinterpret_cast<float *>(smem + R::o_part);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < R::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < R::kSlots; ++i) mbar_init(&sc_full[i], 32);
        for (int i = 0; i < R::kBufs; ++i) {
            mbar_init(&d_full[i], 1);
            mbar_init(&d_empty[i], 8);
        }
        mbar_init(fin, 1);
        *abort_s = *leave_s = 0;
        *left_s = 0x7fffffff;
        fence_mbar_init();
    }
    if (warp == 0) {
        tc::tmem_alloc(tmem_s, R::kCols);
        tc::tmem_relinquish();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *tmem_s;
    pdl_wait();
    pdl_trigger();  // after the allocation: a dependent that allocates first could never be passed
    const bool skip = a.ctrl && ld_ctrl(a.ctrl) <= a.layer;
    const int rank = S > 1 ? (int)cluster_rank() : 0;
    const int first = S > 1 ? blockIdx.x / S : blockIdx.x, step = gridDim.x / S;
    const int kb0 = (int)((long long)a.KB * rank / S), kb1 = (int)((long long)a.KB * (rank + 1) / S);
    const uint32_t blocks = first < a.tiles ? (uint32_t)((a.tiles - 1 - first) / step + 1) * (uint32_t)(kb1 - kb0) : 0u;
    bool failed = false;
    auto wait = [&](uint64_t *bar, uint32_t parity) {  // of one thread
        for (uint32_t i = 0; i < kSpinPolls; ++i)
            if (mbar_test_wait(bar, parity)) return true;
        atomicExch(abort_s, 1);
        failed = true;
        return false;
    };

    if (skip) {
        // nothing to do, in any CTA
    } else if (warp == kLoadW) {
        uint32_t n = 0;
        for (int tile = first; tile < a.tiles && !failed; tile += step) {
            const int tn = tile % a.tiles_n, t0 = tile / a.tiles_n * TT;
            for (int kb = kb0; kb < kb1; ++kb, ++n) {
                const int s = n % R::kStages;
                if (lane == 0 && (n < (uint32_t)R::kStages || wait(&empty[s], (n / R::kStages - 1) & 1))) {
                    uint8_t *st = smem + R::o_ring + s * R::kStage;
                    mbar_arrive_expect_tx(&full[s], R::kStage);
#pragma unroll
                    for (int m = 0; m < NA; ++m) tma_load_2d(st + m * kTileBytes, &a.wmap[m], kb * kG, tn * 128, &full[s]);
                    tma_load_2d(st + NA * kTileBytes, &a.xmap, kb * kG, t0, &full[s]);
                }
                __syncwarp();
                failed = __any_sync(kFull, failed);
                if (failed) break;
                const uint32_t dst = smem_addr(sc + (n % R::kSlots) * R::kScales);
#pragma unroll
                for (int i = 0; i < (TT + 31) / 32; ++i) {
                    const int t = 32 * i + lane;
                    if (t < TT)
                        cp_async_ca<4>(dst + 4 * t, a.xs + (t0 + t < a.T ? (size_t)(t0 + t) * a.KB + kb : 0),
                                       t0 + t < a.T ? 4 : 0);
                }
                if (lane < NA) cp_async_ca<4>(dst + 4 * (TT + lane), a.ws[lane] + (size_t)tn * a.KB + kb, 4);
                cp_async_arrive(&sc_full[n % R::kSlots]);
                __syncwarp();
            }
        }
        cp_async_commit();
        cp_async_wait_all_but<0>();
        // copies that nobody waited for (only after a failure) land before the CTA exits
        if (failed)
            for (uint32_t j = n >= (uint32_t)R::kStages ? n - R::kStages : 0; j < n; ++j)
                mbar_wait_warp(&full[j % R::kStages], (j / R::kStages) & 1);
    } else if (warp == kMmaW) {
        if (lane == 0) {
            const uint32_t idesc = tc::instr_desc(0u, 128, TT), ring = smem_addr(smem + R::o_ring);
            for (uint32_t n = 0; n < blocks; ++n) {
                const int s = n % R::kStages, b = n % R::kBufs;
                if (!wait(&full[s], (n / R::kStages) & 1)) break;
                if (n >= (uint32_t)R::kBufs && !wait(&d_empty[b], (n / R::kBufs - 1) & 1)) break;
                tc::fence_after();
                const uint32_t st = ring + s * R::kStage;
                const uint64_t bd = tc::smem_desc_sw128(st + NA * kTileBytes, 1024);
#pragma unroll
                for (int m = 0; m < NA; ++m) {
                    const uint64_t ad = tc::smem_desc_sw128(st + m * kTileBytes, 1024);
#pragma unroll
                    for (int k = 0; k < kG / 32; ++k)
                        tc::mma_f8(tmem + (b * NA + m) * TT, ad + 2 * k, bd + 2 * k, idesc, k > 0);
                }
                tc::commit(&d_full[b]);
                tc::commit(&empty[s]);
            }
        }
        __syncwarp();
    } else if (warp == kPollW) {
        // waits for each block's scales and product and lets the promoting warps pass the barrier of its buffer
        // (id 2 + buffer); the next arrival there comes after they have released the buffer
        for (uint32_t n = 0; n < blocks; ++n) {
            const int b = n % R::kBufs;
            bool ok = true;
            if (lane == 0 && (!wait(&sc_full[n % R::kSlots], (n / R::kSlots) & 1) || !wait(&d_full[b], (n / R::kBufs) & 1))) {
                ok = false;
                *reinterpret_cast<volatile int *>(leave_s) = 1;
                __threadfence_block();
            }
            __syncwarp();
            ok = __all_sync(kFull, ok);
            asm volatile("bar.arrive %0, 288;" ::"r"(2 + b) : "memory");
            if (!ok) break;
        }
    } else if (warp < 8) {
        const int qd = warp & 3, c0 = (warp >> 2) * CW;  // lane quadrant, first column
        const uint32_t trow = tmem + ((uint32_t)(32 * qd) << 16) + c0;
        const int row = 32 * qd + lane;
        uint32_t n = 0;
        for (int tile = first; tile < a.tiles && !failed; tile += step) {
            const int tn = tile % a.tiles_n, t0 = tile / a.tiles_n * TT;
            const int nt = a.T - t0 < TT ? a.T - t0 : TT;
            unsigned long long acc[NA][CW / 2];
#pragma unroll
            for (int m = 0; m < NA; ++m)
#pragma unroll
                for (int j = 0; j < CW / 2; ++j) acc[m][j] = 0ull;
            for (int kb = kb0; kb < kb1; ++kb, ++n) {
                const int b = n % R::kBufs;
                asm volatile("bar.sync %0, 288;" ::"r"(2 + b) : "memory");
                __syncwarp();
                if (*reinterpret_cast<volatile int *>(leave_s)) {  // the same for all eight warps: set before the arrival
                    failed = true;
                    break;
                }
                tc::fence_after();
                const float *ss = sc + (n % R::kSlots) * R::kScales;
                const uint32_t xa = smem_addr(ss + c0);
                constexpr int C = CW < 16 ? CW : 16;
#pragma unroll
                for (int c = 0; c < CW; c += C) {
                    uint32_t d[NA][C];
#pragma unroll
                    for (int m = 0; m < NA; ++m) {
                        if constexpr (C == 8) tc::ld8(trow + (b * NA + m) * TT + c, d[m]);
                        else tc::ld16(trow + (b * NA + m) * TT + c, d[m]);
                    }
                    unsigned long long x2[C / 2];
#pragma unroll
                    for (int j = 0; j < C; j += 4) {
                        const float4 v = lds_f4(xa + 4 * (c + j));
                        x2[j / 2] = pack2(__float_as_uint(v.x), __float_as_uint(v.y));
                        x2[j / 2 + 1] = pack2(__float_as_uint(v.z), __float_as_uint(v.w));
                    }
#pragma unroll
                    for (int m = 0; m < NA; ++m) {
                        const unsigned long long w2 = dup2(ss[TT + m]);
                        tc::ld_wait(d[m]);
#pragma unroll
                        for (int j = 0; j < C; j += 2)
                            acc[m][(c + j) / 2] = ffma2(pack2(d[m][j], d[m][j + 1]), fmul2(x2[j / 2], w2), acc[m][(c + j) / 2]);
                    }
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&d_empty[b]);
                __syncwarp();  // rejoin the warp (see cta_sync)
            }
            if (failed) {
                *left_s = tile;  // the same of all eight warps
                break;
            }
            if (S > 1 || R::kStaged) {
#pragma unroll
                for (int m = 0; m < NA; ++m)
#pragma unroll
                    for (int j = 0; j < CW; ++j)
                        if (c0 + j < nt)
                            part[(m * TT + c0 + j) * 128 + row] = j & 1 ? hi2(acc[m][j / 2]) : lo2(acc[m][j / 2]);
                if (S == 1) {
                    epi_sync();
                    if constexpr (!GATED) {
                        const int col = tn * 128 + (tid & 127);
                        if (col < a.N) {
#pragma unroll 4
                            for (int t = tid >> 7; t < nt; t += 2) {
                                const size_t at = (size_t)(t0 + t) * a.N + col;
                                float v = part[t * 128 + (tid & 127)];
                                if (a.res) v += load1(a.res, at, a.dtype);
                                store1(a.y, at, v, a.dtype);
                            }
                        }
                    } else {
#pragma unroll 1
                        for (int t = warp; t < nt; t += 8) {
                            const float4 g = lds_f4(smem_addr(part + t * 128 + 4 * lane));
                            const float4 u = lds_f4(smem_addr(part + (TT + t) * 128 + 4 * lane));
                            float h[4] = {silu(g.x) * u.x, silu(g.y) * u.y, silu(g.z) * u.z, silu(g.w) * u.w};
                            gated_store(a, t0 + t, tn, h);
                        }
                    }
                    epi_sync();  // the sums are read before the next tile's are written
                }
            } else if constexpr (!GATED) {
                const int col = tn * 128 + row;
                if (col < a.N) {
#pragma unroll
                    for (int j = 0; j < CW; ++j) {
                        if (c0 + j < nt) {
                            const size_t at = (size_t)(t0 + c0 + j) * a.N + col;
                            float v = j & 1 ? hi2(acc[0][j / 2]) : lo2(acc[0][j / 2]);
                            if (a.res) v += load1(a.res, at, a.dtype);
                            store1(a.y, at, v, a.dtype);
                        }
                    }
                }
            }
        }
    }
    __syncwarp();
    __syncthreads();
    const bool bad = *reinterpret_cast<volatile int *>(abort_s) != 0;
    if (bad) {  // outputs that could not be computed are NaN, so that a call without ctrl tells of it too
        int tile = *reinterpret_cast<volatile int *>(left_s);
        if (S > 1 && tile < a.tiles) {
            for (int e = tid; e < NA * TT * 128; e += kThreads) part[e] = __int_as_float(0x7fffffff);
            __syncwarp();
        }
        if (S == 1)
            for (; tile < a.tiles; tile += step) spoil<GATED>(a, kThreads, tile / a.tiles_n * TT, TT, tile % a.tiles_n * 128, 128);
    }
    if (S > 1) {
        cluster_sync();
        if (!skip) {
            const int tn = first % a.tiles_n, t0 = first / a.tiles_n * TT;
            const int nt = a.T - t0 < TT ? a.T - t0 : TT;
            const uint32_t base = smem_addr(part);
            if constexpr (!GATED) {
#pragma unroll 1
                for (int e = rank * kThreads + tid; e < nt * 32; e += S * kThreads) {
                    const int t = e >> 5, col = tn * 128 + 4 * (e & 31);
                    const float4 f = sum_peers(base + 16 * e, S);
                    const float v[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (col + j < a.N) {
                            const size_t at = (size_t)(t0 + t) * a.N + col + j;
                            store1(a.y, at, a.res ? v[j] + load1(a.res, at, a.dtype) : v[j], a.dtype);
                        }
                    }
                }
            } else {
#pragma unroll 1
                for (int t = rank + S * warp; t < nt; t += S * (kThreads / 32)) {
                    const uint32_t at = base + 4 * (t * 128 + 4 * lane);
                    const float4 g = sum_peers(at, S), u = sum_peers(at + 4 * TT * 128, S);
                    float h[4] = {silu(g.x) * u.x, silu(g.y) * u.y, silu(g.z) * u.z, silu(g.w) * u.w};
                    gated_store(a, t0 + t, tn, h);
                }
            }
        }
        __syncwarp();
        cluster_sync();
    }
    if (bad) {  // MMAs in flight end before tensor memory is given back
        if (tid == 0 && a.ctrl) dev_error(a.ctrl, RL_DEVERR_WAIT_TIMEOUT);
        if (tid == kMmaW * 32) {
            tc::commit(fin);
            mbar_wait(fin, 0);
        }
        __syncwarp();
        __syncthreads();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 0) tc::tmem_dealloc(tmem, R::kCols);
}

// ---- wide: 256 tokens x 256 weight rows per pair of CTAs ----------------------------------------
// A pair shares its weights: each CTA has 128 tokens (its lanes) and loads half of the 256 weight rows, so that a
// block costs an SM 32 KB of shared memory traffic in instead of 48 KB.  Sixteen warps promote, 64 columns
// each.  Two threads issue the MMAs of every other block: one needs about 1200 cycles for a block's two waits, four MMAs
// and two commits beside the promoting warps, the tensor cores 512.
constexpr int kWThreads = 640, kWEpi = 16, kWLoadW = 16, kWMmaW = 17 /* and 18 */, kWPollW = 19;
constexpr int kWStages = 4, kWStage = 2 * kTileBytes;
constexpr int kWScales = 132, kWSlots = 16;                              // a block's scales: 128 tokens, the two halves' weights
constexpr int kWoRing = 1024;
constexpr int kWoOut = kWoRing + kWStages * kWStage;                    // per warp 32 x 33 floats
constexpr int kWOutFloats = 32 * 33;
constexpr int kWoTop = kWoOut + kWEpi * kWOutFloats * 4;                // gated: maxima of [4][128] row quarters
constexpr int kWoSc = kWoTop + 4 * 128 * 4;
constexpr size_t kWBytes = kWoSc + kWSlots * kWScales * 4;
static_assert(kWBytes <= 232448, "shared memory of one CTA");

__device__ __forceinline__ void wide_sync() {  // the sixteen promoting warps
    asm volatile("bar.sync 1, 512;" ::: "memory");
    __syncwarp();
}
// Arrive on an mbarrier of the cluster, by its address there.  Relaxed: what it tells of are reads of tensor memory that
// have returned their values, and it publishes no memory (as a release, 8192 x 8192 x 4096 takes 485 us in place of 253).
// The reads of a block's scales are not ordered by it: they have returned before the warp's multiply-adds of that block
// were issued, those before the next block's values were loaded into the same registers, and a slot of scales is written
// again only after the release of the block three after its own.
__device__ __forceinline__ void arrive_at(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// tma_load_2d into this CTA's shared memory, completing on the mbarrier `bar` of either CTA of the pair
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// 32 values of each lane's row from column n on, the lanes' rows starting at t.  Through shared memory, so that a warp
// stores 32 neighbouring values at a time, wherever rows start: 32768 f32 outputs of 4096 rows from K = 32 take 93 us, with
// pieces of 16 bytes straight from the lanes, 32 rows apart, 288.
template <typename E>
__device__ __forceinline__ void put32_as(void *to, const float *stage, int N, int rows, size_t at) {
    E *y = static_cast<E *>(to) + at;
#pragma unroll 8
    for (int r = 0; r < rows; ++r, y += N) *y = from_float<E>(stage[r * 33]);
}
// the same with a residual
template <typename E>
__device__ __forceinline__ void put32_res(void *to, const void *res, const float *stage, int N, int rows, size_t at) {
    E *y = static_cast<E *>(to) + at;
    const E *e = static_cast<const E *>(res) + at;
    for (int r0 = 0; r0 < rows; r0 += 16) {  // the reads first: res may be y, so they would wait for the stores
        float q[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) q[r] = r0 + r < rows ? to_float(e[(size_t)(r0 + r) * N]) : 0.f;
#pragma unroll
        for (int r = 0; r < 16; ++r)
            if (r0 + r < rows) y[(size_t)(r0 + r) * N] = from_float<E>(stage[(r0 + r) * 33] + q[r]);
    }
}
template <bool RES>
__device__ __forceinline__ void put32(const F8Args &a, float *stage, int t, int n, const unsigned long long (&v)[16]) {
    const int lane = threadIdx.x & 31, rows = a.T - t < 32 ? a.T - t : 32;
#pragma unroll
    for (int j = 0; j < 16; ++j) stage[lane * 33 + 2 * j] = lo2(v[j]), stage[lane * 33 + 2 * j + 1] = hi2(v[j]);
    __syncwarp();
    if (n + lane < a.N && rows > 0) {
        const size_t at = (size_t)t * a.N + n + lane;
        const float *mine = stage + lane;
        if constexpr (RES) {
            if (a.dtype == RL_F32) put32_res<float>(a.y, a.res, mine, a.N, rows, at);
            else if (a.dtype == RL_F16) put32_res<__half>(a.y, a.res, mine, a.N, rows, at);
            else put32_res<__nv_bfloat16>(a.y, a.res, mine, a.N, rows, at);
        } else {
            if (a.dtype == RL_F32) put32_as<float>(a.y, mine, a.N, rows, at);
            else if (a.dtype == RL_F16) put32_as<__half>(a.y, mine, a.N, rows, at);
            else put32_as<__nv_bfloat16>(a.y, mine, a.N, rows, at);
        }
    }
    __syncwarp();
}

// GATED: the 256 weight rows are 128 rows of the gate's matrix and the same 128 of the up matrix.  RES: a residual is added (a
// variant of its own, because the registers of its loads slow the promotion down by 5% even where there is none).
template <bool GATED, bool RES>
__global__ void __launch_bounds__(kWThreads, 1) f8_wide_kernel(const __grid_constant__ F8Args a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    // full and d_empty: of the even CTA, for both; the others: of each CTA
    uint64_t *full = reinterpret_cast<uint64_t *>(smem), *empty = full + 8, *d_full = full + 16, *d_empty = full + 18;
    uint64_t *fin = full + 20, *sc_full = full + 21;
    uint32_t *tmem_s = reinterpret_cast<uint32_t *>(smem + 512);
    int *abort_s = reinterpret_cast<int *>(smem + 516), *leave_s = reinterpret_cast<int *>(smem + 520);
    int *left_s = reinterpret_cast<int *>(smem + 524);  // the first tile without sums
    float *sc = reinterpret_cast<float *>(smem + kWoSc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)cluster_rank();

    if (tid == 0) {
        for (int i = 0; i < kWStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&d_full[i], 1);
            mbar_init(&d_empty[i], 2 * kWEpi);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&sc_full[i], 32);
        mbar_init(fin, 2);
        *abort_s = *leave_s = 0;
        *left_s = 0x7fffffff;
        fence_mbar_init();
    }
    if (warp == 0) {
        tc::tmem_alloc_pair(tmem_s, 512);
        tc::tmem_relinquish_pair();
    }
    tc::fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers and tensor memory are there
    tc::fence_after();
    const uint32_t tmem = *tmem_s;
    pdl_wait();
    pdl_trigger();
    const bool skip = a.ctrl && ld_ctrl(a.ctrl) <= a.layer;
    bool failed = false;
    // Waits of one thread.  A poll occupies the pipe that every shared-memory operation takes: with sixteen warps
    // polling for themselves each load, arrival and read of tensor memory took about 300 cycles.  So one warp waits
    // for the promoting ones, which park at CTA barriers.
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        for (uint32_t i = 0; i < kSpinPolls; ++i)
            if (mbar_test_wait(bar, parity)) return true;
        atomicExch(abort_s, 1);
        failed = true;
        return false;
    };
    const int tiles_t = (a.T + 255) / 256;  // token tiles run fastest: pairs side by side share their weights
    const int first = blockIdx.x >> 1, step = gridDim.x >> 1;

    // registers: 640 threads at 96 = 512 promoting ones at 104 + 128 at 64
    if (warp >= kWEpi) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (!skip && warp == kWLoadW) {
            uint32_t s = 0, par = 1, n = 0;  // stage; parity of its last release (the first round passes); block
            const uint32_t full0 = peer_addr(smem_addr(full), 0);
            // Scales: copied for eight blocks at a time into a ring of sixteen slots (loads by the promoting warps,
            // a block ahead, cost a quarter of the time: every eighth block they wait for L2).  This lane copies for block
            // m = 8 batch + (lane & 7), tokens 4 i + (lane >> 3).
            const uint32_t blocks = (uint32_t)(first < a.tiles ? (a.tiles - 1 - first) / step + 1 : 0) * a.KB;
            uint32_t m = lane & 7;
            int mtile = first, mkb = lane & 7;
            for (int tile = first; tile < a.tiles && !failed; tile += step) {
                const int t0 = tile % tiles_t * 256 + 128 * rank, j = tile / tiles_t;
                const int r0 = GATED ? j * 128 : j * 256 + 128 * rank;  // this CTA's weight rows
                const CUtensorMap *wmap = &a.wmap[GATED ? rank : 0];
                for (int kb = 0; kb < a.KB; ++kb, ++n) {
                    if (lane == 0 && wait(&empty[s], par)) {
                        uint8_t *st = smem + kWoRing + s * kWStage;
                        if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kWStage);
                        tma_load_2d_pair(st, &a.xmap, kb * kG, t0, full0 + 8 * s);
                        tma_load_2d_pair(st + kTileBytes, wmap, kb * kG, r0, full0 + 8 * s);
                    }
                    __syncwarp();
                    if (__any_sync(kFull, failed)) {
                        failed = true;
                        break;
                    }
                    if (++s == kWStages) s = 0, par ^= 1;
                    if ((n & 7) == 0) {
                        // the MMAs of block n - 4 are done, so block n - 6 and the ones before it were released
                        while (mkb >= a.KB) mkb -= a.KB, mtile += step;
                        if (m < blocks) {
                            const int mt = mtile % tiles_t * 256 + 128 * rank, mj = mtile / tiles_t;
                            const uint32_t dst = smem_addr(sc + (m % kWSlots) * kWScales);
#pragma unroll 4
                            for (int i = lane >> 3; i < 128; i += 4)
                                cp_async_ca<4>(dst + 4 * i, a.xs + (mt + i < a.T ? (size_t)(mt + i) * a.KB + mkb : 0), mt + i < a.T ? 4 : 0);
                            if (lane < 16) {  // of both halves of the weight rows (past the end: any, their products are zero)
                                const int half = lane >> 3, last = (a.N - 1) / 128, nb = GATED ? mj : 2 * mj + half;
                                cp_async_ca<4>(dst + 4 * (128 + half), a.ws[GATED ? half : 0] + (size_t)(nb < last ? nb : last) * a.KB + mkb, 4);
                            }
                        }
                        cp_async_arrive(&sc_full[(n >> 3) & 1]);
                        m += 8;
                        mkb += 8;
                        __syncwarp();
                    }
                }
            }
            cp_async_commit();
            cp_async_wait_all_but<0>();
            if (failed)  // copies in flight land within microseconds; nobody waits for them any more
                for (int i = 0; i < 4096; ++i) __nanosleep(1000);
            __syncwarp();
        }
        if (!skip && (warp == kWMmaW || warp == kWMmaW + 1) && rank == 0 && lane == 0) {
            // blocks b, b + 2, .. of all that this CTA goes through, into accumulator b
            const uint32_t b = warp - kWMmaW, idesc = tc::instr_desc(0u, 256, 256), ring = smem_addr(smem + kWoRing);
            const uint32_t blocks = (uint32_t)(first < a.tiles ? (a.tiles - 1 - first) / step + 1 : 0) * a.KB;
            uint32_t s = b, par = 0, dpar = 1;
            for (uint32_t n = b; n < blocks; n += 2) {
                if (!wait(&full[s], par) || !wait(&d_empty[b], dpar)) break;
                tc::fence_after();
                const uint32_t st = ring + s * kWStage;
                const uint64_t ad = tc::smem_desc_sw128(st, 1024), bd = tc::smem_desc_sw128(st + kTileBytes, 1024);
#pragma unroll
                for (int k = 0; k < kG / 32; ++k) tc::mma_f8_pair(tmem + b * 256, ad + 2 * k, bd + 2 * k, idesc, k > 0);
                tc::commit_pair(&d_full[b]);
                tc::commit_pair(&empty[s]);
                dpar ^= 1;
                s += 2;
                if (s >= kWStages) s -= kWStages, par ^= 1;
            }
        }
        if (!skip && warp == kWPollW) {
            // Waits for each block's product and lets the two groups of eight promoting warps pass their barrier of its
            // buffer (ids 2 + buffer and 4 + buffer); the next arrival there comes after both have released the buffer.
            const uint32_t blocks = (uint32_t)(first < a.tiles ? (a.tiles - 1 - first) / step + 1 : 0) * a.KB;
            for (uint32_t n = 0; n < blocks; ++n) {
                bool ok = true;
                if (lane == 0 && (((n & 7) == 0 && !wait(&sc_full[(n >> 3) & 1], (n >> 4) & 1)) || !wait(&d_full[n & 1], (n >> 1) & 1))) {
                    ok = false;
                    *reinterpret_cast<volatile int *>(leave_s) = 1;
                    __threadfence_block();
                }
                __syncwarp();
                ok = __all_sync(kFull, ok);
                asm volatile("bar.arrive %0, 288;\n\tbar.arrive %1, 288;" ::"r"(2 + (n & 1)), "r"(4 + (n & 1)) : "memory");
                if (!ok) break;
            }
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        const int qd = warp & 3, part = warp >> 2, group = warp >> 3, row = 32 * qd + lane;
        // two runs of 32 columns: neighbours, or the same rows of gate and up
        const int col0 = GATED ? 32 * part : 64 * part, col1 = col0 + (GATED ? 128 : 32);
        const uint32_t trow = tmem + ((uint32_t)(32 * qd) << 16);
        const uint32_t release = peer_addr(smem_addr(d_empty), 0);
        float *stage = reinterpret_cast<float *>(smem + kWoOut) + warp * kWOutFloats;
        float *top = reinterpret_cast<float *>(smem + kWoTop);
        uint32_t n = 0;
        for (int tile = skip ? a.tiles : first; tile < a.tiles && !failed; tile += step) {
            const int t = tile % tiles_t * 256 + 128 * rank + row, j = tile / tiles_t;
            unsigned long long acc[2][16];
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[r][i] = 0ull;
            for (int kb = 0; kb < a.KB; ++kb, ++n) {
                const int b = n & 1;
                asm volatile("bar.sync %0, 288;" ::"r"(2 + 2 * group + b) : "memory");
                __syncwarp();
                if (*reinterpret_cast<volatile int *>(leave_s)) {  // the same for all sixteen warps: set before the arrival
                    failed = true;
                    break;
                }
                tc::fence_after();
                const uint32_t db = trow + b * 256;
                const float *ss = sc + (n % kWSlots) * kWScales;
                const float x = ss[row], f0 = x * ss[128 + (GATED ? 0 : group)], f1 = GATED ? x * ss[129] : f0;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t d[16];
                    tc::ld16(db + (c < 2 ? col0 : col1) + 16 * (c & 1), d);
                    tc::ld_wait(d);
                    if (c == 3) {
                        tc::fence_before();
                        __syncwarp();
                        if (lane == 0) arrive_at(release + 8 * b);
                        __syncwarp();  // rejoin the warp (see cta_sync)
                    }
                    const unsigned long long f = dup2(c < 2 ? f0 : f1);
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[c >> 1][8 * (c & 1) + i] = ffma2(pack2(d[2 * i], d[2 * i + 1]), f, acc[c >> 1][8 * (c & 1) + i]);
                }
            }
            if (failed) {
                *left_s = tile;  // the same of all sixteen warps
                break;
            }
            if constexpr (!GATED) {
#pragma unroll
                for (int r = 0; r < 2; ++r) put32<RES>(a, stage, t - lane, j * 256 + 64 * part + 32 * r, acc[r]);
            } else {
                const int i0 = j * 128 + 32 * part;
                float m = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float h0 = silu(lo2(acc[0][i])) * lo2(acc[1][i]), h1 = silu(hi2(acc[0][i])) * hi2(acc[1][i]);
                    if (i0 + 2 * i < a.N) m = max_abs_nan(m, h0);
                    if (i0 + 2 * i + 1 < a.N) m = max_abs_nan(m, h1);
                    acc[0][i] = pack2(__float_as_uint(h0), __float_as_uint(h1));
                }
                if (a.y) put32<false>(a, stage, t - lane, i0, acc[0]);
                if (a.q) {
                    wide_sync();  // every warp has read the last tile's maxima
                    top[128 * part + row] = m;
                    wide_sync();
                    m = max_nan(max_nan(top[row], top[128 + row]), max_nan(top[256 + row], top[384 + row]));
                    const bool bad = !(m < INFINITY);
                    float f = m > 0.f && !bad ? 448.f / m : 0.f, f1 = 1.f;
                    if (f == INFINITY) f1 = 18446744073709551616.f, f = 448.f / (m * f1);  // in two steps
                    if (part == 0 && t < a.T)
                        a.scale[(size_t)t * a.tiles_n + j] = bad ? __int_as_float(0x7fffffff) : m / 448.f;
                    if (t < a.T) {
                        uint8_t *q = a.q + (size_t)t * a.N + i0;
                        const bool vec_q = (a.N & 15) == 0 && i0 + 32 <= a.N && (reinterpret_cast<uintptr_t>(a.q) & 15) == 0;
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            uint32_t w[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const unsigned long long p0 = acc[0][8 * c + 2 * i], p1 = acc[0][8 * c + 2 * i + 1];
                                w[i] = f > 0.f ? pack4_e4m3(lo2(p0) * f1 * f, hi2(p0) * f1 * f, lo2(p1) * f1 * f, hi2(p1) * f1 * f) : 0u;
                            }
                            if (vec_q) {
                                *reinterpret_cast<uint4 *>(q + 16 * c) = make_uint4(w[0], w[1], w[2], w[3]);
                            } else {
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    if (i0 + 16 * c + i < a.N) q[16 * c + i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
                            }
                        }
                    }
                    __syncwarp();
                }
            }
        }
    }
    __syncwarp();
    __syncthreads();
    if (*reinterpret_cast<volatile int *>(abort_s) != 0) {
        for (int tile = *reinterpret_cast<volatile int *>(left_s); tile < a.tiles; tile += step)  // as in f8_rows_kernel
            spoil<GATED>(a, 32 * kWEpi, tile % tiles_t * 256 + 128 * rank, 128, tile / tiles_t * (GATED ? 128 : 256), GATED ? 128 : 256);
        if (tid == 0 && a.ctrl) dev_error(a.ctrl, RL_DEVERR_WAIT_TIMEOUT);
        if (rank == 0 && lane == 0 && (warp == kWMmaW || warp == kWMmaW + 1)) {
            tc::commit_pair(fin);  // MMAs in flight end before tensor memory is given back
            mbar_wait(fin, 0);
        }
        __syncwarp();
        __syncthreads();
    }
    tc::fence_before();
    __syncthreads();
    cluster_sync();  // the other CTA's operands and barriers are no longer used
    tc::fence_after();
    if (warp == 0) tc::tmem_dealloc_pair(tmem, 512);
}

// ---- host side ----------------------------------------------------------------------------------
rl_status byte_map(CUtensorMap *map, const void *base, int rows, int cols, int box_rows, const char *what) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = encode_tiled();
    if (!enc) return fail(RL_ERR_CUDA, "%s: cuTensorMapEncodeTiled unavailable", what);
    const cuuint64_t gdim[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t gstride[1] = {(cuuint64_t)cols};
    const cuuint32_t box[2] = {(cuuint32_t)kG, (cuuint32_t)box_rows};
    const cuuint32_t estride[2] = {1, 1};
    const CUresult cr = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), gdim, gstride, box, estride,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (cr != CUDA_SUCCESS) return fail(RL_ERR_CUDA, "%s: tensor map rejected (error %d)", what, (int)cr);
    return RL_OK;
}

template <typename Kern, typename... Args>
rl_status launch_cluster(Kern kernel, int ctas, int threads, int cluster, size_t smem, cudaStream_t s, const char *what, Args... args) {
    rl_status st = allow_smem((const void *)kernel, smem);
    if (st != RL_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e != cudaSuccess) return fail(RL_ERR_CUDA, "%s: launch failed: %s", what, cudaGetErrorString(e));
    return RL_OK;
}

template <int TT, bool GATED>
rl_status run_rows(F8Args &a, const void *x, cudaStream_t s, const char *what) {
    rl_status st = byte_map(&a.xmap, x, a.T, a.K, TT, what);
    if (st != RL_OK) return st;
    const int sms = sm_count(), tt = (a.T + TT - 1) / TT;
    a.tiles = a.tiles_n * tt;
    int S = 1;
    while (S < kMaxCluster && 2 * S <= a.KB && a.tiles * 2 * S <= sms) S *= 2;
    const int ctas = S > 1 ? a.tiles * S : a.tiles < 2 * sms ? a.tiles : 2 * sms;
    return launch_cluster(f8_rows_kernel<TT, GATED>, ctas, kThreads, S, Rows<TT, GATED>::bytes(S > 1), s, what, a, S);
}

template <bool GATED>
rl_status run_wide(F8Args &a, const void *x, cudaStream_t s, const char *what) {
    rl_status st = byte_map(&a.xmap, x, a.T, a.K, 128, what);
    if (st != RL_OK) return st;
    const int per = GATED ? 128 : 256;
    a.tiles = (a.T + 255) / 256 * ((a.N + per - 1) / per);
    const int pairs = a.tiles < sm_count() / 2 ? a.tiles : sm_count() / 2;
    if (!GATED && a.res) return launch_cluster(f8_wide_kernel<false, true>, 2 * pairs, kWThreads, 2, kWBytes, s, what, a);
    return launch_cluster(f8_wide_kernel<GATED, false>, 2 * pairs, kWThreads, 2, kWBytes, s, what, a);
}

// shared checks; 0 rows: nothing to do
rl_status check(const char *what, const void *const *w, const float *const *ws, int nw, int N, int K, const void *x,
                const float *xs, int T, int32_t layer, const int32_t *ctrl) {
    if (T < 0 || N <= 0 || K <= 0) return fail(RL_ERR_INVALID, "%s: T=%d rows=%d K=%d", what, T, N, K);
    if (K % 16) return fail(RL_ERR_UNSUPPORTED, "%s: K=%d is not a multiple of 16", what, K);
    if (N > (1 << 26) || K > (1 << 20) || T > (1 << 22))
        return fail(RL_ERR_UNSUPPORTED, "%s: T=%d rows=%d K=%d (at most 2^22, 2^26, 2^20)", what, T, N, K);
    if (ctrl && layer < 0) return fail(RL_ERR_INVALID, "%s: layer=%d", what, layer);
    if (T == 0) return RL_OK;
    if (!x || !xs) return fail(RL_ERR_INVALID, "%s: NULL x or x_scale", what);
    uintptr_t p16 = reinterpret_cast<uintptr_t>(x), p4 = reinterpret_cast<uintptr_t>(xs) | reinterpret_cast<uintptr_t>(ctrl);
    for (int i = 0; i < nw; ++i) {
        if (!w[i] || !ws[i]) return fail(RL_ERR_INVALID, "%s: NULL weights or their scales", what);
        p16 |= reinterpret_cast<uintptr_t>(w[i]);
        p4 |= reinterpret_cast<uintptr_t>(ws[i]);
    }
    if (p16 & 15) return fail(RL_ERR_INVALID, "%s: x and the weights must be 16-byte aligned", what);
    if (p4 & 3) return fail(RL_ERR_INVALID, "%s: scales and ctrl must be 4-byte aligned", what);
    return RL_OK;
}

rl_status fill_args(F8Args &a, const void *const *w, const float *const *ws, int nw, int N, int K, const float *xs, int T,
                    int32_t layer, int32_t *ctrl, const char *what) {
    for (int i = 0; i < nw; ++i) {
        rl_status st = byte_map(&a.wmap[i], w[i], N, K, 128, what);
        if (st != RL_OK) return st;
        a.ws[i] = ws[i];
    }
    a.xs = xs;
    a.T = T;
    a.N = N;
    a.K = K;
    a.KB = (K + kG - 1) / kG;
    a.tiles_n = (N + 127) / 128;
    a.layer = layer;
    a.ctrl = ctrl;
    return RL_OK;
}

bool row_type(int dt) { return dt == RL_F32 || dt == RL_F16 || dt == RL_BF16; }

}  // namespace

extern "C" rl_status rl_f8_matmul(const uint8_t *w, const float *w_scale, int32_t N, int32_t K, const uint8_t *x,
                                  const float *x_scale, int32_t T, const void *res, void *y, int32_t y_dtype,
                                  int32_t layer, int32_t *ctrl, void *stream) {
    const char *what = "rl_f8_matmul";
    const void *const ww[1] = {w};
    const float *const ss[1] = {w_scale};
    if (!row_type(y_dtype)) return fail(RL_ERR_INVALID, "%s: y_dtype %d is none of RL_F32, RL_F16, RL_BF16", what, y_dtype);
    rl_status st = check(what, ww, ss, 1, N, K, x, x_scale, T, layer, ctrl);
    if (st != RL_OK || T == 0) return st;
    if (!y) return fail(RL_ERR_INVALID, "%s: NULL y", what);
    if ((reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(res)) % dtype_bytes(y_dtype))
        return fail(RL_ERR_INVALID, "%s: y or res misaligned", what);
    F8Args a = {};
    st = fill_args(a, ww, ss, 1, N, K, x_scale, T, layer, ctrl, what);
    if (st != RL_OK) return st;
    a.y = y;
    a.res = res;
    a.dtype = y_dtype;
    cudaStream_t s = as_stream(stream);
    if (T <= 16) return run_rows<16, false>(a, x, s, what);
    if (T <= 32) return run_rows<32, false>(a, x, s, what);
    if (T <= 64) return run_rows<64, false>(a, x, s, what);
    if (T <= 128) return run_rows<128, false>(a, x, s, what);
    return run_wide<false>(a, x, s, what);
}

extern "C" rl_status rl_f8_gated(const uint8_t *w_gate, const float *gate_scale, const uint8_t *w_up,
                                 const float *up_scale, int32_t I, int32_t K, const uint8_t *x, const float *x_scale,
                                 int32_t T, void *h, int32_t h_dtype, uint8_t *q, float *scale, int32_t layer,
                                 int32_t *ctrl, void *stream) {
    const char *what = "rl_f8_gated";
    const void *const ww[2] = {w_gate, w_up};
    const float *const ss[2] = {gate_scale, up_scale};
    if (h && !row_type(h_dtype)) return fail(RL_ERR_INVALID, "%s: h_dtype %d is none of RL_F32, RL_F16, RL_BF16", what, h_dtype);
    rl_status st = check(what, ww, ss, 2, I, K, x, x_scale, T, layer, ctrl);
    if (st != RL_OK || T == 0) return st;
    if ((q == nullptr) != (scale == nullptr)) return fail(RL_ERR_INVALID, "%s: q and scale come together", what);
    if (!h && !q) return fail(RL_ERR_INVALID, "%s: no output", what);
    if (h && reinterpret_cast<uintptr_t>(h) % dtype_bytes(h_dtype)) return fail(RL_ERR_INVALID, "%s: h misaligned", what);
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(scale)) & 3)
        return fail(RL_ERR_INVALID, "%s: q and scale must be 4-byte aligned", what);
    F8Args a = {};
    st = fill_args(a, ww, ss, 2, I, K, x_scale, T, layer, ctrl, what);
    if (st != RL_OK) return st;
    a.y = h;
    a.dtype = h_dtype;
    a.q = q;
    a.scale = scale;
    cudaStream_t s = as_stream(stream);
    if (T <= 16) return run_rows<16, true>(a, x, s, what);
    if (T <= 32) return run_rows<32, true>(a, x, s, what);
    if (T <= 64) return run_rows<64, true>(a, x, s, what);
    return run_wide<true>(a, x, s, what);
}
