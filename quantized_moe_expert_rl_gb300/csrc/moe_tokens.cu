// moe_tokens.cu - moe_decode_tokens: a whole routed MoE layer for 1 to 32 tokens in ONE launch.
//
//   logits = W_r xn (+ bias),  ids = top-K, weights = softmax over the selection,
//   y[t] (+)= sum_k weights[t][k] * down_k(silu(gate_k xn_t) * (up_k xn_t))
//
// One cooperative CTA per SM: 16 computing warps, three finishing warps and one that issues the weight
// copies.
//   R  every CTA takes up to four router rows (f32 dots with every token, each warp a sixteenth
//      of the columns), and a share of the split of x into bf16 parts;  grid barrier
//   S  every CTA selects for itself (one warp per token, the same code on the same logits): the
//      list of distinct experts, each with its tokens as a bit mask, and from it the whole
//      schedule of weight copies.  CTA 0 writes ids, weights, slots, misses and the flag
//   G  gate and up: tiles of (expert, 16 hidden rows) -> h;  grid barrier (the copies of D's first
//      weights are already under way)
//   D  down: CTA b has output rows 16 b .. 16 b + 15 of every expert, so that the sum over k in
//      selection order needs no further exchange.  (Tiles of 128 rows spread over all SMs, with the
//      outputs exchanged through a third grid barrier, were no faster at 32 tokens and 3 us slower at 1.)
// Work comes in rounds of units, a unit being 16 weight rows x 256 values (one block of every row).  In G
// a computing warp has two units of a round, gate and up of the same rows and block, which share
// the activations; in D it has one.  A G round's block sums go through one of four buffers to a
// finishing warp, which adds them and applies SwiGLU, so that no computing warp waits for another.  Every
// CTA takes a run of consecutive G tiles of equal weight, where a tile weighs one per two tokens of
// its expert; an expert's activations then stay in registers over its tiles.
// For few tokens the launch is a chain of latencies, much of them the first fetch of straight code: a
// combine unrolled to 16 experts took 8.5k cycles where the rolled loop takes 1.2k.  So what runs once
// stays in rolled loops, and the codebook table and the expert tables are built while the first grid
// barrier is pending.  (Running the unit code dry there, to fetch it early, cost 0.7 us at 1 token; one
// copy of the unit code for both phases cost 2 us at 1 token and 15 at 32.)
//
// The matrix arithmetic.  A weight is d * (codebook value) * (sign): the codebook value is an
// 8-bit integer, exact in bf16, so a group's 8 values are one 16-byte table entry whose signs are
// flipped by XOR; 16 weight rows are the A operand of mma.m16n8k16 and d multiplies the f32
// sums of a 256-value block.  An f32 activation is exactly the sum of three bf16 values (its
// leading 8 bits, the next 8, the last 8, each taken by truncation), so three columns of B
// carry it without loss, two tokens share the 8 columns of one MMA, and the products are exact
// before the f32 sums.  On the CUDA cores the same dot needs two unpacking instructions and a packed FMA
// per pair of weights (25 instructions per group against 13 here).
//
// Measured at hidden 2048, 512 experts, top-10, intermediate 512, back to back in a graph: 1 token 22.6 us
// (12.3 MB, 1.8 us at the measured copy rate), 5 drafted tokens with 22 to 24 distinct experts 38.3 us
// (23.8 MB with 24, 3.5 us), 32 independent tokens with 233 to 240 distinct experts 153 us (199 MB with 240,
// 29 us).  DRAM reads are the router and every distinct expert once.  At 1 token, of 41k cycles (clock64 of
// one thread, instrumented): router 4k, first barrier 3k, selection 5.5k, list and first copies 5k, G 5.5k,
// finishing and second barrier 9.5k, D and its first copies 7k, combine 1.4k.  At 32 tokens G takes 121k and
// D 100k of 285k; shared loads (the table's above all) fill 35% of their pipe's slots, issue slots are 57%
// used.  With a given routing (after a fill) the same take 20.6, 35.6 and 141.6 us.  For comparison: T calls of moe_decode_layer take 21 to 23 us each, the grouped prefill path
// (half-precision operands) 58, 119, 201 and 306 us at 1, 5, 16 and 32 tokens.
#include "decode_rows.cuh"
#include "select.cuh"
#include "stack_kernel.cuh"

using namespace rl;

namespace {

constexpr int kMtWarps = 16, kMtFin = 3;            // computing and finishing warps
constexpr int kMtWork = (kMtWarps + kMtFin) * 32;   // threads that meet at the grid barriers
constexpr int kMtThreads = kMtWork + 32;            // and the copying warp
constexpr int kMtRed = 4;                           // buffers between computing and finishing warps
constexpr int kMtMaxT = 32;
constexpr int kMtUnits = 16896;    // bytes of 16 units of 16 rows x 256 values
constexpr int kMtMaxStages = 4;
constexpr int kMtHdr = 256;        // workspace: barrier counter, test knobs (64..71), RMS scales (128..255)

struct MtArgs {
    const float *x, *W, *bias;
    const uint64_t *table;  // the layer's row
    const int8_t *codebook;
    int32_t *ids;
    float *weights;
    uint64_t *slots;
    uint32_t *miss;  // the layer's counter
    int32_t *ctrl;
    float *logits_out, *y;
    unsigned long long *ctr;
    float *rs, *raw;       // [32] RMS scales, [T][512] router dots
    uint16_t *xs, *hs;     // [T][3][H], [T K][3][I] bf16 parts
    float eps;
    int layer, T, H, E, K, I, accumulate, stages, halves;  // ring slots, and 16-unit halves of one (2, or 1)
};

// shared memory: the header (barriers, scalars), the codebook table, then
constexpr int kMtRedB = kMtRed * kMtWarps * 64 * 4;  // [kMtRed][16 warps][gate, up][2 tokens][16 rows] f32
constexpr int kMtORed = 512 + kTabBytes;
constexpr int kMtOList = kMtORed + kMtRedB;          // [512] (expert, first pair, token mask, weight before it)
constexpr int kMtOMask = kMtOList + 512 * 16;        // [512] u32 token masks by expert
constexpr int kMtOSlot = kMtOMask + 512 * 4;         // [512] u64 slots by expert
constexpr int kMtOId = kMtOSlot + 512 * 8;           // [512] i32 selected ids
constexpr int kMtOW = kMtOId + 512 * 4;              // [512] f32 selected logits, then weights
constexpr int kMtOPair = kMtOW + 512 * 4;            // [512] u16 pair number of (t, k)
constexpr int kMtOTok = kMtOPair + 512 * 2;          // [512] u8 token of a pair
// partial outputs [pairs][units per row][16] f32; before that the selection's scratch [16 warps][448] and
// keys [T][512], which reach into the ring behind it
constexpr int kMtOPart = kMtOTok + 512;
constexpr int kMtSelB = kMtWarps * 448;
__host__ __device__ inline int mt_ring(int T, int K, int I) {
    const int part = T * K * (I > 256 ? I / 256 : 1) * 64;
    return (int)align_up(kMtOPart + (part > kMtSelB ? part : kMtSelB), 128);
}

static_assert(kMtWork == 608, "the barriers below count 608 threads");
// all warps but the copying one
__device__ __forceinline__ void workers_sync() {
    asm volatile("bar.sync 1, 608;" ::: "memory");
    __syncwarp();
}
// the same with a vote: true everywhere when any thread brought `pred`
__device__ __forceinline__ bool workers_sync_or(bool pred) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 1, 608, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"(pred ? 1u : 0u)
        : "memory");
    __syncwarp();
    return any != 0u;
}

// The working warps of all CTAs meet (see grid_sync in stack_kernel.cuh; the copying warp does not take
// part), in two halves: what the CTA wrote before its arrival is visible to every CTA after the wait.
__device__ __forceinline__ void grid_arrive(unsigned long long *ctr, unsigned long long &target) {
    workers_sync();
    if (threadIdx.x == 0) {
        unsigned long long old;
        asm volatile("atom.add.release.gpu.global.u64 %0, [%1], 1;" : "=l"(old) : "l"(ctr) : "memory");
        if (target == 0ull) target = old - old % gridDim.x;
        target += gridDim.x;
    }
    __syncwarp();
}
__device__ __forceinline__ bool grid_wait(unsigned long long *ctr, unsigned long long target, volatile int *stop,
                                          int32_t *ctrl, uint32_t cap) {
    if (threadIdx.x == 0) {
        bool ok = false;
#pragma unroll 1
        for (uint32_t i = 0; i < cap; ++i)
            if (ld_acquire_u64(ctr) >= target) {
                ok = true;
                break;
            }
        if (!ok) {
            dev_error(ctrl, RL_DEVERR_WAIT_TIMEOUT);
            *stop = 1;
        }
    }
    workers_sync();
    return *stop == 0;
}

// Bounded wait of a whole warp for phase `parity` of an mbarrier, given up once *stop is set.  The
// warps that mostly wait (SLEEP) sleep between their polls, so that they leave the issue slots to
// the computing warps.
template <bool SLEEP>
__device__ __forceinline__ bool wait_or_stop(uint64_t *bar, uint32_t parity, const volatile int *stop) {
    if (__all_sync(kFull, mbar_test_wait(bar, parity))) return true;
    int ok = 0;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll 1
        for (uint32_t i = 0; i < kSpinCap; ++i) {
            if (mbar_try_wait(bar, parity)) {
                ok = 1;
                break;
            }
            if (*stop) break;
            if (SLEEP) __nanosleep(40);
        }
    }
    __syncwarp();  // rejoin the warp (see cta_sync)
    return __shfl_sync(kFull, ok, 0) != 0;
}

// v = p[0] + p[1] + p[2] exactly, each a bf16 value (truncated, so nothing overflows)
__device__ __forceinline__ void split3(float v, uint32_t (&p)[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const uint32_t b = __float_as_uint(v) & 0xffff0000u;
        p[i] = b >> 16;
        v -= __uint_as_float(b);
    }
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// flip the signs of a table entry's 8 values by the 8-bit mask s (see group_fma2)
__device__ __forceinline__ void flip_signs(uint4 &q, uint32_t s) {
    q.x ^= (s * 0x40008000u) & 0x80008000u;
    q.y ^= (s * 0x10002000u) & 0x80008000u;
    q.z ^= (s * 0x04000800u) & 0x80008000u;
    q.w ^= (s * 0x01000200u) & 0x80008000u;
}
__device__ __forceinline__ uint32_t lds_half(const uint8_t *p) { return *reinterpret_cast<const uint16_t *>(p); }

// Groups of a unit and lanes.  Lane 4 g + t multiplies rows g and g + 8; in step j = 0..7 the four
// lanes of a quad take four groups of 8 values, in any order that the activations share.
//   WIDE: a lane reads its group bytes as aligned words (two groups each) 4 m + t, m = 0..3.  A block is
//   66 bytes, so blocks at an odd multiple of 66 bytes start their groups on a word, (2 w, 2 w + 1) in word
//   w; at an even multiple word w holds (2 w - 1, 2 w), the half before group 0 being the scale d, and
//   group 31 takes its place.  Needs all rows of a unit at the same parity: two blocks or more per row.
//   Else: 16-bit reads of group 4 j + t.
template <bool WIDE>
__device__ __forceinline__ int lane_group(int j, int t, bool even) {
    if (!WIDE) return 4 * j + t;
    const int g = 8 * (j >> 1) + 2 * t + (j & 1) - (even ? 1 : 0);
    return g < 0 ? 31 : g;
}

// What the activations of a unit come from: this lane's column of B (16-byte pieces of one bf16 part
// of one row), or NULL for a column that is not used.
struct BColumn {
    const uint4 *p;
};
// B fragments of two rows of bf16 parts (rowA, rowB: [3][width], rowB may be NULL), values from `at` on:
// lane (n, t) holds its groups of column n.
__device__ __forceinline__ BColumn b_column(const uint16_t *rowA, const uint16_t *rowB, int width, int at) {
    const int n = (threadIdx.x >> 2) & 7;
    const uint16_t *row = (n == 2 || n == 3 || n == 5) ? rowB : rowA;
    const int part = n >= 4 ? 2 : n & 1;
    BColumn c;
    c.p = n < 6 && row != nullptr ? reinterpret_cast<const uint4 *>(row + part * width + at) : nullptr;
    return c;
}
template <bool WIDE>
__device__ __forceinline__ void load_b(uint4 (&b)[8], BColumn c, int steps, bool even) {
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        b[j] = c.p != nullptr && (WIDE || j < steps) ? __ldcg(c.p + lane_group<WIDE>(j, t, even)) : make_uint4(0u, 0u, 0u, 0u);
}

// NU units against two tokens: d * sums of rows g (v[u][0]) and g + 8 (v[u][1]) for token t in lanes t = 0,
// 1.  p[u]: the block's first byte in row g of unit u, `r8` bytes before row g + 8's (`go`: bytes of the
// groups before this lane's, for half blocks).  One straight piece of code: a branch in it (say, to refill
// B half-way) keeps the compiler from overlapping the steps and cost 40% in D.
template <bool WIDE, int NU>
__device__ __forceinline__ void unit_dot(const uint8_t *const (&p)[NU], int r8, int go, int steps, bool even,
                                         const uint4 (&b)[8], const uint4 *tabc, float (&v)[NU][2]) {
    const int t = threadIdx.x & 3;
    float c[NU][2][4] = {};
    auto step = [&](int j, uint32_t (&x)[NU][2]) {  // x: index | sign << 8 in the half (j & 1) of a word
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            const bool hi = WIDE && (j & 1);
            uint4 q = tabc[(hi ? __byte_perm(x[u][0], 0, 0x4442) : x[u][0] & 0xffu) * kTabCopies];
            uint4 r = tabc[(hi ? __byte_perm(x[u][1], 0, 0x4442) : x[u][1] & 0xffu) * kTabCopies];
            flip_signs(q, hi ? x[u][0] >> 24 : __byte_perm(x[u][0], 0, 0x4441));
            flip_signs(r, hi ? x[u][1] >> 24 : __byte_perm(x[u][1], 0, 0x4441));
            mma_bf16(c[u][0], q.x, r.x, q.y, r.y, b[j].x, b[j].y);
            mma_bf16(c[u][1], q.z, r.z, q.w, r.w, b[j].z, b[j].w);
        }
    };
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        uint32_t x[NU][2];
        if (WIDE) {
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint8_t *row = p[u] + h * r8;
                    x[u][h] = *reinterpret_cast<const uint32_t *>(row + (even ? 0 : 2) + 4 * t + 16 * m);
                    if (m == 0) {
                        const uint32_t g31 = lds_half(row + 64);
                        x[u][h] = even && t == 0 ? __byte_perm(x[u][h], g31, 0x3254) : x[u][h];
                    }
                }
            step(2 * m, x);
            step(2 * m + 1, x);
        } else {
#pragma unroll
            for (int j = 2 * m; j < 2 * m + 2; ++j)
                if (j < steps) {
#pragma unroll
                    for (int u = 0; u < NU; ++u)
#pragma unroll
                        for (int h = 0; h < 2; ++h) x[u][h] = lds_half(p[u] + h * r8 + go + 2 + 8 * j + 2 * t);
                    step(j, x);
                }
        }
    }
    // columns 0, 1: token 0 leading and middle parts; 2, 3: token 1; 4: token 0 last part; 5: token 1
    const int src = (threadIdx.x & 28) | 2;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
        const float c0 = c[u][0][0] + c[u][1][0], c1 = c[u][0][1] + c[u][1][1];
        const float c2 = c[u][0][2] + c[u][1][2], c3 = c[u][0][3] + c[u][1][3];
        const float l0 = __shfl_sync(kFull, c0, src), l1 = __shfl_sync(kFull, c1, src);
        const float l2 = __shfl_sync(kFull, c2, src), l3 = __shfl_sync(kFull, c3, src);
        v[u][0] = fp16_bits_to_float(lds_half(p[u])) * ((c0 + c1) + (t == 0 ? l0 : l1));
        v[u][1] = fp16_bits_to_float(lds_half(p[u] + r8)) * ((c2 + c3) + (t == 0 ? l2 : l3));
    }
}

// The K best of the E keys in shared memory (key, then lower index; E <= 512, key[e] = 0 from E on) by
// one warp: lane r < K gets the r-th.  The threshold is the K-th largest of the 32 lane maxima (so at
// least K keys reach it); the few keys at or above it are ranked exactly, and with more than 32 of
// them (heavy ties) K rounds of arg-max take over.  As warp_topk_thr, in rolled loops over
// shared memory: this code runs once per launch, and fetching it costs more than executing it.
__device__ __noinline__ void warp_topk_smem(const uint32_t *key, int E, int K, uint8_t *scratch, int &my_id,
                                            float &my_val) {
    const int lane = threadIdx.x & 31;
    uint32_t *wm = reinterpret_cast<uint32_t *>(scratch);
    uint2 *cand = reinterpret_cast<uint2 *>(scratch + 128);
    int *sel = reinterpret_cast<int *>(scratch + 384);
    const uint4 *k4 = reinterpret_cast<const uint4 *>(key) + lane;  // keys 128 j + 4 lane + c
    uint32_t m = 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint4 v = k4[32 * j];
        m = max(max(m, max(v.x, v.y)), max(v.z, v.w));
    }
    wm[lane] = m;
    __syncwarp();
    int rank = 0;
#pragma unroll 4
    for (int q = 0; q < 32; ++q) rank += wm[q] > m || (wm[q] == m && q < lane) ? 1 : 0;
    const uint32_t thr = __shfl_sync(kFull, m, __ffs(__ballot_sync(kFull, rank == K - 1)) - 1);
    int n = 0;
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
        const uint4 v = k4[32 * j];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t k = c == 0 ? v.x : c == 1 ? v.y : c == 2 ? v.z : v.w;
            const int e = 128 * j + 4 * lane + c;
            const bool in = e < E && k >= thr;
            const unsigned bal = __ballot_sync(kFull, in);
            const int at = n + __popc(bal & ((1u << lane) - 1u));
            if (in && at < 32) cand[at] = make_uint2(k, (uint32_t)e);
            n += __popc(bal);
        }
    }
    __syncwarp();
    my_id = 0;
    my_val = 0.f;
    if (n <= 32) {
        const uint2 me = lane < n ? cand[lane] : make_uint2(0u, 0x7fffffffu);
        int r = 0;
#pragma unroll 4
        for (int d = 0; d < n; ++d) {
            const uint2 o = cand[d];
            r += precedes(o.x, (int)o.y, me.x, (int)me.y) ? 1 : 0;
        }
        if (lane < n && r < K) sel[r] = lane;
        __syncwarp();
        if (lane < K) {
            const uint2 c = cand[sel[lane]];
            my_id = (int)c.y;
            my_val = key_value(c.x);
        }
    } else {
        unsigned taken = 0u;  // bit i: this lane's expert lane + 32 i
#pragma unroll 1
        for (int r = 0; r < K; ++r) {
            uint32_t bk = 0u;
            int bi = 0x7fffffff;
#pragma unroll 1
            for (int i = 0; i < 16; ++i) {
                const int e = lane + 32 * i;
                if (e < E && !((taken >> i) & 1u) && precedes(key[e], e, bk, bi)) bk = key[e], bi = e;
            }
            __syncwarp();
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const uint32_t ok = __shfl_xor_sync(kFull, bk, o);
                const int oi = __shfl_xor_sync(kFull, bi, o);
                if (precedes(ok, oi, bk, bi)) bk = ok, bi = oi;
            }
            if (lane == r) my_id = bi, my_val = key_value(bk);
            if ((bi & 31) == lane) taken |= 1u << (bi >> 5);
        }
    }
    __syncwarp();
}

// First tile of CTA b's run: tiles are numbered expert by expert, 2^lg each; expert i's tiles weigh
// (tokens + 1) / 2 each and list[i].w is the weight of the experts before it, per tile.
__device__ __forceinline__ int run_start(const int4 *list, int n, int total, int lg, int b, int G) {
    const int pos = (int)((uint32_t)((total << lg) * b) / (uint32_t)G);  // at most 512 << 7, times 152
    int at = 0, left = n;
#pragma unroll 1
    while (left > 1) {
        const int h = left >> 1;
        if (list[at + h].w << lg <= pos) at += h, left -= h;
        else left = h;
    }
    const int c = (__popc((uint32_t)list[at].z) + 1) >> 1, in = pos - (list[at].w << lg);
    return (at << lg) + (in + c - 1) / c;
}

template <bool WIDE>
__global__ void __launch_bounds__(kMtThreads, 1) moe_tokens_kernel(const __grid_constant__ MtArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t *full = reinterpret_cast<uint64_t *>(smem), *empty = full + kMtMaxStages;
    uint64_t *redfull = empty + kMtMaxStages, *redempty = redfull + kMtRed;
    volatile int *stop_s = reinterpret_cast<volatile int *>(smem + 192);
    int *bad_s = reinterpret_cast<int *>(smem + 196);    // bit 0: a slot is absent, 1: misaligned, 2: bad id, 3: NaN
    int *nd_s = reinterpret_cast<int *>(smem + 200);
    int *weight_s = reinterpret_cast<int *>(smem + 204);   // weight of all experts' tiles, per tile
    int *run_s = reinterpret_cast<int *>(smem + 208);      // [2] this CTA's run of G tiles: first, last + 1
    float *rs_s = reinterpret_cast<float *>(smem + 224);   // [32] RMS scales (to 352)
    uint4 *tab = reinterpret_cast<uint4 *>(smem + 512);
    float *red = reinterpret_cast<float *>(smem + kMtORed);
    int4 *list = reinterpret_cast<int4 *>(smem + kMtOList);
    uint32_t *mask_s = reinterpret_cast<uint32_t *>(smem + kMtOMask);
    uint64_t *slot_s = reinterpret_cast<uint64_t *>(smem + kMtOSlot);
    int *id_s = reinterpret_cast<int *>(smem + kMtOId);
    float *w_s = reinterpret_cast<float *>(smem + kMtOW);
    uint16_t *pair_s = reinterpret_cast<uint16_t *>(smem + kMtOPair);
    uint8_t *ptok_s = smem + kMtOTok;
    float *part = reinterpret_cast<float *>(smem + kMtOPart);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = gridDim.x, cta = blockIdx.x;
    const int T = a.T, H = a.H, E = a.E, K = a.K, I = a.I, lgH = 31 - __clz(H);
    uint8_t *ring = smem + mt_ring(T, K, I);
    const bool routed = a.W != nullptr;  // else ids, weights and slots are given
    const int flag = ld_ctrl(a.ctrl);    // the same for every thread: this launch raises it to `layer` at most
    if (routed ? flag < a.layer : flag <= a.layer) return;
    const uint2 knob = *reinterpret_cast<const uint2 *>(reinterpret_cast<const uint32_t *>(a.ctr) + 16);  // test knobs
    const uint32_t cap = knob.x ? knob.x : kSpinCap;

    // R: the router rows of this CTA (row r: expert cta + r G); warp w holds columns [w H/16, (w + 1) H/16)
    const int rcol = warp * (H >> 4) + 4 * lane;
    const bool rmine = routed && warp < kMtWarps && 4 * lane < (H >> 4);
    unsigned long long target = 0ull;
    bool ok = true;
    if (tid < kMtWork) {
        if (routed && warp < kMtWarps) {
            float4 wv[4];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                wv[r] = rmine && cta + r * G < E ? __ldg(reinterpret_cast<const float4 *>(a.W + (size_t)(cta + r * G) * H + rcol))
                                                 : make_float4(0.f, 0.f, 0.f, 0.f);
            float4 xv[4];
            auto load_x = [&](int t0) {
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    xv[u] = rmine && t0 + u < T ? *reinterpret_cast<const float4 *>(a.x + (size_t)(t0 + u) * H + rcol)
                                                : make_float4(0.f, 0.f, 0.f, 0.f);
            };
            load_x(0);
#pragma unroll 1
            for (int t0 = 0; t0 < T; t0 += 4) {
                float s[16];  // [token][row]
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        s[4 * u + r] = fmaf(wv[r].x, xv[u].x, fmaf(wv[r].y, xv[u].y, fmaf(wv[r].z, xv[u].z, wv[r].w * xv[u].w)));
                load_x(t0 + 4);
                // transposing reduction: each step halves the values a lane holds; lane l ends with value l & 15
#pragma unroll
                for (int h = 8; h > 0; h >>= 1) {
                    const bool up = (lane & h) != 0;
#pragma unroll
                    for (int i = 0; i < h; ++i) {
                        const float give = up ? s[i] : s[i + h], keep = up ? s[i + h] : s[i];
                        s[i] = keep + __shfl_xor_sync(kFull, give, h);
                    }
                }
                s[0] += __shfl_xor_sync(kFull, s[0], 16);
                // partial dots [16 warps][32 tokens][4 rows] in the (still unused) reduction buffers
                if (lane < 16) red[(warp * 32 + t0) * 4 + lane] = s[0];
                __syncwarp();
            }
        }
        // x as bf16 parts, 8 values at a time over the whole grid
#pragma unroll 1
        for (int i = cta * kMtWork + tid; i < T * H / 8; i += G * kMtWork) {
            const int t = i >> (lgH - 3), h = (i << 3) & (H - 1);
            const float4 v0 = *reinterpret_cast<const float4 *>(a.x + (size_t)t * H + h);
            const float4 v1 = *reinterpret_cast<const float4 *>(a.x + (size_t)t * H + h + 4);
            const float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
            uint32_t p[8][3];
#pragma unroll
            for (int j = 0; j < 8; ++j) split3(v[j], p[j]);
#pragma unroll
            for (int k = 0; k < 3; ++k)
                __stcg(reinterpret_cast<uint4 *>(a.xs + ((size_t)t * 3 + k) * H + h),
                       make_uint4(p[0][k] | p[1][k] << 16, p[2][k] | p[3][k] << 16, p[4][k] | p[5][k] << 16,
                                  p[6][k] | p[7][k] << 16));
        }
        // RMS scale of token t by CTA G - 1 - t (the CTAs with the fewest router rows)
        if (warp == kMtWarps && G - 1 - cta < T) {
            const int t = G - 1 - cta;
            bool range = false;
            const float r = a.eps >= 0.f ? rms_scale_warp(a.x + (size_t)t * H, H, a.eps, &range) : 1.f;
            if (lane == 0) {
                __stcg(a.rs + t, r);
                if (range) dev_error(a.ctrl, RL_DEVERR_RANGE);
            }
            __syncwarp();
        }
        if (tid == 0) {
            *stop_s = 0;
            *bad_s = 0;
        }
        workers_sync();
        if (routed && tid < 4 * T) {
            const int t = tid >> 2, r = tid & 3, e = cta + r * G;
            if (e < E) {
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < kMtWarps; ++w) v += red[(w * 32 + t) * 4 + r];
                __stcg(a.raw + t * 512 + e, v);
            }
        }
        if ((int)knob.y - 1 == cta) {  // test knob: this CTA leaves before its arrival
            if (tid == 0) *stop_s = 1;
            cta_sync();
            return;
        }
        grid_arrive(a.ctr, target);
        // while the others arrive: the barriers, the expert tables, the codebook table
        if (tid == 32) {
#pragma unroll 1
            for (int s = 0; s < a.stages; ++s) {
                mbar_init(full + s, 1);
                mbar_init(empty + s, kMtWarps);
            }
#pragma unroll 1
            for (int s = 0; s < kMtRed; ++s) {
                mbar_init(redfull + s, kMtWarps);
                mbar_init(redempty + s, 1);
            }
            fence_mbar_init();
        }
        if (tid >= 64 && tid < 320) {
            const int e = tid - 64;
            const uint2 q = reinterpret_cast<const uint2 *>(a.codebook)[e];
            uint32_t w[4];
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const uint32_t two = (p < 2 ? q.x : q.y) >> (16 * (p & 1));
                w[p] = bf16_bits((int8_t)(two & 0xffu)) | (bf16_bits((int8_t)((two >> 8) & 0xffu)) << 16);
            }
#pragma unroll
            for (int c = 0; c < kTabCopies; ++c)  // rotated so one store instruction hits 8 bank quads
                tab[e * kTabCopies + ((c + tid) & (kTabCopies - 1))] = make_uint4(w[0], w[1], w[2], w[3]);
        } else if (tid >= 352) {
            for (int e = tid - 352; e < 512; e += 256) {
                mask_s[e] = 0u;
                if (routed && e < E) slot_s[e] = a.table[e];
            }
        }
        __syncwarp();
    } else {
        // the copying warp
        cta_sync();
        if (*stop_s || (*bad_s & 7)) return;
        cta_sync();
        const int nD = *nd_s, nb = H >> 8, rowb = nb * kBlockBytes, tpr = 8 * a.halves / nb, tileb = 32 * rowb;
        const int lgG = 31 - __clz(I >> 4), upe = I > 256 ? I >> 8 : 1, epr = kMtWarps / upe, dnb = I * kBlockBytes / 16;
        const int g0 = run_s[0], g1 = run_s[1];
        const int gr = (g1 - g0 + tpr - 1) / tpr, dr = cta < H / 16 ? (nD + epr - 1) / epr : 0;
        const size_t mat = (size_t)I * rowb;
        int slot = 0, turn = 0, issued = 0;
#pragma unroll 1
        for (int r = 0; r < gr + dr; ++r) {
            if (turn > 0 && !wait_or_stop<true>(empty + slot, (turn - 1) & 1, stop_s)) {
                if (lane == 0) dev_error(a.ctrl, RL_DEVERR_WAIT_TIMEOUT);
                break;
            }
            uint8_t *dst = ring + slot * a.halves * kMtUnits;
            if (r < gr) {
                const int n = min(tpr, g1 - g0 - r * tpr);
                if (lane == 0) mbar_arrive_expect_tx(full + slot, n * tileb);
                __syncwarp();
                if (lane < 2 * n) {
                    const int tile = g0 + r * tpr + (lane >> 1);
                    const uint8_t *rec = reinterpret_cast<const uint8_t *>(slot_s[list[tile >> lgG].x]);
                    bulk_g2s(dst + (lane >> 1) * tileb + (lane & 1) * 16 * rowb,
                             rec + (lane & 1) * mat + (size_t)(tile & ((1 << lgG) - 1)) * 16 * rowb, 16 * rowb, full + slot);
                }
            } else {
                const int e0 = (r - gr) * epr, n = min(epr, nD - e0);
                if (lane == 0) mbar_arrive_expect_tx(full + slot, n * dnb);
                __syncwarp();
                if (lane < n) {
                    const uint8_t *rec = reinterpret_cast<const uint8_t *>(slot_s[list[e0 + lane].x]);
                    bulk_g2s(dst + lane * dnb, rec + 2 * mat + (size_t)cta * dnb, dnb, full + slot);
                }
            }
            __syncwarp();
            ++issued;
            if (++slot == a.stages) slot = 0, ++turn;
        }
        // every copy issued has landed before the CTA's shared memory goes away
#pragma unroll 1
        for (int r = max(0, issued - a.stages); r < issued; ++r) mbar_wait_warp(full + r % a.stages, (r / a.stages) & 1);
        return;
    }

    const int g = lane >> 2, t4 = lane & 3, nb = H >> 8, rowb = nb * kBlockBytes, tpr = 8 * a.halves / nb, tileb = 32 * rowb;
    const int lgnb = 31 - __clz(nb), lgG = 31 - __clz(I >> 4), upe = I > 256 ? I >> 8 : 1, lgu = 31 - __clz(upe);
    const int epr = kMtWarps >> lgu, dnb = I * kBlockBytes / 16;
    const uint4 *tabc = tab + (lane & (kTabCopies - 1));
    int slot = 0, turn = 0, s = 0, g0 = 0, g1 = 0, nD = 0;
    uint4 b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) b[j] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
    for (int ph = 0; ph < 2; ++ph) {  // 0: S and G, 1: D
        const bool down = ph == 1;
        if (ph == 0) {
            ok = grid_wait(a.ctr, target, stop_s, a.ctrl, cap);
            // S: selection.  Keys of every (token, expert) into shared memory, then one warp per token.
            uint32_t *keys = reinterpret_cast<uint32_t *>(smem + kMtOPart + kMtSelB);
            if (ok) {
                if (tid < T) rs_s[tid] = __ldcg(a.rs + tid);
                if (routed) {
#pragma unroll 4
                    for (int i = tid; i < 128 * T; i += kMtWork) {
                        const int t = i >> 7, e = (i & 127) * 4;
                        const float rs = __ldcg(a.rs + t);
                        const float4 r = __ldcg(reinterpret_cast<const float4 *>(a.raw + t * 512 + e));
                        float v[4] = {rs * r.x, rs * r.y, rs * r.z, rs * r.w};
                        uint32_t k[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            k[c] = 0u;
                            if (e + c < E) {
                                if (a.bias) v[c] += a.bias[e + c];
                                if (v[c] != v[c]) atomicOr(bad_s, 8);
                                k[c] = order_key(v[c]);
                                if (a.logits_out && cta == 0) a.logits_out[(size_t)t * E + e + c] = v[c];
                            }
                        }
                        *reinterpret_cast<uint4 *>(keys + t * 512 + e) = make_uint4(k[0], k[1], k[2], k[3]);
                    }
                }
            }
            workers_sync();
            if (ok && warp < kMtWarps) {
#pragma unroll 1
                for (int t = warp; t < T; t += kMtWarps) {
                    int my_id = 0;
                    float my_val = 0.f;
                    uint64_t at = 1;
                    if (routed) {
                        warp_topk_smem(keys + 512 * t, E, K, smem + kMtOPart + warp * 448, my_id, my_val);
                        if (lane < K) at = slot_s[my_id];
                    } else if (lane < K) {
                        my_id = a.ids[t * K + lane];
                        my_val = a.weights[t * K + lane];
                        at = a.slots[t * K + lane];
                        if (my_id < 0 || my_id >= E) {
                            atomicOr(bad_s, 4);
                            my_id = 0;
                        }
                        slot_s[my_id] = at;
                    }
                    __syncwarp();
                    if (lane < K) {
                        id_s[t * K + lane] = my_id;
                        w_s[t * K + lane] = my_val;
                        atomicOr(mask_s + my_id, 1u << t);
                        if (at == 0) atomicOr(bad_s, 1);
                        if (at & 15) atomicOr(bad_s, 2);
                    }
                    __syncwarp();
                }
            }
            fence_proxy_async_smem();  // the ring's copies come after the keys
            cta_sync();
            if (*stop_s) return;
            const int bad = *bad_s;
            if (!(bad & 7)) {
                // The list of distinct experts in index order: thread e holds expert e; its pairs (expert,
                // token) are numbered in token order, and `w` is the weight of the experts before it.
                int *scan = reinterpret_cast<int *>(red);  // [16 warps][2]
                const uint32_t m = tid < 512 ? mask_s[tid] : 0u;
                const uint32_t own = (uint32_t)__popc(m) | (uint32_t)((__popc(m) + 1) >> 1) << 16;  // pairs | weight
                uint32_t incl = own;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t v = __shfl_up_sync(kFull, incl, o);
                    if (lane >= o) incl += v;
                }
                const unsigned has = __ballot_sync(kFull, m != 0u);
                if (lane == 31 && warp < kMtWarps) {
                    scan[2 * warp] = __popc(has);
                    scan[2 * warp + 1] = (int)incl;
                }
                __syncwarp();
                workers_sync();
                int at = 0;
                uint32_t before = 0u;
#pragma unroll 4
                for (int w = 0; w < kMtWarps; ++w)
                    if (w < warp) {
                        at += scan[2 * w];
                        before += (uint32_t)scan[2 * w + 1];
                    }
                if (tid == kMtWarps * 32 - 1) {  // the last expert's thread knows the totals
                    *nd_s = at + __popc(has);
                    *weight_s = (int)((before + incl) >> 16);
                }
                if (m) {
                    at += __popc(has & ((1u << lane) - 1u));
                    before += incl - own;
                    list[at] = make_int4(tid, (int)(before & 0xffffu), (int)m, (int)(before >> 16));
                    uint32_t left = m;
#pragma unroll 1
                    for (int i = (int)(before & 0xffffu); left; ++i, left &= left - 1u) ptok_s[i] = (uint8_t)(__ffs(left) - 1);
                }
                __syncwarp();
                workers_sync();
                if (tid < 2) run_s[tid] = run_start(list, *nd_s, *weight_s, lgG, cta + tid, G);
                __syncwarp();
                cta_sync();
                nD = *nd_s;
                g0 = run_s[0];
                g1 = run_s[1];
            }
            // the outputs of the selection, by the finishing warps of CTA 0
            if (routed && cta == 0 && warp >= kMtWarps) {
#pragma unroll 1
                for (int t = warp - kMtWarps; t < T; t += kMtFin) {
                    const float w = topk_weight(lane < K ? w_s[t * K + lane] : 0.f, K);
                    uint64_t at = 1;
                    if (lane < K) {
                        const int e = id_s[t * K + lane];
                        at = slot_s[e];
                        a.ids[t * K + lane] = e;
                        a.weights[t * K + lane] = w;
                        a.slots[t * K + lane] = at;
                    }
                    const int nmiss = __popc(__ballot_sync(kFull, lane < K && at == 0));
                    if (lane == 0 && nmiss > 0) {
                        atomicAdd(a.miss, (uint32_t)nmiss);
                        atomicMin(a.ctrl, a.layer);
                    }
                    __syncwarp();
                }
            }
            if (bad && tid == 0 && cta == 0) {
                const int bits = ((bad & 1) && !routed ? RL_DEVERR_MISSING : 0) | (bad & 2 ? RL_DEVERR_SLOT_ALIGN : 0) |
                                 (bad & 4 ? RL_DEVERR_BAD_ID : 0) | (bad & 8 ? RL_DEVERR_NAN : 0);
                if (bits) dev_error(a.ctrl, bits);
            }
            if (bad & 7) return;
        }
        const int gr = (g1 - g0 + tpr - 1) / tpr, dr = cta < H / 16 ? (nD + epr - 1) >> (4 - lgu) : 0;
        const int rounds = down ? dr : gr;
        // passes (two tokens each) of a G round: as many as its most shared expert needs
        auto passes_of = [&](int r) {
            int n = 1;
#pragma unroll 1
            for (int i = 0; i < tpr; ++i) {
                const int tile = g0 + r * tpr + i;
                if (tile < g1) n = max(n, (__popc((uint32_t)list[tile >> lgG].z) + 1) >> 1);
            }
            return n;
        };
        if (warp >= kMtWarps) {
            // finishing warps: h of every third pass of G
#pragma unroll 1
            for (int r = 0; r < (down ? 0 : rounds) && ok; ++r) {
                const int passes = passes_of(r);
#pragma unroll 1
                for (int p = 0; p < passes && ok; ++p, ++s) {
                    if (s % kMtFin != warp - kMtWarps) continue;
                    const int buf = s % kMtRed;
                    ok = wait_or_stop<true>(redfull + buf, (s / kMtRed) & 1, stop_s);
                    if (!ok) break;
                    const int row = lane & 15, tk = 2 * p + (lane >> 4);  // lane = 16 token + row
#pragma unroll 1
                    for (int i = 0; i < tpr; ++i) {
                        const int tl = g0 + r * tpr + i;
                        if (tl >= g1) break;
                        const int4 q = list[tl >> lgG];
                        if (tk < __popc((uint32_t)q.z)) {
                            const float *v = red + (buf * kMtWarps + i * nb) * 64 + lane;
                            float gv = 0.f, uv = 0.f;
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                if (k < nb) {
                                    gv += v[k * 64];
                                    uv += v[k * 64 + 32];
                                }
                            const float rs = rs_s[ptok_s[q.y + tk]];
                            uint32_t h3[3];
                            split3(silu(rs * gv) * (rs * uv), h3);
                            uint16_t *h = a.hs + (size_t)(q.y + tk) * 3 * I + ((tl & ((1 << lgG) - 1)) << 4) + row;
#pragma unroll
                            for (int k = 0; k < 3; ++k)
                                __stcg(reinterpret_cast<unsigned short *>(h + (size_t)k * I), (unsigned short)h3[k]);
                        }
                        __syncwarp();
                    }
                    if (lane == 0) mbar_arrive(redempty + buf);
                    __syncwarp();
                }
            }
            if (down) {  // weights and pair numbers, for the combine
#pragma unroll 1
                for (int t = warp - kMtWarps; t < (routed ? T : 0); t += kMtFin) {
                    const float w = topk_weight(lane < K ? w_s[t * K + lane] : 0.f, K);
                    if (lane < K) w_s[t * K + lane] = w;
                    __syncwarp();
                }
#pragma unroll 1
                for (int i = tid - kMtWarps * 32; i < T * K; i += kMtFin * 32) {
                    const int e = id_s[i];
                    int at = 0, n = nD;  // position of e in the list (sorted by expert)
                    while (n > 1) {
                        const int h = n >> 1;
                        if (list[at + h].x <= e) at += h, n -= h;
                        else n = h;
                    }
                    pair_s[i] = (uint16_t)(list[at].y + __popc((uint32_t)list[at].z & ((1u << (i / K)) - 1u)));
                }
                __syncwarp();
            }
        } else {
            // this warp's units: G (gate and up of tile ti of the round, block blk), D (expert ti, block)
            const int ti = down ? warp >> lgu : warp >> lgnb, blk = down ? warp & (upe - 1) : warp & (nb - 1);
            const int width = down ? I : H, steps = down && I < 256 ? 4 : 8, go = down && I < 256 ? 32 * (g & 1) : 0;
            const bool even = (blk & 1) == 0;
            // byte of row g in the slot, and from there to row g + 8; a row of 128 values is half a block (rows
            // 2 i and 2 i + 1 share block i)
            const int off = !down ? ti * tileb + g * rowb + blk * kBlockBytes
                                  : ti * dnb + (I >= 256 ? (g << lgu) + blk : g >> 1) * kBlockBytes;
            const int r8 = !down ? 8 * rowb : (I >= 256 ? 8 << lgu : 4) * kBlockBytes;
            int haveA = -1, haveB = -1, ntok = 0, first = 0;  // B's rows; tokens and first pair of the round's expert
            auto find = [&](int r) {
                const int at = down ? r * epr + ti : (g0 + r * tpr + ti) >> lgG;
                const bool in = r < rounds && (down ? at < nD : ti < tpr && g0 + r * tpr + ti < g1);
                const int4 l = list[in ? at : 0];
                ntok = in ? __popc((uint32_t)l.z) : 0;
                first = l.y;
            };
            // the columns of pass p of the round found last; false where B stays as it is
            auto columns = [&](int p, BColumn &c) {
                if (2 * p >= ntok) return false;
                const int at = first + 2 * p;
                const int rA = down ? at : ptok_s[at];
                const int rB = 2 * p + 1 >= ntok ? -1 : down ? at + 1 : ptok_s[at + 1];
                if (rA == haveA && rB == haveB) return false;
                const uint16_t *src = down ? a.hs : a.xs;
                c = b_column(src + (size_t)rA * 3 * width, rB < 0 ? nullptr : src + (size_t)rB * 3 * width, width, blk * 256);
                haveA = rA;
                haveB = rB;
                return true;
            };
            BColumn next = {nullptr};
            find(0);
            if (columns(0, next)) load_b<WIDE>(b, next, steps, even);
#pragma unroll 1
            for (int r = 0; r < rounds && ok; ++r) {
                const int n = ntok, pair = first;
                const int passes = down ? max(1, (n + 1) >> 1) : passes_of(r);
                const uint8_t *st = ring + slot * a.halves * kMtUnits + off;
                ok = wait_or_stop<false>(full + slot, turn & 1, stop_s);
#pragma unroll 1
                for (int p = 0; p < passes && ok; ++p) {
                    const bool last = p == passes - 1;
                    if (!down) {
                        float v[2][2] = {};
                        if (2 * p < n) {
                            const uint8_t *const rows[2] = {st, st + 16 * rowb};
                            unit_dot<WIDE, 2>(rows, r8, 0, 8, even, b, tabc, v);
                        }
                        __syncwarp();
                        if (last && lane == 0) mbar_arrive(empty + slot);
                        if (last) find(r + 1);
                        if (columns(last ? 0 : p + 1, next)) load_b<WIDE>(b, next, steps, even);
                        const int buf = s % kMtRed;
                        if (s >= kMtRed) ok = wait_or_stop<false>(redempty + buf, (s / kMtRed - 1) & 1, stop_s);
                        if (t4 < 2 && 2 * p < n) {
                            float *o = red + (buf * kMtWarps + warp) * 64 + t4 * 16 + g;
                            o[0] = v[0][0];
                            o[8] = v[0][1];
                            o[32] = v[1][0];
                            o[40] = v[1][1];
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(redfull + buf);
                        ++s;
                    } else {
                        float v[1][2] = {};
                        if (2 * p < n) {
                            const uint8_t *const rows[1] = {st};
                            unit_dot<WIDE, 1>(rows, r8, go, steps, even, b, tabc, v);
                        }
                        __syncwarp();
                        if (last && lane == 0) mbar_arrive(empty + slot);
                        if (last) find(r + 1);
                        if (columns(last ? 0 : p + 1, next)) load_b<WIDE>(b, next, steps, even);
                        if (t4 < 2 && 2 * p + t4 < n) {
                            float *o = part + (((pair + 2 * p + t4) << lgu) + blk) * 16 + g;
                            o[0] = v[0][0];
                            o[8] = v[0][1];
                        }
                    }
                }
                if (++slot == a.stages) slot = 0, ++turn;
            }
        }
        if (!ok && lane == 0) {
            dev_error(a.ctrl, RL_DEVERR_WAIT_TIMEOUT);
            *stop_s = 1;
        }
        __syncwarp();
        if (workers_sync_or(!ok)) return;
        if (down) break;
        grid_arrive(a.ctr, target);
        if (!grid_wait(a.ctr, target, stop_s, a.ctrl, cap)) return;
    }
    if (cta >= H / 16) return;
#pragma unroll 1
    for (int i = tid; i < 16 * T; i += kMtWork) {
        const int t = i >> 4, row = i & 15;
        float *y = a.y + (size_t)t * H + cta * 16 + row;
        const float base = a.accumulate ? *y : 0.f;
        float acc = 0.f;
        int at = pair_s[t * K];
#pragma unroll 1
        for (int k = 0; k < K; ++k) {
            const float *v = part + (at << lgu) * 16 + row;
            at = pair_s[t * K + (k + 1 < K ? k + 1 : k)];
            const float w = w_s[t * K + k];
            float o = v[0];
            if (upe > 1) o += v[16];
#pragma unroll 1
            for (int j = 2; j < upe; ++j) o += v[j * 16];
            acc = fmaf(w, o, acc);
        }
        *y = a.accumulate ? base + acc : acc;
    }
}

size_t mt_raw_bytes(int T) { return (size_t)T * 512 * sizeof(float); }
size_t mt_x_bytes(int T, int H) { return align_up((size_t)T * 3 * H * sizeof(uint16_t), 256); }

}  // namespace

extern "C" size_t moe_decode_tokens_workspace_bytes(const rl_moe_shape *shp, int32_t T) {
    if (check_shape(shp) != RL_OK || T <= 0 || T > kMtMaxT) return 0;
    return kMtHdr + mt_raw_bytes(T) + mt_x_bytes(T, shp->hidden) +
           mt_x_bytes(T * shp->top_k, shp->inter);
}

extern "C" rl_status moe_decode_tokens(const rl_moe_shape *shp, int32_t layer, int32_t T, const float *x,
                                       float norm_eps, const float *w_router, const float *bias,
                                       const uint64_t *residency, const int8_t *codebook, int32_t *ids, float *weights,
                                       uint64_t *slots, uint32_t *miss, int32_t *ctrl, float *logits_out, float *y,
                                       int32_t accumulate, void *ws, size_t ws_bytes, void *stream) {
    const rl_status st = check_shape(shp);
    if (st != RL_OK) return st;
    if (layer < 0 || layer >= shp->n_layers)
        return fail(RL_ERR_INVALID, "moe_decode_tokens: layer %d outside [0, %d)", layer, shp->n_layers);
    if (T < 0) return fail(RL_ERR_INVALID, "moe_decode_tokens: T=%d", T);
    if (T > kMtMaxT) return fail(RL_ERR_UNSUPPORTED, "moe_decode_tokens: T=%d > %d (rl_route and moe_prefill_chunk take more)", T, kMtMaxT);
    if (T == 0) return RL_OK;
    if (!x || !codebook || !ids || !weights || !slots || !ctrl || !y)
        return fail(RL_ERR_INVALID, "moe_decode_tokens: NULL buffer");
    if (w_router && (!residency || !miss)) return fail(RL_ERR_INVALID, "moe_decode_tokens: NULL residency or miss");
    if (!w_router && logits_out) return fail(RL_ERR_INVALID, "moe_decode_tokens: logits_out without w_router");
    const size_t need = moe_decode_tokens_workspace_bytes(shp, T);
    if (!ws || ws_bytes < need)
        return fail(RL_ERR_INVALID, "moe_decode_tokens: workspace of %zu B needed, %zu given", need, ws_bytes);
    if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(w_router) | reinterpret_cast<uintptr_t>(ws)) & 15)
        return fail(RL_ERR_INVALID, "moe_decode_tokens: x, w_router and ws must be 16-byte aligned");
    MtArgs a = {};
    a.x = x;
    a.W = w_router;
    a.bias = bias;
    a.table = residency ? residency + (size_t)layer * shp->n_experts : nullptr;
    a.codebook = codebook;
    a.ids = ids;
    a.weights = weights;
    a.slots = slots;
    a.miss = miss ? miss + layer : nullptr;
    a.ctrl = ctrl;
    a.logits_out = logits_out;
    a.y = y;
    uint8_t *w8 = static_cast<uint8_t *>(ws);
    a.ctr = reinterpret_cast<unsigned long long *>(w8);
    a.rs = reinterpret_cast<float *>(w8 + 128);
    a.raw = reinterpret_cast<float *>(w8 + kMtHdr);
    a.xs = reinterpret_cast<uint16_t *>(w8 + kMtHdr + mt_raw_bytes(T));
    a.hs = reinterpret_cast<uint16_t *>(w8 + kMtHdr + mt_raw_bytes(T) + mt_x_bytes(T, shp->hidden));
    a.eps = norm_eps;
    a.layer = layer;
    a.T = T;
    a.H = shp->hidden;
    a.E = shp->n_experts;
    a.K = shp->top_k;
    a.I = shp->inter;
    a.accumulate = accumulate != 0;
    // two 16-unit halves per ring slot, one where the partial outputs leave too little room
    const int ring = mt_ring(T, a.K, a.I), room = (227 * 1024 - ring) / kMtUnits;
    a.halves = room >= 4 ? 2 : 1;
    a.stages = room / a.halves < kMtMaxStages ? room / a.halves : kMtMaxStages;
    const size_t smem = ring + (size_t)a.stages * a.halves * kMtUnits;
    if (a.stages < 1) return fail(RL_ERR_UNSUPPORTED, "moe_decode_tokens: T=%d top_k=%d inter=%d does not fit", T, a.K, a.I);
    const int G = sm_count();
    if (G < 128) return fail(RL_ERR_UNSUPPORTED, "moe_decode_tokens: needs a GPU of 128 SMs or more");
    // 32-bit reads of the group bytes need two blocks or more per matrix row
    const void *kernel = a.H >= 512 && a.I >= 512 ? (const void *)moe_tokens_kernel<true> : (const void *)moe_tokens_kernel<false>;
    const rl_status sa = allow_smem(kernel, smem);
    if (sa != RL_OK) return sa;
    void *args[] = {&a};
    const cudaError_t e = cudaLaunchCooperativeKernel(kernel, dim3(G), dim3(kMtThreads), args, smem, as_stream(stream));
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(RL_ERR_CUDA, "moe_decode_tokens: launch failed: %s", cudaGetErrorString(e));
    }
    return RL_OK;
}
