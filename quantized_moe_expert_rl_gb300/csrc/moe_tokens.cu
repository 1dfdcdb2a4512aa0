// moe_tokens.cu - moe_decode_tokens: a whole routed MoE layer for 1 to 32 tokens in ONE launch.
//
//   logits = W_r xn (+ bias),  ids = top-K, weights = softmax over the selection,
//   y[t] (+)= sum_k weights[t][k] * down_k(silu(gate_k xn_t) * (up_k xn_t))
//
// One cooperative CTA per SM: 16 computing warps and one warp that issues the weight copies.
//   R  every CTA takes up to four router rows (a quarter row per warp, f32 dots with every
//      token), and a share of the split of x into bf16 parts;  grid barrier
//   S  every CTA selects for itself (one warp per token, the same code on the same logits): the
//      list of distinct experts, each with its tokens as a bit mask, and from it the whole
//      schedule of weight copies.  CTA 0 writes ids, weights, slots, misses and the flag
//   G  the (expert, 16 hidden rows) tiles of gate and up, in equal runs over the CTAs -> h
//      grid barrier (the copies of D's weights are already under way)
//   D  CTA b: output rows 16 b .. 16 b + 15 of every expert's down matrix; the partial outputs stay
//      in shared memory, so the sum over k in selection order needs no further exchange.
//
// The matrix arithmetic.  A weight is d * (codebook value) * (sign): the codebook value is an
// 8-bit integer, exact in bf16, so a group's 8 values are one 16-byte table entry whose signs are
// flipped by XOR; 16 weight rows are the A operand of mma.m16n8k16 and d multiplies the f32
// sums of a 256-value block.  An f32 activation is exactly the sum of three bf16 values (its
// leading 8 bits, the next 8, the last 8, each taken by truncation), so three columns of B
// carry it without loss, two tokens share the 8 columns of one MMA, and the products are exact
// before the f32 sums.  On the CUDA cores the same dot needs two unpacking instructions and a packed FMA
// per pair of weights (25 instructions per group against 13 here).
#include "decode_rows.cuh"
#include "select.cuh"
#include "stack_kernel.cuh"

using namespace rl;

namespace {

constexpr int kMtWarps = 16, kMtThreads = kMtWarps * 32 + 32;
constexpr int kMtMaxT = 32;
constexpr int kMtStage = 16896;    // one round of weights: 16 units of 16 rows x 256 values
constexpr int kMtMaxStages = 8;
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
    float *rs, *raw;       // [32] RMS scales, [T][E] router dots
    uint16_t *xs, *hs;     // [T][3][H], [T K][3][I] bf16 parts
    float eps;
    int layer, T, H, E, K, I, accumulate, stages;
};

struct MtLayout {
    uint32_t o_red, o_list, o_mask, o_slot, o_id, o_w, o_pair, o_ptok, o_sel, o_part, o_ring, total;
    __host__ __device__ MtLayout(int T, int K, int I, int stages) {
        const uint32_t P = T * K;
        o_red = 512 + kTabBytes;                       // [2][16 warps][2 tokens][16 rows] f32
        o_list = o_red + 2 * kMtWarps * 32 * 4;        // [512] (expert, first pair, token mask, -)
        o_mask = o_list + 512 * 16;                    // [512] u32
        o_slot = o_mask + 512 * 4;                     // [512] u64
        o_id = o_slot + 512 * 8;                       // [P] i32
        o_w = o_id + 512 * 4;                          // [P] f32
        o_pair = o_w + 512 * 4;                        // [P] u16 pair index of (t, k)
        o_ptok = o_pair + 512 * 2;                     // [P] u8 token of a pair
        o_sel = o_ptok + 512;                          // [16 warps] selection scratch
        o_part = o_sel + kMtWarps * 448;               // [P][units per expert][16] f32
        o_ring = (uint32_t)align_up(o_part + P * (I > 256 ? I / 256 : 1) * 64, 128);
        total = o_ring + stages * kMtStage;
    }
};

__device__ __forceinline__ void workers_sync() {
    asm volatile("bar.sync 1, 512;" ::: "memory");
    __syncwarp();
}
// the same with a vote: true in every computing warp when any of them brought `pred`
__device__ __forceinline__ bool workers_sync_or(bool pred) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 1, 512, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"(pred ? 1u : 0u)
        : "memory");
    __syncwarp();
    return any != 0u;
}

// The computing warps of all CTAs meet (see grid_sync in stack_kernel.cuh; the copying warp does not
// take part).
__device__ __forceinline__ bool workers_grid_sync(unsigned long long *ctr, unsigned long long &target, int *ok_s,
                                                  int32_t *ctrl, uint32_t cap) {
    workers_sync();
    if (threadIdx.x == 0) {
        unsigned long long old;
        asm volatile("atom.add.release.gpu.global.u64 %0, [%1], 1;" : "=l"(old) : "l"(ctr) : "memory");
        if (target == 0ull) target = old - old % gridDim.x;
        target += gridDim.x;
        bool ok = false;
        for (uint32_t i = 0; i < cap; ++i)
            if (ld_acquire_u64(ctr) >= target) {
                ok = true;
                break;
            }
        if (!ok) dev_error(ctrl, RL_DEVERR_WAIT_TIMEOUT);
        *ok_s = ok;
    }
    workers_sync();
    return *ok_s != 0;
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

// the 8 signed codebook values of the group bytes gs (index | sign mask << 8) as bf16 pairs
__device__ __forceinline__ uint4 signed_group(uint32_t gs, const uint4 *tabc) {
    uint4 q = tabc[(gs & 0xffu) * kTabCopies];
    const uint32_t s = gs >> 8;
    q.x ^= (s * 0x40008000u) & 0x80008000u;
    q.y ^= (s * 0x10002000u) & 0x80008000u;
    q.z ^= (s * 0x04000800u) & 0x80008000u;
    q.w ^= (s * 0x01000200u) & 0x80008000u;
    return q;
}

// One unit: 16 rows x 32 STEPS values against two tokens.  p0, p1: this lane's first group bytes of
// rows g and g + 8 (lane = 4 g + t, group 4 j + t in step j); b: its B fragments.  Returns, in lanes
// t = 0, 1, token t's sums for rows g (v0) and g + 8 (v1), without the block scale.
template <int STEPS>
__device__ __forceinline__ void unit_dot(const uint8_t *p0, const uint8_t *p1, const uint4 (&b)[8], const uint4 *tabc,
                                         float &v0, float &v1) {
    float c[4] = {0.f, 0.f, 0.f, 0.f}, e[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
        const uint4 q = signed_group(*reinterpret_cast<const uint16_t *>(p0 + 8 * j), tabc);
        const uint4 r = signed_group(*reinterpret_cast<const uint16_t *>(p1 + 8 * j), tabc);
        mma_bf16(c, q.x, r.x, q.y, r.y, b[j].x, b[j].y);
        mma_bf16(e, q.z, r.z, q.w, r.w, b[j].z, b[j].w);
    }
    // columns 0, 1: token 0 leading and middle parts; 2, 3: token 1; 4: token 0 last part; 5: token 1
    const int src = (threadIdx.x & 28) | 2, t = threadIdx.x & 3;
    const float c0 = c[0] + e[0], c1 = c[1] + e[1], c2 = c[2] + e[2], c3 = c[3] + e[3];
    const float l0 = __shfl_sync(kFull, c0, src), l1 = __shfl_sync(kFull, c1, src);
    const float l2 = __shfl_sync(kFull, c2, src), l3 = __shfl_sync(kFull, c3, src);
    v0 = (c0 + c1) + (t == 0 ? l0 : l1);
    v1 = (c2 + c3) + (t == 0 ? l2 : l3);
}

// B fragments of two rows of bf16 parts (rowA, rowB: [3][width], rowB may be NULL), values from
// `at` on: lane (n, t) holds column n's groups 4 j + t.
template <int STEPS>
__device__ __forceinline__ void load_b(uint4 (&b)[8], const uint16_t *rowA, const uint16_t *rowB, int width, int at) {
    const int n = (threadIdx.x >> 2) & 7, t = threadIdx.x & 3;
    const uint16_t *row = (n == 2 || n == 3 || n == 5) ? rowB : rowA;
    const int part = n >= 4 ? 2 : n & 1;
    const bool in = n < 6 && row != nullptr;
    const uint4 *p = reinterpret_cast<const uint4 *>(row + part * width + at) + t;
#pragma unroll
    for (int j = 0; j < STEPS; ++j) b[j] = in ? __ldcg(p + 4 * j) : make_uint4(0u, 0u, 0u, 0u);
}

__global__ void __launch_bounds__(kMtThreads, 1) moe_tokens_kernel(const __grid_constant__ MtArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    const MtLayout lay(a.T, a.K, a.I, a.stages);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem), *empty = full + kMtMaxStages;
    int *ok_s = reinterpret_cast<int *>(smem + 128);
    volatile int *stop_s = reinterpret_cast<volatile int *>(smem + 132);
    int *bad_s = reinterpret_cast<int *>(smem + 136);    // bit 0: a slot is absent, bit 1: misaligned, bit 2: bad id
    int *scan_s = reinterpret_cast<int *>(smem + 160);   // [16][2] warp totals of the list
    uint32_t *cap_s = reinterpret_cast<uint32_t *>(smem + 140);
    int *skip_s = reinterpret_cast<int *>(smem + 144);
    int *nd_s = reinterpret_cast<int *>(smem + 148);
    int *hold_s = reinterpret_cast<int *>(smem + 152);
    uint4 *tab = reinterpret_cast<uint4 *>(smem + 512);
    float *red = reinterpret_cast<float *>(smem + lay.o_red);
    int4 *list = reinterpret_cast<int4 *>(smem + lay.o_list);
    uint32_t *mask_s = reinterpret_cast<uint32_t *>(smem + lay.o_mask);
    uint64_t *slot_s = reinterpret_cast<uint64_t *>(smem + lay.o_slot);
    int *id_s = reinterpret_cast<int *>(smem + lay.o_id);
    float *w_s = reinterpret_cast<float *>(smem + lay.o_w);
    uint16_t *pair_s = reinterpret_cast<uint16_t *>(smem + lay.o_pair);
    uint8_t *ptok_s = smem + lay.o_ptok;
    float *part = reinterpret_cast<float *>(smem + lay.o_part);
    uint8_t *ring = smem + lay.o_ring;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = gridDim.x, cta = blockIdx.x;
    const int T = a.T, H = a.H, E = a.E, K = a.K, I = a.I;
    const bool routed = a.W != nullptr;  // else ids, weights and slots are given

    if (tid == 0) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, kMtWarps);
        }
        fence_mbar_init();
        *stop_s = 0;
        *bad_s = 0;
        const uint32_t *knob = reinterpret_cast<const uint32_t *>(a.ctr) + 16;
        *cap_s = knob[0] ? knob[0] : kSpinCap;
        *hold_s = (int)knob[1];
        const int flag = ld_ctrl(a.ctrl);
        *skip_s = routed ? flag < a.layer : flag <= a.layer;
    }
    // R: the router rows of this CTA (row r -> expert cta + r G), a quarter of a row per warp
    const int q4 = H / 4, wrow = warp >> 2, wexp = cta + wrow * G, wcol = (warp & 3) * q4 + 4 * lane;
    const bool wmine = routed && warp < kMtWarps && wexp < E;
    float4 wv[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        wv[j] = wmine && 128 * j + 4 * lane < q4
                    ? __ldg(reinterpret_cast<const float4 *>(a.W + (size_t)wexp * H + wcol + 128 * j))
                    : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int e = tid; e < 512; e += kMtThreads) mask_s[e] = 0u;
    build_pair_table(tab, a.codebook, nullptr);  // ends with a CTA barrier
    if (*skip_s) return;
    unsigned long long target = 0ull;
    if (warp < kMtWarps) {
        if (wmine)
            for (int t0 = 0; t0 < T; t0 += 4) {
                float s[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    s[u] = 0.f;
                    const int t = t0 + u < T ? t0 + u : T - 1;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (128 * j + 4 * lane < q4) {
                            const float4 v = *reinterpret_cast<const float4 *>(a.x + (size_t)t * H + wcol + 128 * j);
                            s[u] = fmaf(wv[j].x, v.x, fmaf(wv[j].y, v.y, fmaf(wv[j].z, v.z, fmaf(wv[j].w, v.w, s[u]))));
                        }
                }
                __syncwarp();
#pragma unroll
                for (int u = 0; u < 4; ++u) s[u] = warp_sum(s[u]);
                // partial dots [4 rows][4 quarters][32 tokens] in the (still unused) reduction buffer
                if (lane < 4 && t0 + lane < T)
                    red[warp * 32 + t0 + lane] = lane == 0 ? s[0] : lane == 1 ? s[1] : lane == 2 ? s[2] : s[3];
            }
        // x as bf16 parts, 8 values at a time over the whole grid
        for (int i = cta * 512 + tid; i < T * H / 8; i += G * 512) {
            const int t = i / (H / 8), h = (i - t * (H / 8)) * 8;
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
        if (warp == kMtWarps - 1 && G - 1 - cta < T) {
            const int t = G - 1 - cta;
            bool range = false;
            const float r = a.eps >= 0.f ? rms_scale_warp(a.x + (size_t)t * H, H, a.eps, &range) : 1.f;
            if (lane == 0) {
                __stcg(a.rs + t, r);
                if (range) dev_error(a.ctrl, RL_DEVERR_RANGE);
            }
            __syncwarp();
        }
        workers_sync();
        if (routed && tid < 4 * T) {
            const int r = tid / T, t = tid - r * T, e = cta + r * G;
            if (e < E)
                __stcg(a.raw + (size_t)t * E + e, (red[(4 * r) * 32 + t] + red[(4 * r + 1) * 32 + t]) +
                                                      (red[(4 * r + 2) * 32 + t] + red[(4 * r + 3) * 32 + t]));
        }
        bool ok = *hold_s - 1 != cta;  // test knob: this CTA leaves before its arrival
        if (ok) ok = workers_grid_sync(a.ctr, target, ok_s, a.ctrl, *cap_s);
        if (!ok && tid == 0) *stop_s = 1;
        // S: selection, one warp per token
        if (ok)
            for (int t = warp; t < T; t += kMtWarps) {
                int my_id = 0;
                float my_val = 0.f, w = 0.f;
                uint64_t slot = 1;
                if (routed) {
                    const float rs = __ldcg(a.rs + t);
                    uint32_t key[16];
                    bool nan = false;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const int e = sel_id(lane, j);
                        float v = 0.f;
                        key[j] = 0u;
                        if (e < E) {
                            v = rs * __ldcg(a.raw + (size_t)t * E + e) + (a.bias ? a.bias[e] : 0.f);
                            nan |= v != v;
                            key[j] = order_key(v);
                            if (a.logits_out && cta == 0) a.logits_out[(size_t)t * E + e] = v;
                        }
                    }
                    if (__any_sync(kFull, nan) && lane == 0 && cta == 0) dev_error(a.ctrl, RL_DEVERR_NAN);
                    __syncwarp();
                    uint8_t *sc = smem + lay.o_sel + warp * 448;
                    warp_topk_thr(key, E, K, reinterpret_cast<uint32_t *>(sc), reinterpret_cast<uint2 *>(sc + 128),
                                  reinterpret_cast<int *>(sc + 384), my_id, my_val);
                    w = topk_weight(my_val, K);
                    if (lane < K) slot = a.table[my_id];
                } else if (lane < K) {
                    my_id = a.ids[t * K + lane];
                    w = a.weights[t * K + lane];
                    slot = a.slots[t * K + lane];
                    if (my_id < 0 || my_id >= E) {
                        atomicOr(bad_s, 4);
                        my_id = 0;
                    }
                }
                __syncwarp();
                if (lane < K) {
                    id_s[t * K + lane] = my_id;
                    w_s[t * K + lane] = w;
                    slot_s[my_id] = slot;
                    atomicOr(mask_s + my_id, 1u << t);
                    if (slot == 0) atomicOr(bad_s, 1);
                    if (slot & 15) atomicOr(bad_s, 2);
                    if (routed && cta == 0) {
                        a.ids[t * K + lane] = my_id;
                        a.weights[t * K + lane] = w;
                        a.slots[t * K + lane] = slot;
                    }
                }
                const int nmiss = __popc(__ballot_sync(kFull, lane < K && slot == 0));
                if (lane == 0 && nmiss > 0 && cta == 0 && routed) {
                    atomicAdd(a.miss, (uint32_t)nmiss);
                    atomicMin(a.ctrl, a.layer);
                }
                __syncwarp();
            }
    }
    cta_sync();
    if (*stop_s) return;
    if (*bad_s) {
        if (tid == 0 && cta == 0) {
            const int b = *bad_s;
            const int bits = ((b & 1) && !routed ? RL_DEVERR_MISSING : 0) | (b & 2 ? RL_DEVERR_SLOT_ALIGN : 0) |
                             (b & 4 ? RL_DEVERR_BAD_ID : 0);
            if (bits) dev_error(a.ctrl, bits);
        }
        return;
    }
    // The list of distinct experts in index order: thread e holds expert e; its pairs (expert, token)
    // are numbered in token order from `off`.
    uint32_t m = 0u;
    int incl = 0;
    if (warp < kMtWarps) {
        m = tid < E ? mask_s[tid] : 0u;
        incl = __popc(m);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += v;
        }
        const unsigned has = __ballot_sync(kFull, m != 0u);
        if (lane == 31) {
            scan_s[2 * warp] = __popc(has);
            scan_s[2 * warp + 1] = incl;
        }
        __syncwarp();
        workers_sync();
        int at = __popc(has & ((1u << lane) - 1u)), off = incl - __popc(m);
        for (int w = 0; w < warp; ++w) {
            at += scan_s[2 * w];
            off += scan_s[2 * w + 1];
        }
        if (m) {
            list[at] = make_int4(tid, off, (int)m, 0);
            uint32_t left = m;
            for (int i = 0; left; ++i, left &= left - 1u) ptok_s[off + i] = (uint8_t)(__ffs(left) - 1);
        }
        __syncwarp();
        if (tid == 0) {
            int n = 0;
            for (int w = 0; w < kMtWarps; ++w) n += scan_s[2 * w];
            *nd_s = n;
        }
    }
    cta_sync();
    const int nD = *nd_s;
    // schedule: gate/up tiles [g0, g1) of this CTA, then the down rows of every expert
    const int RT = I / 16, nb = H / 256, rowb = nb * kBlockBytes, tpr = 8 / nb, tileb = 32 * rowb;
    const int tiles = nD * RT, g0 = (int)((long long)cta * tiles / G), g1 = (int)((long long)(cta + 1) * tiles / G);
    const int gr = (g1 - g0 + tpr - 1) / tpr;
    const int upe = I > 256 ? I / 256 : 1, epr = kMtWarps / upe, dnb = I * kBlockBytes / 16;
    const int dr = cta < H / 16 ? (nD + epr - 1) / epr : 0;

    if (warp == kMtWarps) {  // the copying warp
        const size_t mat = (size_t)I * rowb;
        int slot = 0, turn = 0;
        bool ok = true;
        int issued = 0;
        for (int r = 0; r < gr + dr && ok; ++r) {
            if (turn > 0) {
                ok = false;
                for (uint32_t i = 0; i < kSpinCap && !ok; ++i) {
                    ok = mbar_try_wait(empty + slot, (turn - 1) & 1);
                    if (*stop_s) break;
                }
                ok = __all_sync(kFull, ok) != 0;
                if (!ok) {
                    if (lane == 0) dev_error(a.ctrl, RL_DEVERR_WAIT_TIMEOUT);
                    break;
                }
            }
            uint8_t *dst = ring + slot * kMtStage;
            if (r < gr) {
                const int n = min(tpr, g1 - g0 - r * tpr);
                if (lane == 0) mbar_arrive_expect_tx(full + slot, n * tileb);
                __syncwarp();
                if (lane < 2 * n) {
                    const int tile = g0 + r * tpr + (lane >> 1), ei = tile / RT, rt = tile - ei * RT;
                    const uint8_t *rec = reinterpret_cast<const uint8_t *>(slot_s[list[ei].x]);
                    bulk_g2s(dst + (lane >> 1) * tileb + (lane & 1) * 16 * rowb,
                             rec + (lane & 1) * mat + (size_t)rt * 16 * rowb, 16 * rowb, full + slot);
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
        for (int r = max(0, issued - a.stages); r < issued; ++r) mbar_wait_warp(full + r % a.stages, (r / a.stages) & 1);
        return;
    }

    // pair numbers of (t, k)
    for (int e = tid; e < nD; e += 512) mask_s[list[e].x] = (uint32_t)e;  // expert -> position in the list
    workers_sync();
    for (int i = tid; i < T * K; i += 512) {
        const int4 l = list[mask_s[id_s[i]]];
        pair_s[i] = (uint16_t)(l.y + __popc((uint32_t)l.z & ((1u << (i / K)) - 1u)));
    }
    const int g = lane >> 2, t4 = lane & 3;
    const uint4 *tabc = tab + (lane & (kTabCopies - 1));
    int slot = 0, turn = 0, buf = 0, haveA = -1, haveB = -1;
    uint4 b[8];
    bool ok = true;
    // G: gate and up
    for (int r = 0; r < gr && ok; ++r) {
        const int ti = warp / (2 * nb), tile = g0 + r * tpr + ti, ei = tile / RT;
        const bool mine = tile < g1;
        const int4 l = mine ? list[ei] : make_int4(0, 0, 0, 0);
        const int ntok = __popc((uint32_t)l.z);
        int passes = 1;  // two tokens each; the same for every warp of the CTA
        for (int i = 0; i < tpr; ++i)
            if (g0 + r * tpr + i < g1) passes = max(passes, (__popc((uint32_t)list[(g0 + r * tpr + i) / RT].z) + 1) / 2);
        const int blk = warp % nb;
        const uint8_t *base = ring + slot * kMtStage + ti * tileb + ((warp / nb) & 1) * 16 * rowb + blk * kBlockBytes;
        const uint8_t *p0 = base + g * rowb, *p1 = p0 + 8 * rowb;
        for (int p = 0; p < passes; ++p) {
            if (mine && 2 * p < ntok) {
                const int tA = ptok_s[l.y + 2 * p], tB = 2 * p + 1 < ntok ? ptok_s[l.y + 2 * p + 1] : -1;
                if (tA != haveA || tB != haveB) {
                    load_b<8>(b, a.xs + (size_t)tA * 3 * H, tB < 0 ? nullptr : a.xs + (size_t)tB * 3 * H, H, blk * 256);
                    haveA = tA;
                    haveB = tB;
                }
            }
            if (p == 0) ok = mbar_wait_warp(full + slot, turn & 1);
            if (mine && 2 * p < ntok && ok) {
                float v0, v1;
                unit_dot<8>(p0 + 2 + 2 * t4, p1 + 2 + 2 * t4, b, tabc, v0, v1);
                const float d0 = fp16_bits_to_float(*reinterpret_cast<const uint16_t *>(p0));
                const float d1 = fp16_bits_to_float(*reinterpret_cast<const uint16_t *>(p1));
                if (t4 < 2) {
                    float *o = red + (buf * kMtWarps + warp) * 32 + t4 * 16;
                    o[g] = d0 * v0;
                    o[g + 8] = d1 * v1;
                }
            }
            __syncwarp();
            if (p == passes - 1 && lane == 0) mbar_arrive(empty + slot);
            ok = !workers_sync_or(!ok);
            if (!ok) break;
            // h of tile i by one warp: lane = 16 token + row
            for (int i = 0; i < tpr; ++i) {
                const int tl = g0 + r * tpr + i;
                if (tl >= g1 || ((r + p) * tpr + i) % kMtWarps != warp) continue;
                const int4 q = list[tl / RT];
                const int row = lane & 15, s = lane >> 4, tk = 2 * p + s;
                if (tk < __popc((uint32_t)q.z)) {
                    const float *o = red + (buf * kMtWarps + i * 2 * nb) * 32 + s * 16 + row;
                    float gv = 0.f, uv = 0.f;
                    for (int k = 0; k < nb; ++k) {
                        gv += o[k * 32];
                        uv += o[(nb + k) * 32];
                    }
                    const float rs = __ldcg(a.rs + ptok_s[q.y + tk]);
                    uint32_t h3[3];
                    split3(silu(rs * gv) * (rs * uv), h3);
                    uint16_t *h = a.hs + (size_t)(q.y + tk) * 3 * I + (tl % RT) * 16 + row;
#pragma unroll
                    for (int k = 0; k < 3; ++k) __stcg(reinterpret_cast<unsigned short *>(h + (size_t)k * I), (unsigned short)h3[k]);
                }
                __syncwarp();
            }
            buf ^= 1;
        }
        if (++slot == a.stages) slot = 0, ++turn;
    }
    if (!ok) {
        if (lane == 0) {
            dev_error(a.ctrl, RL_DEVERR_WAIT_TIMEOUT);
            *stop_s = 1;
        }
        return;
    }
    if (!workers_grid_sync(a.ctr, target, ok_s, a.ctrl, *cap_s)) {
        if (tid == 0) *stop_s = 1;
        return;
    }
    if (dr == 0) return;
    // D: this CTA's 16 output rows of every expert
    const int ui = warp / upe, blk = warp % upe;
    for (int r = 0; r < dr; ++r) {
        const int ei = r * epr + ui;
        const bool mine = ei < nD;
        const int4 l = mine ? list[ei] : make_int4(0, 0, 0, 0);
        const int ntok = __popc((uint32_t)l.z);
        const uint8_t *base = ring + slot * kMtStage + ui * dnb;
        // a row of 128 values is half a block: rows 2 i and 2 i + 1 share block i
        const uint8_t *p0 = I >= 256 ? base + g * (I / 256 * kBlockBytes) + blk * kBlockBytes : base + (g >> 1) * kBlockBytes;
        const uint8_t *p1 = p0 + (I >= 256 ? 8 * (I / 256) : 4) * kBlockBytes;
        const int go = I >= 256 ? 0 : 32 * (g & 1);
        for (int p = 0; 2 * p < ntok || p == 0; ++p) {
            if (mine) {
                const int pa = l.y + 2 * p;
                const uint16_t *A = a.hs + (size_t)pa * 3 * I, *B = 2 * p + 1 < ntok ? A + 3 * I : nullptr;
                if (I >= 256) load_b<8>(b, A, B, I, blk * 256);
                else load_b<4>(b, A, B, I, 0);
            }
            if (p == 0) ok = mbar_wait_warp(full + slot, turn & 1);
            if (mine && ok) {
                float v0, v1;
                if (I >= 256) unit_dot<8>(p0 + 2 + 2 * t4, p1 + 2 + 2 * t4, b, tabc, v0, v1);
                else unit_dot<4>(p0 + go + 2 + 2 * t4, p1 + go + 2 + 2 * t4, b, tabc, v0, v1);
                const float d0 = fp16_bits_to_float(*reinterpret_cast<const uint16_t *>(p0));
                const float d1 = fp16_bits_to_float(*reinterpret_cast<const uint16_t *>(p1));
                if (t4 < 2 && 2 * p + t4 < ntok) {
                    float *o = part + ((size_t)(l.y + 2 * p + t4) * upe + blk) * 16;
                    o[g] = d0 * v0;
                    o[g + 8] = d1 * v1;
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + slot);
        if (!ok) break;
        if (++slot == a.stages) slot = 0, ++turn;
    }
    if (!ok && lane == 0) {
        dev_error(a.ctrl, RL_DEVERR_WAIT_TIMEOUT);
        *stop_s = 1;
    }
    __syncwarp();
    if (workers_sync_or(!ok)) return;
    for (int i = tid; i < 16 * T; i += 512) {
        const int t = i >> 4, row = i & 15;
        float acc = 0.f;
        for (int k = 0; k < K; ++k) {
            const float *o = part + (size_t)pair_s[t * K + k] * upe * 16 + row;
            float v = 0.f;
            for (int j = 0; j < upe; ++j) v += o[j * 16];
            acc = fmaf(w_s[t * K + k], v, acc);
        }
        float *y = a.y + (size_t)t * H + cta * 16 + row;
        *y = a.accumulate ? *y + acc : acc;
    }
}

size_t mt_raw_bytes(int T, int E) { return align_up((size_t)T * E * sizeof(float), 256); }
size_t mt_x_bytes(int T, int H) { return align_up((size_t)T * 3 * H * sizeof(uint16_t), 256); }

}  // namespace

extern "C" size_t moe_decode_tokens_workspace_bytes(const rl_moe_shape *shp, int32_t T) {
    if (check_shape(shp) != RL_OK || T <= 0 || T > kMtMaxT) return 0;
    return kMtHdr + mt_raw_bytes(T, shp->n_experts) + mt_x_bytes(T, shp->hidden) +
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
    a.xs = reinterpret_cast<uint16_t *>(w8 + kMtHdr + mt_raw_bytes(T, shp->n_experts));
    a.hs = reinterpret_cast<uint16_t *>(w8 + kMtHdr + mt_raw_bytes(T, shp->n_experts) + mt_x_bytes(T, shp->hidden));
    a.eps = norm_eps;
    a.layer = layer;
    a.T = T;
    a.H = shp->hidden;
    a.E = shp->n_experts;
    a.K = shp->top_k;
    a.I = shp->inter;
    a.accumulate = accumulate != 0;
    for (a.stages = kMtMaxStages; a.stages > 2; --a.stages)
        if (MtLayout(T, a.K, a.I, a.stages).total <= 227 * 1024) break;
    const size_t smem = MtLayout(T, a.K, a.I, a.stages).total;
    const int G = sm_count();
    if (G < 128 || smem > 227 * 1024)
        return fail(RL_ERR_UNSUPPORTED, "moe_decode_tokens: needs 128 SMs and 227 KB of shared memory");
    const rl_status sa = allow_smem((const void *)moe_tokens_kernel, smem);
    if (sa != RL_OK) return sa;
    void *args[] = {&a};
    const cudaError_t e = cudaLaunchCooperativeKernel((const void *)moe_tokens_kernel, dim3(G), dim3(kMtThreads), args,
                                                      smem, as_stream(stream));
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(RL_ERR_CUDA, "moe_decode_tokens: launch failed: %s", cudaGetErrorString(e));
    }
    return RL_OK;
}
