// logprobs.cu - rl_logprobs: log probability of given tokens, entropy and the n most probable
// tokens of each row of logits, one pass over the logits.
//
//   lse = m + log S,  S = sum e^(x - m),  U = sum (x - m) e^(x - m),  m = max x
//   logprob = x_target - lse,  entropy = log S - U / S
//
// The logits of all rows are one long array, cut into equal runs, one per CTA (three CTAs per SM), so
// that any number of rows keeps the GPU evenly busy.  A CTA streams its run in tiles of 4096 values;
// every thread copies the 16-byte pieces that it will read itself, three tiles
// ahead and on across the rows, so that no barrier stands between the copies and their use.  Rows
// that lie whole in a run are finished at once.  Every thread keeps a running (m, S, U), to which a tile's 16
// terms are added as one sum; when a tile raises m by d, S and U are rescaled by e^-d (U loses d S first).  The pieces of a row cut by a run's end meet in the last of their CTAs to
// finish (a completion counter in the workspace), which merges them in row order, so results do not
// depend on arrival order.
//
// Top n.  A candidate is a 64-bit key, order-preserving logit above ~index, so that keys are
// distinct and equal logits go to the lower index.  Only keys above a threshold are kept, in a buffer
// that is cut back to its n best whenever it holds more than 64, by counting for every key the
// larger ones.  A row's first tile sets the threshold: the CTA's 64 groups of 4 threads each publish
// their largest logit, and the n-th largest of the 64 bounds the tile's n-th largest from below.  The
// survivors (a few more than n) go into the buffer without a barrier; every fourth tile the CTA meets
// and cuts the buffer back if need be.  If it overflowed (rising logits, masses of equal ones) the CTA
// goes through those tiles again with the groups' largest keys, which are distinct, so that a tile
// leaves at most n groups x 64 of them.
//
// Measured back to back in a graph: 512 x 131072 f32 (268.5 MB, 39.6 us at the measured copy rate) 72.3 us
// with the 20 best tokens, 53.8 without any; 912 rows without any 71.8 us, 6.7 TB/s.  What is left are the
// rows cut by the runs' ends (with 512 rows every CTA has two: two publications and a merge; 456 rows, which
// have none, take 51.1 us with the 20 best and 38.6 without) and the insertions.  One row of 131072 takes 9.7 us, 16 rows of 100003 bf16 11.7 us: a chain of latencies
// (launch, tile, first threshold, publication, merge).
#include <math.h>

#include "qdot.cuh"
#include "row_types.cuh"
#include "select.cuh"

using namespace rl;

namespace {

constexpr int kLpThreads = 256, kLpEpt = 16, kLpTile = kLpThreads * kLpEpt;
constexpr int kLpMaxN = 32;
constexpr int kLpMaxCtas = 3 * 152;
constexpr int kLpMaxPieces = 64;                    // of one row
constexpr int kLpDepth = 3;                         // tiles on their way
constexpr int kLpTurn = 4;                          // tiles between two meetings of the CTA
constexpr int kLpKeep = 64;                         // the buffer is cut back beyond this many
constexpr int kLpCap = kLpKeep + 64 * kLpMaxN;      // and never holds more than this
constexpr float kLog2e = 1.4426950408889634f;

struct LpArgs {
    const void *x;
    const int32_t *targets;
    float *logprob, *entropy;
    int32_t *top_ids;
    float *top_logprob;
    float *part;               // [CTAs][2][4] (m, S, U) of the run's first and last piece
    unsigned long long *keys;  // [CTAs][2][n]
    uint32_t *done;            // [CTAs], by the CTA of a row's first piece; zero between calls
    long long total, run;      // values in all, per CTA
    int V, n, per_row;         // per_row > 0: that many CTAs per row, none over a row's end
};

struct LpShared {
    unsigned long long cand[kLpCap];
    unsigned long long sorted[kLpMaxN];
    unsigned long long heads[64];
    unsigned long long thr;
    float red[3][kLpThreads / 32], xt[2];
    int count, merge[2];
};

__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ unsigned long long dup2(float v) { return pack2(__float_as_uint(v), __float_as_uint(v)); }
__device__ __forceinline__ unsigned long long fadd2(unsigned long long a, unsigned long long b) {
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ unsigned long long fmul2(unsigned long long a, unsigned long long b) {
    unsigned long long d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// (m, S, U) of two disjoint parts
__device__ __forceinline__ void lp_merge(float &m, float &S, float &U, float m2, float S2, float U2) {
    const float mm = fmaxf(m, m2);
    if (mm == __int_as_float(0xff800000)) {  // nothing but -inf on both sides (a NaN keeps S)
        S += S2;
        U += U2;
        return;
    }
    const float d1 = fmaxf(m - mm, -1e4f), d2 = fmaxf(m2 - mm, -1e4f);
    const float f1 = ex2(d1 * kLog2e), f2 = ex2(d2 * kLog2e);
    // a side of -inf only has S = U = 0
    U = f1 * fmaf(d1, S, U) + f2 * fmaf(d2, S2, U2);
    S = f1 * S + f2 * S2;
    m = mm;
}

// The n largest of the `cnt` (> 0) keys in sh.cand, in descending order, into sh.sorted; with
// `keep` also back into sh.cand with the threshold at the n-th.  Whole CTA.
__device__ __noinline__ void lp_sort(LpShared &sh, int cnt, int n, bool keep) {
    for (int i0 = 0; i0 < cnt; i0 += kLpThreads / 8) {  // 8 lanes per key
        const int i = i0 + (threadIdx.x >> 3);
        const unsigned long long k = i < cnt ? sh.cand[i] : 0ull;
        int rank = 0;
#pragma unroll 4
        for (int j = threadIdx.x & 7; j < cnt; j += 8) rank += sh.cand[j] > k ? 1 : 0;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) rank += __shfl_xor_sync(kFull, rank, o);
        if (i < cnt && rank < n && (threadIdx.x & 7) == 0) sh.sorted[rank] = k;
    }
    cta_sync();
    if (keep) {
        if (threadIdx.x < n && threadIdx.x < cnt) sh.cand[threadIdx.x] = sh.sorted[threadIdx.x];
        if (threadIdx.x == 0) {
            sh.count = cnt < n ? cnt : n;
            if (cnt >= n) sh.thr = sh.sorted[n - 1];
        }
        cta_sync();
    }
}

// Raise the threshold to just below the n-th largest of the 64 groups' (of 4 threads) largest keys, m
// being this thread's (0: none).  Whole CTA.
__device__ __noinline__ void lp_raise(LpShared &sh, unsigned long long m, int n) {
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        const unsigned long long v = __shfl_xor_sync(kFull, m, o);
        m = v > m ? v : m;
    }
    if ((threadIdx.x & 3) == 0) sh.heads[threadIdx.x >> 2] = m;
    cta_sync();
    // rank of this group's head, 16 comparisons per lane (equal heads are all 0)
    int rank = 0;
#pragma unroll 4
    for (int j = threadIdx.x & 3; j < 64; j += 4) rank += sh.heads[j] > m ? 1 : 0;
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) rank += __shfl_xor_sync(kFull, rank, o);
    // one below the n-th head, so that the head itself passes
    if ((threadIdx.x & 3) == 0 && rank == n - 1 && m > 0ull && m - 1ull > sh.thr) sh.thr = m - 1ull;
    cta_sync();
}
// The first tile's threshold: just below every key whose logit (as an order-preserving integer) reaches
// the n-th largest of the groups' largest, m being this thread's.  Whole CTA; true where any thread brought
// `pred` (nothing is raised then).
__device__ __forceinline__ bool lp_first(LpShared &sh, uint32_t m, int n, bool pred) {
    uint32_t *heads = reinterpret_cast<uint32_t *>(sh.heads);
    m = max(m, __shfl_xor_sync(kFull, m, 1));
    m = max(m, __shfl_xor_sync(kFull, m, 2));
    const int group = threadIdx.x >> 2;
    if ((threadIdx.x & 3) == 0) heads[group] = m;
    if (cta_sync_or(pred)) return true;
    int rank = 0;  // among equal heads the lower group comes first; 16 comparisons per lane
#pragma unroll 4
    for (int j = threadIdx.x & 3; j < 64; j += 4) rank += heads[j] > m || (heads[j] == m && j < group) ? 1 : 0;
    rank += __shfl_xor_sync(kFull, rank, 1);
    rank += __shfl_xor_sync(kFull, rank, 2);
    if ((threadIdx.x & 3) == 0 && rank == n - 1) sh.thr = ((unsigned long long)m << 32) - 1ull;
    cta_sync();
    return false;
}
// After insertions by the whole CTA: cut the buffer back to its n best if it holds more than kLpKeep.
__device__ __forceinline__ void lp_settle(LpShared &sh, int n) {
    cta_sync();
    const int cnt = sh.count;
    cta_sync();  // everybody has read the count
    if (cnt > kLpKeep) lp_sort(sh, cnt, n, true);
}

__device__ __forceinline__ unsigned long long lp_key(float v, int idx) {
    return ((unsigned long long)order_key(v) << 32) | (uint32_t)~idx;
}

// one value at a shared-window address
template <typename E>
__device__ __forceinline__ float lds_value(uint32_t at) {
    if constexpr (sizeof(E) == 4) {
        float v;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at));
        return v;
    } else {
        const unsigned short b = (unsigned short)lds_u16(at);
        return to_float(*reinterpret_cast<const E *>(&b));
    }
}

// Where the 16-byte pieces of a tile lie in a row: piece j of this thread starts at value
// t0 + (256 j + tid) EV of the row; -inf outside [lo, hi).
template <typename E>
struct LpTile {
    static constexpr int EV = 16 / sizeof(E), NV = kLpEpt / EV;  // values per piece, pieces per thread
    // first tile of values from l on: pieces start at aligned addresses, up to EV - 1 values before l
    static __device__ __forceinline__ int first(const E *p, int l) {
        return l - (int)((reinterpret_cast<uintptr_t>(p + l) & 15) / sizeof(E));
    }
    static __device__ __forceinline__ uint4 edge(const E *p, int l, int h, int i0) {
        E e[EV];
#pragma unroll
        for (int k = 0; k < EV; ++k) e[k] = i0 + k >= l && i0 + k < h ? p[i0 + k] : from_float<E>(-INFINITY);
        return *reinterpret_cast<const uint4 *>(e);
    }
    static __device__ __forceinline__ void unpack(const uint4 (&q)[NV], float (&v)[kLpEpt]) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t w[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                if constexpr (sizeof(E) == 4) {
                    v[j * EV + p] = __uint_as_float(w[p]);
                } else {
                    const float2 f = unpack2(w[p], E());
                    v[j * EV + 2 * p] = f.x, v[j * EV + 2 * p + 1] = f.y;
                }
            }
        }
    }
};

// The cold parts are functions of their own, so that the tile loop keeps its registers.

// Tiles t0, t0 + kLpTile, .. t1 into the buffer, from the logits' memory, with the threshold raised tile by
// tile.  Whole CTA.
template <typename E>
__device__ __noinline__ void lp_robust(LpShared &sh, const E *x, int lo, int hi, int t0, int t1, int n) {
    using Tile = LpTile<E>;
    constexpr int EV = Tile::EV;
#pragma unroll 1
    for (int tt = t0; tt <= t1; tt += kLpTile) {
        unsigned long long best = 0ull;
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {  // this thread's largest key; then the keys above the threshold
            const unsigned long long thr = sh.thr;
#pragma unroll 1
            for (int j = 0; j < Tile::NV; ++j) {
                const int i0 = tt + (j * kLpThreads + threadIdx.x) * EV;
                const uint4 q = i0 >= lo && i0 + EV <= hi ? *reinterpret_cast<const uint4 *>(x + i0) : Tile::edge(x, lo, hi, i0);
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int k = 0; k < EV; ++k) {
                    float v;
                    if constexpr (sizeof(E) == 4) {
                        v = __uint_as_float(w[k]);
                    } else {
                        const float2 f = unpack2(w[k >> 1], E());
                        v = k & 1 ? f.y : f.x;
                    }
                    const int idx = i0 + k;
                    const unsigned long long key = lp_key(v, idx);
                    if (idx >= lo && idx < hi) {
                        if (pass == 0) best = key > best ? key : best;
                        else if (key > thr) sh.cand[atomicAdd(&sh.count, 1)] = key;
                    }
                }
            }
            __syncwarp();
            if (pass == 0) lp_raise(sh, best, n);
        }
        lp_settle(sh, n);
    }
    cta_sync();
}

// Final outputs of a row from its (m, S, U), its target's logit xt (thread t = 0; NaN for a target outside
// the vocabulary) and its n best keys in order (thread t has the t-th)
__device__ __forceinline__ void lp_finish(const LpArgs &a, int t, unsigned long long k, int row, float m, float S,
                                          float U, float xt) {
    const float ninf = -INFINITY, nan = __int_as_float(0x7fffffff);
    // a row of -inf only: no distribution; -inf for every token, entropy 0
    const bool empty = m == ninf && S == 0.f;
    const float ls = logf(S);
    if (t == 0) {
        if (a.entropy) a.entropy[row] = empty ? 0.f : ls - U / S;
        if (a.logprob) a.logprob[row] = S != S || xt != xt ? nan : empty ? ninf : (xt - m) - ls;
    }
    if (t < a.n) {
        const uint32_t hi = (uint32_t)(k >> 32);
        a.top_ids[(size_t)row * a.n + t] = (int)~(uint32_t)k;
        a.top_logprob[(size_t)row * a.n + t] = S != S || hi == 0u ? nan : empty ? ninf : (key_value(hi) - m) - ls;
    }
}

// the lanes' triples as one, in a fixed order; every lane ends with the same bits
__device__ __forceinline__ void lp_merge_lanes(float &m, float &S, float &U) {
    float M = m;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
    // a side of -inf only has S = U = 0 (or NaN, which stays)
    const float d = fmaxf(m - M, -1e4f), f = ex2(d * kLog2e);
    U = f * fmaf(d, S, U);
    S *= f;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        S += __shfl_xor_sync(kFull, S, o);
        U += __shfl_xor_sync(kFull, U, o);
    }
    m = M;
}

// The end of a piece: the CTA's triple and its n best keys; a whole row is finished, another is
// published in slot `at`.  Leaves the buffer empty.
__device__ __noinline__ void lp_piece_end(const LpArgs &a, LpShared &sh, int row, bool whole, int at, float m, float S,
                                          float U, float xt) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = a.n;
    lp_merge_lanes(m, S, U);
    if (lane == 0) sh.red[0][warp] = m, sh.red[1][warp] = S, sh.red[2][warp] = U;
    cta_sync();
    const int mine = sh.count;
    if (n > 0) lp_sort(sh, mine, n, false);
    if (warp == 0) {  // the warps' triples, lane w holding warp w's
        m = lane < kLpThreads / 32 ? sh.red[0][lane] : -INFINITY;
        S = lane < kLpThreads / 32 ? sh.red[1][lane] : 0.f;
        U = lane < kLpThreads / 32 ? sh.red[2][lane] : 0.f;
        lp_merge_lanes(m, S, U);
        if (whole) {
            lp_finish(a, lane, lane < n ? sh.sorted[lane] : 0ull, row, m, S, U, xt);
        } else {
            if (lane < n) __stcg(a.keys + (size_t)at * n + lane, lane < mine ? sh.sorted[lane] : 0ull);
            if (lane == 0) {
                __stcg(a.part + 4 * at, m);
                __stcg(a.part + 4 * at + 1, S);
                __stcg(a.part + 4 * at + 2, U);
                sh.xt[at & 1] = xt;
            }
        }
        __syncwarp();
    }
    cta_sync();
    if (tid == 0) {
        sh.count = 0;
        sh.thr = 0ull;
    }
    cta_sync();
}

// The rows of this run's first and last pieces (r0, r1; -1: none) that other CTAs hold pieces of: the last of
// a row's CTAs to arrive merges them all, slot 1 of CTA c0, where the row begins, and slot 0 of the CTAs
// after it up to c1.
__device__ __noinline__ void lp_cut_rows(const LpArgs &a, LpShared &sh, int r0, int r1) {
    const int tid = threadIdx.x, lane = tid & 31, n = a.n;
    const int k = (tid >> 5) & 1, r = k ? r1 : r0;  // warp 0 takes r0, warp 1 r1
    const long long at = (long long)(r < 0 ? 0 : r) * a.V;
    const int c0 = a.per_row ? r * a.per_row : (int)(at / a.run);
    const int c1 = a.per_row ? c0 + a.per_row - 1 : (int)((at + a.V - 1) / a.run);
    const int total = (c1 - c0 + 1) * n;
    const unsigned long long *keys = a.keys + (size_t)2 * c0 * n;
    auto key_at = [&](int j) {  // piece 0 is slot 2 c0 + 1, piece i slot 2 (c0 + i)
        return j < total ? __ldcg(keys + (j < n ? n + j : j / n * 2 * n + j % n)) : 0ull;
    };
    auto triple = [&](float &m, float &S, float &U) {
        m = -INFINITY, S = 0.f, U = 0.f;
        for (int c = c0 + lane; c <= c1; c += 32) {
            const float *p = a.part + 4 * (2 * (size_t)c + (c == c0 ? 1 : 0));
            lp_merge(m, S, U, __ldcg(p), __ldcg(p + 1), __ldcg(p + 2));
        }
        __syncwarp();
        lp_merge_lanes(m, S, U);
    };
    if (tid < 64) {
        int last = 0;
        if (r >= 0 && lane == 0) {
            // release what the CTA wrote (before its last barrier), acquire what the others did
            uint32_t old;
            asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(a.done + c0) : "memory");
            last = old == (uint32_t)(c1 - c0);
            if (last) a.done[c0] = 0u;
        }
        last = __shfl_sync(kFull, last, 0);
        __syncwarp();  // lane 0's acquire holds for the loads of every lane (a shuffle orders no memory)
        if (last && total <= 64) {  // few keys: a warp ranks them by itself
            unsigned long long *cand = sh.cand + k * 64;
            unsigned long long key[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                key[i] = n > 0 ? key_at(lane + 32 * i) : 0ull;
                cand[lane + 32 * i] = key[i];
            }
            float m, S, U;
            triple(m, S, U);
            __syncwarp();
            int rank[2] = {};
#pragma unroll 4
            for (int j = 0; j < total; ++j) {
                const unsigned long long o = cand[j];
#pragma unroll
                for (int i = 0; i < 2; ++i) rank[i] += o > key[i] ? 1 : 0;
            }
            if (lane == 0 && n == 0) lp_finish(a, 0, 0ull, r, m, S, U, sh.xt[k]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (key[i] != 0ull && rank[i] < n) lp_finish(a, rank[i], key[i], r, m, S, U, sh.xt[k]);
            last = 0;
        }
        if (lane == 0) sh.merge[k] = last;
        __syncwarp();
    }
    cta_sync();
    // many pieces: the CTA finds the best keys together
#pragma unroll 1
    for (int q = 0; q < 2; ++q) {
        if (!sh.merge[q]) continue;
        if (n > 0) {
            const int rr = q ? r1 : r0, cc = a.per_row ? rr * a.per_row : (int)((long long)rr * a.V / a.run);
            const int ce = a.per_row ? cc + a.per_row - 1 : (int)(((long long)rr * a.V + a.V - 1) / a.run);
            const unsigned long long *kk = a.keys + (size_t)2 * cc * n;
            const int tt = (ce - cc + 1) * n;
            constexpr int M = 4;
            auto at = [&](int j) { return j < tt ? __ldcg(kk + (j < n ? n + j : j / n * 2 * n + j % n)) : 0ull; };
            if (tt <= kLpThreads) {
                sh.cand[tid] = at(tid);
                if (tid == 0) sh.count = tt;
                cta_sync();
            } else {
#pragma unroll 1
                for (int base = 0; base < tt; base += M * kLpThreads) {
                    unsigned long long key[M];
#pragma unroll
                    for (int i = 0; i < M; ++i) key[i] = at(base + i * kLpThreads + tid);
                    unsigned long long best = 0ull;
#pragma unroll
                    for (int i = 0; i < M; ++i) best = key[i] > best ? key[i] : best;
                    lp_raise(sh, best, n);
#pragma unroll
                    for (int i = 0; i < M; ++i)
                        if (key[i] > sh.thr) sh.cand[atomicAdd(&sh.count, 1)] = key[i];
                    __syncwarp();
                    lp_settle(sh, n);
                }
            }
            lp_sort(sh, sh.count, n, false);
        }
        if ((tid >> 5) == q) {
            float m, S, U;
            triple(m, S, U);
            lp_finish(a, lane, lane < n ? sh.sorted[lane] : 0ull, r, m, S, U, sh.xt[k]);
        }
        cta_sync();
        if (tid == 0) {
            sh.count = 0;
            sh.thr = 0ull;
        }
        cta_sync();
    }
}

template <typename E>
__global__ void __launch_bounds__(kLpThreads, 3) logprobs_kernel(const __grid_constant__ LpArgs a) {
    using Tile = LpTile<E>;
    constexpr int EV = Tile::EV, NV = Tile::NV;
    constexpr float kNinf = -INFINITY;
    __shared__ LpShared sh;
    extern __shared__ __align__(16) uint8_t ring_s[];
    const int tid = threadIdx.x, n = a.n, V = a.V;
    int row, lo;
    long long left;  // values of the run from here on
    if (a.per_row) {
        row = blockIdx.x / a.per_row;
        lo = (blockIdx.x - row * a.per_row) * (int)a.run;
        left = lo + a.run < V ? a.run : V - lo;
    } else {
        const long long pos = a.run * blockIdx.x;
        row = (int)(pos / V);
        lo = (int)(pos - (long long)row * V);
        left = pos + a.run < a.total ? a.run : a.total - pos;
    }
    const E *x = static_cast<const E *>(a.x) + (size_t)row * V;
    int hi = lo + left < V ? (int)(lo + left) : V, r0 = -1, r1 = -1;
    if (tid == 0) {
        sh.count = 0;
        sh.thr = 0ull;
    }
    pdl_wait();
    pdl_trigger();
    // this thread's pieces of tile k of the run lie in slot k % kLpDepth; the cursor runs ahead across rows
    const uint32_t ring = smem_addr(ring_s) + tid * 16;
    constexpr uint32_t kPiece = kLpThreads * 16, kSlot = kPiece * NV;
    int t0 = Tile::first(x, lo);
    const E *px = x;
    int plo = lo, phi = hi, pt0 = t0;
    long long pleft = left;
    uint32_t pslot = ring, slot = ring;
    auto issue = [&]() {
        if (pleft > 0) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int i0 = pt0 + (j * kLpThreads + tid) * EV;
                if (i0 >= plo && i0 + EV <= phi) cp_async16(pslot + j * kPiece, px + i0, 16);
            }
            pt0 += kLpTile;
            if (pt0 >= phi) {
                pleft -= phi - plo;
                px += V;
                plo = 0;
                phi = pleft < V ? (int)pleft : V;
                pt0 = Tile::first(px, 0);
            }
        }
        pslot = pslot == ring + (kLpDepth - 1) * kSlot ? ring : pslot + kSlot;
        cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < kLpDepth; ++k) issue();
    cta_sync();
#pragma unroll 1
    for (;;) {  // the rows of the run
        float m = kNinf, xt = __int_as_float(0x7fffffff);
        if (tid == 0 && a.logprob) {  // the target's logit, while the first tile is on its way
            const int t = a.targets[row];
            if (t >= 0 && t < V) xt = to_float(x[t]);
        }
        unsigned long long S2 = 0ull, U2 = 0ull;  // packed pairs of partial sums
        int since = 0, tb = t0, before = 0;       // tiles since the last meeting, the first of them, keys before it
        const int begin = t0;
#pragma unroll 1
        for (; t0 < hi; t0 += kLpTile) {  // its tiles
            float v[kLpEpt];
            cp_async_wait_all_but<kLpDepth - 1>();
            {
                uint4 q[NV];
                if (t0 >= lo && t0 + kLpTile <= hi) {
#pragma unroll
                    for (int j = 0; j < NV; ++j) q[j] = lds128(slot + j * kPiece);
                } else {  // pieces that reach over the ends are read value by value
#pragma unroll
                    for (int j = 0; j < NV; ++j) {
                        const int i0 = t0 + (j * kLpThreads + tid) * EV;
                        if (i0 >= lo && i0 + EV <= hi) q[j] = lds128(slot + j * kPiece);
                        else q[j] = Tile::edge(x, lo, hi, i0);
                    }
                }
                Tile::unpack(q, v);
            }
            float tm = v[0];
#pragma unroll
            for (int i = 1; i < kLpEpt; ++i) tm = max_nan(tm, v[i]);
            const bool nan = tm != tm;
            if (nan) {  // the row's sums are NaN; its top values still come from the numbers
                tm = kNinf;
#pragma unroll
                for (int i = 0; i < kLpEpt; ++i) tm = fmaxf(tm, v[i]);
                S2 = U2 = 0x7fffffff7fffffffull;
            }
            if (tm > m) {
                if (m > kNinf) {
                    const float d = fmaxf(m - tm, -1e4f), f = ex2(d * kLog2e);
                    U2 = fmul2(dup2(f), ffma2(dup2(d), S2, U2));
                    S2 = fmul2(dup2(f), S2);
                }
                m = tm;
            }
            if (m > kNinf) {
                // The tile's terms are added among themselves first: one by one, those below half a step of a
                // running sum that holds a large term would all be lost.
                const unsigned long long nm = dup2(-m), l2 = dup2(kLog2e);
                unsigned long long s = 0ull, w = 0ull;
#pragma unroll
                for (int i = 0; i < kLpEpt; i += 2) {
                    const unsigned long long d = fadd2(pack2(__float_as_uint(v[i]), __float_as_uint(v[i + 1])), nm);
                    const unsigned long long t = fmul2(d, l2);
                    const unsigned long long e = pack2(__float_as_uint(ex2(__uint_as_float((uint32_t)t))),
                                                       __float_as_uint(ex2(__uint_as_float((uint32_t)(t >> 32)))));
                    s = i == 0 ? e : fadd2(s, e);
                    w = i == 0 ? fmul2(d, e) : ffma2(d, e, w);
                }
                const float u = hsum2(w);
                if (u != u) {  // a value of -inf (its 0 * -inf contributes 0), or a NaN
                    w = 0ull;
#pragma unroll
                    for (int i = 0; i < kLpEpt; i += 2) {
                        const float d0 = v[i] - m, d1 = v[i + 1] - m;
                        const float c0 = fmaxf(d0, -1e4f) * ex2(d0 * kLog2e), c1 = fmaxf(d1, -1e4f) * ex2(d1 * kLog2e);
                        w = fadd2(w, pack2(__float_as_uint(c0), __float_as_uint(c1)));
                    }
                }
                S2 = fadd2(S2, s);
                U2 = fadd2(U2, w);
            }
            bool again = false;  // the first tile, with a NaN in it
            if (n > 0 && t0 == begin) again = lp_first(sh, order_key(tm), n, nan);
            if (n > 0 && !again) {
                const unsigned long long thr = sh.thr;
                const uint32_t th = (uint32_t)(thr >> 32);
                if (nan || order_key(tm) >= th) {
                    const float tv = th ? key_value(th) : __int_as_float(0x7fffffff);
                    uint32_t pass = 0u;
#pragma unroll
                    for (int i = 0; i < kLpEpt; ++i) pass |= v[i] < tv ? 0u : 1u << i;
                    while (pass) {  // a value in thousands: read again where it lies
                        const int i = __ffs(pass) - 1, idx = t0 + ((i / EV) * kLpThreads + tid) * EV + i % EV;
                        pass &= pass - 1u;
                        if (idx < lo || idx >= hi) continue;
                        const uint32_t at_s = slot + (i / EV) * kPiece + (i % EV) * (int)sizeof(E);
                        const bool inner = idx - i % EV >= lo && idx - i % EV + EV <= hi;  // else not in the ring
                        const float w = !inner ? to_float(x[idx]) : lds_value<E>(at_s);
                        const unsigned long long k = lp_key(w, idx);
                        if (k > thr) {
                            const int at = atomicAdd(&sh.count, 1);
                            if (at < kLpCap) sh.cand[at] = k;
                        }
                    }
                }
                __syncwarp();  // rejoin the warp (see cta_sync): here, where every lane comes by
            }
            slot = slot == ring + (kLpDepth - 1) * kSlot ? ring : slot + kSlot;
            issue();  // into the slot just read
            if (n == 0) continue;
            if (++since == kLpTurn || t0 == begin || t0 + kLpTile >= hi) {
                cta_sync();
                const int cnt = sh.count;
                cta_sync();  // everybody has read the count
                if (again || cnt > kLpCap) {  // again, from the tiles' memory
                    if (tid == 0) sh.count = before;
                    cta_sync();
                    lp_robust(sh, x, lo, hi, tb, t0, n);
                } else if (cnt > kLpKeep) {
                    lp_sort(sh, cnt, n, true);
                }
                before = sh.count;
                since = 0;
                tb = t0 + kLpTile;
                cta_sync();
            }
        }
        const bool whole = lo == 0 && hi == V;
        if (!whole) {
            if (lo == 0) r1 = row;
            else r0 = row;
        }
        lp_piece_end(a, sh, row, whole, 2 * blockIdx.x + (lo == 0 ? 1 : 0), m, hsum2(S2), hsum2(U2), xt);
        left -= hi - lo;
        if (left <= 0) break;
        ++row;
        x += V;
        lo = 0;
        hi = left < V ? (int)left : V;
        t0 = Tile::first(x, 0);
    }
    if (r0 >= 0 || r1 >= 0) lp_cut_rows(a, sh, r0, r1);
}

// Few values: every row in pieces of about one tile (4096 values, what a CTA reads in one round trip),
// a CTA each.  Else equal runs over as many CTAs as the GPU holds at once (three per SM), but none
// shorter than 1/62 of a row, so that a row has at most kLpMaxPieces pieces.
void lp_runs(int T, int V, LpArgs &a, int &ctas) {
    const long long total = (long long)T * V, tiles = (V + kLpTile - 1) / kLpTile;
    const int most = kLpMaxPieces - 2, pieces = (int)(tiles < most ? tiles : most);
    if ((long long)T * pieces <= kLpMaxCtas) {
        a.run = (long long)align_up((V + pieces - 1) / pieces, 16);
        a.per_row = (int)((V + a.run - 1) / a.run);
        ctas = T * a.per_row;
        return;
    }
    a.per_row = 0;
    a.run = (total + kLpMaxCtas - 1) / kLpMaxCtas;
    if (a.run < (V + most - 1) / most) a.run = (V + most - 1) / most;
    ctas = (int)((total + a.run - 1) / a.run);
}

// Workspace: the completion counters (zero between calls, at the same place whatever the sizes),
// then the triples and the keys of two pieces per CTA.
constexpr size_t kLpDoneBytes = (kLpMaxCtas * sizeof(uint32_t) + 255) / 256 * 256;
constexpr size_t kLpPartBytes = (kLpMaxCtas * 2 * 4 * sizeof(float) + 255) / 256 * 256;

}  // namespace

extern "C" size_t rl_logprobs_workspace_bytes(int32_t T, int32_t V, int32_t top_n) {
    if (T <= 0 || V <= 0 || top_n < 0 || top_n > kLpMaxN) return 0;
    return kLpDoneBytes + kLpPartBytes + (size_t)kLpMaxCtas * 2 * top_n * sizeof(unsigned long long);
}

extern "C" rl_status rl_logprobs(const void *logits, int32_t dtype, int32_t T, int32_t V, const int32_t *targets,
                                 float *logprob, float *entropy, int32_t top_n, int32_t *top_ids, float *top_logprob,
                                 void *ws, size_t ws_bytes, void *stream) {
    if (dtype != RL_F32 && dtype != RL_F16 && dtype != RL_BF16)
        return fail(RL_ERR_INVALID, "rl_logprobs: dtype %d is none of RL_F32, RL_F16, RL_BF16", dtype);
    if (T < 0 || V <= 0 || top_n < 0) return fail(RL_ERR_INVALID, "rl_logprobs: T=%d V=%d top_n=%d", T, V, top_n);
    if (V > (1 << 30)) return fail(RL_ERR_UNSUPPORTED, "rl_logprobs: V=%d > 2^30", V);
    if (top_n > kLpMaxN) return fail(RL_ERR_UNSUPPORTED, "rl_logprobs: top_n=%d > %d", top_n, kLpMaxN);
    if (top_n > V) return fail(RL_ERR_INVALID, "rl_logprobs: top_n=%d > V=%d", top_n, V);
    if (T == 0) return RL_OK;
    if (!logits) return fail(RL_ERR_INVALID, "rl_logprobs: NULL logits");
    if ((targets == nullptr) != (logprob == nullptr))
        return fail(RL_ERR_INVALID, "rl_logprobs: targets and logprob come together");
    if ((top_n > 0) != (top_ids != nullptr) || (top_n > 0) != (top_logprob != nullptr))
        return fail(RL_ERR_INVALID, "rl_logprobs: top_ids and top_logprob come with top_n > 0");
    if (!logprob && !entropy && top_n == 0) return fail(RL_ERR_INVALID, "rl_logprobs: no output");
    const uintptr_t es = dtype_bytes(dtype);
    if (reinterpret_cast<uintptr_t>(logits) % es) return fail(RL_ERR_INVALID, "rl_logprobs: logits misaligned");
    if ((reinterpret_cast<uintptr_t>(targets) | reinterpret_cast<uintptr_t>(logprob) |
         reinterpret_cast<uintptr_t>(entropy) | reinterpret_cast<uintptr_t>(top_ids) |
         reinterpret_cast<uintptr_t>(top_logprob)) & 3)
        return fail(RL_ERR_INVALID, "rl_logprobs: targets and outputs must be 4-byte aligned");
    const size_t need = rl_logprobs_workspace_bytes(T, V, top_n);
    if (!ws || ws_bytes < need) return fail(RL_ERR_INVALID, "rl_logprobs: workspace of %zu B needed, %zu given", need, ws_bytes);
    if (reinterpret_cast<uintptr_t>(ws) & 15) return fail(RL_ERR_INVALID, "rl_logprobs: ws must be 16-byte aligned");
    uint8_t *w8 = static_cast<uint8_t *>(ws);
    LpArgs a = {};
    a.x = logits;
    a.targets = targets;
    a.logprob = logprob;
    a.entropy = entropy;
    a.top_ids = top_ids;
    a.top_logprob = top_logprob;
    a.done = reinterpret_cast<uint32_t *>(w8);
    a.part = reinterpret_cast<float *>(w8 + kLpDoneBytes);
    a.keys = reinterpret_cast<unsigned long long *>(w8 + kLpDoneBytes + kLpPartBytes);
    a.total = (long long)T * V;
    a.V = V;
    a.n = top_n;
    int ctas = 0;
    lp_runs(T, V, a, ctas);
    const dim3 grid(ctas), block(kLpThreads);
    cudaStream_t s = as_stream(stream);
    const size_t smem = (size_t)kLpDepth * kLpTile * es;
    if (dtype == RL_F32) return launch_pdl(logprobs_kernel<float>, grid, block, smem, s, "rl_logprobs", a);
    if (dtype == RL_F16) return launch_pdl(logprobs_kernel<__half>, grid, block, smem, s, "rl_logprobs", a);
    return launch_pdl(logprobs_kernel<__nv_bfloat16>, grid, block, smem, s, "rl_logprobs", a);
}
