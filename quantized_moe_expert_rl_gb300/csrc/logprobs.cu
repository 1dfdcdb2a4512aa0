// logprobs.cu - rl_logprobs: log probability of given tokens, entropy and the n most probable
// tokens of each row of logits, one pass over the logits.
//
//   lse = m + log S,  S = sum e^(x - m),  U = sum (x - m) e^(x - m),  m = max x
//   logprob = x_target - lse,  entropy = log S - U / S
//
// A row is split into segments, one CTA each; a CTA streams its segment in tiles of 4096 values
// held in registers.  Every thread keeps a running (m, S, U): when a tile raises m by d, S and U
// are rescaled by e^-d (U loses d S first).  The segments' triples meet in the row's last CTA to
// finish (a completion counter in the workspace), which merges them in segment order, so results
// do not depend on arrival order.
//
// Top n.  A candidate is a 64-bit key, order-preserving logit above ~index, so that keys are
// distinct and equal logits go to the lower index.  Only keys above a threshold are kept, in a buffer
// that is cut back to its n best whenever it holds more than 128, by counting for every key the
// larger ones.  The first tile sets the threshold: the CTA's 64 groups of 4 threads each publish
// their largest key, and the n-th largest of the 64 bounds the tile's n-th largest from below, which
// leaves at most n groups x 64 values.  Later tiles put their few survivors straight into the buffer;
// a tile that overflows it (rising logits) is taken back and goes the first tile's way.
#include "qdot.cuh"
#include "row_types.cuh"
#include "select.cuh"

using namespace rl;

namespace {

constexpr int kLpThreads = 256, kLpEpt = 16, kLpTile = kLpThreads * kLpEpt;
constexpr int kLpMaxN = 32, kLpMaxSeg = 32;
constexpr int kLpMaxRows = 4096;                    // rows of one launch (more rows: more launches)
constexpr int kLpCtas = 8 * 152;
constexpr int kLpKeep = 128;                        // the buffer is cut back beyond this many
constexpr int kLpCap = kLpKeep + 64 * kLpMaxN;      // and never holds more than this
constexpr float kLog2e = 1.4426950408889634f;

struct LpArgs {
    const void *x;
    const int32_t *targets;
    float *logprob, *entropy;
    int32_t *top_ids;
    float *top_logprob;
    float *part;               // [T][segs][4] (m, S, U)
    unsigned long long *keys;  // [T][segs][n]
    uint32_t *done;            // [T], zero between calls
    int V, n, segs, seglen;
};

struct LpShared {
    unsigned long long cand[kLpCap];
    unsigned long long sorted[kLpMaxN];
    unsigned long long heads[64];
    unsigned long long thr;
    float red[3][kLpThreads / 32];
    int count, last;
};

__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
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
__device__ __forceinline__ void lp_sort(LpShared &sh, int cnt, int n, bool keep) {
    for (int i = threadIdx.x; i < cnt; i += kLpThreads) {
        const unsigned long long k = sh.cand[i];
        int rank = 0;
        for (int j = 0; j < cnt; ++j) rank += sh.cand[j] > k ? 1 : 0;
        if (rank < n) sh.sorted[rank] = k;
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

// Put the keys (0 = none) above the threshold into the buffer.  Whole CTA; the buffer holds at
// most kLpKeep keys before the call and fewer than or as many after it.
template <int M>
__device__ __forceinline__ void lp_insert(LpShared &sh, const unsigned long long (&key)[M], int n) {
    const int lane = threadIdx.x & 31;
    const unsigned long long thr = sh.thr;
    const int before = sh.count;
    int c = 0;
#pragma unroll
    for (int i = 0; i < M; ++i) c += key[i] > thr ? 1 : 0;
    int total = c;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
    cta_sync();  // everybody has read thr and count
    if (lane == 0 && total) atomicAdd(&sh.count, total);
    cta_sync();
    const bool over = sh.count - before > kLpKeep;
    cta_sync();
    if (threadIdx.x == 0) sh.count = before;
    if (over) {  // raise the threshold to the n-th largest of the 64 groups' largest keys
        unsigned long long m = 0ull;
#pragma unroll
        for (int i = 0; i < M; ++i) m = key[i] > m ? key[i] : m;
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            const unsigned long long v = __shfl_xor_sync(kFull, m, o);
            m = v > m ? v : m;
        }
        if ((threadIdx.x & 3) == 0) sh.heads[threadIdx.x >> 2] = m;
        cta_sync();
        if (threadIdx.x < 64) {
            const unsigned long long k = sh.heads[threadIdx.x];
            int rank = 0;
            for (int j = 0; j < 64; ++j) rank += (sh.heads[j] > k || (sh.heads[j] == k && j < threadIdx.x)) ? 1 : 0;
            // one below the n-th head, so that the head itself passes
            if (rank == n - 1 && k > 0ull && k - 1ull > thr) sh.thr = k - 1ull;
        }
    }
    cta_sync();
    const unsigned long long t2 = sh.thr;
#pragma unroll
    for (int i = 0; i < M; ++i)
        if (key[i] > t2) sh.cand[atomicAdd(&sh.count, 1)] = key[i];
    cta_sync();
    const int cnt = sh.count;
    if (cnt > kLpKeep) lp_sort(sh, cnt, n, true);
}

__device__ __forceinline__ unsigned long long lp_key(float v, int idx) {
    return ((unsigned long long)order_key(v) << 32) | (uint32_t)~idx;
}

// Final outputs of a row from its (m, S, U) and the n sorted keys in sh.sorted
template <typename E>
__device__ __forceinline__ void lp_finish(const LpArgs &a, LpShared &sh, int row, float m, float S, float U) {
    const float ninf = __int_as_float(0xff800000);
    // a row of -inf only: no distribution; -inf for every token, entropy 0
    const bool empty = m == ninf && S == 0.f;
    const float ls = logf(S);
    if (threadIdx.x == 0) {
        if (a.entropy) a.entropy[row] = empty ? 0.f : ls - U / S;
        if (a.logprob) {
            const int t = a.targets[row];
            float v = __int_as_float(0x7fffffff);
            if (t >= 0 && t < a.V) {
                const float x = to_float(static_cast<const E *>(a.x)[(size_t)row * a.V + t]);
                v = empty ? ninf : (x - m) - ls;
                if (S != S) v = S;
            }
            a.logprob[row] = v;
        }
    }
    if (threadIdx.x < a.n) {
        const unsigned long long k = sh.sorted[threadIdx.x];
        const uint32_t hi = (uint32_t)(k >> 32);
        a.top_ids[(size_t)row * a.n + threadIdx.x] = (int)~(uint32_t)k;
        float v = hi == 0u ? __int_as_float(0x7fffffff) : (empty ? ninf : (key_value(hi) - m) - ls);
        if (S != S) v = S;
        a.top_logprob[(size_t)row * a.n + threadIdx.x] = v;
    }
}

template <typename E>
__global__ void __launch_bounds__(kLpThreads, 4) logprobs_kernel(const LpArgs a) {
    __shared__ LpShared sh;
    const int row = blockIdx.y, seg = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int EV = 16 / sizeof(E);       // values per 16-byte load
    constexpr int NV = kLpEpt / EV;          // loads per thread and tile
    if (tid == 0) {
        sh.count = 0;
        sh.thr = 0ull;
    }
    pdl_wait();
    pdl_trigger();
    const E *x = static_cast<const E *>(a.x) + (size_t)row * a.V;
    const int lo = seg * a.seglen, hi = min(a.V, lo + a.seglen);
    // 16-byte loads start at aligned addresses: `mis` values of the first one lie before `lo`
    const int mis = (int)((reinterpret_cast<uintptr_t>(x + lo) & 15) / sizeof(E));
    float m = __int_as_float(0xff800000), S = 0.f, U = 0.f;
    cta_sync();
    for (int t0 = lo - mis; t0 < hi; t0 += kLpTile) {
        float v[kLpEpt];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i0 = t0 + (j * kLpThreads + tid) * EV;
            if (i0 >= lo && i0 + EV <= hi) {
                const uint4 q = __ldcs(reinterpret_cast<const uint4 *>(x + i0));
                if constexpr (sizeof(E) == 4) {
                    v[j * EV] = __uint_as_float(q.x), v[j * EV + 1] = __uint_as_float(q.y);
                    v[j * EV + 2] = __uint_as_float(q.z), v[j * EV + 3] = __uint_as_float(q.w);
                } else {
                    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const float2 f = unpack2(w[p], E());
                        v[j * EV + 2 * p] = f.x, v[j * EV + 2 * p + 1] = f.y;
                    }
                }
            } else {
#pragma unroll
                for (int p = 0; p < EV; ++p) {
                    const int i = i0 + p;
                    v[j * EV + p] = i >= lo && i < hi ? to_float(x[i]) : __int_as_float(0xff800000);
                }
            }
        }
        float tm = v[0];
#pragma unroll
        for (int i = 1; i < kLpEpt; ++i) tm = max_nan(tm, v[i]);
        const bool nan = tm != tm;
        if (nan) {  // the row's sums are NaN; its top values still come from the numbers
            tm = __int_as_float(0xff800000);
#pragma unroll
            for (int i = 0; i < kLpEpt; ++i) tm = fmaxf(tm, v[i]);
            S = U = __int_as_float(0x7fffffff);
        }
        if (tm > m) {
            if (S > 0.f) {
                const float d = fmaxf(m - tm, -1e4f), f = ex2(d * kLog2e);
                U = f * fmaf(d, S, U);
                S *= f;
            }
            m = tm;
        }
        if (m > __int_as_float(0xff800000)) {
#pragma unroll
            for (int i = 0; i < kLpEpt; ++i) {
                const float d = v[i] - m, e = ex2(d * kLog2e);
                S += e;
                U = fmaf(fmaxf(d, -1e4f), e, U);  // -inf contributes 0
            }
        }
        if (a.n == 0) continue;
        auto key_at = [&](int i) {
            const int idx = t0 + ((i / EV) * kLpThreads + tid) * EV + i % EV;
            return idx >= lo && idx < hi ? lp_key(v[i], idx) : 0ull;
        };
        bool robust = t0 <= lo;  // the first tile
        if (!robust) {
            const unsigned long long thr = sh.thr;
            const int before = sh.count;
            const bool pass = nan || order_key(tm) >= (uint32_t)(thr >> 32);
            // a vote on both sides of the insertions: nobody inserts before everybody has read the count
            if (!cta_sync_or(pass)) continue;
            if (pass) {
#pragma unroll
                for (int i = 0; i < kLpEpt; ++i) {
                    const unsigned long long k = key_at(i);
                    if (k > thr) {
                        const int at = atomicAdd(&sh.count, 1);
                        if (at < kLpCap) sh.cand[at] = k;
                    }
                }
            }
            cta_sync();
            const int cnt = sh.count;
            if (cnt <= kLpKeep) continue;
            robust = cnt > kLpCap;
            cta_sync();
            if (robust) {  // take the tile's insertions back
                if (tid == 0) sh.count = before;
                cta_sync();
            } else {
                lp_sort(sh, cnt, a.n, true);
            }
        }
        if (robust) {
            unsigned long long key[kLpEpt];
#pragma unroll
            for (int i = 0; i < kLpEpt; ++i) key[i] = key_at(i);
            lp_insert(sh, key, a.n);
        }
    }
    // the CTA's triple
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(kFull, m, o), S2 = __shfl_xor_sync(kFull, S, o), U2 = __shfl_xor_sync(kFull, U, o);
        // the same order on both sides, so that every lane ends with the same bits
        float ma = lane & o ? m2 : m, Sa = lane & o ? S2 : S, Ua = lane & o ? U2 : U;
        lp_merge(ma, Sa, Ua, lane & o ? m : m2, lane & o ? S : S2, lane & o ? U : U2);
        m = ma, S = Sa, U = Ua;
    }
    if (lane == 0) sh.red[0][warp] = m, sh.red[1][warp] = S, sh.red[2][warp] = U;
    cta_sync();
    m = sh.red[0][0], S = sh.red[1][0], U = sh.red[2][0];
#pragma unroll
    for (int w = 1; w < kLpThreads / 32; ++w) lp_merge(m, S, U, sh.red[0][w], sh.red[1][w], sh.red[2][w]);
    const int mine = sh.count;
    if (a.n > 0 && mine > 0) lp_sort(sh, mine, a.n, false);
    if (a.segs == 1) {
        lp_finish<E>(a, sh, row, m, S, U);
        return;
    }
    // publish, then the last CTA of the row merges
    const size_t at = (size_t)row * a.segs + seg;
    if (tid < a.n) __stcg(a.keys + at * a.n + tid, tid < mine ? sh.sorted[tid] : 0ull);
    if (tid == 0) {
        __stcg(a.part + 4 * at, m);
        __stcg(a.part + 4 * at + 1, S);
        __stcg(a.part + 4 * at + 2, U);
    }
    __threadfence();
    cta_sync();
    if (tid == 0) sh.last = atomicAdd(a.done + row, 1u) == (uint32_t)a.segs - 1u;
    cta_sync();
    if (!sh.last) return;
    __threadfence();
    if (tid == 0) {
        a.done[row] = 0u;
        sh.count = 0;
        sh.thr = 0ull;
    }
    cta_sync();
    if (a.n > 0) {
        constexpr int M = kLpMaxSeg * kLpMaxN / kLpThreads;
        unsigned long long key[M];
#pragma unroll
        for (int i = 0; i < M; ++i) {
            const int j = i * kLpThreads + tid;
            key[i] = j < a.segs * a.n ? __ldcg(a.keys + (size_t)row * a.segs * a.n + j) : 0ull;
        }
        lp_insert(sh, key, a.n);
        lp_sort(sh, sh.count, a.n, false);
    }
    const float *p = a.part + 4 * (size_t)row * a.segs;
    m = __ldcg(p), S = __ldcg(p + 1), U = __ldcg(p + 2);
    for (int s = 1; s < a.segs; ++s) lp_merge(m, S, U, __ldcg(p + 4 * s), __ldcg(p + 4 * s + 1), __ldcg(p + 4 * s + 2));
    lp_finish<E>(a, sh, row, m, S, U);
}

// Segments per row: about eight CTAs per SM over all rows, but no segment shorter than one tile
// (4096 values), which is what a single CTA reads in one round trip.
int lp_segments(int T, int V) {
    const int want = (kLpCtas + T - 1) / T, most = (V + kLpTile - 1) / kLpTile;
    const int s = want < most ? want : most;
    return s > kLpMaxSeg ? kLpMaxSeg : s;
}

// Workspace: the completion counters (zero between calls, at the same place whatever the sizes),
// then the triples and the keys of a launch's segments.
constexpr size_t kLpDoneBytes = kLpMaxRows * sizeof(uint32_t);
size_t lp_part_bytes(int T, int V) { return align_up((size_t)T * lp_segments(T, V) * 4 * sizeof(float), 256); }

}  // namespace

extern "C" size_t rl_logprobs_workspace_bytes(int32_t T, int32_t V, int32_t top_n) {
    if (T <= 0 || V <= 0 || top_n < 0 || top_n > kLpMaxN) return 0;
    size_t most = 0;  // the last launch of many rows may hold few rows in more segments
    for (int t = T; t > 0; t -= kLpMaxRows) {
        const int rows = t < kLpMaxRows ? t : kLpMaxRows;
        const size_t b = lp_part_bytes(rows, V) + (size_t)rows * lp_segments(rows, V) * top_n * sizeof(unsigned long long);
        most = b > most ? b : most;
    }
    return kLpDoneBytes + most;
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
    for (int t0 = 0; t0 < T; t0 += kLpMaxRows) {
        LpArgs a = {};
        a.x = static_cast<const uint8_t *>(logits) + (size_t)t0 * V * es;
        a.targets = targets ? targets + t0 : nullptr;
        a.logprob = logprob ? logprob + t0 : nullptr;
        a.entropy = entropy ? entropy + t0 : nullptr;
        a.top_ids = top_ids ? top_ids + (size_t)t0 * top_n : nullptr;
        a.top_logprob = top_logprob ? top_logprob + (size_t)t0 * top_n : nullptr;
        const int rows = T - t0 < kLpMaxRows ? T - t0 : kLpMaxRows;
        a.done = reinterpret_cast<uint32_t *>(w8);
        a.part = reinterpret_cast<float *>(w8 + kLpDoneBytes);
        a.keys = reinterpret_cast<unsigned long long *>(w8 + kLpDoneBytes + lp_part_bytes(rows, V));
        a.V = V;
        a.n = top_n;
        a.segs = lp_segments(rows, V);
        a.seglen = (int)align_up((V + a.segs - 1) / a.segs, 16);
        a.segs = (V + a.seglen - 1) / a.seglen;
        const dim3 grid(a.segs, rows), block(kLpThreads);
        cudaStream_t s = as_stream(stream);
        const rl_status st = dtype == RL_F32   ? launch_pdl(logprobs_kernel<float>, grid, block, 0, s, "rl_logprobs", a)
                             : dtype == RL_F16 ? launch_pdl(logprobs_kernel<__half>, grid, block, 0, s, "rl_logprobs", a)
                                               : launch_pdl(logprobs_kernel<__nv_bfloat16>, grid, block, 0, s, "rl_logprobs", a);
        if (st != RL_OK) return st;
    }
    return RL_OK;
}
