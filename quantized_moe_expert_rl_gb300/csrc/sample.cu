// sample.cu - rl_sample: the next token of each row of logits, by temperature, top-k, top-p and min-p, from
// given random numbers.
//
// Order: logits descending, equal ones by index.  A token's place in it is the 64-bit key (order-preserving
// logit above ~index), so that a border is one key and a token is kept when its key is not below.
//
//   w(l) = 2^((l - max) log2(e) / temperature), as an integer multiple of 2^-s (s = 46 for up to 2^17 tokens)
//   top-k border: the k-th key;  top-p border: the first key at which the sum of w reaches p times that of
//   all (of the k);  min-p border: the smallest logit whose w is min_p of the largest;  the highest of them counts
//   the token: the first one in index order at which the sum of the kept w passes u times their total
//
// Why integers: whether a token next to a border is in, and which one u meets, must depend neither on the order
// of summation nor on the rounding of 32-bit sums (over 512 rows of 131072 flat logits 32-bit sums pick another
// token about once).  w is good to 2^-30 of itself: the exponent is a pair of f32, its fraction's first five bits go
// through a table of 2^(j / 32) (one entry per bank, so lookups never conflict), the rest through the series of e^x.
//
// Fewer rows than SMs: a row is held by a cluster of up to 8 CTAs in shared memory and read from HBM once; rows that do not fit
// are streamed by the cluster in every pass.  From as many rows as SMs on, two CTAs (one for rows below 128 KB) stream a row in
// every pass, all but the first from L2 (512 rows of 131072: 294 us held, 192 streamed, since a cluster's barriers leave its SMs
// idle); rows of up to 32 KB are held there too.  Passes: the
// maximum; then, where nothing is filtered, the sums of w per warp (a warp holds neighbouring tokens), and the warp that
// holds the token goes through its share once more.  With top-k or top-p:
//   1. The candidates above a bound go into a list: for top-k the k-th largest of the warps' largest logits (for larger k the
//      smallest of the warps' j-th largest lane maxima, j = k / warps), so that the k-th token is in it; for top-p alone the
//      bound at three quarters of the warps, which a peaked row's share p lies above.  One CTA sorts up to 2048 of them (by
//      counting the larger ones up to 128, else bitonic) and finds the border on their running sum; all kept tokens are in
//      the list, whose w give the warps' sums.
//   2. Where that does not hold the border (flat rows, large k): counts of the tokens in 2048 bins of the logit, of those above
//      (1 - p) M' / V (all below together have less than 1 - p of the sum; M' is the sum of w of the warps' maxima).  For
//      top-k the counts name the bin; for top-p an estimate from the bins' middles names a few bins, whose tokens are sorted
//      while those above are summed up exactly, which also tells whether the estimate was right.
//   3. Else (top-k and top-p with more than 2048 candidates; thousands of equal logits at the border; an estimate that missed): the
//      range of keys is narrowed by histograms of counts and of 64-bit sums until 2048 keys are left or a single logit, whose
//      tokens have equal w and are counted off by index.
//
// Measured back to back in a graph: 1 x 131072 f32 9.7 us greedy, 12 unfiltered, 21 with k = 50 and p = 0.9; with p = 0.95 30 for
// a peaked row and 50 for normally distributed logits; k = 5000 and p = 0.9 77 and 92; 76 to 190 where all logits are equal; 512 x
// 131072 f32 182 unfiltered (the copy rate allows 40; the row's maximum parts the pass that loads from the one that weighs, so
// neither HBM, 25%, nor the issue slots, 41%, are full), 428 with p = 0.95 and a quarter of the rows nearly flat (L2 passes, and one
// CTA sorting while the others wait).  A batch takes as long as its slowest row.
#include <math.h>

#include "qdot.cuh"
#include "row_types.cuh"
#include "select.cuh"

using namespace rl;

namespace {

typedef unsigned long long u64;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxC = 8;                  // CTAs of a cluster
constexpr int kCap = 2048;                // candidates that are sorted
constexpr int kBins = 2048;               // of border_by_ranges()
constexpr int kCounts = 2048;             // of border_by_counts()
constexpr int kFixedBytes = 2 * kCap * 8 + kCounts * 4;  // shared memory beside the row
constexpr int kMaxV = 1 << 26;

struct Pow2Table {
    int32_t v[32];  // 2^(j / 32 + 30)
};
constexpr Pow2Table make_table() {
    double r = 2.0;  // 2^(1 / 32): five square roots of 2, by Newton's iteration
    for (int i = 0; i < 5; ++i) {
        double s = 1.0;
        for (int k = 0; k < 60; ++k) s = 0.5 * (s + r / s);
        r = s;
    }
    Pow2Table t = {};
    double p = 1073741824.0;
    for (int j = 0; j < 32; ++j) {
        t.v[j] = (int32_t)(p + 0.5);
        p *= r;
    }
    return t;
}
__device__ constexpr Pow2Table kPow2 = make_table();

struct SampleArgs {
    const void *x;
    const float *u, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int32_t *ids;
    float *logprob;
    int V, C, per, iters, shift;  // pieces of 16 bytes per CTA and per thread; w = multiples of 2^-shift
};

// log2(e) / temperature as (hi + lo * pre) * s (pre: 1, or 2^-24 where lo by itself would leave f32's normal range).  s: 1, or 1 / 2
// at temperatures that see no differences but those of logits near the largest f32, whose difference as such may be twice that:
// there logits are halved before they are subtracted.
struct Factor {
    float hi, lo, pre, s;
};

struct Shared {
    u64 mass[kMaxC];         // by CTA of the cluster
    u64 wmass[kWarps], wabove[kWarps];
    u64 border;              // kept: key >= border
    u64 above_mass, target;
    float wtop[kMaxC * kWarps], wjth[kMaxC * kWarps];  // by warp of the cluster
    uint32_t count[kMaxC];
    uint32_t wcount[kWarps];
    uint32_t klo, khi;       // the range of keys (upper halves) that holds the border
    uint32_t above, inside;  // tokens above the range, in it
    int mine, found;
    Factor fac;
    float bound;
    int32_t table[32];
    int k;
    float p, u, min_p;
};

__device__ __forceinline__ void cluster_sync_all(int C) {
    if (C == 1) {
        cta_sync();
        return;
    }
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    __syncwarp();
}
__device__ __forceinline__ uint32_t peer(uint32_t a, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}
__device__ __forceinline__ void put32(void *p, int rank, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer(smem_addr(p), rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void put64(void *p, int rank, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(peer(smem_addr(p), rank)), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t get32(const void *p, int rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(peer(smem_addr(p), rank)) : "memory");
    return v;
}
__device__ __forceinline__ u64 get64(const void *p, int rank) {
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(peer(smem_addr(p), rank)) : "memory");
    return v;
}
__device__ __forceinline__ u64 warp_sum64(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}
__device__ __forceinline__ u64 warp_scan64(u64 v) {  // inclusive
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 w = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += w;
    }
    return v;
}
__device__ __forceinline__ u64 make_key(uint32_t k, int idx) { return ((u64)k << 32) | (uint32_t)~idx; }

// log2(w) of a logit as a pair, for l <= m
__device__ __forceinline__ void exponent(float l, float m, Factor c, float &t, float &t_lo) {
    l *= c.s, m *= c.s;
    const float d = l - m, b = d + m, e = (l - b) + ((b - d) - m);  // d + e = l - m exactly (two-sum)
    t = d * c.hi;
    t_lo = fmaf(e, c.hi, fmaf(d * c.pre, c.lo, fmaf(d, c.hi, -t)));
}

// ceil(p * total) and floor(p * total) for 0 <= p < 1, exactly: p is an integer over a power of two
__device__ __forceinline__ u64 share(float p, u64 total, bool up) {
    const uint32_t bits = __float_as_uint(p), ex = bits >> 23;
    const u64 mant = ex ? (bits & 0x7fffffu) | 0x800000u : bits;
    const int sh = ex ? 150 - (int)ex : 149;  // p = mant / 2^sh, sh >= 24
    const u64 lo = mant * total, hi = __umul64hi(mant, total);
    u64 q, rest;
    if (sh < 64) {
        q = (hi << (64 - sh)) | (lo >> sh);
        rest = lo & ((1ull << sh) - 1ull);
    } else {
        const int s2 = sh - 64;
        q = s2 < 64 ? hi >> s2 : 0ull;
        rest = lo | (s2 < 64 ? hi & ((1ull << s2) - 1ull) : hi);
    }
    return q + (up && rest ? 1ull : 0ull);
}

// The steps of w(l) for two logits (packed f32 pairs); one logit is the same with both halves alike.  Valid for
// t = (l - m) log2(e) / temperature in [-shift, 0]; anything else gives any value (the callers leave out what is below `least`).
//   d + e = s l - s m exactly (two-sum, -b in place of b);  k / 32 = t rounded (the magic sum leaves k in the low bits);  r = t - k / 32
//   P = 2^32 (e^(r ln 2) - 1), |r| <= 1 / 64: the fifth term of the series is below 2^-39
//   w = 2^(k / 32 + shift) (1 + P / 2^32), truncated and made odd, which is off by at most a unit to either side and not
//   on the average (131072 truncations would sum up to 2^-30 of the largest w)
struct Weigh {
    u64 s, nm, hi, lo, pre;
    int sh;
    uint32_t table;
    static constexpr float kMagic = 393216.f;  // 1.5 * 2^18: sums with it are rounded to multiples of 1 / 32
    static __device__ __forceinline__ u64 both(float v) { return pack2(__float_as_uint(v), __float_as_uint(v)); }
    static __device__ __forceinline__ u64 add2(u64 a, u64 b) {
        u64 d;
        asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
        return d;
    }
    static __device__ __forceinline__ u64 mul2(u64 a, u64 b) {
        u64 d;
        asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
        return d;
    }
    __device__ __forceinline__ void set(float max, Factor c, int shift, const int32_t *tab) {
        s = both(c.s), nm = both(-max * c.s), hi = both(c.hi), lo = both(c.lo), pre = both(c.pre);
        sh = 62 - shift + (__float_as_int(kMagic) >> 5);
        table = smem_addr(tab);
    }
    __device__ __forceinline__ u64 finish(uint32_t kf, uint32_t p) const {
        const int P = __float2int_rn(__uint_as_float(p));
        int32_t T;
        asm volatile("ld.shared.s32 %0, [%1];" : "=r"(T) : "r"(table + ((kf & 31u) << 2)));
        const u64 e = (u64)((long long)T * P + ((long long)T << 32));  // 2^62 ... 2^63
        return (e >> ((sh - (int)(kf >> 5)) & 63)) | 1ull;
    }
    __device__ __forceinline__ void pair(float l0, float l1, u64 &w0, u64 &w1) const {
        const u64 l = pack2(__float_as_uint(l0), __float_as_uint(l1)), neg = both(-1.f), magic = both(kMagic);
        const u64 d = ffma2(l, s, nm), nb = ffma2(d, neg, nm), e = add2(ffma2(l, s, nb), ffma2(add2(nb, d), neg, nm));
        const u64 kf = ffma2(d, hi, magic);
        u64 r = ffma2(d, hi, ffma2(kf, neg, magic));
        r = ffma2(mul2(d, pre), lo, ffma2(e, hi, r));
        u64 q = ffma2(r, both(9.618129e-3f * 4294967296.f), both(5.550411e-2f * 4294967296.f));
        q = ffma2(q, r, both(0.24022651f * 4294967296.f));
        q = mul2(ffma2(q, r, both(0.69314718f * 4294967296.f)), r);
        w0 = finish((uint32_t)kf, (uint32_t)q);
        w1 = finish((uint32_t)(kf >> 32), (uint32_t)(q >> 32));
    }
    __device__ __forceinline__ u64 one(float l) const {
        u64 a, b;
        pair(l, l, a, b);
        return a;
    }
};

// The row's pieces of 16 bytes.  Piece i of the row starts at value i EV - skew, so that it lies on a 16-byte
// boundary; values outside the row are -infinity.  Warp w of CTA c takes the pieces from (16 c + w) 32 iters on.
template <typename E, bool HELD>
struct Row {
    static constexpr int EV = 16 / sizeof(E);
    const E *x;
    int V, skew, first;      // first: value index of this lane's piece 0
    uint32_t held;           // shared memory of this lane's piece 0
    __device__ __forceinline__ int at(int it) const { return first + it * 32 * EV; }
    __device__ __forceinline__ bool inner(int i0) const { return i0 >= 0 && i0 <= V - EV; }
    static __device__ __noinline__ uint4 edge_of(const E *x, int V, int i0) {
        alignas(16) E e[EV];
#pragma unroll
        for (int k = 0; k < EV; ++k) e[k] = i0 + k >= 0 && i0 + k < V ? x[i0 + k] : from_float<E>(-INFINITY);
        return *reinterpret_cast<const uint4 *>(e);
    }
    __device__ __forceinline__ uint4 edge(int i0) const { return edge_of(x, V, i0); }
    __device__ __forceinline__ void load(int iters) const {  // HELD: into shared memory
        for (int it = 0; it < iters; ++it) {
            const int i0 = at(it);
            const uint32_t dst = held + it * 512;
            if (inner(i0)) {
                cp_async16(dst, x + i0, 16);
            } else {
                const uint4 q = edge(i0);
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(q.x), "r"(q.y), "r"(q.z), "r"(q.w) : "memory");
            }
        }
        cp_async_commit();
        __syncwarp();
    }
    __device__ __forceinline__ uint4 raw(int it) const {
        if constexpr (HELD) return lds128(held + it * 512);
        else return inner(at(it)) ? __ldg(reinterpret_cast<const uint4 *>(x + at(it))) : edge(at(it));
    }
    static __device__ __forceinline__ void unpack(const uint4 &q, float (&v)[EV]) {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            if constexpr (sizeof(E) == 4) {
                v[p] = __uint_as_float(w[p]);
            } else {
                const float2 f = unpack2(w[p], E());
                v[2 * p] = f.x, v[2 * p + 1] = f.y;
            }
        }
    }
    __device__ __forceinline__ void get(int it, float (&v)[EV]) const { unpack(raw(it), v); }
    // f(it, values) for this lane's pieces; from memory with four loads in flight
    template <typename F>
    __device__ __forceinline__ void each(int iters, F f) const {
        constexpr int B = HELD ? 1 : 4;
#pragma unroll 1
        for (int i0 = 0; i0 < iters; i0 += B) {
            uint4 q[B];
#pragma unroll
            for (int b = 0; b < B; ++b) q[b] = raw(i0 + b);  // (past the last: beyond the row or a neighbour's, not used)
#pragma unroll
            for (int b = 0; b < B; ++b) {
                if (i0 + b < iters) {
                    float v[EV];
                    unpack(q[b], v);
                    f(i0 + b, v);
                }
            }
        }
    }
};

// ---- the sort of the candidates ----------------------------------------------------------------
// EPT * kThreads keys in buf, descending.  Element e kThreads + tid is in this thread's register e: exchanges
// at a distance of kThreads and more stay in the thread, below 32 in the warp, the others go through buf.
template <int EPT>
__device__ __noinline__ void sort_keys(u64 *buf) {
    const int tid = threadIdx.x;
    u64 v[EPT];
#pragma unroll
    for (int e = 0; e < EPT; ++e) v[e] = buf[e * kThreads + tid];
    cta_sync();
#pragma unroll 1
    for (int k = 2; k <= EPT * kThreads; k <<= 1) {
#pragma unroll 1
        for (int j = k >> 1; j > 0; j >>= 1) {
            if (j >= kThreads) {
#pragma unroll
                for (int e = 0; e < EPT; ++e) {
                    const int o = e ^ (j / kThreads);
                    if (o > e && o < EPT) {
                        const bool desc = ((e * kThreads + tid) & k) == 0;
                        const u64 a = v[e], b = v[o];
                        if ((a < b) == desc) v[e] = b, v[o] = a;
                    }
                }
                continue;
            }
            u64 w[EPT];
            if (j < 32) {
#pragma unroll
                for (int e = 0; e < EPT; ++e) w[e] = __shfl_xor_sync(kFull, v[e], j);
            } else {
#pragma unroll
                for (int e = 0; e < EPT; ++e) buf[e * kThreads + tid] = v[e];
                cta_sync();
#pragma unroll
                for (int e = 0; e < EPT; ++e) w[e] = buf[e * kThreads + (tid ^ j)];
                cta_sync();
            }
#pragma unroll
            for (int e = 0; e < EPT; ++e) {
                const int i = e * kThreads + tid;
                const bool larger = ((i & k) == 0) == ((i & j) == 0);  // this place takes the larger one
                v[e] = (v[e] > w[e]) == larger ? v[e] : w[e];
            }
        }
    }
#pragma unroll
    for (int e = 0; e < EPT; ++e) buf[e * kThreads + tid] = v[e];
    cta_sync();
}

template <typename E, bool HELD>
struct Sampler {
    using R = Row<E, HELD>;
    static constexpr int EV = R::EV;
    const SampleArgs &a;
    Shared &sh;
    u64 *list, *sorted;                  // kCap keys each; together the histograms of border_by_ranges()
    uint32_t *counts;                    // kCounts
    R row;
    int rank, lane, warp;
    float m, least;                      // least: the smallest logit that has a weight
    Factor fac;
    Weigh weigh;
    float bin_scale;                     // bins per unit of the logit

    // bins of equal width in the logit, 0 at the maximum; monotone
    __device__ __forceinline__ int bin(float l) const { return min((int)((m - l) * bin_scale), kCounts - 1); }
    // the sum that the tokens kept by top-p reach: a share p < 1 of `total`, at least the first token's
    __device__ __forceinline__ u64 share_of(u64 total) const {
        const u64 t = share(sh.p, total, true);
        return t > 0ull ? t : 1ull;
    }
    __device__ __forceinline__ u64 w_of(float l) const { return weigh.one(l); }
    // the sum of w over the values j of a piece with in[j]
    static __device__ __forceinline__ u64 sum_in(const Weigh &weigh, const float (&v)[EV], const bool (&in)[EV]) {
        u64 sum = 0ull;
#pragma unroll
        for (int j = 0; j < EV; j += 2) {
            u64 w0, w1;
            weigh.pair(v[j], v[j + 1], w0, w1);
            if (in[j]) sum += w0;
            if (in[j + 1]) sum += w1;
        }
        return sum;
    }
    static __device__ __forceinline__ bool at_least(const float (&v)[EV], float lo, bool (&in)[EV]) {
        bool any = false;
#pragma unroll
        for (int j = 0; j < EV; ++j) {
            in[j] = v[j] >= lo;
            any = any || in[j];
        }
        return any;
    }
    // in[j]: value j of the piece at `i0` is kept: its logit is not below `lo`, the border's; where the border divides
    // equal logits (its lower half is not 0), its key is not below.  True if any is.
    static __device__ __forceinline__ bool kept(const float (&v)[EV], int i0, float lo, u64 border, bool (&in)[EV]) {
        bool any = at_least(v, lo, in);
        if ((uint32_t)border != 0u && any) {
            any = false;
#pragma unroll
            for (int j = 0; j < EV; ++j) {
                in[j] = in[j] && (v[j] > lo || make_key(order_key(lo), i0 + j) >= border);
                any = any || in[j];
            }
        }
        __syncwarp();
        return any;
    }

    // Tokens whose logit's key lies in [klo, khi] and that are not below `floor` into this CTA's list; sh.count
    // has their numbers after the next cluster barrier (anything beyond kCap where they are more).  With ALL also
    // the sums of all w (sh.mass), with ABOVE the sums of the w of the tokens above khi (sh.mass, and sh.wabove by warp).
    template <bool ALL, bool ABOVE = false>
    __device__ __noinline__ void collect(uint32_t klo, uint32_t khi, u64 floor) {
        // (the members in registers: they lie in local memory, where every use in a loop would load them again)
        const Weigh weigh = this->weigh;
        const R row = this->row;
        const int iters = a.iters;
        const float least = this->least;
        u64 *const list = this->list;
        if (threadIdx.x == 0) sh.mine = 0;
        cta_sync();
        const float lo = key_value(klo), hi = key_value(khi);
        u64 sum = 0ull;
        row.each(iters, [&](int it, const float (&v)[EV]) {
            if (ALL) {
                bool all[EV];
                if (__any_sync(kFull, at_least(v, least, all))) sum += sum_in(weigh, v, all);
            }
            if (ABOVE) {
                bool over[EV], any = false;
#pragma unroll
                for (int j = 0; j < EV; ++j) {
                    over[j] = v[j] > hi;
                    any = any || over[j];
                }
                if (__any_sync(kFull, any)) sum += sum_in(weigh, v, over);
            }
            uint32_t in = 0u;
#pragma unroll
            for (int j = 0; j < EV; ++j) in |= v[j] >= lo && v[j] <= hi ? 1u << j : 0u;
            if (!__any_sync(kFull, in != 0u)) return;
            // beyond kCap the number does not matter: the list is not used
            if (in && *reinterpret_cast<volatile int *>(&sh.mine) <= kCap) {
#pragma unroll 1
                while (in) {
                    const int j = __ffs(in) - 1;
                    in &= in - 1u;
                    float l = v[0];
#pragma unroll
                    for (int i = 1; i < EV; ++i) l = i == j ? v[i] : l;
                    const uint32_t k = order_key(l);
                    const u64 key = make_key(k, row.at(it) + j);
                    if (k > khi || key < floor) continue;
                    const int at = atomicAdd(&sh.mine, 1);
                    if (at < kCap) list[at] = key;
                }
            }
            __syncwarp();
        });
        if (ALL || ABOVE) {
            sum = warp_sum64(sum);
            if (lane == 0) (ABOVE ? sh.wabove : sh.wmass)[warp] = sum;
        }
        cta_sync();
        if (warp == 0) {
            u64 t = (ALL || ABOVE) && lane < kWarps ? (ABOVE ? sh.wabove : sh.wmass)[lane] : 0ull;
            if (ALL || ABOVE) t = warp_sum64(t);
            if (lane < a.C) {
                put32(&sh.count[rank], lane, (uint32_t)sh.mine);
                if (ALL || ABOVE) put64(&sh.mass[rank], lane, t);
            }
            __syncwarp();
        }
    }

    // Sorts the candidates of all lists (n <= kCap, all that they hold: every caller counts the keys that collect() takes) and
    // finds the border: the k-th token of the order (k > 0) and the first at which the sum reaches p times `total` (of the k
    // tokens' sum with k > 0), counted from `above` tokens and a sum of `above_mass` that lie before the candidates.
    // Leader CTA; the border goes to all CTAs.  whole: nothing that has a weight lies behind the candidates; else a sum that
    // does not get there leaves sh.found 0.
    __device__ __noinline__ void border_of_list(int n, uint32_t above, u64 above_mass, int k, bool by_p, u64 total, bool total_of_k, bool whole) {
        const int tid = threadIdx.x;
        for (int i = tid; i < n; i += kThreads) {
            int c = 0, at = i;
            while (at >= (int)sh.count[c]) at -= (int)sh.count[c++];
            sorted[i] = get64(&list[at], c);
        }
        constexpr int kMost = kCap / kThreads;
        const int ept = n <= kThreads ? 1 : n <= 2 * kThreads ? 2 : kMost;
        for (int i = n + tid; i < ept * kThreads; i += kThreads) sorted[i] = 0ull;
        cta_sync();
        if (n <= 128) {  // by counting the larger ones, several lanes per key
            constexpr int L = kThreads / 128;
            const int i = tid / L;
            const u64 mine = sorted[i];
            int rank = 0;
#pragma unroll 4
            for (int j = tid % L; j < n; j += L) rank += sorted[j] > mine ? 1 : 0;
#pragma unroll
            for (int o = 1; o < L; o <<= 1) rank += __shfl_xor_sync(kFull, rank, o);
            cta_sync();
            if (i < n && tid % L == 0) sorted[rank] = mine;
            cta_sync();
        } else if (ept == 1) sort_keys<1>(sorted);
        else if (ept == 2) sort_keys<2>(sorted);
        else sort_keys<kMost>(sorted);
        // running sums: thread t has the places ept t .. ept t + ept - 1
        u64 key[kMost], w[kMost], sum = 0ull;
        for (int e = 0; e < kMost; ++e) {
            const int i = ept * tid + e;
            key[e] = e < ept && i < n ? sorted[i] : 0ull;
            w[e] = key[e] ? w_of(key_value((uint32_t)(key[e] >> 32))) : 0ull;
            sum += w[e];
        }
        const u64 incl = warp_scan64(sum);
        if (lane == 31) sh.wmass[warp] = incl;
        cta_sync();
        u64 before = above_mass + incl - sum;
        for (int i = 0; i < warp; ++i) before += sh.wmass[i];
        const long long kpos = k > 0 ? (long long)k - above : (long long)n;  // places kept by top-k, 1 at least
        const int last = (int)(kpos < n ? kpos : n) - 1;
        if (total_of_k) {  // the sum of the first k
            u64 b = before;
            for (int e = 0; e < ept; ++e) {
                b += w[e];
                if (ept * tid + e == last) sh.target = b;
            }
            cta_sync();
            total = sh.target;
            cta_sync();
        }
        if (tid == 0) {
            sh.target = by_p ? share_of(total) : ~0ull;
            sh.border = 0ull;
            sh.found = 0;
        }
        cta_sync();
        const u64 target = sh.target;
        for (int e = 0; e < ept; ++e) {
            const int i = ept * tid + e;
            // the last place of the run: the sum before it is below the target, with it not, or top-k ends
            if (i <= last && before < target && ((i == last && (whole || !by_p)) || before + w[e] >= target)) {
                sh.border = key[e];
                sh.found = 1;
            }
            before += w[e];
        }
        cta_sync();
        if (tid < a.C) {
            put64(&sh.border, tid, sh.border);
            put32(&sh.found, tid, (uint32_t)sh.found);
        }
        __syncwarp();
    }

    // the CTA's sum, of the warps', to all CTAs
    __device__ __forceinline__ void publish_sums() {
        cta_sync();
        if (warp == 0) {
            const u64 t = warp_sum64(lane < kWarps ? sh.wmass[lane] : 0ull);
            if (lane < a.C) put64(&sh.mass[rank], lane, t);
            __syncwarp();
        }
        cluster_sync_all(a.C);
    }

    // The border from the counts of the tokens of [sh.bound, m] by bin(): k > 0: the bin of the k-th token;
    // else a run of bins around the place where the sum, estimated from the counts and the bins' middles, reaches
    // p times `total`.  The tokens above it are summed up exactly, those in it sorted.  False (nothing decided): the
    // run is too large or, by the exact sums, does not hold the border.  Whole cluster.
    __device__ __noinline__ bool border_by_counts(int k, u64 total) {
        const int tid = threadIdx.x;
        uint32_t *const cnt = counts;
        {
            const R row = this->row;
            const float low = sh.bound, m = this->m, bin_scale = this->bin_scale;
            for (int i = tid; i < kCounts; i += kThreads) cnt[i] = 0u;
            cta_sync();
            row.each(a.iters, [&](int, const float (&v)[EV]) {
                bool some[EV];
                if (!__any_sync(kFull, at_least(v, low, some))) return;
#pragma unroll
                for (int j = 0; j < EV; ++j)
                    if (some[j]) atomicAdd(&cnt[min((int)((m - v[j]) * bin_scale), kCounts - 1)], 1u);
                __syncwarp();
            });
            cluster_sync_all(a.C);
        }
        const bool by_k = k > 0;
        constexpr int Q = kCounts / kThreads;
        const int part = kCounts / a.C;
        uint32_t c4[Q];
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            c4[i] = 0u;
            if (tid + i * kThreads < part)
                for (int c = 0; c < a.C; ++c) c4[i] += get32(&cnt[rank * part + tid + i * kThreads], c);
        }
        __syncwarp();
        cluster_sync_all(a.C);
#pragma unroll
        for (int i = 0; i < Q; ++i)
            if (tid + i * kThreads < part) put32(&cnt[rank * part + tid + i * kThreads], 0, c4[i]);
        __syncwarp();
        cluster_sync_all(a.C);
        if (rank == 0) {
            // thread t has the bins Q t .. Q t + Q - 1
            const float octaves = fac.hi * fac.s / bin_scale, one = (float)(1ull << a.shift);
            uint32_t n[Q], csum = 0u;
            float e[Q], esum = 0.f;
            for (int i = 0; i < Q; ++i) {
                n[i] = cnt[Q * tid + i];
                e[i] = (float)n[i] * exp2f(-octaves * ((float)(Q * tid + i) + 0.5f));
                csum += n[i];
                esum += e[i];
            }
            uint32_t cincl = csum;
            float eincl = esum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t c = __shfl_up_sync(kFull, cincl, o);
                const float f = __shfl_up_sync(kFull, eincl, o);
                if (lane >= o) cincl += c, eincl += f;
            }
            if (lane == 31) sh.wcount[warp] = cincl, sh.wtop[warp] = eincl;
            if (tid == 0) sh.found = 0;
            cta_sync();
            uint32_t c0 = cincl - csum;
            float e0 = eincl - esum;
            for (int i = 0; i < warp; ++i) c0 += sh.wcount[i], e0 += sh.wtop[i];
            const float want = sh.p * ((float)total / one);
            for (int i = 0; i < Q; ++i) {
                const bool here = by_k ? c0 < (uint32_t)k && c0 + n[i] >= (uint32_t)k : e0 < want && e0 + e[i] >= want && n[i] > 0u;
                if (here) {
                    sh.found = 1;
                    sh.klo = sh.khi = Q * tid + i;  // bins, for now
                    sh.above = c0;
                    sh.inside = n[i];
                }
                c0 += n[i];
                e0 += e[i];
            }
            cta_sync();
            if (sh.found) {
                if (!by_k && tid == 0) {  // a bin or more to both sides
                    int b0 = (int)sh.klo, b1 = b0;
                    uint32_t in = sh.inside;
                    for (int i = 0; i < 8 && in <= 64; ++i) {
                        if (b0 > 0) --b0, in += cnt[b0], sh.above -= cnt[b0];
                        if (b1 < kCounts - 1) ++b1, in += cnt[b1];
                    }
                    if (b0 > 0 && b0 == (int)sh.klo && in + cnt[b0 - 1] <= kCap) --b0, in += cnt[b0], sh.above -= cnt[b0];
                    if (b1 < kCounts - 1 && b1 == (int)sh.klo && in + cnt[b1 + 1] <= kCap) ++b1, in += cnt[b1];
                    sh.klo = b1, sh.khi = b0, sh.inside = in;  // higher bins hold smaller logits
                }
                cta_sync();
                const uint32_t b = warp == 0 ? sh.klo : sh.khi, bottom = order_key(sh.bound), top = order_key(m);
                cta_sync();
                if (warp < 2) {
                    // warp 0: the smallest key whose bin is not beyond klo's; warp 1: the smallest whose bin is before khi's,
                    // less one.  32 places of the range at a time.
                    uint32_t x0 = bottom, x1 = warp == 0 ? top : top + 1u;
                    const int limit = (int)__shfl_sync(kFull, b, 0) - warp;  // the first key with a bin of at most this
                    while (x0 < x1) {
                        const uint32_t x = x0 + (uint32_t)((u64)(x1 - x0) * (uint32_t)lane >> 5);
                        const unsigned in = __ballot_sync(kFull, bin(key_value(x)) <= limit);
                        const int at = in ? __ffs(in) - 1 : 32;
                        const uint32_t below = __shfl_sync(kFull, x, at > 0 ? at - 1 : 0), above = __shfl_sync(kFull, x, at & 31);
                        if (at < 32) x1 = above;
                        if (at > 0) x0 = below + 1u;
                    }
                    if (lane == 0) {
                        if (warp == 0) sh.klo = x0;
                        else sh.khi = x0 - 1u;
                    }
                }
                __syncwarp();
                cta_sync();
            }
            if (tid < a.C && tid > 0) {
                put32(&sh.found, tid, (uint32_t)sh.found);
                put32(&sh.klo, tid, sh.klo);
                put32(&sh.khi, tid, sh.khi);
                put32(&sh.inside, tid, sh.inside);
            }
            __syncwarp();
        }
        cluster_sync_all(a.C);
        if (!sh.found) {
            if (!by_k) return false;
            if (tid == 0) sh.border = 0ull;  // fewer tokens than k have a weight
            cta_sync();
            return true;
        }
        const uint32_t klo = sh.klo, khi = sh.khi, inside = sh.inside;
        if (inside > (uint32_t)kCap) return false;
        // the sums above the run, and its tokens
        if (by_k) collect<false>(klo, khi, 0ull);
        else collect<false, true>(klo, khi, 0ull);
        cluster_sync_all(a.C);
        if (rank == 0) {
            u64 above_mass = 0ull;
            for (int c = 0; c < a.C; ++c) above_mass += sh.mass[c];
            border_of_list((int)inside, sh.above, above_mass, k, !by_k, total, false, false);
        }
        cluster_sync_all(a.C);
        return sh.found != 0;
    }
    // sum_kept() from the lists, on top of the sums in sh.wabove: after border_by_counts() of top-p (those above the run), or
    // where all kept tokens are in the lists.
    __device__ __noinline__ void sum_listed(u64 border) {
        for (int i = threadIdx.x; i < sh.mine; i += kThreads) {
            const u64 key = list[i];
            if (key >= border) {
                const int piece = (int)(~(uint32_t)key + (uint32_t)row.skew) / EV;
                atomicAdd(&sh.wabove[piece / (32 * a.iters) - rank * kWarps], w_of(key_value((uint32_t)(key >> 32))));
            }
        }
        __syncwarp();
        cta_sync();
        if (lane == 0) sh.wmass[warp] = sh.wabove[warp];
        publish_sums();
    }

    // The border among more keys than can be sorted: k > 0: the k-th token; else the first token at which the sum of w
    // reaches p times `total`, over the tokens not below `floor`.  Whole cluster; sh.border in every CTA at the end.
    // Keys outside [key of low, key of m] are left out: they hold no border.
    __device__ __noinline__ void border_by_ranges(int k, u64 total, float low, u64 floor) {
        const int tid = threadIdx.x, iters = a.iters;
        const R row = this->row;
        const Weigh weigh = this->weigh;
        const float m = this->m;
        uint32_t *cnt = reinterpret_cast<uint32_t *>(sorted);  // [kBins]
        u64 *mass = list;                                      // [kBins]
        uint32_t klo = order_key(low), khi = order_key(m);
        u64 above_mass = 0ull;
        uint32_t above = 0u;
        const bool by_k = k > 0;
        if (tid == 0) sh.target = by_k ? 0ull : share_of(total);
        cta_sync();
        const u64 target = sh.target;
        const float scale = fminf(kBins / fmaxf(m - low, 1e-37f), 1e37f);
        bool linear = true;
#pragma unroll 1
        for (;;) {
            const int sh_bits = max(0, 32 - __clz((khi - klo) | 1u) - 11);
            // bin 0 holds the largest logits; both maps are monotone
            auto bin_of = [&](float l, uint32_t key) {
                return linear ? min((int)((m - l) * scale), kBins - 1) : (int)((khi - key) >> sh_bits);
            };
            for (int i = tid; i < kBins; i += kThreads) cnt[i] = 0u, mass[i] = 0ull;
            cta_sync();
#pragma unroll 1
            for (int it = 0; it < iters; ++it) {
                float v[EV];
                row.get(it, v);
#pragma unroll 1
                for (int j = 0; j < EV; ++j) {
                    float l = v[0];
#pragma unroll
                    for (int i = 1; i < EV; ++i) l = i == j ? v[i] : l;
                    const uint32_t key = order_key(l);
                    if (key >= klo && key <= khi && l > -INFINITY && make_key(key, row.at(it) + j) >= floor) {
                        const int b = bin_of(l, key);
                        atomicAdd(&cnt[b], 1u);
                        if (!by_k) atomicAdd(&mass[b], weigh.one(l));
                    }
                    __syncwarp();
                }
            }
            cluster_sync_all(a.C);
            // CTA r adds up its share of the bins over the cluster; the leader gets the sums
            const int share = kBins / a.C;
            uint32_t c4[kBins / kThreads];
            u64 m4[kBins / kThreads];
#pragma unroll
            for (int i = 0; i < kBins / kThreads; ++i) {
                const int b = tid + i * kThreads;
                c4[i] = 0u;
                m4[i] = 0ull;
                if (b >= share) continue;
                for (int c = 0; c < a.C; ++c) {
                    const int at = rank * share + b;
                    c4[i] += get32(&cnt[at], c);
                    m4[i] += get64(&mass[at], c);
                }
            }
            __syncwarp();
            cluster_sync_all(a.C);
#pragma unroll
            for (int i = 0; i < kBins / kThreads; ++i) {
                const int b = tid + i * kThreads;
                if (b >= share) continue;
                put32(&cnt[rank * share + b], 0, c4[i]);
                put64(&mass[rank * share + b], 0, m4[i]);
            }
            __syncwarp();
            cluster_sync_all(a.C);
            if (rank == 0) {
                // thread t has the bins 4 t .. 4 t + 3; the first one at which the count or the sum gets there
                constexpr int Q = kBins / kThreads;
                u64 val[Q], sum = 0ull, csum = 0ull;
                if (tid == 0) sh.found = 0;
                for (int i = 0; i < Q; ++i) {
                    const int b = Q * tid + i;
                    val[i] = by_k ? (u64)cnt[b] : mass[b];
                    sum += val[i];
                    csum += cnt[b];
                }
                const u64 incl = warp_scan64(sum), cincl = warp_scan64(csum);
                if (lane == 31) sh.wmass[warp] = incl, sh.wcount[warp] = (uint32_t)cincl;
                cta_sync();
                u64 b0 = (by_k ? (u64)above : above_mass) + incl - sum;
                uint32_t c0 = above + (uint32_t)(cincl - csum);
                for (int i = 0; i < warp; ++i) b0 += sh.wmass[i], c0 += sh.wcount[i];
                const u64 want = by_k ? (u64)k : target;
                for (int i = 0; i < Q; ++i) {
                    const int b = Q * tid + i;
                    if (b0 < want && b0 + val[i] >= want) {
                        sh.found = 1;
                        sh.above = c0;
                        sh.above_mass = b0;
                        sh.inside = cnt[b];
                        // the keys of this bin, by bisection of the monotone map
                        uint32_t lo = klo, hi = khi;
                        if (linear) {
                            uint32_t x0 = klo, x1 = khi;  // smallest key whose bin is <= b
                            while (x0 < x1) {
                                const uint32_t mid = x0 + (x1 - x0) / 2;
                                if (bin_of(key_value(mid), mid) <= b) x1 = mid;
                                else x0 = mid + 1;
                            }
                            lo = x0;
                            x0 = lo, x1 = khi;            // largest key whose bin is >= b
                            while (x0 < x1) {
                                const uint32_t mid = x1 - (x1 - x0) / 2;
                                if (bin_of(key_value(mid), mid) >= b) x0 = mid;
                                else x1 = mid - 1;
                            }
                            hi = x0;
                        } else {
                            hi = khi - ((uint32_t)b << sh_bits);
                            const uint32_t width = (1u << sh_bits) - 1u;
                            lo = hi - klo > width ? hi - width : klo;
                        }
                        sh.klo = lo;
                        sh.khi = hi;
                    }
                    b0 += val[i];
                    c0 += cnt[b];
                }
                __syncwarp();
                cta_sync();
                if (tid > 0 && tid < a.C) {
                    put32(&sh.found, tid, (uint32_t)sh.found);
                    put32(&sh.klo, tid, sh.klo);
                    put32(&sh.khi, tid, sh.khi);
                    put32(&sh.above, tid, sh.above);
                    put32(&sh.inside, tid, sh.inside);
                    put64(&sh.above_mass, tid, sh.above_mass);
                }
                __syncwarp();
            }
            cluster_sync_all(a.C);
            if (!sh.found) {  // fewer tokens than k above `low`: everything that has a weight is kept
                if (tid == 0) sh.border = 0ull;
                cluster_sync_all(a.C);
                return;
            }
            klo = sh.klo, khi = sh.khi, above = sh.above;
            above_mass = by_k ? 0ull : sh.above_mass;
            const uint32_t inside = sh.inside;
            linear = false;
            if (inside <= (uint32_t)kCap) {
                collect<false>(klo, khi, floor);
                cluster_sync_all(a.C);
                if (rank == 0) border_of_list((int)inside, above, above_mass, k, !by_k, total, false, true);
                cluster_sync_all(a.C);
                return;
            }
            if (klo == khi) {
                const u64 w = w_of(key_value(klo));
                u64 need = by_k ? (u64)k - above : (target - above_mass + w - 1ull) / w;
                if (need > inside) need = inside;
                nth_equal(klo, (uint32_t)need, floor);
                return;
            }
            cta_sync();
        }
    }

    // Border at the need-th (from 1) token, by index, of those with logit key k (and not below `floor`).
    // Whole cluster.
    __device__ __noinline__ void nth_equal(uint32_t k, uint32_t need, u64 floor) {
        const R row = this->row;
        const int iters = a.iters;
        auto tokens = [&](int it, int j, float l) {
            return order_key(l) == k && row.at(it) + j >= 0 && row.at(it) + j < a.V && make_key(k, row.at(it) + j) >= floor;
        };
        uint32_t n = 0u;
#pragma unroll 1
        for (int it = 0; it < iters; ++it) {
            float v[EV];
            row.get(it, v);
#pragma unroll
            for (int j = 0; j < EV; ++j) n += tokens(it, j, v[j]) ? 1u : 0u;
        }
        n = __reduce_add_sync(kFull, n);
        if (lane == 0) sh.wcount[warp] = n;
        cta_sync();
        if (warp == 0) {
            const uint32_t t = __reduce_add_sync(kFull, lane < kWarps ? sh.wcount[lane] : 0u);
            if (lane < a.C) put32(&sh.count[rank], lane, t);
            __syncwarp();
        }
        cluster_sync_all(a.C);
        uint32_t before = 0u;
        for (int c = 0; c < rank; ++c) before += sh.count[c];
        for (int i = 0; i < warp; ++i) before += sh.wcount[i];
        if (before < need && need <= before + sh.wcount[warp]) {  // warp-uniform
#pragma unroll 1
            for (int it = 0; it < iters && before < need; ++it) {
                float v[EV];
                row.get(it, v);
                uint32_t c = 0u;
#pragma unroll
                for (int j = 0; j < EV; ++j) c += tokens(it, j, v[j]) ? 1u : 0u;
                uint32_t incl = c;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t w = __shfl_up_sync(kFull, incl, o);
                    if (lane >= o) incl += w;
                }
                uint32_t at = before + incl - c;
                if (at < need && need <= at + c) {
#pragma unroll
                    for (int j = 0; j < EV; ++j) {
                        if (tokens(it, j, v[j]) && ++at == need)
                            for (int r = 0; r < a.C; ++r) put64(&sh.border, r, make_key(k, row.at(it) + j));
                    }
                }
                __syncwarp();
                before += __shfl_sync(kFull, incl, 31);
            }
        }
        __syncwarp();
        cluster_sync_all(a.C);
    }

    __device__ __forceinline__ float border_logit(u64 border) const {
        const uint32_t bk = (uint32_t)(border >> 32);
        return bk ? fmaxf(key_value(bk), least) : least;
    }
    // Sums of the w of the kept tokens (key >= border) per warp (sh.wmass) and, after the cluster barrier that
    // ends it, per CTA (sh.mass).
    __device__ __forceinline__ void sum_kept(u64 border) {
        const Weigh weigh = this->weigh;
        const R row = this->row;
        const int iters = a.iters;
        const float lo = border_logit(border);
        u64 sum = 0ull;
        row.each(iters, [&](int it, const float (&v)[EV]) {
            bool in[EV];
            if (__any_sync(kFull, kept(v, row.at(it), lo, border, in))) sum += sum_in(weigh, v, in);
        });
        sum = warp_sum64(sum);
        if (lane == 0) sh.wmass[warp] = sum;
        publish_sums();
    }

    __device__ __forceinline__ void run(int t) {
        const int tid = threadIdx.x;
        const R row = this->row;
        const int iters = a.iters;
        // this thread's maximum, the warps' and their j-th lane maxima
        float mine = -INFINITY;
        if (HELD) {
            cp_async_wait_all_but<0>();
            __syncwarp();
        }
        row.each(iters, [&](int, const float (&v)[EV]) {
#pragma unroll
            for (int j = 0; j < EV; ++j) mine = max_nan(mine, v[j]);
        });
        const int warps = a.C * kWarps, k0 = sh.k;
        // warps whose share lies in the row for certain; `full * jth` lane maxima bound the k-th logit
        const int full = max(1, min(warps, (a.V - EV) / (EV * 32 * a.iters)));
        const int jth = k0 > 1 && k0 < a.V ? (k0 + full - 1) / full : 0;
        float wm = mine;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) wm = max_nan(wm, __shfl_xor_sync(kFull, wm, o));
        float wj = wm;
        if (jth > 1 && jth <= 32) {
            uint32_t key = order_key(mine);
            for (int i = 1; i < jth; ++i) {
                const uint32_t top = __reduce_max_sync(kFull, key);
                if (lane == __ffs(__ballot_sync(kFull, key == top)) - 1) key = 0u;
                __syncwarp();
            }
            wj = key_value(__reduce_max_sync(kFull, key));
        }
        // every CTA of the cluster runs (it arrived as it began) before its shared memory is written to
        if (a.C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (lane < a.C) {
            put32(&sh.wtop[rank * kWarps + warp], lane, __float_as_uint(wm));
            put32(&sh.wjth[rank * kWarps + warp], lane, __float_as_uint(wj));
        }
        __syncwarp();
        cluster_sync_all(a.C);
        float mm = -INFINITY;
        for (int i = lane; i < warps; i += 32) mm = max_nan(mm, sh.wtop[i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mm = max_nan(mm, __shfl_xor_sync(kFull, mm, o));
        m = mm;
        fac = sh.fac;
        if (!(m < INFINITY) || m == -INFINITY) {  // no distribution (uniform over the cluster)
            if (rank == 0 && tid == 0) {
                a.ids[t] = -1;
                if (a.logprob) a.logprob[t] = __int_as_float(0x7fffffff);
            }
            return;
        }
        const float p = sh.p;
        const bool greedy = !(fac.hi > 0.f) || k0 == 1, by_k = jth > 0, by_p = p < 1.f;
        // rounded up (towards m): below it the integer weight's shift would pass 63 and wrap, and the logit next below the exact
        // border may be several temperatures away from it
        least = __fsub_ru(m * fac.s, __fdiv_rd((float)a.shift, fac.hi));
        least = greedy ? m : fmaxf(fac.s < 1.f ? least + least : least, -3.4028234e38f);
        weigh.set(m, fac, a.shift, sh.table);
        u64 border = 0ull, total = 0ull;
        bool summed = false, in_list = false;  // the kept tokens' sums: above a run already; all of them are in the lists
        if (greedy) {
            border = (u64)order_key(m) << 32;
        } else if (by_k || by_p) {
            // A bound for the list: the k-th largest of the warps' maxima (for top-p alone, three quarters of their number:
            // a few hundred tokens, which mostly hold the share p), or the smallest j-th largest lane maximum.
            const int nth = by_k ? jth == 1 ? k0 : 0 : max(1, full * 3 / 4);
            if (tid == 0) sh.bound = -INFINITY;
            cta_sync();
            if (nth > 0) {
                const int i = tid >> 2;  // 4 threads for each warp
                const float own = i < warps ? sh.wtop[i] : 0.f;
                int above = 0;
                if (i < warps)
                    for (int q = tid & 3; q < warps; q += 4) above += sh.wtop[q] > own || (sh.wtop[q] == own && q < i) ? 1 : 0;
                above += __shfl_xor_sync(kFull, above, 1);
                above += __shfl_xor_sync(kFull, above, 2);
                if (i < warps && (tid & 3) == 0 && above == nth - 1) sh.bound = own;
            } else if (jth <= 32 && warp == 0) {
                float lo = INFINITY;
                for (int i = lane; i < full; i += 32) lo = fminf(lo, sh.wjth[i]);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) lo = fminf(lo, __shfl_xor_sync(kFull, lo, o));
                if (lane == 0) sh.bound = lo;
            }
            // Top-p: all tokens below w = (1 - p) M' / V together have less than 1 - p of the sum, M' being what the warps'
            // maxima alone add up to.
            float sum = 0.f;
            for (int i = lane; i < warps; i += 32) sum += exp2f((sh.wtop[i] * fac.s - m * fac.s) * fac.hi);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
            const float low_p = fmaxf(fminf(m + (log2f((1.f - p) * sum / (float)a.V) - 0.05f) / (fac.hi * fac.s), m), least);
            __syncwarp();
            cta_sync();
            float bound = fmaxf(sh.bound, least), low = by_k ? bound : low_p;
            if (a.V <= kCap) bound = low;
            bound = fmaxf(bound, low);
            bin_scale = fminf(kCounts / fmaxf(m - low, 1e-37f), 1e37f);
            cta_sync();
            if (tid == 0) sh.bound = low;
            // the candidates; by top-p alone also the sum of all
            if (by_k) collect<false>(order_key(bound), order_key(m), 0ull);
            else collect<true>(order_key(bound), order_key(m), 0ull);
            cluster_sync_all(a.C);
            uint32_t n = 0u;
            for (int c = 0; c < a.C; ++c) {
                n += sh.count[c];
                total += by_k ? 0ull : sh.mass[c];
            }
            // by top-k the list holds the k-th token (or all that have a weight); by top-p alone it may end too early
            // (it does for certain where its tokens, at a weight of one each, do not add up to p of the sum)
            bool done = false;
            if (n <= (uint32_t)kCap && (by_k || bound == low || (float)n >= p * (float)(total >> a.shift) * 0.999f)) {
                if (rank == 0) border_of_list((int)n, 0u, 0ull, by_k ? k0 : 0, by_p, total, by_k, by_k || bound == low);
                cluster_sync_all(a.C);
                done = sh.found != 0;
            }
            if (done) {
                border = sh.border;
                in_list = true;
            } else if (by_k != by_p && border_by_counts(by_k ? k0 : 0, total)) {
                border = sh.border;
                summed = by_p;
            } else {
                cluster_sync_all(a.C);
                u64 floor = 0ull;
                if (by_k) {
                    border_by_ranges(k0, 0ull, low, 0ull);
                    floor = border = sh.border;
                }
                if (by_p) {
                    if (by_k) {
                        sum_kept(floor);
                        total = 0ull;
                        for (int c = 0; c < a.C; ++c) total += sh.mass[c];
                        cluster_sync_all(a.C);  // everybody has read the sums
                    }
                    border_by_ranges(0, total, by_k ? least : low_p, floor);
                    border = sh.border > floor ? sh.border : floor;
                }
            }
        }
        if (!greedy && sh.min_p > 0.f) {
            // the smallest logit whose w is at least min_p times the largest: 32 places of the range at a time
            const u64 want = sh.min_p < 1.f ? share(sh.min_p, 1ull << a.shift, true) : 1ull << a.shift;
            uint32_t x0 = order_key(least), x1 = order_key(m);
            if (warp == 0) {
                while (x0 < x1) {
                    const uint32_t x = x0 + (uint32_t)((u64)(x1 - x0) * (uint32_t)lane >> 5);
                    const unsigned in = __ballot_sync(kFull, w_of(key_value(x)) >= want);
                    const int at = in ? __ffs(in) - 1 : 32;
                    const uint32_t below = __shfl_sync(kFull, x, at > 0 ? at - 1 : 0), above = __shfl_sync(kFull, x, at & 31);
                    if (at < 32) x1 = above;
                    if (at > 0) x0 = below + 1u;
                }
                if (lane == 0) sh.klo = x0;
            }
            cta_sync();
            const u64 b = (u64)sh.klo << 32;
            summed = summed && b <= border;
            border = b > border ? b : border;
        }
        cta_sync();
        if (in_list && tid < kWarps) sh.wabove[tid] = 0ull;
        cta_sync();
        if (summed || in_list) sum_listed(border);
        else sum_kept(border);
        u64 S = 0ull, before = 0ull;
        for (int c = 0; c < a.C; ++c) {
            const u64 v = sh.mass[c];
            S += v;
            before += c < rank ? v : 0ull;
        }
        if (tid == 0) {
            const float u = greedy ? 0.f : fmaxf(sh.u, 0.f);
            sh.target = u < 1.f ? share(u, S, false) : S - 1ull;
        }
        cta_sync();
        const u64 target = sh.target;  // the first token at which the sum exceeds it
        for (int i = 0; i < warp; ++i) before += sh.wmass[i];
        if (before <= target && target < before + sh.wmass[warp]) {  // one warp of the cluster
            const Weigh weigh = this->weigh;
            const float lo = border_logit(border);
#pragma unroll 1
            for (int it = 0; it < iters; ++it) {
                float v[EV];
                row.get(it, v);
                bool in[EV];
                if (!__any_sync(kFull, kept(v, row.at(it), lo, border, in))) continue;
                u64 w[EV], sum = 0ull;
#pragma unroll
                for (int j = 0; j < EV; j += 2) {
                    weigh.pair(v[j], v[j + 1], w[j], w[j + 1]);
                    w[j] = in[j] ? w[j] : 0ull;
                    w[j + 1] = in[j + 1] ? w[j + 1] : 0ull;
                    sum += w[j] + w[j + 1];
                }
                const u64 incl = warp_scan64(sum);
                u64 at = before + incl - sum;
                const bool here = at <= target && target < at + sum;
                if (here) {
                    bool done = false;
#pragma unroll
                    for (int j = 0; j < EV; ++j) {
                        if (!done && target < at + w[j]) {
                            done = true;
                            a.ids[t] = row.at(it) + j;
                            if (a.logprob) {
                                float e, e_lo;
                                exponent(v[j], m, fac, e, e_lo);
                                // the total as a pair of f32, in units of the largest w
                                const u64 one = 1ull << a.shift, whole = S >> a.shift;
                                const float s_hi = (float)whole, s_lo = (float)(S & (one - 1ull)) * (1.f / (float)one);
                                const float s = s_hi + s_lo, rest = s_lo - (s - s_hi);
                                a.logprob[t] = greedy || w[j] == S ? 0.f : (e + e_lo) * 0.69314718f - (logf(s) + rest / s);
                            }
                        }
                        at += w[j];
                    }
                }
                __syncwarp();
                if (__any_sync(kFull, here)) break;
                before += __shfl_sync(kFull, incl, 31);
            }
        }
        __syncwarp();
    }
};

template <typename E, bool HELD>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a) {
    constexpr int EV = 16 / sizeof(E);
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Shared sh;
    const int tid = threadIdx.x;
    const int t = blockIdx.x / a.C, rank = blockIdx.x - t * a.C;
    u64 *list = reinterpret_cast<u64 *>(smem), *sorted = list + kCap;
    if (a.C > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    pdl_wait();
    pdl_trigger();
    const E *x = static_cast<const E *>(a.x) + (size_t)t * a.V;
    const int skew = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(E));
    const int warp = tid >> 5, lane = tid & 31;
    Row<E, HELD> row;
    row.x = x;
    row.V = a.V;
    row.skew = skew;
    row.first = (((rank * kWarps + warp) * a.iters) * 32 + lane) * EV - skew;
    row.held = smem_addr(smem) + kFixedBytes + (warp * a.iters * 32 + lane) * 16;
    float heat = 1.f, mp = 0.f, p = 1.f, u = 0.f;
    int k = 0;
    if (tid == 0) {
        if (a.temperature) heat = a.temperature[t];
        if (a.min_p) mp = a.min_p[t];
        if (a.top_k) k = a.top_k[t];
        if (a.top_p) p = a.top_p[t];
        u = a.u[t];
    }
    if (HELD) row.load(a.iters);
    if (tid < 32) sh.table[tid] = kPow2.v[tid];
    if (tid == 0) {
        sh.k = k;
        sh.p = p < 1.f ? fmaxf(p, 0.f) : 1.f;  // NaN: off
        sh.u = u;
        if (heat > 0.f) {
            // log2(e) / heat in two parts: the quotient of the significands and its remainder's
            const float h = fminf(fmaxf(heat, 8.5e-39f), 3.4028234e38f);
            int ex;
            const float f = 2.f * frexpf(h, &ex), q = 1.44269504f / f;
            const float rest = (fmaf(-q, f, 1.44269504f) + 1.9259630e-8f) / f;
            const bool tiny = ex > 60;
            sh.fac.s = ex > 100 ? 0.5f : 1.f;
            if (ex > 100) --ex;
            sh.fac.hi = ldexpf(q, 1 - ex);
            sh.fac.lo = ldexpf(rest, 1 - ex + (tiny ? 24 : 0)) + (tiny ? ldexpf(ldexpf(q, 25 - ex) - ldexpf(sh.fac.hi, 24), 0) : 0.f);
            sh.fac.pre = tiny ? 5.9604644775390625e-8f : 1.f;
        } else {
            sh.fac = Factor{0.f, 0.f, 0.f, 1.f};
        }
        sh.min_p = mp > 0.f ? fminf(mp, 1.f) : 0.f;
    }
    cta_sync();
    Sampler<E, HELD> s{a, sh, list, sorted, reinterpret_cast<uint32_t *>(sorted + kCap), row, rank, lane, warp, 0.f, 0.f, Factor{}, Weigh{}, 0.f};
    s.run(t);
    __syncwarp();
    cluster_sync_all(a.C);  // nobody leaves while others may still reach for its shared memory
}

template <typename E, bool HELD>
rl_status launch_sample(SampleArgs &a, int T, cudaStream_t s) {
    auto kernel = sample_kernel<E, HELD>;
    a.iters = (a.per + kThreads - 1) / kThreads;
    const size_t smem = kFixedBytes + (HELD ? (size_t)a.iters * kThreads * 16 : 0);
    rl_status st = allow_smem((const void *)kernel, smem);
    if (st != RL_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(T * a.C);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.C;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    if (e != cudaSuccess) return fail(RL_ERR_CUDA, "rl_sample: launch failed: %s", cudaGetErrorString(e));
    return RL_OK;
}

template <typename E>
rl_status run_sample(SampleArgs &a, int T, cudaStream_t s) {
    constexpr int EV = 16 / sizeof(E);
    // pieces of 16 bytes of a row, one more where rows do not start on 16-byte boundaries
    const bool even = (size_t)a.V * sizeof(E) % 16 == 0 && (reinterpret_cast<uintptr_t>(a.x) & 15) == 0;
    const int pieces = even ? a.V / EV : (a.V + 2 * (EV - 1)) / EV;
    // CTAs per row: held, 64 KB of it each, and with few rows as many as still leave every thread a piece; streamed (from as
    // many rows as SMs on) two, whose waves are finer than one's (512 x 131072: 198 against 220 us, four 218)
    const int sms = sm_count();
    const bool streamed = T >= sms;
    a.C = streamed && pieces >= 16 * kThreads ? 2 : 1;
    while (!streamed && a.C < kMaxC && (pieces > a.C * 8 * kThreads || ((long long)T * a.C * 2 <= sms && pieces > a.C * kThreads))) a.C *= 2;
    a.per = (pieces + a.C - 1) / a.C;
    a.shift = 63;
    for (int v = 1; v < a.V; v *= 2) --a.shift;  // the sum of V weights stays below 2^64
    if (a.shift > 46) a.shift = 46;
    // 227 KB of shared memory per CTA: 22 times 8 KB of a row beside the lists (streamed rows of up to 32 KB are held too)
    if (a.per <= (streamed ? 4 : 22) * kThreads) return launch_sample<E, true>(a, T, s);
    return launch_sample<E, false>(a, T, s);
}

}  // namespace

extern "C" rl_status rl_sample(const void *logits, int32_t dtype, int32_t T, int32_t V, const float *uniform,
                               const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
                               int32_t *ids, float *logprob, void *stream) {
    if (dtype != RL_F32 && dtype != RL_F16 && dtype != RL_BF16)
        return fail(RL_ERR_INVALID, "rl_sample: dtype %d is none of RL_F32, RL_F16, RL_BF16", dtype);
    if (T < 0 || V <= 0) return fail(RL_ERR_INVALID, "rl_sample: T=%d V=%d", T, V);
    if (V > kMaxV) return fail(RL_ERR_UNSUPPORTED, "rl_sample: V=%d > 2^26", V);
    if (T > (1 << 24)) return fail(RL_ERR_UNSUPPORTED, "rl_sample: T=%d > 2^24", T);
    if (T == 0) return RL_OK;
    if (!logits || !uniform || !ids) return fail(RL_ERR_INVALID, "rl_sample: NULL logits, uniform or ids");
    if (reinterpret_cast<uintptr_t>(logits) % dtype_bytes(dtype)) return fail(RL_ERR_INVALID, "rl_sample: logits misaligned");
    if ((reinterpret_cast<uintptr_t>(uniform) | reinterpret_cast<uintptr_t>(temperature) | reinterpret_cast<uintptr_t>(top_k) |
         reinterpret_cast<uintptr_t>(top_p) | reinterpret_cast<uintptr_t>(min_p) | reinterpret_cast<uintptr_t>(ids) |
         reinterpret_cast<uintptr_t>(logprob)) & 3)
        return fail(RL_ERR_INVALID, "rl_sample: settings and outputs must be 4-byte aligned");
    SampleArgs a = {};
    a.x = logits;
    a.u = uniform;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.ids = ids;
    a.logprob = logprob;
    a.V = V;
    cudaStream_t s = as_stream(stream);
    if (dtype == RL_F32) return run_sample<float>(a, T, s);
    if (dtype == RL_F16) return run_sample<__half>(a, T, s);
    return run_sample<__nv_bfloat16>(a, T, s);
}
