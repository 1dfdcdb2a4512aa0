// sample.cu - rl_sample: the next token of each row of logits, by temperature, top-k, top-p and min-p, from
// given random numbers.
//
// Order: logits descending, equal ones by index.  A token's place in it is the 64-bit key (order-preserving
// logit above ~index), so that a border is one key and a token is kept when its key is not below.
//
//   w(l) = 2^((l - max) log2(e) / temperature), as an integer multiple of 2^-s (s = 45 for 2^17 tokens)
//   top-k border: the k-th key;  top-p border: the first key at which the sum of w reaches p times that of
//   all (of the k);  min-p border: logit max + temperature ln(min_p);  the highest of them counts
//   the token: the first one in index order at which the sum of the kept w passes u times their total
//
// Why integers: whether a token next to a border is in, and which one u meets, must depend neither on the order
// of summation nor on the rounding of 32-bit sums (over 512 rows of 131072 flat logits 32-bit sums pick another
// token about once).  w is good to 2^-30 of itself: the exponent is a pair of f32, its fraction's first five bits go
// through a table of 2^(j / 32) (one entry per bank, so lookups never conflict), the rest through the series of e^x.
//
// A row is held by a cluster of up to 8 CTAs in shared memory and read from HBM once (rows beyond what
// fits are read again in each pass).  Passes over it: the maximum; the sum of all w (top-p without top-k)
// and the candidates above a bound that the border cannot lie below; the sums of the kept w per warp (a
// warp holds neighbouring tokens); and the warp that holds the token goes through its share once more.
//   bound for top-k: the k-th largest of the warps' largest logits (or, for larger k, the smallest of the
//   warps' j-th largest lane maxima, j = k / warps);  for top-p: (1 - p) / V of the largest w, because all
//   tokens below it together have less than 1 - p of the sum.
// Up to 2048 candidates are sorted by one CTA (bitonic, in registers and through shared memory), which finds
// the border on their running sum.  With more of them (flat rows, large k) the range of keys that holds the border is
// narrowed by histograms of counts and sums, 2048 bins of equal width in the logit first and of equal width in the key
// after that, until 2048 keys are left or a single logit, whose tokens have equal w and are counted off by index.
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
constexpr int kBins = 2048;
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
    int V, C, iters, shift;  // iters: pieces of 16 bytes per thread; w = multiples of 2^-shift
};

// log2(e) / temperature as hi + lo * pre (pre: 1, or 2^-24 where lo by itself would leave f32's normal range)
struct Factor {
    float hi, lo, pre;
};

struct Shared {
    u64 mass[kMaxC];         // by CTA of the cluster
    u64 wmass[kWarps];
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
    double gap;              // -temperature ln(min_p), or negative: off
    int32_t table[32];
    int k;
    float p, u;
};

__device__ __forceinline__ void cluster_sync_all() {
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
    const float d = l - m, b = d + m, e = (l - b) + ((b - d) - m);  // d + e = l - m exactly (two-sum)
    t = d * c.hi;
    t_lo = fmaf(e, c.hi, fmaf(d * c.pre, c.lo, fmaf(d, c.hi, -t)));
}
// w(l) in multiples of 2^-shift, rounded to the nearest; 0 from 2^-shift down and for -infinity
__device__ __forceinline__ u64 weight(float l, float m, Factor c, int shift, const int32_t *table) {
    float t, t_lo;
    exponent(l, m, c, t, t_lo);
    const bool none = !(t > -(float)shift);
    t = none ? 0.f : t;
    const float kf = t + 393216.f;  // 1.5 * 2^18: the nearest multiple of 1 / 32
    const int k = __float_as_int(kf) - __float_as_int(393216.f);
    const float r = (t - (kf - 393216.f)) + (none ? 0.f : t_lo);
    // e^(r ln 2) - 1, |r| <= 1 / 64: the fifth term is below 2^-39
    const float p = r * fmaf(r, fmaf(r, fmaf(r, 9.618129e-3f, 5.550411e-2f), 0.24022651f), 0.69314718f);
    const int P = __float2int_rn(p * 4294967296.f);
    const int32_t T = table[k & 31];
    const u64 e = (u64)((long long)T * P + ((long long)T << 32));  // 2^62 ... 2^63
    return none ? 0ull : ((e >> (61 - shift - (k >> 5))) + 1ull) >> 1;
}

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
    __device__ __forceinline__ uint4 edge(int i0) const {
        E e[EV];
#pragma unroll
        for (int k = 0; k < EV; ++k) e[k] = i0 + k >= 0 && i0 + k < V ? x[i0 + k] : from_float<E>(-INFINITY);
        return *reinterpret_cast<const uint4 *>(e);
    }
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
    __device__ __forceinline__ void get(int it, float (&v)[EV]) const {
        uint4 q;
        if constexpr (HELD) q = lds128(held + it * 512);
        else q = inner(at(it)) ? __ldg(reinterpret_cast<const uint4 *>(x + at(it))) : edge(at(it));
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
};

// ---- the sort of the candidates ----------------------------------------------------------------
// N = EPT * kThreads keys in buf, descending.  Element e kThreads + tid is in this thread's register e: exchanges
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
    u64 *list, *sorted;                  // kCap keys each; together the histograms
    R row;
    int rank, lane, warp;
    float m;
    Factor fac;

    // the sum that the tokens kept by top-p reach: a share p < 1 of `total`, at least the first token's
    __device__ __forceinline__ u64 share_of(u64 total) const {
        const u64 t = (u64)ceil((double)sh.p * (double)total);
        return t > 0ull ? t : 1ull;
    }
    __device__ __forceinline__ u64 w_of(float l) const { return weight(l, m, fac, a.shift, sh.table); }

    // Tokens whose logit's key lies in [klo, khi] and that are not below `floor` into this CTA's list; sh.count
    // has their numbers after the next cluster barrier, also beyond kCap.  With ALL also the sums of all w
    // (sh.mass).
    template <bool ALL>
    __device__ __noinline__ void collect(uint32_t klo, uint32_t khi, u64 floor) {
        if (threadIdx.x == 0) sh.mine = 0;
        cta_sync();
        const float lo = key_value(klo);
        u64 sum = 0ull;
#pragma unroll 1
        for (int it = 0; it < a.iters; ++it) {
            float v[EV];
            row.get(it, v);
            bool any = false;
#pragma unroll
            for (int j = 0; j < EV; ++j) any = any || v[j] >= lo;
            if (ALL) {
#pragma unroll
                for (int j = 0; j < EV; ++j) sum += w_of(v[j]);
            }
            if (!__any_sync(kFull, any)) continue;
#pragma unroll 1
            for (int j = 0; j < EV; ++j) {
                float l = v[0];
#pragma unroll
                for (int i = 1; i < EV; ++i) l = i == j ? v[i] : l;
                const uint32_t k = order_key(l);
                const bool in = k >= klo && k <= khi && l > -INFINITY && make_key(k, row.at(it) + j) >= floor;
                const unsigned mask = __ballot_sync(kFull, in);
                if (mask == 0u) continue;
                int base = 0;
                if (lane == 0) base = atomicAdd(&sh.mine, __popc(mask));
                base = __shfl_sync(kFull, base, 0) + __popc(mask & ((1u << lane) - 1u));
                if (in && base < kCap) list[base] = make_key(k, row.at(it) + j);
                __syncwarp();
            }
        }
        if (ALL) {
            sum = warp_sum64(sum);
            if (lane == 0) sh.wmass[warp] = sum;
        }
        cta_sync();
        if (warp == 0) {
            u64 t = ALL && lane < kWarps ? sh.wmass[lane] : 0ull;
            if (ALL) t = warp_sum64(t);
            if (lane < a.C) {
                put32(&sh.count[rank], lane, (uint32_t)sh.mine);
                if (ALL) put64(&sh.mass[rank], lane, t);
            }
            __syncwarp();
        }
    }

    // Sorts the candidates of all lists (n <= kCap) and finds the border: the k-th token of the order (k > 0)
    // and the first at which the sum reaches p times `total` (of the k tokens' sum with k > 0), counted from
    // `above` tokens and a sum of `above_mass` that lie before the candidates.  Leader CTA; the border goes to
    // all CTAs.
    __device__ __noinline__ void border_of_list(int n, uint32_t above, u64 above_mass, int k, bool by_p, u64 total, bool total_of_k) {
        const int tid = threadIdx.x;
        int at = 0;
        for (int c = 0; c < a.C; ++c) {
            const int cnt = (int)sh.count[c];
            for (int i = tid; i < cnt; i += kThreads) sorted[at + i] = get64(&list[i], c);
            at += cnt;
        }
        const int ept = n <= kThreads ? 1 : n <= 2 * kThreads ? 2 : 4;
        for (int i = n + tid; i < ept * kThreads; i += kThreads) sorted[i] = 0ull;
        cta_sync();
        if (ept == 1) sort_keys<1>(sorted);
        else if (ept == 2) sort_keys<2>(sorted);
        else sort_keys<4>(sorted);
        // running sums: thread t has the places ept t .. ept t + ept - 1
        u64 key[4], w[4], sum = 0ull;
        for (int e = 0; e < 4; ++e) {
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
        }
        cta_sync();
        const u64 target = sh.target;
        for (int e = 0; e < ept; ++e) {
            const int i = ept * tid + e;
            // the last place of the run: the sum before it is below the target, with it not, or top-k ends
            if (i <= last && (i == 0 || before < target) && (i == last || before + w[e] >= target)) sh.border = key[e];
            before += w[e];
        }
        cta_sync();
        if (tid < a.C) put64(&sh.border, tid, sh.border);
        __syncwarp();
    }

    // The border among more keys than can be sorted: k > 0: the k-th token; else the first token at which the sum of w
    // reaches p times `total`, over the tokens not below `floor`.  Whole cluster; sh.border in every CTA at the end.
    // Keys outside [key of low, key of m] are left out: they hold no border.
    __device__ __noinline__ void border_by_ranges(int k, u64 total, float low, u64 floor) {
        const int tid = threadIdx.x;
        uint32_t *cnt = reinterpret_cast<uint32_t *>(sorted);  // [kBins]
        u64 *mass = list;                                      // [kBins]
        uint32_t klo = order_key(low), khi = order_key(m);
        u64 above_mass = 0ull;
        uint32_t above = 0u;
        const bool by_k = k > 0;
        if (tid == 0) sh.target = by_k ? 0ull : share_of(total);
        cta_sync();
        const u64 target = sh.target;
        const float scale = kBins / fmaxf(m - low, 1e-37f);
        bool linear = scale < INFINITY;
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
            for (int it = 0; it < a.iters; ++it) {
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
                        if (!by_k) atomicAdd(&mass[b], w_of(l));
                    }
                    __syncwarp();
                }
            }
            cluster_sync_all();
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
            cluster_sync_all();
#pragma unroll
            for (int i = 0; i < kBins / kThreads; ++i) {
                const int b = tid + i * kThreads;
                if (b >= share) continue;
                put32(&cnt[rank * share + b], 0, c4[i]);
                put64(&mass[rank * share + b], 0, m4[i]);
            }
            __syncwarp();
            cluster_sync_all();
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
            cluster_sync_all();
            if (!sh.found) {  // fewer tokens than k above `low`: everything that has a weight is kept
                if (tid == 0) sh.border = 0ull;
                cluster_sync_all();
                return;
            }
            klo = sh.klo, khi = sh.khi, above = sh.above;
            above_mass = by_k ? 0ull : sh.above_mass;
            const uint32_t inside = sh.inside;
            linear = false;
            if (inside <= (uint32_t)kCap) {
                collect<false>(klo, khi, floor);
                cluster_sync_all();
                if (rank == 0) border_of_list((int)inside, above, above_mass, k, !by_k, total, false);
                cluster_sync_all();
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
        auto tokens = [&](int it, int j, float l) {
            return order_key(l) == k && row.at(it) + j >= 0 && row.at(it) + j < a.V && make_key(k, row.at(it) + j) >= floor;
        };
        uint32_t n = 0u;
#pragma unroll 1
        for (int it = 0; it < a.iters; ++it) {
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
        cluster_sync_all();
        uint32_t before = 0u;
        for (int c = 0; c < rank; ++c) before += sh.count[c];
        for (int i = 0; i < warp; ++i) before += sh.wcount[i];
        if (before < need && need <= before + sh.wcount[warp]) {  // warp-uniform
#pragma unroll 1
            for (int it = 0; it < a.iters && before < need; ++it) {
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
        cluster_sync_all();
    }

    // Sums of the w of the kept tokens (key >= border) per warp (sh.wmass) and, after the cluster barrier that
    // ends it, per CTA (sh.mass).
    __device__ __forceinline__ void sum_kept(u64 border) {
        const uint32_t bk = (uint32_t)(border >> 32);
        const float lo = bk ? key_value(bk) : -INFINITY;
        u64 sum = 0ull;
#pragma unroll 1
        for (int it = 0; it < a.iters; ++it) {
            float v[EV];
            row.get(it, v);
            bool any = false;
#pragma unroll
            for (int j = 0; j < EV; ++j) any = any || v[j] >= lo;
            if (!__any_sync(kFull, any)) continue;
#pragma unroll
            for (int j = 0; j < EV; ++j) {
                const u64 w = w_of(v[j]);
                if (v[j] > lo || make_key(order_key(v[j]), row.at(it) + j) >= border) sum += w;
            }
        }
        sum = warp_sum64(sum);
        if (lane == 0) sh.wmass[warp] = sum;
        cta_sync();
        if (warp == 0) {
            const u64 t = warp_sum64(lane < kWarps ? sh.wmass[lane] : 0ull);
            if (lane < a.C) put64(&sh.mass[rank], lane, t);
            __syncwarp();
        }
        cluster_sync_all();
    }

    __device__ __forceinline__ void run(int t) {
        const int tid = threadIdx.x;
        // this thread's maximum, the warps' and their j-th lane maxima
        float mine = -INFINITY;
        if (HELD) {
            cp_async_wait_all_but<0>();
            __syncwarp();
        }
#pragma unroll 1
        for (int it = 0; it < a.iters; ++it) {
            float v[EV];
            row.get(it, v);
#pragma unroll
            for (int j = 0; j < EV; ++j) mine = max_nan(mine, v[j]);
        }
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
        if (lane < a.C) {
            put32(&sh.wtop[rank * kWarps + warp], lane, __float_as_uint(wm));
            put32(&sh.wjth[rank * kWarps + warp], lane, __float_as_uint(wj));
        }
        __syncwarp();
        cluster_sync_all();
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
        u64 border = 0ull, total = 0ull;
        if (greedy) {
            border = (u64)order_key(m) << 32;
        } else if (by_k || by_p) {
            if (tid == 0) sh.bound = -INFINITY;
            cta_sync();
            if (by_k && jth == 1) {
                // the k-th largest of the warps' maxima, 4 threads for each
                const int i = tid >> 2;
                const float own = i < warps ? sh.wjth[i] : 0.f;
                int above = 0;
                if (i < warps)
                    for (int q = tid & 3; q < warps; q += 4) above += sh.wjth[q] > own || (sh.wjth[q] == own && q < i) ? 1 : 0;
                above += __shfl_xor_sync(kFull, above, 1);
                above += __shfl_xor_sync(kFull, above, 2);
                if (i < warps && (tid & 3) == 0 && above == k0 - 1) sh.bound = own;
            } else if (by_k && jth <= 32) {
                if (warp == 0) {
                    float lo = INFINITY;
                    for (int i = lane; i < full; i += 32) lo = fminf(lo, sh.wjth[i]);
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) lo = fminf(lo, __shfl_xor_sync(kFull, lo, o));
                    if (lane == 0) sh.bound = lo;
                }
            } else if (!by_k && tid == 0) {
                sh.bound = m + (log2f((1.f - p) / (float)a.V) - 0.05f) / fac.hi;
            }
            __syncwarp();
            cta_sync();
            const float bound = sh.bound;
            const float weightless = m - ((float)a.shift + 1.f) / fac.hi;  // tokens below have w = 0
            const float low = fmaxf(fmaxf(bound, weightless), -3.4028234e38f);
            // the candidates; by top-p alone also the sum of all
            const bool listed = !by_k || bound > -INFINITY || a.V <= kCap;
            if (!by_k) collect<true>(order_key(low), order_key(m), 0ull);
            else if (listed) collect<false>(order_key(low), order_key(m), 0ull);
            cluster_sync_all();
            uint32_t n = 0u;
            for (int c = 0; c < a.C; ++c) {
                n += listed ? sh.count[c] : 0u;
                total += by_k ? 0ull : sh.mass[c];
            }
            if (listed && n <= (uint32_t)kCap) {
                if (rank == 0) border_of_list((int)n, 0u, 0ull, by_k ? k0 : 0, by_p, total, by_k);
                cluster_sync_all();
                border = sh.border;
            } else {
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
                        cluster_sync_all();  // everybody has read the sums
                    }
                    const float low_p = fmaxf(m + (log2f((1.f - p) / (float)a.V) - 0.05f) / fac.hi, fmaxf(weightless, -3.4028234e38f));
                    border_by_ranges(0, total, low_p, floor);
                    border = sh.border > floor ? sh.border : floor;
                }
            }
        }
        if (!greedy && sh.gap >= 0.) {
            const u64 b = (u64)order_key(__double2float_ru((double)m - sh.gap)) << 32;
            border = b > border ? b : border;
        }
        cta_sync();
        sum_kept(border);
        u64 S = 0ull, before = 0ull;
        for (int c = 0; c < a.C; ++c) {
            const u64 v = sh.mass[c];
            S += v;
            before += c < rank ? v : 0ull;
        }
        if (tid == 0) {
            const double u = greedy ? 0. : fmin(fmax((double)sh.u, 0.), 1.);
            const u64 g = (u64)(u * (double)S);
            sh.target = g < S ? g : S - 1ull;
        }
        cta_sync();
        const u64 target = sh.target;  // the first token at which the sum exceeds it
        for (int i = 0; i < warp; ++i) before += sh.wmass[i];
        if (before <= target && target < before + sh.wmass[warp]) {  // one warp of the cluster
            const uint32_t bk = (uint32_t)(border >> 32);
            const float lo = bk ? key_value(bk) : -INFINITY;
#pragma unroll 1
            for (int it = 0; it < a.iters; ++it) {
                float v[EV];
                row.get(it, v);
                u64 w[EV], sum = 0ull;
#pragma unroll
                for (int j = 0; j < EV; ++j) {
                    w[j] = v[j] > lo || make_key(order_key(v[j]), row.at(it) + j) >= border ? w_of(v[j]) : 0ull;
                    sum += w[j];
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
                                a.logprob[t] = greedy ? 0.f : (e + e_lo) * 0.69314718f - (logf(s) + rest / s);
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
__global__ void __launch_bounds__(kThreads, HELD ? 2 : 1) sample_kernel(const __grid_constant__ SampleArgs a) {
    constexpr int EV = 16 / sizeof(E);
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Shared sh;
    const int tid = threadIdx.x;
    const int t = blockIdx.x / a.C, rank = blockIdx.x - t * a.C;
    u64 *list = reinterpret_cast<u64 *>(smem), *sorted = list + kCap;
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
    row.held = smem_addr(smem) + 2 * kCap * 8 + (warp * a.iters * 32 + lane) * 16;
    if (HELD) row.load(a.iters);
    if (tid < 32) sh.table[tid] = kPow2.v[tid];
    if (tid == 0) {
        const float heat = a.temperature ? a.temperature[t] : 1.f;
        const float mp = a.min_p ? a.min_p[t] : 0.f;
        sh.k = a.top_k ? a.top_k[t] : 0;
        sh.p = a.top_p ? a.top_p[t] : 1.f;
        sh.u = a.u[t];
        sh.p = sh.p < 1.f ? fmaxf(sh.p, 0.f) : 1.f;  // NaN: off
        if (heat > 0.f) {
            const double c = fmin(1.4426950408889634 / (double)fminf(heat, 3.4028234e38f), 1.7e38);
            const bool tiny = c < 1e-18;
            sh.fac.hi = (float)c;
            sh.fac.lo = (float)((c - (double)sh.fac.hi) * (tiny ? 16777216. : 1.));
            sh.fac.pre = tiny ? 5.9604644775390625e-8f : 1.f;
        } else {
            sh.fac = Factor{0.f, 0.f, 0.f};
        }
        sh.gap = mp > 0.f ? -(double)heat * log(fmin((double)mp, 1.)) : -1.;
    }
    cta_sync();
    Sampler<E, HELD> s{a, sh, list, sorted, row, rank, lane, warp, 0.f, Factor{}};
    cluster_sync_all();  // every CTA of the cluster runs before its shared memory is written to
    s.run(t);
    __syncwarp();
    cluster_sync_all();  // nobody leaves while others may still reach for its shared memory
}

template <typename E, bool HELD>
rl_status launch_sample(SampleArgs &a, int T, cudaStream_t s) {
    auto kernel = sample_kernel<E, HELD>;
    const size_t smem = 2 * kCap * 8 + (HELD ? (size_t)a.iters * kThreads * 16 : 0);
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
    // CTAs per row: 64 KB of it each; with few rows as many as still leave every thread a piece
    const int sms = sm_count();
    a.C = 1;
    while (a.C < kMaxC && (pieces > a.C * 8 * kThreads || ((long long)T * a.C * 2 <= sms && pieces > a.C * kThreads))) a.C *= 2;
    const int per = (pieces + a.C - 1) / a.C;
    a.iters = (per + kThreads - 1) / kThreads;
    a.shift = 62;
    for (int v = 1; v < a.V; v *= 2) --a.shift;  // the sum of V weights stays below 2^62
    if (a.shift > 45) a.shift = 45;
    // 227 KB of shared memory per CTA: 24 pieces of 8 KB beside the lists
    if (a.iters <= 22) return launch_sample<E, true>(a, T, s);
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
