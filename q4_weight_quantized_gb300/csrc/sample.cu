// Sampling with temperature, top-k, top-p and min-p from given random numbers.
//
// The row's weights are whole numbers w = floor(2^(40 - d)), d = (z_max - z) / (T ln 2),
// so sums are exact in any order and every decision (which tokens top-p keeps, which
// one the random number falls on) is an integer comparison: the token does not depend
// on how the work is split.  What top-k and top-p keep is a prefix in rank (logit
// descending, index ascending), so all that has to be found is where it ends.
//
// A cluster of CTAs owns a row: each keeps its contiguous share of the logits in shared
// memory, so the row is read from global memory once, and the CTAs exchange bins, sums
// and cuts through distributed shared memory.
//   1. load, largest logits of 128 parts of the row: its largest, and a bound below the k-th
//      (at least k logits are as large as the k-th of these);
//   2. where top-k (k <= 96) or min-p can be seen to leave few tokens, those are gathered in
//      one CTA by index, the row's weight is summed meanwhile if top-p asks for it, and that CTA
//      ranks them, where a cut may lie among them, and draws.  If they are many, but top-p ends beyond what min-p keeps, step 5
//      follows.  Otherwise:
//   3. the number and the weight of the tokens in bins of d.  With top-k or min-p the cut
//      is near the top: 64 bins to each of 16 octaves, and with top-k what lies below is not
//      even weighed.  Otherwise 32 to each of 32; the rest is added up without bins.  If the cut
//      turns out to lie below, again with 16 bins to each of all 41 octaves;
//   4. the tokens of the bin in which top-k (then top-p) ends are gathered in one CTA, narrowed
//      there by histograms over their keys, and the last few ranked against each other;
//      if they are too many to be gathered, the whole cluster narrows them the same way
//      first; equal logits are counted off by index;
//   5. the sum of what is kept, the target, and the token by a scan in index order.
// Where the tokens down to the first cut's bin are few, one CTA gathers them all after step
// 3 and does the rest with them alone.
// A bin never crosses an octave, so its tokens' weights have one scale: they are summed as
// two 12-bit halves of a 24-bit number by 32-bit atomics without a result.
// Bound for many rows by the arithmetic of the weights (half of it on two logits at once) and
// the exchanges that two CTAs on an SM do not hide, for one row by the exchanges and the fetch
// of instructions that are used once.  Measured: 9.6 us for a row of 128001 with top-k 50 and
// top-p (13.1 without step 2), 133 us for 256 rows of 151936 with top-p and min-p.

#include <cuda_runtime.h>

#include "decode_ops.h"
#include "q4k_ptx.cuh"

namespace q4k {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr int kList = 768;           // tokens of a bin that one CTA gathers
constexpr int kFew = 256;            // tokens that are ranked against each other
constexpr int kMaxCluster = 8;
constexpr int kBests = 128;          // parts of a row whose largest logits bound the k-th from below
constexpr int kTop = 96;             // the largest k for that: some 180 of independent logits lie above the bound
constexpr int kCached = 19328;       // logits of a CTA that stay in shared memory with two CTAs on an SM
constexpr int kCachedOne = 47000;    // and with one
constexpr float kAll = 41.f;         // from this d on the weight is 0
constexpr uint32_t kOne = 1u << 24;
constexpr uint32_t kFull = 0xFFFFFFFFu;

typedef unsigned long long u64;

__device__ __forceinline__ uint32_t key_of(float z) {
    const uint32_t u = __float_as_uint(z);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k >> 31 ? k ^ 0x80000000u : ~k); }
// The negative of a logit, as the row is kept: that of NaN is +inf, that of either zero +0.
__device__ __forceinline__ float stored(float z) { return fminf(0.f - z, INFINITY); }

// Logits 4 i .. 4 i + 3 of a row's part, negated; places outside head .. n - 1 count as -inf.
__device__ __forceinline__ float4 fetch(const float *z, int i, int head, int n) {
    float v[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) v[x] = 4 * i + x >= head && 4 * i + x < n ? stored(__ldg(z + 4 * i + x)) : INFINITY;
    return make_float4(v[0], v[1], v[2], v[3]);
}

// Where the largest logit or 1 / temperature is infinite, every distance is 0 or infinite: the
// row then counts as one of zeros and -inf.  least: the largest logit, negated.
__device__ __forceinline__ float flat(float v, float least) { return v == least ? 0.f : INFINITY; }

// Two fp32 operations at once, each rounded on its own.  A packed product and a packed sum behind it would be compiled
// into one fused operation, .rn or not, which rounds once: the sum of what may be a product is therefore itself written as
// a fused operation, x * one + y, with a 1 that only the launch knows.  (256 rows of 151936 with top-p and min-p: 133 us;
// 126 as it was compiled before, one weight in ten off by a unit; scalar operations, which the compiler leaves alone, take
// 3 % longer than this.)
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    u64 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(*reinterpret_cast<u64 *>(&a)), "l"(*reinterpret_cast<u64 *>(&b)));
    return *reinterpret_cast<float2 *>(&r);
}
__device__ __forceinline__ float2 sum2(float2 a, float2 b) {  // (of no product)
    u64 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(*reinterpret_cast<u64 *>(&a)), "l"(*reinterpret_cast<u64 *>(&b)));
    return *reinterpret_cast<float2 *>(&r);
}
__device__ __forceinline__ float2 fma2_down(float2 a, float2 b, float2 c) {
    u64 r;
    asm("fma.rm.f32x2 %0, %1, %2, %3;"
        : "=l"(r)
        : "l"(*reinterpret_cast<u64 *>(&a)), "l"(*reinterpret_cast<u64 *>(&b)), "l"(*reinterpret_cast<u64 *>(&c)));
    return *reinterpret_cast<float2 *>(&r);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// floor(2^24 2^-f) and n of two distances 0 <= d < 2^22, n = floor(d), f = d - n: the series
// of 2^-f about f = 1/2, coefficients 2^-1/2 (-ln 2)^i / i!.  It lies in [1/2, 1] for every f, where the
// bits of an fp32 number p are 2^24 p + 0x3E800000.
__device__ __forceinline__ void mantissa2(float2 d, float one, uint32_t (&w)[2], uint32_t (&n)[2]) {
    // 2^23 + d, rounded down, is 2^23 + n
    const float2 t = fma2_down(d, both(one), both(8388608.f));
    n[0] = __float_as_uint(t.x) & 0x7FFFFF, n[1] = __float_as_uint(t.y) & 0x7FFFFF;
    const float2 f = sum2(fma2(sum2(t, both(-8388608.f)), both(-1.f), d), both(-0.5f));  // (d - n is exact)
    float2 p = both(-1.0785311133076902e-05f);
    p = fma2(mul2(p, f), both(one), both(0.00010891940473811701f));
    p = fma2(mul2(p, f), both(one), both(-0.0009428249322809279f));
    p = fma2(mul2(p, f), both(one), both(0.006801044102758169f));
    p = fma2(mul2(p, f), both(one), both(-0.03924733027815819f));
    p = fma2(mul2(p, f), both(one), both(0.16986578702926636f));
    p = fma2(mul2(p, f), both(one), both(-0.4901290833950043f));
    p = fma2(mul2(p, f), both(one), both(0.7071067690849304f));
    w[0] = __float_as_uint(p.x) - 0x3E800000u, w[1] = __float_as_uint(p.y) - 0x3E800000u;
}
__device__ __forceinline__ u64 scaled(uint32_t w, uint32_t n) { return ((u64)w << 16) >> n; }
__device__ __forceinline__ u64 weight_of(float d, float one) {  // d < kAll
    uint32_t w[2], n[2];
    mantissa2(both(d), one, w, n);
    return scaled(w[0], n[0]);
}
// floor(total * share / 2^24)
__device__ __forceinline__ u64 part_of(u64 total, uint32_t share) {
    return (total >> 24) * share + (((total & (kOne - 1)) * share) >> 24);
}
// floor(x * 2^24) of x clamped to [0, 1]; NaN gives `none`
__device__ __forceinline__ uint32_t share_of(float x, uint32_t none) {
    return x != x ? none : (uint32_t)(fminf(fmaxf(x, 0.f), 1.f) * 16777216.f);
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}
__device__ __forceinline__ uint32_t peer(const uint32_t *p, uint32_t rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_shared_rank(smem_u32(p), rank)) : "memory");
    return v;
}
__device__ __forceinline__ void peer_store(u64 *p, uint32_t rank, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(map_shared_rank(smem_u32(p), rank)), "l"(v) : "memory");
}
__device__ __forceinline__ void peer_store(uint32_t *p, uint32_t rank, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_shared_rank(smem_u32(p), rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void peer_store(uint4 *p, uint32_t rank, uint4 v) {
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(map_shared_rank(smem_u32(p), rank)), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ u64 list_weight(uint4 t) { return (u64)t.w << 32 | t.z; }
__device__ __forceinline__ uint32_t peer_add(uint32_t *p, uint32_t rank, uint32_t v) {
    uint32_t old;
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(map_shared_rank(smem_u32(p), rank)), "r"(v) : "memory");
    return old;
}

struct Shared {
    uint32_t cnt[kBins], lo[kBins], hi[kBins];  // this CTA's bins: counts, and the halves of 24-bit weights
    uint32_t all_cnt[kBins];                    // the cluster's bins
    u64 all_sum[kBins];
    uint4 list[kList];  // key, index, weight (CTA 0's is used)
    u64 warp_u64[kWarps];
    u64 slot[2][3 * kMaxCluster];  // exchanged values
    alignas(16) uint32_t best[kBests];       // largest keys of parts of the row
    u64 found_sum, ranked_sum;
    uint32_t warp_u32[kWarps];
    uint32_t list_n[2];  // tokens that came for the list (CTA 0's are used): two counters in turn
    uint32_t list_left, own_n;
    uint32_t found_bin, found_cnt, ranked_key, ranked_idx;
};

static_assert(2 * (sizeof(Shared) + 4 * kCached + 1024) <= 233472, "two CTAs on an SM");
static_assert(sizeof(Shared) + 4 * kCachedOne + 1024 <= 233472, "one CTA on an SM");

// A prefix in rank: logits above z, and those equal to it up to index idx.
struct Cut {
    float z;
    uint32_t idx;
    u64 sum;  // its weight
};

template <bool CACHED>
struct Row {
    Shared &s;
    // this CTA's share in groups of four, aligned as the row is in global memory: places outside head .. n - 1
    // hold no logits.  CACHED: in shared memory, negated, +inf in those places
    const float *z;
    uint32_t base;     // index of place 0 (mod 2^32)
    int head, n, n4;   // n4: groups
    uint32_t rank, ctas;
    float top, c;      // largest logit; log2(e) / temperature
    float one;         // 1 (see mul2)
    float infinite;    // not CACHED: the row is to be flattened (see there) about this, unless NaN
    int per_octave;    // log2 of the bins of an octave
    float span;        // bins cover d < span
    int turn, counter;

    // logits 4 i .. 4 i + 3, negated
    __device__ __forceinline__ float4 four(int i) const {
        if constexpr (CACHED) {
            return reinterpret_cast<const float4 *>(z)[i];
        } else {
            float4 v = fetch(z, i, head, n);
            if (infinite == infinite) v = make_float4(flat(v.x, infinite), flat(v.y, infinite), flat(v.z, infinite), flat(v.w, infinite));
            return v;
        }
    }
    // distances of two negated logits; not < kAll (inf or NaN) for a weight of 0
    __device__ __forceinline__ float2 dist2(float a, float b) const {
        return mul2(sum2(both(top), make_float2(a, b)), both(c));
    }
    __device__ __forceinline__ float dist(float a) const { return dist2(a, a).x; }
    // floor(d 2^per_octave) for d < span (the sum has its last bit at 2^-per_octave)
    __device__ __forceinline__ int bin_of(float d) const {
        const float magic = __uint_as_float((uint32_t)(127 + 23 - per_octave) << 23);
        return (int)(__float_as_uint(__fadd_rd(d, magic)) & 0x7FFFFF);
    }
    __device__ __forceinline__ void cover(int log_bins) {
        per_octave = log_bins;
        span = fminf(kAll, (float)(kBins >> log_bins));
    }

    // Every CTA's value (or up to three) to all CTAs, by rank.  Two slots in turn, so one barrier an
    // exchange is enough.
    __device__ __forceinline__ const u64 *exchange(u64 v, u64 v2 = 0, u64 v3 = 0) {
        u64 *slot = s.slot[turn];
        turn ^= 1;
        if (threadIdx.x < ctas) {
            peer_store(slot + rank, threadIdx.x, v);
            peer_store(slot + kMaxCluster + rank, threadIdx.x, v2);
            peer_store(slot + 2 * kMaxCluster + rank, threadIdx.x, v3);
        }
        cluster_sync();
        return slot;
    }
    // The largest of all threads' keys; and those of kBests parts of the row, for kth_best.
    __device__ __forceinline__ uint32_t cluster_best(uint32_t v) {
        const int tid = threadIdx.x, lane = tid & 31;
        const int lanes = (int)ctas * (kThreads / kBests);  // of a part: 4 to 32
        static_assert(kMaxCluster * (kThreads / kBests) == 32 && kBests == 128, "a part within a warp");
        for (int o = 1; o < lanes; o <<= 1) v = max(v, __shfl_xor_sync(kFull, v, o));
        const int mate = tid & (lanes - 1);
        if (mate < (int)ctas) peer_store(&s.best[(rank * kThreads + tid) / lanes], mate, v);
        cluster_sync();
        const uint4 b = reinterpret_cast<const uint4 *>(s.best)[lane];
        return __reduce_max_sync(kFull, max(max(b.x, b.y), max(b.z, b.w)));
    }
    // The k-th largest of the parts' largest keys, 0 < k <= kBests: at least k logits are as large.
    __device__ __forceinline__ uint32_t kth_best(int k) {
        constexpr int TEAM = kThreads / kBests;
        const int i = threadIdx.x / TEAM, mate = threadIdx.x % TEAM;
        const uint32_t me = s.best[i];
        int before = 0;
#pragma unroll
        for (int x = 0; x < kBests / TEAM; x += 4) {
            const int j = x * TEAM + 4 * mate;
            const uint4 b = reinterpret_cast<const uint4 *>(s.best)[j / 4];
            before += (b.x > me || (b.x == me && j < i)) + (b.y > me || (b.y == me && j + 1 < i)) +
                      (b.z > me || (b.z == me && j + 2 < i)) + (b.w > me || (b.w == me && j + 3 < i));
        }
#pragma unroll
        for (int o = 1; o < TEAM; o <<= 1) before += __shfl_xor_sync(kFull, before, o);
        if (mate == 0 && before == k - 1) s.ranked_key = me;
        __syncthreads();
        return s.ranked_key;
    }
    __device__ __forceinline__ u64 block_sum(u64 v) {
        v = warp_sum(v);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) s.warp_u64[threadIdx.x >> 5] = v;
        __syncthreads();
        const int lane = threadIdx.x & 31;
        return warp_sum(lane < kWarps ? s.warp_u64[lane] : 0);
    }
    __device__ __forceinline__ u64 cluster_sum(u64 v) {
        const u64 *all = exchange(block_sum(v));
        u64 t = 0;
        for (uint32_t r = 0; r < ctas; ++r) t += all[r];
        return t;
    }
    __device__ __forceinline__ uint32_t cluster_max(uint32_t v) {
        v = __reduce_max_sync(kFull, v);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) s.warp_u32[threadIdx.x >> 5] = v;
        __syncthreads();
        const int lane = threadIdx.x & 31;
        const u64 *all = exchange(__reduce_max_sync(kFull, lane < kWarps ? s.warp_u32[lane] : 0));
        uint32_t t = 0;
        for (uint32_t r = 0; r < ctas; ++r) t = max(t, (uint32_t)all[r]);
        return t;
    }

    __device__ __forceinline__ void clear_bins() {
        for (int i = threadIdx.x; i < kBins; i += kThreads) s.cnt[i] = s.lo[i] = s.hi[i] = 0;
        __syncthreads();
    }
    __device__ __forceinline__ void into_bin(int bin, uint32_t w, uint32_t n) {
        const uint32_t v = n <= 16 ? w : w >> (n - 16);
        atomicAdd(&s.cnt[bin], 1u);
        atomicAdd(&s.lo[bin], v & 0xFFFu);
        atomicAdd(&s.hi[bin], v >> 12);
    }
    // The CTAs' bins, joined, into all_cnt and all_sum of every CTA; octave(bin): n of its tokens.
    template <typename Octave>
    __device__ __forceinline__ void join_bins(Octave &&octave) {
        cluster_sync();
        // CTA r joins bins [r, r + 1) * share and hands them to all, some threads to a bin, each for
        // some of the CTAs
        const int share = kBins / (int)ctas, team = max(1, kThreads / share), mate = threadIdx.x % team;
        for (int i = threadIdx.x / team; i < share; i += kThreads / team) {
            const int b = (int)rank * share + i;
            u64 w = 0;
            uint32_t k = 0;
#pragma unroll 2
            for (uint32_t r = mate; r < ctas; r += team) {
                const uint32_t kr = peer(&s.cnt[b], r), hr = peer(&s.hi[b], r), lr = peer(&s.lo[b], r);
                k += kr;
                w += ((u64)hr << 12) + lr;
            }
            for (int o = 1; o < team; o <<= 1) {  // (teams lie within a warp, and all of them are here)
                k += __shfl_xor_sync(kFull, k, o);
                w += __shfl_xor_sync(kFull, w, o);
            }
            w <<= max(0, 16 - octave(b));
            for (uint32_t r = mate; r < ctas; r += team) {
                peer_store(&s.all_cnt[b], r, k);
                peer_store(&s.all_sum[b], r, w);
            }
        }
        cluster_sync();
    }
    // Bins of d < edge (edge <= span) over the row, from cleared ones.  Returns this thread's part of the
    // weight beyond (if beyond).
    __device__ __forceinline__ u64 histogram(float edge, bool beyond) {
        u64 tail = 0;
        const float limit = beyond ? kAll : edge;
        for (int i = threadIdx.x; i < n4; i += kThreads) {
            const float4 v = four(i);
            const float x[4] = {v.x, v.y, v.z, v.w};
            u64 below = 0;
#pragma unroll
            for (int h = 0; h < 4; h += 2) {
                const float2 d = dist2(x[h], x[h + 1]);
                if (!(d.x < limit || d.y < limit)) continue;
                uint32_t w[2], oct[2];
                mantissa2(make_float2(d.x < kAll ? d.x : 0.f, d.y < kAll ? d.y : 0.f), one, w, oct);
                const float dd[2] = {d.x, d.y};
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (dd[e] < edge) into_bin(bin_of(dd[e]), w[e], oct[e]);
                    else if (dd[e] < limit) below += scaled(w[e], oct[e]);
                }
            }
            tail += below;
        }
        join_bins([&](int b) { return b >> per_octave; });
        return tail;
    }

    // The bin in which the running count (by_sum: weight), beginning with cnt (sum), reaches
    // `need`, or bin `last` before that: its number, and the count and weight before it in cnt and sum.
    // -1: none does.  own: of this CTA's bins (weights scaled by 2^up), otherwise of the cluster's.
    __device__ __forceinline__ int find_bin(bool by_sum, u64 need, int last, u64 &cnt, u64 &sum, bool own = false, int up = 0) {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        static_assert(kBins == 2 * kThreads, "two bins a thread");
        uint32_t k[2];
        u64 w[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            k[x] = own ? s.cnt[2 * tid + x] : s.all_cnt[2 * tid + x];
            w[x] = own ? (((u64)s.hi[2 * tid + x] << 12) + s.lo[2 * tid + x]) << up : s.all_sum[2 * tid + x];
        }
        uint32_t ki = k[0] + k[1];
        u64 wi = w[0] + w[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t kt = __shfl_up_sync(kFull, ki, o);
            const u64 wt = __shfl_up_sync(kFull, wi, o);
            if (lane >= o) ki += kt, wi += wt;
        }
        __syncthreads();
        if (lane == 31) s.warp_u32[warp] = ki, s.warp_u64[warp] = wi;
        if (tid == 0) s.found_bin = kBins;
        __syncthreads();
        const uint32_t kb = __reduce_add_sync(kFull, lane < warp ? s.warp_u32[lane] : 0u);
        const u64 wb = warp_sum(lane < warp ? s.warp_u64[lane] : 0ull);
        u64 c0 = cnt + kb + ki - k[0] - k[1], s0 = sum + wb + wi - w[0] - w[1];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const u64 at = by_sum ? s0 : c0, to = at + (by_sum ? w[x] : k[x]);
            if (at < need && (2 * tid + x == last || (need <= to && 2 * tid + x < last))) {
                s.found_bin = 2 * tid + x;
                s.found_cnt = (uint32_t)c0;
                s.found_sum = s0;
            }
            c0 += k[x], s0 += w[x];
        }
        __syncthreads();
        const int bin = (int)s.found_bin;
        if (bin == kBins) return -1;
        cnt = s.found_cnt;
        sum = s.found_sum;
        return bin;
    }

    // Where, by index, the running sum of value4(negated logits, index, values) over the whole row
    // first exceeds target(total).  Returns true, in one warp of one CTA, with the index and its value.
    template <typename Value, typename Target>
    __device__ __forceinline__ bool locate(Value &&value4, Target &&target, uint32_t &idx, u64 &val, u64 &total) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int per = (n4 + kThreads - 1) / kThreads * 32;  // a warp's run of groups
        const int i0 = min(warp * per, n4), i1 = min(i0 + per, n4);
        u64 sum = 0;
        for (int i = i0 + lane; i < i1; i += 32) {
            u64 v[4];
            value4(four(i), base + 4 * i, v);
            sum += v[0] + v[1] + v[2] + v[3];
        }
        const u64 *all = exchange(block_sum(sum));
        u64 before = 0;
        total = 0;
        for (uint32_t r = 0; r < ctas; ++r) {
            if (r < rank) before += all[r];
            total += all[r];
        }
        const u64 goal = target(total);
        before += warp_sum(lane < warp ? s.warp_u64[lane] : 0ull);
        const u64 mine = s.warp_u64[warp];
        if (!(before <= goal && goal < before + mine)) return false;
        for (int j = i0; j < i1; j += 32) {
            const int i = j + lane;
            u64 v[4] = {0, 0, 0, 0};
            if (i < i1) value4(four(i), base + 4 * i, v);
            const u64 own = v[0] + v[1] + v[2] + v[3];
            u64 inc = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 t = __shfl_up_sync(kFull, inc, o);
                if (lane >= o) inc += t;
            }
            const uint32_t over = __ballot_sync(kFull, before + inc > goal);
            if (over) {
                u64 run = before + inc - own;
                int x = 0;
#pragma unroll
                for (int y = 0; y < 3; ++y)
                    if (x == y && run + v[y] <= goal) run += v[y], ++x;
                const u64 mine_v = x == 0 ? v[0] : x == 1 ? v[1] : x == 2 ? v[2] : v[3];
                const int l = __ffs(over) - 1;
                idx = __shfl_sync(kFull, base + 4 * i + x, l);
                val = __shfl_sync(kFull, mine_v, l);
                return true;
            }
            before += __shfl_sync(kFull, inc, 31);
        }
        return false;
    }

    // Tokens from <= d < to, of a key in [lo, hi]: their number, and themselves in CTA 0's list as far as it
    // holds them.  visit(index, key, d)
    template <typename Visit>
    __device__ __forceinline__ void each(float from, float to, uint32_t lo, uint32_t hi, Visit &&visit) {
        for (int i = threadIdx.x; i < n4; i += kThreads) {
            const float4 v = four(i);
            const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int h = 0; h < 4; h += 2) {
                const float2 d = dist2(x[h], x[h + 1]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float de = e ? d.y : d.x;
                    if (!(de >= from && de < to)) continue;
                    const uint32_t key = key_of(-x[h + e]);
                    if (key >= lo && key <= hi) visit(base + 4 * i + h + e, key, de);
                }
            }
        }
    }
    __device__ __forceinline__ int gather(float from, float to, uint32_t lo, uint32_t hi) {
        each(from, to, lo, hi, [&](uint32_t idx, uint32_t key, float d) {
            const uint32_t at = peer_add(&s.list_n[counter], 0, 1);
            if (at < kList) {
                const u64 w = weight_of(d, one);
                peer_store(&s.list[at], 0, make_uint4(key, idx, (uint32_t)w, (uint32_t)(w >> 32)));
            }
        });
        cluster_sync();
        const int m = (int)peer(&s.list_n[counter], 0);
        counter ^= 1;  // the other one's readers are past the barrier, and its next users behind another
        if (rank == 0 && threadIdx.x == 0) s.list_n[counter] = 0;
        return m;
    }
    // Tokens of d < to and no logit below -zc, into CTA 0's list by index, if they are at most kFew: their
    // number.  weigh: their weight and the row's, too.
    __device__ __forceinline__ int collect(float zc, float to, bool weigh, u64 &reach, u64 &whole) {
        u64 *own = s.all_sum;  // (not in use before the bins are joined, and after the last look at them)
        u64 sum = 0, in = 0;
        for (int i = threadIdx.x; i < n4; i += kThreads) {
            const float4 v = four(i);
            const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int h = 0; h < 4; h += 2) {
                const float2 d = dist2(x[h], x[h + 1]);
                u64 w[2] = {0, 0};
                if (weigh) {
                    uint32_t wm[2], oct[2];
                    mantissa2(make_float2(fminf(d.x, 60.f), fminf(d.y, 60.f)), one, wm, oct);  // (from kAll on, 0)
                    w[0] = scaled(wm[0], oct[0]), w[1] = scaled(wm[1], oct[1]);
                    sum += w[0] + w[1];
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (!(x[h + e] <= zc && (e ? d.y : d.x) < to)) continue;
                    const uint32_t at = atomicAdd(&s.own_n, 1u);
                    if (at < kFew) own[at] = (u64)__float_as_uint(x[h + e]) << 32 | (base + 4 * i + h + e);
                    in += w[e];
                }
            }
        }
        sum = block_sum(sum);
        if (weigh) in = block_sum(in);
        const int m = (int)s.own_n;
        const u64 *all = exchange(sum, m, in);
        if (threadIdx.x == 0) s.own_n = 0;
        int n = 0, at = 0;
        for (uint32_t r = 0; r < ctas; ++r) {
            if (r < rank) at += (int)all[kMaxCluster + r];
            n += (int)all[kMaxCluster + r];
            if (weigh) whole += all[r], reach += all[2 * kMaxCluster + r];
        }
        if (n > kFew) return n;
        int team = 1;  // neighbouring lanes that count the tokens before one
        while (team < 32 && 2 * team * m <= kThreads) team *= 2;
        const int mate = threadIdx.x & (team - 1), i = threadIdx.x / team;
        static_assert(kFew <= kThreads, "one token a thread");
        if (m > 0) {
            const u64 me = own[min(i, m - 1)];
            int before = 0;
            for (int j = mate; j < m; j += team) before += (uint32_t)own[j] < (uint32_t)me ? 1 : 0;
            for (int o = 1; o < team; o <<= 1) before += __shfl_xor_sync(kFull, before, o);
            if (i < m && mate == 0) {
                const float x = __uint_as_float((uint32_t)(me >> 32));
                const u64 w = weight_of(dist(x), one);
                peer_store(&s.list[at + before], 0, make_uint4(key_of(-x), (uint32_t)me, (uint32_t)w, (uint32_t)(w >> 32)));
            }
        }
        cluster_sync();
        return n;
    }
    // Over the m tokens of CTA 0's list (m < 2^16; every thread of it calls): done(i, t, count, sum) for
    // each token t, with the number and the weight of the tokens that before(other, t) names.  A token is
    // the work of a few neighbouring lanes, one of which calls done.
    template <typename Before, typename Done>
    __device__ __forceinline__ void compare_all(int m, Before &&before, Done &&done) {
        int team = 1;
        while (team < 32 && 2 * team * m <= kThreads) team *= 2;
        const int mate = threadIdx.x & (team - 1);
        for (int i0 = 0; i0 < m; i0 += kThreads / team) {
            const int i = i0 + threadIdx.x / team;
            const uint4 me = s.list[min(i, m - 1)];
            uint32_t k = 0;
            u64 w = 0;
#pragma unroll 8
            for (int j = mate; j < m; j += team) {
                const uint4 t = s.list[j];
                const bool is = before(t, me);
                k += is ? 1u : 0u;
                w += is ? list_weight(t) : 0ull;
            }
            for (int o = 1; o < team; o <<= 1) {
                k += __shfl_xor_sync(kFull, k, o);
                w += __shfl_xor_sync(kFull, w, o);
            }
            if (i < m && mate == 0) done(i, me, k, w);
        }
    }
    static __device__ __forceinline__ bool ranks_before(uint4 a, uint4 b) { return a.x > b.x || (a.x == b.x && a.y < b.y); }

    // The token of bin `bin` (of d) with which the running count (weight) reaches `need`, cnt and
    // sum being those before the bin.
    __device__ __forceinline__ Cut refine(bool by_sum, int bin, u64 need, u64 cnt, u64 sum) {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        const int octave = bin >> per_octave;
        uint32_t lo = 0, hi = 0xFFFFFFFFu;  // keys of the bin that are left
        const float from = ldexpf((float)bin, -per_octave), to = fminf(span, ldexpf((float)(bin + 1), -per_octave));
        for (;;) {
            int m = gather(from, to, lo, hi);  // in CTA 0, if they are few
            if (m <= kList) {
                if (rank == 0) {
                    const int up = max(0, 16 - octave);
                    while (m > kFew) {
                        // narrow by a histogram over the keys, from the largest down
                        uint32_t a = 0, b = 0;
                        for (int i = tid; i < m; i += kThreads) {
                            const uint32_t key = s.list[i].x;
                            if (key >= lo && key <= hi) a = max(a, key), b = max(b, ~key);
                        }
                        a = __reduce_max_sync(kFull, a), b = __reduce_max_sync(kFull, b);
                        if (lane == 0) s.warp_u64[warp] = (u64)a << 32 | b;
                        clear_bins();
                        a = __reduce_max_sync(kFull, (uint32_t)(s.warp_u64[lane & (kWarps - 1)] >> 32));
                        b = __reduce_max_sync(kFull, (uint32_t)s.warp_u64[lane & (kWarps - 1)]);
                        hi = a, lo = ~b;
                        if (lo == hi) break;  // equal logits: ranked by index below
                        const int shift = max(0, 32 - __clz(hi - lo) - 10);
                        for (int i = tid; i < m; i += kThreads) {
                            const uint4 t = s.list[i];
                            if (t.x < lo || t.x > hi) continue;
                            const int bin = (int)((hi - t.x) >> shift);
                            const uint32_t v = (uint32_t)(list_weight(t) >> up);
                            atomicAdd(&s.cnt[bin], 1u);
                            atomicAdd(&s.lo[bin], v & 0xFFFu);
                            atomicAdd(&s.hi[bin], v >> 12);
                        }
                        __syncthreads();
                        const uint32_t sub = (uint32_t)max(find_bin(by_sum, need, kBins, cnt, sum, true, up), 0);
                        hi -= sub << shift;
                        lo = hi - min(hi - lo, (1u << shift) - 1);
                        // the tokens of that bin alone stay in the list
                        uint4 t[(kList + kThreads - 1) / kThreads];
#pragma unroll
                        for (int x = 0; x < (kList + kThreads - 1) / kThreads; ++x) t[x] = s.list[min(tid + x * kThreads, m - 1)];
                        if (tid == 0) s.list_left = 0;
                        __syncthreads();
#pragma unroll
                        for (int x = 0; x < (kList + kThreads - 1) / kThreads; ++x)
                            if (tid + x * kThreads < m && t[x].x >= lo && t[x].x <= hi) s.list[atomicAdd(&s.list_left, 1u)] = t[x];
                        __syncthreads();
                        m = (int)s.list_left;
                        __syncthreads();  // (list_left and warp_u64 are written again)
                    }
                    // what is left is ranked against all of it
                    compare_all(m, ranks_before, [&](int, uint4 t, uint32_t k, u64 w) {
                        const u64 w1 = sum + w + list_weight(t);
                        if (by_sum ? sum + w < need && need <= w1 : cnt + k + 1 == need)
                            for (uint32_t r = 0; r < ctas; ++r) {
                                peer_store(&s.ranked_key, r, t.x);
                                peer_store(&s.ranked_idx, r, t.y);
                                peer_store(&s.ranked_sum, r, w1);
                            }
                    });
                }
                cluster_sync();
                return {of_key(s.ranked_key), s.ranked_idx, s.ranked_sum};
            }
            // many: a histogram over their keys, from the largest down
            uint32_t a = 0, b = 0;
            each(from, to, lo, hi, [&](uint32_t, uint32_t key, float) { a = max(a, key), b = max(b, ~key); });
            a = cluster_max(a);
            lo = ~cluster_max(b);
            hi = a;
            if (lo == hi) break;
            const int shift = max(0, 32 - __clz(hi - lo) - 10);
            clear_bins();
            each(from, to, lo, hi, [&](uint32_t, uint32_t key, float d) {
                uint32_t w[2], oct[2];
                mantissa2(both(d), one, w, oct);
                into_bin((int)((hi - key) >> shift), w[0], oct[0]);
            });
            join_bins([&](int) { return octave; });
            const uint32_t sub = (uint32_t)max(find_bin(by_sum, need, kBins, cnt, sum), 0);
            hi -= sub << shift;
            lo = hi - min(hi - lo, (1u << shift) - 1);
        }
        // equal logits: the q-th by index
        const float z0 = of_key(hi);
        const u64 w = weight_of(dist(-z0), one);
        const u64 q = by_sum ? (need - sum + w - 1) / w : need - cnt;
        uint32_t idx;
        u64 val, total;
        const bool here = locate(
            [&](float4 v, uint32_t, u64 (&is)[4]) { is[0] = -v.x == z0, is[1] = -v.y == z0, is[2] = -v.z == z0, is[3] = -v.w == z0; },
            [&](u64) { return q - 1; }, idx, val, total);
        if (here && (uint32_t)lane < ctas) peer_store(&s.ranked_idx, lane, idx);
        cluster_sync();
        return {z0, s.ranked_idx, sum + q * w};
    }
};

struct Settings {
    int32_t k;
    uint32_t p_share, m_share, u;
    bool by_k, by_p;
};

// The row's token from the n tokens of CTA 0's list alone, which are in order and hold everything that
// top-k, or without it top-p, or min-p keeps.  whole: without top-k, the weight of the row; reach: the
// tokens' own, or 0.
template <typename R>
__device__ __forceinline__ void finish_few(R &r, const SampleArgs &a, int64_t m, const Settings &set, int n, u64 whole, u64 reach, u64 least) {
    Shared &s = r.s;
    if (r.rank != 0) return;  // (no CTA touches another's memory from here on)
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint4 mine = s.list[min(tid, kList - 1)];
    u64 weight = tid < n ? list_weight(mine) : 0;
    // each token's rank, and the weight before it, where a cut may lie among them
    u64 need = set.by_p ? max(part_of(whole, set.p_share), (u64)1) : 0;
    if (set.by_k ? set.by_p || n > set.k : set.by_p && (reach == 0 || reach > need)) {
        r.compare_all(n, R::ranks_before, [&](int i, uint4, uint32_t k, u64 w) { s.all_cnt[i] = k, s.all_sum[i] = w; });
        __syncthreads();
        if (set.by_k) {
            if (tid < n && s.all_cnt[tid] >= (uint32_t)set.k) weight = 0;
            if (set.by_p) need = max(part_of(r.block_sum(weight), set.p_share), (u64)1);
        }
        if (set.by_p && tid < n && s.all_sum[tid] >= need) weight = 0;
    }
    if (weight < least) weight = 0;
    const u64 total = r.block_sum(weight), goal = part_of(total, set.u);
    u64 to = weight;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 t = __shfl_up_sync(kFull, to, o);
        if (lane >= o) to += t;
    }
    to += warp_sum(lane < warp ? s.warp_u64[lane] : 0ull);
    if (to - weight <= goal && goal < to) {
        a.token[m] = (int32_t)mine.y;
        if (a.prob) a.prob[m] = __fdiv_rn((float)weight, (float)total);
    }
}

// The row's cut and its token, after the load.
template <typename R>
__device__ __forceinline__ void finish(R &r, const SampleArgs &a, int64_t m, const Settings &set, bool finite) {
    Shared &s = r.s;
    const int tid = threadIdx.x, lane = tid & 31;
    Cut cut = {-INFINITY, 0xFFFFFFFFu, 0};
    // First the cut of top-k, if any, then that of top-p: each phase's code is there once (inlined twice, a
    // single row waits longer for instructions than for anything else).
    bool by_sum = !set.by_k, bins = false, all = false;
    u64 part = 0, whole = 0, reach = 0;  // whole: what top-k keeps
    const u64 least = (u64)set.m_share << 16;  // (the largest weight is 2^40)
    // from this d on, w is below 2^(40 - limit) <= least / 2 (the series errs by far less than a factor 2)
    const float limit = least > 0 ? fminf(kAll, 41.f - (float)(63 - __clzll((long long)least))) : kAll;
    const bool bounded = limit < 16.f;
    // Where top-k or min-p can be seen to leave few tokens, those alone.
    int few = kFew + 1;
    const bool by_best = finite && set.by_k && set.k <= kTop, last_k = !set.by_p, weigh = !set.by_k && set.by_p;
    if (by_best || (bounded && !set.by_k))
        few = r.collect(by_best ? -of_key(r.kth_best(set.k)) : INFINITY, weigh || last_k ? limit : kAll, weigh, reach, whole);
    r.cover(set.by_k || bounded ? 6 : 5);
    // (nor need a cut of top-p be found that lies beyond what min-p keeps)
    while (few > kFew && (set.by_k || (set.by_p && !(weigh && bounded && reach < part_of(whole, set.p_share))))) {
        // where the last cut lies beyond what min-p keeps, it need not be found
        const int last = bounded && (by_sum || !set.by_p) ? r.bin_of(limit) : kBins;
        if (!bins) part = r.histogram(fminf(r.span, ldexpf((float)(last + 1), -r.per_octave)), !set.by_k && whole == 0);
        bins = true;
        if (by_sum && whole == 0) {
            if (r.rank == 0)  // (the bins are the cluster's)
                for (int i = tid; i < kBins; i += kThreads) part += s.all_sum[i];
            whole = r.cluster_sum(part);
        }
        const u64 need = by_sum ? max(part_of(whole, set.p_share), (u64)1) : (u64)set.k;
        u64 cnt = 0, sum = 0;
        const int bin = r.find_bin(by_sum, need, last, cnt, sum);
        if (bin < 0 && !all) {
            // beyond the bins: bins of every weight
            all = true;
            bins = false;
            r.cover(4);
            r.clear_bins();
            continue;
        }
        if (bin >= 0 && by_sum != set.by_k && cnt + s.all_cnt[bin] <= (u64)kFew) {
            reach = 0;
            few = r.collect(INFINITY, fminf(r.span, ldexpf((float)(bin + 1), -r.per_octave)), false, reach, part);
            break;
        }
        // (-1: fewer than k tokens have any weight)
        if (bin >= 0 && (by_sum ? sum + s.all_sum[bin] : cnt + s.all_cnt[bin]) >= need) {
            // where there are too many to gather, bins over keys take the place of those over d
            bins = !by_sum && s.all_cnt[bin] <= kList;
            cut = r.refine(by_sum, bin, need, cnt, sum);
            whole = cut.sum;
            if (!bins) r.clear_bins();
        }
        if (by_sum || !set.by_p) break;
        by_sum = true;
    }
    if (few <= kFew) {
        finish_few(r, a, m, set, few, whole, reach, least);
        return;
    }
    // ---- the token
    const float zc = -cut.z;
    uint32_t idx;
    u64 w, total;
    const bool here = r.locate(
        [&](float4 v, uint32_t i, u64 (&x)[4]) {
            const float z[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int h = 0; h < 4; h += 2) {
                x[h] = x[h + 1] = 0;
                const float2 d = r.dist2(z[h], z[h + 1]);
                if (!((z[h] <= zc && d.x < limit) || (z[h + 1] <= zc && d.y < limit))) continue;
                uint32_t wm[2], n[2];
                mantissa2(make_float2(d.x < kAll ? d.x : 0.f, d.y < kAll ? d.y : 0.f), r.one, wm, n);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const bool in = z[h + e] < zc || (z[h + e] == zc && i + h + e <= cut.idx);
                    const u64 we = scaled(wm[e], n[e]);
                    if (in && (e ? d.y : d.x) < limit && we >= least) x[h + e] = we;
                }
            }
        },
        [&](u64 all) { return part_of(all, set.u); }, idx, w, total);
    if (here && lane == 0) {
        a.token[m] = (int32_t)idx;
        if (a.prob) a.prob[m] = __fdiv_rn((float)w, (float)total);
    }
}

template <bool CACHED>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a, int per) {
    extern __shared__ __align__(16) uint8_t dyn[];
    Shared &s = *reinterpret_cast<Shared *>(dyn);
    float *own = reinterpret_cast<float *>(dyn + (sizeof(Shared) + 15) / 16 * 16);
    const int tid = threadIdx.x;
    const uint32_t rank = cluster_ctarank(), ctas = a.ctas;
    if (tid == 0) s.list_n[0] = s.list_n[1] = s.own_n = 0;
    for (int i = tid; i < kBins; i += kThreads) s.cnt[i] = s.lo[i] = s.hi[i] = 0;
    cluster_arrive();  // (waited for before the first access to another CTA's memory)
    pdl_wait();
    pdl_trigger();
    const int64_t m = blockIdx.x / ctas;
    const int64_t i0 = min((int64_t)rank * per, (int64_t)a.V), i1 = min(i0 + per, (int64_t)a.V);
    const float *row = a.logits + m * a.ldl + i0;
    const int head = (int)(reinterpret_cast<uintptr_t>(row) % 16 / 4), n = (int)(i1 - i0) + head;
    row -= head;
    Row<CACHED> r = {s, CACHED ? own : row, (uint32_t)i0 - head, head, n, (n + 3) / 4, rank, ctas, 0.f, 0.f, a.one, NAN, 0, 0.f, 0, 0};
    // ---- the row's settings
    float t = a.temperature ? __ldg(a.temperature + m) : 1.f;
    const bool greedy = !(t > 0.f);
    if (greedy) t = 1.f;
    r.c = __fmul_rn(__fdiv_rn(1.f, t), 1.4426950408889634f);
    Settings set;
    set.k = greedy ? 1 : a.top_k ? __ldg(a.top_k + m) : 0;
    set.p_share = greedy || !a.top_p ? kOne : share_of(__ldg(a.top_p + m), kOne);
    set.m_share = greedy || !a.min_p ? 0 : share_of(__ldg(a.min_p + m), 0);
    set.u = min(share_of(__ldg(a.u + m), 0), kOne - 1);
    set.by_k = set.k > 0 && set.k < a.V;
    set.by_p = set.p_share < kOne;
    // ---- load; the largest logit
    float best = INFINITY;  // (of the negated ones, the smallest)
    auto take = [&](int i, float4 v) {
        if (CACHED) reinterpret_cast<float4 *>(own)[i] = v;
        best = fminf(fminf(best, fminf(v.x, v.y)), fminf(v.z, v.w));
    };
    const int whole0 = head > 0 ? 1 : 0, whole1 = n / 4;  // groups full of logits
#pragma unroll 4
    for (int i = whole0 + tid; i < whole1; i += kThreads) {
        const float4 v = __ldg(reinterpret_cast<const float4 *>(row) + i);
        take(i, make_float4(stored(v.x), stored(v.y), stored(v.z), stored(v.w)));
    }
    if (tid < 2) {  // the first and the last group, where they are not
        const int i = tid == 0 ? 0 : whole1;
        if (tid == 0 ? whole0 > 0 : whole1 < r.n4) take(i, fetch(row, i, head, n));
    }
    cluster_wait();
    r.top = of_key(r.cluster_best(key_of(-best)));
    if (r.top == -INFINITY) {
        if (rank == 0 && tid == 0) {
            a.token[m] = -1;
            if (a.prob) a.prob[m] = 0.f;
        }
        return;
    }
    const bool finite = !isinf(r.top) && !isinf(r.c);
    if (!finite) {
        const float least = -r.top;
        __syncthreads();
        if (CACHED)
            for (int i = tid; i < r.n4 * 4; i += kThreads) own[i] = flat(own[i], least);
        else r.infinite = least;
        r.top = 0.f, r.c = 1.f;
        __syncthreads();
    }
    finish(r, a, m, set, finite);
}

}  // namespace

cudaError_t launch_sample(const DeviceInfo &di, const SampleArgs &args, cudaStream_t s) {
    SampleArgs a = args;
    a.one = 1.f;
    // CTAs of a row: up to eight, a few thousand logits each at least; fewer where the rows fill the
    // device by themselves, as long as a row stays in shared memory
    a.ctas = a.V <= 4096 ? 1 : a.V <= 8192 ? 2 : a.V <= 16384 ? 4 : 8;
    while (a.ctas > 1 && a.M * a.ctas > 2 * di.sm_count && a.V <= (int64_t)(a.ctas / 2) * (kCached - 8)) a.ctas /= 2;
    const int per = ((a.V + a.ctas - 1) / a.ctas + 3) / 4 * 4;
    // A share stays in shared memory where that costs no CTA its place on an SM (the other way about, 10 rows
    // of 164899 with top-k 400 took 44 us instead of 30, 174 of 176233 took 334 instead of 232).  It may
    // begin inside a group.
    const bool cached = per + 4 <= (a.M * a.ctas <= di.sm_count ? kCachedOne : kCached);
    const int smem = (int)((sizeof(Shared) + 15) / 16 * 16) + (cached ? (per + 4) * 4 : 0);
    auto kern = cached ? sample_kernel<true> : sample_kernel<false>;
    cudaError_t e = ensure_smem((const void *)kern, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3((unsigned)(a.M * a.ctas)), dim3(kThreads), smem, s, dim3(a.ctas), a, per);
}

}  // namespace q4k
