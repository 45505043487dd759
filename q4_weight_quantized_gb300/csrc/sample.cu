// Sampling with temperature, top-k, top-p and min-p from given random numbers.
//
// The row's weights are whole numbers w = floor(2^(40 - d)), d = (z_max - z) / (T ln 2),
// so sums are exact in any order and every decision (which tokens top-p keeps, which
// one the random number falls on) is an integer comparison: the token does not depend
// on how the work is split.  What is kept by top-k and top-p is a prefix in rank (logit
// descending, index ascending), so all that has to be found is where it ends.
//
// A cluster of CTAs owns a row: each keeps its contiguous share of the logits in shared
// memory, so the row is read from global memory once, and the CTAs exchange bins, sums
// and cuts through distributed shared memory.
//   1. load, largest logit;
//   2. counts and weights per bin of d (monotone in the logit), at first only for d <
//      kHead: the tail's weight, which rarely matters for the cut, is added up in
//      registers without atomics; if the cut turns out to lie in the tail, again with
//      all of d < 41;
//   3. the bin in which top-k (then top-p) ends; its tokens, if few, are ranked against
//      each other; if many, the bin is narrowed by histograms over their keys first;
//      equal logits are counted off by index;
//   4. the sum of what is kept, the target, and the token by a scan in index order.
// Bound by the arithmetic of the weights (about 40 instructions a logit) for many rows
// and by the latency of the cluster's exchanges for one.
#include <cuda_runtime.h>

#include "decode_ops.h"
#include "q4k_ptx.cuh"

namespace q4k {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr int kList = 512;             // tokens of a bin that are ranked against each other
constexpr int kMaxCluster = 8;
constexpr int kCached = 19456;         // logits of a CTA that stay in shared memory with two CTAs on an SM
constexpr float kHead = 12.f;          // d below which a token's bin is counted at once
constexpr float kAll = 41.f;           // from here on the weight is 0
constexpr uint32_t kOne = 1u << 24;

typedef unsigned long long u64;

__device__ __forceinline__ uint32_t key_of(float z) {
    const uint32_t u = __float_as_uint(z);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float clean(float z) { return z != z ? -INFINITY : z + 0.f; }  // NaN is -inf, -0 is +0

// 2^-1/2 (-ln 2)^i / i!: the series of 2^-f about f = 1/2
__device__ __forceinline__ u64 weight_of(float d) {
    const float n = floorf(d), f = __fsub_rn(__fsub_rn(d, n), 0.5f);
    float p = -1.0785311133076902e-05f;
    p = __fadd_rn(__fmul_rn(p, f), 0.00010891940473811701f);
    p = __fadd_rn(__fmul_rn(p, f), -0.0009428249322809279f);
    p = __fadd_rn(__fmul_rn(p, f), 0.006801044102758169f);
    p = __fadd_rn(__fmul_rn(p, f), -0.03924733027815819f);
    p = __fadd_rn(__fmul_rn(p, f), 0.16986578702926636f);
    p = __fadd_rn(__fmul_rn(p, f), -0.4901290833950043f);
    p = __fadd_rn(__fmul_rn(p, f), 0.7071067690849304f);
    return ((u64)(uint32_t)__fmul_rn(p, 16777216.f) << 16) >> (int)n;
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
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
template <typename T>
__device__ __forceinline__ T peer(T *p, uint32_t rank) {
    const uint32_t at = map_shared_rank(smem_u32(p), rank);
    T v;
    if constexpr (sizeof(T) == 8) {
        u64 t;
        asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(t) : "r"(at) : "memory");
        v = *reinterpret_cast<T *>(&t);
    } else {
        uint32_t t;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(t) : "r"(at) : "memory");
        v = *reinterpret_cast<T *>(&t);
    }
    return v;
}
__device__ __forceinline__ void peer_store(u64 *p, uint32_t rank, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(map_shared_rank(smem_u32(p), rank)), "l"(v) : "memory");
}
__device__ __forceinline__ void peer_store(uint32_t *p, uint32_t rank, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_shared_rank(smem_u32(p), rank)), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t peer_add(uint32_t *p, uint32_t rank, uint32_t v) {
    uint32_t old;
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(map_shared_rank(smem_u32(p), rank)), "r"(v) : "memory");
    return old;
}

struct Shared {
    uint32_t cnt[kBins], lo[kBins], hi[kBins];  // this CTA's bins: counts, and weights as two words carried by hand
    uint32_t all_cnt[kBins];                    // the cluster's bins
    u64 all_sum[kBins];
    uint32_t list_key[kList], list_idx[kList];  // (CTA 0's are used)
    u64 list_w[kList];
    uint32_t list_n;
    uint32_t warp_u32[kWarps];
    u64 warp_u64[kWarps];
    u64 slot[2][kMaxCluster];  // exchanged values
    u64 found_sum, ranked_sum;
    uint32_t found_bin, found_cnt, ranked_key, ranked_idx;
    int has;
};

// A prefix in rank: the bins below `bin` whole, and of bin `bin` the keys above `key` and
// those equal to it up to index `idx`.  bin = kBins + 1: no cut.
struct Cut {
    int bin;
    uint32_t key, idx;
    u64 sum;  // its weight
};

template <bool CACHED>
struct Row {
    Shared &s;
    const float *z;  // this CTA's share of the logits: in shared memory, or the row itself
    uint32_t base;   // index of its first
    int n;
    uint32_t rank, ctas;
    float top, c;    // largest logit; log2(e) / temperature
    float span, scale;  // bins cover d < span
    int turn;

    __device__ __forceinline__ float at(int i) const { return CACHED ? z[i] : clean(__ldg(z + i)); }
    __device__ __forceinline__ float dist(float v) const { return v == top ? 0.f : __fmul_rn(__fsub_rn(top, v), c); }
    __device__ __forceinline__ int bin_of(float d) const { return d < span ? min((int)(d * scale), kBins - 1) : kBins; }

    // Every CTA's value (its thread 0's) to all CTAs, by rank.  Two slots in turn, so one
    // barrier an exchange is enough.
    __device__ __forceinline__ const u64 *exchange(u64 v) {
        u64 *slot = s.slot[turn];
        turn ^= 1;
        if (threadIdx.x < ctas) peer_store(slot + rank, threadIdx.x, v);
        cluster_sync();
        return slot;
    }
    __device__ __forceinline__ u64 block_sum(u64 v) {
        v = warp_sum(v);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) s.warp_u64[threadIdx.x >> 5] = v;
        __syncthreads();
        return warp_sum(s.warp_u64[threadIdx.x & 31]);
    }
    __device__ __forceinline__ u64 cluster_sum(u64 v) {
        const u64 *all = exchange(block_sum(v));
        u64 t = 0;
        for (uint32_t r = 0; r < ctas; ++r) t += all[r];
        return t;
    }
    __device__ __forceinline__ uint32_t cluster_max(uint32_t v) {
        v = __reduce_max_sync(0xFFFFFFFFu, v);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) s.warp_u32[threadIdx.x >> 5] = v;
        __syncthreads();
        const u64 *all = exchange(__reduce_max_sync(0xFFFFFFFFu, s.warp_u32[threadIdx.x & 31]));
        uint32_t t = 0;
        for (uint32_t r = 0; r < ctas; ++r) t = max(t, (uint32_t)all[r]);
        return t;
    }

    // Counts and weights of the bins that pick(logit, bin, w) names (false: none), joined over
    // the cluster into all_cnt and all_sum of every CTA.
    template <typename Pick>
    __device__ __forceinline__ void histogram(Pick &&pick) {
        const int tid = threadIdx.x;
        for (int i = tid; i < kBins; i += kThreads) s.cnt[i] = s.lo[i] = s.hi[i] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kThreads) {
            int bin;
            u64 w;
            if (!pick(at(i), bin, w)) continue;
            atomicAdd(&s.cnt[bin], 1u);
            const uint32_t low = (uint32_t)w, old = atomicAdd(&s.lo[bin], low);
            const uint32_t high = (uint32_t)(w >> 32) + (old + low < old ? 1u : 0u);
            if (high) atomicAdd(&s.hi[bin], high);
        }
        cluster_sync();
        // CTA r joins bins [r, r + 1) * kBins / ctas and hands them to all
        const int share = kBins / (int)ctas;
        for (int i = tid; i < share; i += kThreads) {
            const int b = (int)rank * share + i;
            u64 w = 0;
            uint32_t k = 0;
            for (uint32_t r = 0; r < ctas; ++r) {
                k += peer(&s.cnt[b], r);
                w += ((u64)peer(&s.hi[b], r) << 32) + peer(&s.lo[b], r);
            }
            for (uint32_t r = 0; r < ctas; ++r) {
                peer_store(&s.all_cnt[b], r, k);
                peer_store(&s.all_sum[b], r, w);
            }
        }
        cluster_sync();
    }

    // The bin in which the running count (BY_SUM: weight), beginning with cnt (sum), reaches
    // `need`: its number, and the count and weight before it in cnt and sum.  -1: none does.
    template <bool BY_SUM>
    __device__ __forceinline__ int find_bin(u64 need, u64 &cnt, u64 &sum) {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        static_assert(kBins == kThreads, "a bin per thread");
        const uint32_t k = s.all_cnt[tid];
        const u64 w = s.all_sum[tid];
        uint32_t ki = k;
        u64 wi = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t kt = __shfl_up_sync(0xFFFFFFFFu, ki, o);
            const u64 wt = __shfl_up_sync(0xFFFFFFFFu, wi, o);
            if (lane >= o) ki += kt, wi += wt;
        }
        __syncthreads();
        if (lane == 31) s.warp_u32[warp] = ki, s.warp_u64[warp] = wi;
        if (tid == 0) s.found_bin = kBins;
        __syncthreads();
        const uint32_t kb = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? s.warp_u32[lane] : 0u);
        const u64 wb = warp_sum(lane < warp ? s.warp_u64[lane] : 0ull);
        const u64 c1 = cnt + kb + ki, s1 = sum + wb + wi, c0 = c1 - k, s0 = s1 - w;
        if (BY_SUM ? s0 < need && need <= s1 : c0 < need && need <= c1) {
            s.found_bin = tid;
            s.found_cnt = (uint32_t)c0;
            s.found_sum = s0;
        }
        __syncthreads();
        const int bin = (int)s.found_bin;
        if (bin == kBins) return -1;
        cnt = s.found_cnt;
        sum = s.found_sum;
        return bin;
    }

    // Where, by index, the running sum of value(logit, index) over the whole row first exceeds
    // target(total).  Returns true, in one warp of one CTA, with the index and its value.
    template <typename Value, typename Target>
    __device__ __forceinline__ bool locate(Value &&value, Target &&target, uint32_t &idx, u64 &val, u64 &total) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int per = ((n + kWarps - 1) / kWarps + 31) / 32 * 32;  // a warp's run of indices
        const int i0 = min(warp * per, n), i1 = min(i0 + per, n);
        u64 sum = 0;
        for (int i = i0 + lane; i < i1; i += 32) sum += value(at(i), base + i);
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
            const u64 v = i < i1 ? value(at(i), base + i) : 0;
            u64 inc = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 t = __shfl_up_sync(0xFFFFFFFFu, inc, o);
                if (lane >= o) inc += t;
            }
            const uint32_t over = __ballot_sync(0xFFFFFFFFu, before + inc > goal);
            if (over) {
                const int l = __ffs(over) - 1;
                idx = base + j + l;
                val = __shfl_sync(0xFFFFFFFFu, v, l);
                return true;
            }
            before += __shfl_sync(0xFFFFFFFFu, inc, 31);
        }
        return false;
    }

    // The token of bin `bin` (of d) with which the running count (weight) reaches `need`, cnt and
    // sum being those before the bin.
    template <bool BY_SUM>
    __device__ __forceinline__ Cut refine(int bin, u64 need, u64 cnt, u64 sum) {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        uint32_t in = s.all_cnt[bin], lo = 0, hi = 0xFFFFFFFFu;
        auto inside = [&](float v, uint32_t &key) {
            const float d = dist(v);
            key = key_of(v);
            return d < kAll && bin_of(d) == bin && key >= lo && key <= hi;
        };
        while (in > kList) {
            // too many to be ranked: a histogram over their keys, from the largest down
            uint32_t a = 0, b = 0, key;
            for (int i = tid; i < n; i += kThreads)
                if (inside(at(i), key)) a = max(a, key), b = max(b, ~key);
            hi = cluster_max(a);
            lo = ~cluster_max(b);
            if (lo == hi) break;
            const int shift = max(0, 32 - __clz(hi - lo) - 10);
            histogram([&](float v, int &to, u64 &w) {
                uint32_t k;
                if (!inside(v, k)) return false;
                to = (int)((hi - k) >> shift);
                w = weight_of(dist(v));
                return true;
            });
            const uint32_t sub = (uint32_t)max(find_bin<BY_SUM>(need, cnt, sum), 0);
            in = s.all_cnt[sub];
            hi -= sub << shift;
            lo = hi - min(hi - lo, (1u << shift) - 1);
        }
        if (in > kList) {
            // equal logits: the q-th by index
            const float v0 = __uint_as_float(hi >> 31 ? hi ^ 0x80000000u : ~hi);
            const u64 w = weight_of(dist(v0));
            const u64 q = BY_SUM ? (need - sum + w - 1) / w : need - cnt;
            uint32_t idx;
            u64 val, total;
            const bool here = locate([&](float v, uint32_t) { return (u64)(v == v0); }, [&](u64) { return q - 1; }, idx, val, total);
            if (here && (uint32_t)lane < ctas) peer_store(&s.ranked_idx, lane, idx);
            cluster_sync();
            return {bin, hi, s.ranked_idx, sum + q * w};
        }
        // few: CTA 0 gathers them, and each warp ranks some of them against all
        for (int i = tid; i < n; i += kThreads) {
            uint32_t key;
            const float v = at(i);
            if (!inside(v, key)) continue;
            const uint32_t to = peer_add(&s.list_n, 0, 1);
            if (to < kList) {
                peer_store(&s.list_key[to], 0, key);
                peer_store(&s.list_idx[to], 0, base + i);
                peer_store(&s.list_w[to], 0, weight_of(dist(v)));
            }
        }
        cluster_sync();
        if (rank == 0) {
            const int m = min((int)s.list_n, kList);
            for (int i = warp; i < m; i += kWarps) {
                const uint32_t key = s.list_key[i], idx = s.list_idx[i];
                uint32_t k = 0;
                u64 w = 0;
                for (int j = lane; j < m; j += 32) {
                    const uint32_t kj = s.list_key[j];
                    if (kj > key || (kj == key && s.list_idx[j] < idx)) ++k, w += s.list_w[j];
                }
                k = __reduce_add_sync(0xFFFFFFFFu, k);
                w = warp_sum(w);
                const u64 w1 = sum + w + s.list_w[i];
                const bool is = BY_SUM ? sum + w < need && need <= w1 : cnt + k + 1 == need;
                if (is && (uint32_t)lane < ctas) {
                    peer_store(&s.ranked_key, lane, key);
                    peer_store(&s.ranked_idx, lane, idx);
                    peer_store(&s.ranked_sum, lane, w1);
                }
            }
            __syncthreads();
            if (tid == 0) s.list_n = 0;
        }
        cluster_sync();
        return {bin, s.ranked_key, s.ranked_idx, s.ranked_sum};
    }
};

template <bool CACHED>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs a, int per) {
    extern __shared__ __align__(16) uint8_t dyn[];
    Shared &s = *reinterpret_cast<Shared *>(dyn);
    float *own = reinterpret_cast<float *>(dyn + (sizeof(Shared) + 15) / 16 * 16);
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31;
    const uint32_t rank = cluster_ctarank(), ctas = a.ctas;
    const int64_t m = blockIdx.x / ctas;
    const int64_t i0 = min((int64_t)rank * per, (int64_t)a.V), i1 = min(i0 + per, (int64_t)a.V);
    const float *row = a.logits + m * a.ldl + i0;
    Row<CACHED> r = {s, CACHED ? own : row, (uint32_t)i0, (int)(i1 - i0), rank, ctas, 0.f, 0.f, kHead, kBins / kHead, 0};
    if (tid == 0) s.list_n = 0;
    cluster_arrive();  // (waited for before the first access to another CTA's memory)
    // ---- load; the largest logit
    uint32_t best = 0;
    if (CACHED && (reinterpret_cast<uintptr_t>(row) & 15) == 0) {
        const float4 *row4 = reinterpret_cast<const float4 *>(row);
#pragma unroll 4
        for (int i = tid; i < r.n / 4; i += kThreads) {
            float4 v = __ldg(row4 + i);
            v.x = clean(v.x), v.y = clean(v.y), v.z = clean(v.z), v.w = clean(v.w);
            reinterpret_cast<float4 *>(own)[i] = v;
            best = max(max(best, max(key_of(v.x), key_of(v.y))), max(key_of(v.z), key_of(v.w)));
        }
        for (int i = r.n / 4 * 4 + tid; i < r.n; i += kThreads) {
            own[i] = clean(__ldg(row + i));
            best = max(best, key_of(own[i]));
        }
    } else {
#pragma unroll 8
        for (int i = tid; i < r.n; i += kThreads) {
            const float v = clean(__ldg(row + i));
            if (CACHED) own[i] = v;
            best = max(best, key_of(v));
        }
    }
    cluster_wait();
    best = r.cluster_max(best);
    r.top = __uint_as_float(best >> 31 ? best ^ 0x80000000u : ~best);
    if (r.top == -INFINITY) {
        if (rank == 0 && tid == 0) {
            a.token[m] = -1;
            if (a.prob) a.prob[m] = 0.f;
        }
        return;
    }
    // ---- the row's settings
    float t = a.temperature ? __ldg(a.temperature + m) : 1.f;
    const bool greedy = !(t > 0.f);
    if (greedy) t = 1.f;
    r.c = __fmul_rn(__fdiv_rn(1.f, t), 1.4426950408889634f);
    const int64_t k = greedy ? 1 : a.top_k ? __ldg(a.top_k + m) : 0;
    const uint32_t p_share = greedy || !a.top_p ? kOne : share_of(__ldg(a.top_p + m), kOne);
    const uint32_t m_share = greedy || !a.min_p ? 0 : share_of(__ldg(a.min_p + m), 0);
    const uint32_t u = min(share_of(__ldg(a.u + m), 0), kOne - 1);
    const bool by_k = k > 0 && k < a.V, by_p = p_share < kOne;
    // ---- the cut
    Cut cut = {kBins + 1, 0, 0xFFFFFFFFu, 0};
    if (by_k || by_p) {
        for (;;) {
            u64 tail = 0;
            r.histogram([&](float v, int &bin, u64 &w) {
                const float d = r.dist(v);
                if (!(d < kAll)) return false;
                bin = r.bin_of(d);
                if (bin < kBins) {
                    w = weight_of(d);
                    return true;
                }
                if (by_p && !by_k) tail += weight_of(d);
                return false;
            });
            const bool all = r.span == kAll;
            u64 sum = 0, cnt = 0;
            cut.bin = kBins + 1;
            if (by_k) {
                const int bin = r.template find_bin<false>((u64)k, cnt, sum);
                const bool many = bin >= 0 && s.all_cnt[bin] > kList;
                if (bin >= 0) cut = r.template refine<false>(bin, (u64)k, cnt, sum);
                else if (!all) {
                    r.span = kAll, r.scale = kBins / kAll;
                    continue;
                }
                if (by_p && many) {
                    // the bins over keys have taken the place of those over d
                    r.histogram([&](float v, int &to, u64 &w) {
                        const float d = r.dist(v);
                        to = r.bin_of(d);
                        if (!(d < kAll) || to >= kBins) return false;
                        w = weight_of(d);
                        return true;
                    });
                }
            }
            if (by_p) {
                u64 whole = cut.sum;
                if (cut.bin > kBins) {
                    u64 in_bins = 0;
                    for (int i = tid; i < kBins; i += kThreads) in_bins += s.all_sum[i];
                    // (the bins are the cluster's already: one CTA's sum of them is enough)
                    whole = r.cluster_sum(tail + (rank == 0 ? in_bins : 0));
                }
                const u64 need = max(part_of(whole, p_share), (u64)1);
                cnt = sum = 0;
                const int bin = r.template find_bin<true>(need, cnt, sum);
                if (bin < 0) {
                    // beyond the bins (never once they cover every weight)
                    if (all) break;
                    r.span = kAll, r.scale = kBins / kAll;
                    continue;
                }
                cut = r.template refine<true>(bin, need, cnt, sum);
            }
            break;
        }
    }
    // ---- the token
    const u64 least = part_of(weight_of(0.f), m_share);
    uint32_t idx;
    u64 w, total;
    const bool here = r.locate(
        [&](float v, uint32_t i) -> u64 {
            const float d = r.dist(v);
            if (!(d < kAll)) return 0;
            if (cut.bin <= kBins) {
                const int bin = r.bin_of(d);
                if (bin > cut.bin) return 0;
                if (bin == cut.bin) {
                    const uint32_t key = key_of(v);
                    if (key < cut.key || (key == cut.key && i > cut.idx)) return 0;
                }
            }
            const u64 x = weight_of(d);
            return x >= least ? x : 0;
        },
        [&](u64 sum) { return part_of(sum, u); }, idx, w, total);
    if (here && lane == 0) {
        a.token[m] = (int32_t)idx;
        if (a.prob) a.prob[m] = __fdiv_rn((float)w, (float)total);
    }
}

}  // namespace

cudaError_t launch_sample(const DeviceInfo &di, const SampleArgs &args, cudaStream_t s) {
    (void)di;
    SampleArgs a = args;
    // CTAs of a row: up to eight, a few thousand logits each at least
    a.ctas = a.V <= 4096 ? 1 : a.V <= 8192 ? 2 : a.V <= 16384 ? 4 : 8;
    const int per = ((a.V + a.ctas - 1) / a.ctas + 3) / 4 * 4;
    const bool cached = per <= kCached;
    const int smem = (int)((sizeof(Shared) + 15) / 16 * 16) + (cached ? per * 4 : 0);
    auto kern = cached ? sample_kernel<true> : sample_kernel<false>;
    cudaError_t e = ensure_smem((const void *)kern, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3((unsigned)(a.M * a.ctas)), dim3(kThreads), smem, s, dim3(a.ctas), a, per);
}

}  // namespace q4k
