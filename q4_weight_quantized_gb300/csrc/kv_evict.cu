// Eviction from a paged cache by accumulated attention weight.
//
// Of the n slots of one KV head, the n - budget with the smallest (protected?, weight,
// slot) go; the slots freed below budget are filled with the kept ones above it, both
// in increasing order.  Filling holes moves a key and value only where it must: the
// kept slots below budget stay, and sources (>= budget) and destinations (< budget)
// never meet, so all moves run at once.
//
// select_kernel, a CTA per sequence and head: weights become order-preserving 32-bit
// keys in shared memory; a histogram over the range of the keys that are left, narrowed
// to the bin that holds the wanted rank, finds the cut in two or three rounds; then
// each warp walks a contiguous run of slots, so ranks in slot order are prefix sums of
// ballots.  Bound by latency (a few block-wide rounds); the reads are 8 bytes a slot.
// move_kernel copies the rows, 16 bytes a lane: bound by HBM.
#include <cuda_runtime.h>

#include "decode_ops.h"
#include "q4k_ptx.cuh"

namespace q4k {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kCached = 20480;  // slots whose keys fit beside the histogram with two CTAs on an SM
constexpr int kMoveThreads = 256;

// Order-preserving key: smaller weight, smaller key; -0 as +0; NaN above everything.
__device__ __forceinline__ uint32_t key_of(float w) {
    if (w != w) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

__device__ __forceinline__ uint32_t block_sum(uint32_t v, uint32_t *scratch) {
    v = __reduce_add_sync(0xFFFFFFFFu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    return __reduce_add_sync(0xFFFFFFFFu, scratch[threadIdx.x & 31]);
}
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t *scratch) {
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    return __reduce_max_sync(0xFFFFFFFFu, scratch[threadIdx.x & 31]);
}
// Sum of the warps before this one of a value that every lane of a warp holds; *total
// the sum of all.
__device__ __forceinline__ uint32_t warps_before(uint32_t v, uint32_t *scratch, uint32_t *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();
    if (lane == 0) scratch[warp] = v;
    __syncthreads();
    const uint32_t w = scratch[lane];
    *total = __reduce_add_sync(0xFFFFFFFFu, w);
    return __reduce_add_sync(0xFFFFFFFFu, lane < warp ? w : 0u);
}

// CACHED: keys and protection bits lie in shared memory; otherwise both are formed
// again from the arrays on every pass.
template <bool CACHED>
__global__ void __launch_bounds__(kThreads) select_kernel(const EvictArgs a) {
    extern __shared__ uint32_t dyn[];
    __shared__ uint32_t hist[kBins];
    __shared__ uint32_t scratch[kWarps + 1];
    __shared__ uint32_t found[2];
    uint32_t *keys = dyn, *bits = dyn + kCached;  // [kCached], [kCached / 32]
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bh = blockIdx.x, b = bh / a.c.heads;
    const float *w = a.weights + (int64_t)bh * a.ld_meta;
    const int32_t *p = a.positions + (int64_t)bh * a.ld_meta;
    float *w_out = a.weights_out + (int64_t)bh * a.ld_meta;
    int32_t *p_out = a.positions_out + (int64_t)bh * a.ld_meta;
    const int raw = a.seq_lens[b];
    const int n = max(0, min(raw, a.cap)), keep = min(n, a.budget);
    if (tid == 0 && raw > a.cap) atomicOr(a.c.status, kDevIndex);
    if (n <= a.budget) {
        if (tid == 0) a.count[bh] = 0;
        if (w_out != w)
            for (int j = tid; j < n; j += kThreads) w_out[j] = w[j];
        if (p_out != p)
            for (int j = tid; j < n; j += kThreads) p_out[j] = p[j];
        return;
    }
    // ---- newest position; positions as offset binary, so that the unsigned maximum serves
    uint32_t top = 0;
    for (int j = tid; j < n; j += kThreads) {
        top = max(top, (uint32_t)p[j] ^ 0x80000000u);
        if (CACHED) keys[j] = key_of(w[j]);
    }
    const int64_t newest = (int32_t)(block_max(top, scratch) ^ 0x80000000u);
    auto is_protected = [&](int32_t pos) { return pos < a.sinks || (int64_t)pos > newest - a.recent; };
    auto key_at = [&](int j) { return CACHED ? keys[j] : key_of(w[j]); };
    auto prot_at = [&](int j) { return CACHED ? (bits[j >> 5] >> (j & 31) & 1) != 0 : is_protected(p[j]); };
    // ---- protected slots
    uint32_t free_slots = 0;
    for (int j0 = warp * 32; j0 < n; j0 += kThreads) {
        const int j = j0 + lane;
        const bool prot = j < n && is_protected(p[j]);
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, prot);
        if (CACHED && lane == 0) bits[j0 >> 5] = m;
        free_slots += j < n && !prot;
    }
    free_slots = block_sum(free_slots, scratch);  // (its barriers order the bits, too)
    // ---- the class in which the cut lies: unprotected slots, or, if these are not enough, protected ones
    uint32_t need = n - a.budget;
    const bool in_prot = need > free_slots;
    if (in_prot) need -= free_slots;
    // ---- the cut: in that class, keys < cut go, and the first `ties` slots of key == cut
    uint32_t lo = 0xFFFFFFFFu, hi = 0;
    for (int j = tid; j < n; j += kThreads)
        if (prot_at(j) == in_prot) {
            const uint32_t k = key_at(j);
            lo = min(lo, k);
            hi = max(hi, k);
        }
    lo = ~block_max(~lo, scratch);
    hi = block_max(hi, scratch);
    uint32_t cut, ties;
    for (;;) {
        const uint32_t width = hi - lo;
        const int shift = max(0, 32 - __clz(width) - 11);  // at most 2048 bins
        for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
        __syncthreads();
        for (int j = tid; j < n; j += kThreads) {
            const uint32_t k = key_at(j);
            if (k >= lo && k <= hi && prot_at(j) == in_prot) atomicAdd(&hist[(k - lo) >> shift], 1u);
        }
        __syncthreads();
        // bins 2 tid, 2 tid + 1: the one in which the need-th smallest key lies
        const uint32_t c0 = hist[2 * tid], c1 = hist[2 * tid + 1];
        uint32_t inc = c0 + c1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += v;
        }
        uint32_t all;
        const uint32_t before = warps_before(__shfl_sync(0xFFFFFFFFu, inc, 31), scratch, &all) + inc - c0 - c1;
        if (before < need && need <= before + c0) found[0] = 2 * tid, found[1] = before;
        else if (before + c0 < need && need <= before + c0 + c1) found[0] = 2 * tid + 1, found[1] = before + c0;
        __syncthreads();
        const uint32_t bin = found[0], left = need - found[1], in_bin = hist[bin];
        lo += bin << shift;
        hi = lo + min(hi - lo, (1u << shift) - 1);
        need = left;
        if (shift == 0 || in_bin == left) {
            // one key left, or the whole bin goes
            cut = hi;
            ties = in_bin == left ? 0xFFFFFFFFu : left;
            break;
        }
        __syncthreads();
    }
    // ---- ranks in slot order: warp `warp` walks slots [s0, s1)
    const int per = ((n + kWarps - 1) / kWarps + 31) / 32 * 32;
    const int s0 = min(warp * per, n), s1 = min(s0 + per, n);
    uint32_t all;
    uint32_t tie0 = 0;
    if (ties != 0xFFFFFFFFu) {
        for (int j0 = s0; j0 < s1; j0 += 32) {
            const int j = j0 + lane;
            tie0 += __popc(__ballot_sync(0xFFFFFFFFu, j < s1 && key_at(j) == cut && prot_at(j) == in_prot));
        }
        tie0 = warps_before(tie0, scratch, &all);
    }
    auto walk = [&](auto &&visit) {
        uint32_t tie = tie0;
        for (int j0 = s0; j0 < s1; j0 += 32) {
            const int j = j0 + lane;
            bool gone = false, is_tie = false;
            if (j < s1) {
                const bool prot = prot_at(j);
                const uint32_t k = key_at(j);
                is_tie = prot == in_prot && k == cut;
                gone = prot == in_prot ? k < cut || (is_tie && ties == 0xFFFFFFFFu) : in_prot;
            }
            const uint32_t m = __ballot_sync(0xFFFFFFFFu, is_tie);
            if (is_tie && tie + __popc(m & ((1u << lane) - 1)) < ties) gone = true;
            tie += __popc(m);
            visit(j, gone);
        }
    };
    uint32_t holes = 0, fill = 0;
    walk([&](int j, bool gone) {
        holes += __popc(__ballot_sync(0xFFFFFFFFu, j < s1 && gone && j < keep));
        fill += __popc(__ballot_sync(0xFFFFFFFFu, j < s1 && !gone && j >= keep));
    });
    uint32_t moves;
    uint32_t hole = warps_before(holes, scratch, &moves);
    uint32_t from = warps_before(fill, scratch, &all);
    int2 *list = a.moves + (int64_t)bh * a.max_moves;
    walk([&](int j, bool gone) {
        const bool to = j < s1 && gone && j < keep, src = j < s1 && !gone && j >= keep;
        const uint32_t mt = __ballot_sync(0xFFFFFFFFu, to), ms = __ballot_sync(0xFFFFFFFFu, src), lt = (1u << lane) - 1;
        if (to) list[hole + __popc(mt & lt)].x = j;
        if (src) list[from + __popc(ms & lt)].y = j;
        hole += __popc(mt);
        from += __popc(ms);
        if (j < s1 && j < keep && !gone) {
            if (w_out != w) w_out[j] = w[j];
            if (p_out != p) p_out[j] = p[j];
        }
    });
    __syncthreads();
    for (uint32_t i = tid; i < moves; i += kThreads) {
        const int2 m = list[i];
        w_out[m.x] = w[m.y];
        p_out[m.x] = p[m.y];
    }
    if (tid == 0) a.count[bh] = (int32_t)moves;
}

// `per_head` blocks for each sequence and head.  A row is `chunks` 16-byte chunks, a thread
// each, of a key and of a value.
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const EvictArgs a, int chunks, int per_head) {
    pdl_wait();
    pdl_trigger();
    const int bh = blockIdx.x / per_head, b = bh / a.c.heads, h = bh % a.c.heads, part = blockIdx.x % per_head;
    if (part == 0 && h == 0 && threadIdx.x == 0) a.new_lens[b] = max(0, min(min(a.seq_lens[b], a.cap), a.budget));
    const int n = a.count[bh];
    const int2 *list = a.moves + (int64_t)bh * a.max_moves;
    const int32_t *table = a.c.table + b * a.c.ld_table;
    const int rows = kMoveThreads / chunks, ch = threadIdx.x % chunks;
    for (int i = part * rows + threadIdx.x / chunks; i < n; i += per_head * rows) {
        const int2 m = list[i];
        const uint32_t pt = page_of(a.c, m.x), ps = page_of(a.c, m.y);
        const int32_t to = __ldg(table + pt), from = __ldg(table + ps);
        if (!page_ok(a.c, to) || !page_ok(a.c, from)) {
            atomicOr(a.c.status, kDevIndex);
            continue;
        }
        const int64_t dst = row_bytes_at(a.c, to, h, (uint32_t)m.x - pt * a.c.page_size) + ch * 16;
        const int64_t src = row_bytes_at(a.c, from, h, (uint32_t)m.y - ps * a.c.page_size) + ch * 16;
        const uint4 k = *reinterpret_cast<const uint4 *>(a.c.k + src);
        const uint4 v = *reinterpret_cast<const uint4 *>(a.c.v + src);
        *reinterpret_cast<uint4 *>(a.c.k + dst) = k;
        *reinterpret_cast<uint4 *>(a.c.v + dst) = v;
    }
}

}  // namespace

cudaError_t launch_kv_evict(const DeviceInfo &di, const EvictArgs &a, cudaStream_t s) {
    const bool cached = a.cap <= kCached;
    const int smem = cached ? (kCached + kCached / 32) * 4 : 0;
    auto kern = cached ? select_kernel<true> : select_kernel<false>;
    cudaError_t e = cudaSuccess;
    if (cached) e = ensure_smem((const void *)kern, smem);
    if (e != cudaSuccess) return e;
    const int bh = a.c.batch * a.c.heads;
    e = launch_pdl(kern, dim3(bh), dim3(kThreads), smem, s, dim3(1), a);
    if (e != cudaSuccess) return e;
    const int chunks = a.c.dim * (a.c.e4m3 ? 1 : 2) / 16, rows = kMoveThreads / chunks;
    // a few rounds of copies per block, but no more blocks than fill the GPU a few times over
    int64_t per_head = (a.max_moves + 4 * rows - 1) / (4 * rows);
    const int64_t most = ((int64_t)di.sm_count * 32 + bh - 1) / bh;
    if (per_head > most) per_head = most;
    if (per_head < 1) per_head = 1;
    return launch_pdl(move_kernel, dim3((unsigned)(per_head * bh)), dim3(kMoveThreads), 0, s, dim3(1), a, chunks, (int)per_head);
}

}  // namespace q4k
