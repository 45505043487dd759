// Eviction from a paged cache by accumulated attention weight.
//
// Of the n slots of one KV head, the n - budget with the smallest (protected?, weight,
// slot) go; the slots freed below budget are filled with the kept ones above it, both
// in increasing order.  Filling holes moves a key and value only where it must: the
// kept slots below budget stay, and sources (>= budget) and destinations (< budget)
// never meet, so all moves run at once.
//
// select_kernel, a CTA per sequence and head: weights become order-preserving 32-bit
// keys in shared memory.  A histogram over the range of the keys narrows it to the bin
// that holds the wanted rank; once a few slots are left they are ranked against each
// other, which also settles equal weights by slot.  The last pass takes the slots in
// order, a run to a thread, and numbers holes and fillers by one scan.  Bound by
// latency (some fifteen block-wide steps, which fewer threads take faster); the reads are 8 bytes a slot.
// move_kernel copies the rows, 16 bytes a lane, and their weights and positions: bound by HBM (two or
// four rows a thread cost more in occupancy than their overlapping loads gave: 62 and 70 us against 59).
// Measured: 9.0 us for 32 caches of 8 heads with one slot over 2048 (5 of them the selection), 81 us for
// 16 caches of 9001 to 16384 slots to 8192 (15 the selection, 59 the copies: 333 MB at 5.7 TB/s), 337 us for one of 8
// heads of 200001 slots to half (beyond kCached, where every pass of a head's one CTA reads both arrays again).

#include <cuda_runtime.h>

#include <type_traits>

#include "decode_ops.h"
#include "q4k_ptx.cuh"

namespace q4k {
namespace {

constexpr int kSmall = 4096;    // slots that 256 threads hold in registers
constexpr int kMid = 8192;      // 512 threads, of which two CTAs share an SM (256 caches of 8000: 20.6 us, with 1024 23.6)
constexpr int kHeld = 20480;    // slots that 1024 threads hold in registers, and whose keys leave room for two CTAs
constexpr int kCached = 49152;  // slots whose keys fit in shared memory
constexpr int kFew = 128;       // slots that are ranked against each other
constexpr int kMoveThreads = 256;
constexpr uint32_t kFull = 0xFFFFFFFFu;

// Order-preserving key: smaller weight, smaller key; -0 as +0; NaN above everything.
__device__ __forceinline__ uint32_t key_of(float w) {
    if (w != w) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

template <int THREADS>
struct Block {
    static constexpr int WARPS = THREADS / 32;
    // Sum of a value over the threads before this one; total: over all.  Two scratch arrays in turn, so
    // that one barrier a scan is enough.
    static __device__ __forceinline__ uint32_t scan(uint32_t v, uint32_t *scratch, uint32_t &total) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        uint32_t inc = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t t = __shfl_up_sync(kFull, inc, o);
            if (lane >= o) inc += t;
        }
        if (lane == 31) scratch[warp] = inc;
        __syncthreads();
        const uint32_t w = lane < WARPS ? scratch[lane] : 0u;
        total = __reduce_add_sync(kFull, w);
        return __reduce_add_sync(kFull, lane < warp ? w : 0u) + inc - v;
    }
};

// KEYS: the slots whose keys and protection bits lie in shared memory; 0: both are formed again from the
// arrays on every pass.  HELD: a thread holds slots tid, tid + THREADS, ... in registers, too, loaded before
// anything waits for one.
template <int THREADS, int KEYS, bool HELD>
__global__ void __launch_bounds__(THREADS) select_kernel(const EvictArgs a) {
    using B = Block<THREADS>;
    constexpr int BINS = 2 * THREADS, LOG_BINS = THREADS == 1024 ? 11 : THREADS == 512 ? 10 : 9;
    constexpr bool CACHED = KEYS > 0;
    static_assert(BINS == 1 << LOG_BINS, "two bins a thread");
    extern __shared__ __align__(16) uint32_t dyn[];
    __shared__ uint32_t hist[BINS];
    __shared__ uint32_t scratch[2][32], red[5][32];
    __shared__ uint2 list[kFew];
    __shared__ uint32_t found[2], listed;
    uint32_t *keys = dyn, *bits = dyn + KEYS;  // [KEYS], [KEYS / 32]
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bh = blockIdx.x, b = bh / a.c.heads;
    const float *w = a.weights + (int64_t)bh * a.ld_meta;
    const int32_t *p = a.positions + (int64_t)bh * a.ld_meta;
    float *w_out = a.weights_out + (int64_t)bh * a.ld_meta;
    int32_t *p_out = a.positions_out + (int64_t)bh * a.ld_meta;
    const int raw = a.seq_lens[b];
    // (unsigned: of up to 2^31 - 1 slots, the last steps of a pass end beyond 2^31)
    const uint32_t n = max(0, min(raw, a.cap)), keep = min(n, (uint32_t)a.budget);
    if (tid == 0 && raw > a.cap) atomicOr(a.c.status, kDevIndex);
    if (n == keep) {
        if (tid == 0) a.count[bh] = 0;
        if (w_out != w)
            for (uint32_t j = tid; j < n; j += THREADS) w_out[j] = w[j];
        if (p_out != p)
            for (uint32_t j = tid; j < n; j += THREADS) p_out[j] = p[j];
        return;
    }
    // ---- newest position (as offset binary, so that the unsigned maximum serves), and the keys; what
    // stays below keep goes over at once, the holes among it are overwritten at the end
    constexpr int PER = HELD ? KEYS / THREADS : 1;
    const bool copy_w = w_out != w, copy_p = p_out != p;
    uint32_t top = 0, mine[PER];
    int32_t pos[PER];
    if constexpr (HELD) {
        float wj[PER];
#pragma unroll
        for (int x = 0; x < PER; ++x) {
            if (x * THREADS >= n) break;
            const uint32_t j = min((uint32_t)(x * THREADS + tid), n - 1);
            pos[x] = p[j], wj[x] = w[j];
        }
#pragma unroll
        for (int x = 0; x < PER; ++x) {
            if (x * THREADS >= n) break;
            const uint32_t j = x * THREADS + tid;
            top = max(top, (uint32_t)pos[x] ^ 0x80000000u);
            mine[x] = key_of(wj[x]);
            keys[j] = mine[x];  // (past n: never looked at)
            if (copy_w && j < keep) w_out[j] = wj[x];
            if (copy_p && j < keep) p_out[j] = pos[x];
        }
    } else {
        constexpr int kAhead = 8;  // loads before the first store
        for (uint32_t j0 = tid; j0 < n; j0 += kAhead * THREADS) {
            int32_t pj[kAhead];
            float wj[kAhead];
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {
                const uint32_t j = min(j0 + x * THREADS, n - 1);
                pj[x] = p[j], wj[x] = w[j];
            }
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {
                const uint32_t j = j0 + x * THREADS;
                top = max(top, (uint32_t)pj[x] ^ 0x80000000u);
                if (CACHED && j < n) keys[j] = key_of(wj[x]);
                if (copy_w && j < keep) w_out[j] = wj[x];
                if (copy_p && j < keep) p_out[j] = pj[x];
            }
        }
    }
    top = __reduce_max_sync(kFull, top);
    if (lane == 0) red[0][warp] = top;
    __syncthreads();
    const int64_t newest = (int32_t)(__reduce_max_sync(kFull, lane < B::WARPS ? red[0][lane] : 0u) ^ 0x80000000u);
    auto is_protected = [&](int32_t pos) { return pos < a.sinks || (int64_t)pos > newest - a.recent; };
    auto key_at = [&](uint32_t j) { return CACHED ? keys[j] : key_of(w[j]); };
    auto prot_at = [&](uint32_t j) { return CACHED ? (bits[j >> 5] >> (j & 31) & 1) != 0 : is_protected(p[j]); };
    // ---- protected slots; number and range of the keys of either class
    uint32_t free_slots = 0, low[2] = {kFull, kFull}, high[2] = {0, 0}, prots = 0;  // prots: of this thread's slots
    auto of_either = [&](uint32_t k, bool prot) {
        free_slots += !prot;
        low[0] = prot ? low[0] : min(low[0], k), high[0] = prot ? high[0] : max(high[0], k);
        low[1] = prot ? min(low[1], k) : low[1], high[1] = prot ? max(high[1], k) : high[1];
    };
    if constexpr (HELD) {
#pragma unroll
        for (int x = 0; x < PER; ++x) {
            if (x * THREADS >= n) break;
            const uint32_t j = x * THREADS + tid;
            const bool prot = is_protected(pos[x]);
            const uint32_t m = __ballot_sync(kFull, prot);
            if (lane == 0) bits[j >> 5] = m;
            prots |= prot ? 1u << x : 0u;
            if (j < n) of_either(mine[x], prot);
        }
    } else {
        constexpr int kAhead = 8;  // loads before the first is looked at
        for (uint32_t j0 = 0; j0 < n; j0 += kAhead * THREADS) {
            int32_t pj[kAhead];
#pragma unroll
            for (int x = 0; x < kAhead; ++x) pj[x] = p[min(j0 + x * THREADS + tid, n - 1)];
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {
                const uint32_t j = j0 + x * THREADS + tid;
                const bool prot = j < n && is_protected(pj[x]);
                if (CACHED) {
                    const uint32_t m = __ballot_sync(kFull, prot);
                    if (lane == 0 && j < n) bits[j >> 5] = m;
                }
                if (j < n) of_either(CACHED ? keys[j] : key_of(w[j]), prot);
            }
        }
    }
    // visit(slot, key) for every slot of class `of` with a key in [lo, hi]
    auto each = [&](bool of, uint32_t lo, uint32_t hi, auto &&visit) {
        if constexpr (HELD) {
#pragma unroll
            for (int x = 0; x < PER; ++x) {
                if (x * THREADS >= n) break;
                const uint32_t j = x * THREADS + tid;
                if (j < n && mine[x] >= lo && mine[x] <= hi && ((prots >> x & 1) != 0) == of) visit(j, mine[x]);
            }
        } else if constexpr (CACHED) {
            for (uint32_t j = 4 * tid; j < n; j += 4 * THREADS) {
                const uint4 t = *reinterpret_cast<const uint4 *>(keys + j);  // (past n: whatever is there)
                const uint32_t k[4] = {t.x, t.y, t.z, t.w}, prot = bits[j >> 5] >> (j & 31);
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    if (j + x < n && k[x] >= lo && k[x] <= hi && ((prot >> x & 1) != 0) == of) visit(j + x, k[x]);
            }
        } else {
#pragma unroll 4
            for (uint32_t j = tid; j < n; j += THREADS) {
                const uint32_t k = key_at(j);
                if (k >= lo && k <= hi && prot_at(j) == of) visit(j, k);
            }
        }
    };
    free_slots = __reduce_add_sync(kFull, free_slots);
#pragma unroll
    for (int x = 0; x < 2; ++x) low[x] = __reduce_min_sync(kFull, low[x]), high[x] = __reduce_max_sync(kFull, high[x]);
    __syncthreads();
    if (lane == 0) red[0][warp] = free_slots, red[1][warp] = low[0], red[2][warp] = high[0], red[3][warp] = low[1], red[4][warp] = high[1];
    if (tid == 0) listed = 0;
    __syncthreads();
    const int rl = min(lane, B::WARPS - 1);
    free_slots = __reduce_add_sync(kFull, lane < B::WARPS ? red[0][lane] : 0u);
    // ---- the class in which the cut lies: unprotected slots, or, if these are not enough, protected ones
    uint32_t need = n - a.budget, in = free_slots;
    const bool in_prot = need > free_slots;
    if (in_prot) need -= free_slots, in = n - free_slots;
    uint32_t lo = __reduce_min_sync(kFull, red[in_prot ? 3 : 1][rl]), hi = __reduce_max_sync(kFull, red[in_prot ? 4 : 2][rl]);
    // ---- the cut: of that class, slots with a smaller (key, slot) than (cut, cut_slot) go, and this one
    uint32_t cut, cut_slot = kFull;
    bool gathered = false;
    if (need == 1) {  // one token more, one token less: the smallest key
        hi = lo;
        in = 1;  // (if only one slot has it; the list finds out)
    }
    for (;;) {
        if (need == in && hi != lo) {  // all of them go
            cut = hi;
            break;
        }
        if (in <= kFew && !gathered) {
            gathered = true;
            each(in_prot, lo, hi, [&](uint32_t j, uint32_t k) {
                const uint32_t at = atomicAdd(&listed, 1u);
                if (at < kFew) list[at] = make_uint2(k, j);
            });
            __syncthreads();
            in = listed;
            if (in <= kFew) {
                // ranked against each other, a slot by a few neighbouring lanes
                constexpr int TEAM = THREADS / kFew;
                const uint2 me = list[min((uint32_t)(tid / TEAM), in - 1)];
                uint32_t before = 0;
                for (uint32_t i = tid % TEAM; i < in; i += TEAM) {
                    const uint2 t = list[i];
                    before += t.x < me.x || (t.x == me.x && t.y < me.y) ? 1u : 0u;
                }
#pragma unroll
                for (int o = 1; o < TEAM; o <<= 1) before += __shfl_xor_sync(kFull, before, o);
                if (tid / TEAM < in && tid % TEAM == 0 && before + 1 == need) found[0] = me.x, found[1] = me.y;
                __syncthreads();
                cut = found[0], cut_slot = found[1];
                break;
            }
        }
        if (lo == hi) {
            // many equal keys: the need-th of them by slot
            cut = lo;
            uint32_t run = 0;
            int turn = 0;
            for (uint32_t j0 = 0; j0 < n && run < need; j0 += 4 * THREADS, turn ^= 1) {
                const uint32_t j = j0 + 4 * tid;
                uint32_t is = 0, total;
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    if (j + x < n && key_at(j + x) == cut && prot_at(j + x) == in_prot) is |= 1u << x;
                uint32_t before = run + B::scan(__popc(is), scratch[turn], total);
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    if ((is >> x & 1) && ++before == need) found[0] = j + x;
                run += total;
            }
            __syncthreads();
            cut_slot = found[0];
            break;
        }
        const int shift = max(0, 32 - __clz(hi - lo) - LOG_BINS);
        for (int i = tid; i < BINS; i += THREADS) hist[i] = 0;
        __syncthreads();
        each(in_prot, lo, hi, [&](uint32_t, uint32_t k) { atomicAdd(&hist[(k - lo) >> shift], 1u); });
        __syncthreads();
        // bins 2 tid, 2 tid + 1: the one in which the need-th smallest key lies
        const uint32_t c0 = hist[2 * tid], c1 = hist[2 * tid + 1];
        uint32_t all;
        const uint32_t before = B::scan(c0 + c1, scratch[0], all);
        if (before < need && need <= before + c0) found[0] = 2 * tid, found[1] = before;
        else if (before + c0 < need && need <= before + c0 + c1) found[0] = 2 * tid + 1, found[1] = before + c0;
        __syncthreads();
        const uint32_t bin = found[0];
        need -= found[1];
        in = hist[bin];
        lo += bin << shift;
        hi = lo + min(hi - lo, (1u << shift) - 1);
        __syncthreads();
    }
    // ---- holes below keep and fillers from there on, numbered in slot order: a run of slots a thread, so long that one
    // scan is enough for the slots in shared memory (4, 12, 20, ...: then the threads' 16-byte reads meet in no bank).
    // The list, at most half as many pairs as slots, then takes the keys' place, from where it goes out in whole sectors
    int2 *list_out = a.moves + (int64_t)bh * a.max_moves;
    uint32_t holes = 0, fills = 0;
    const uint32_t per = CACHED ? ((n + THREADS - 1) / THREADS + 3) / 8 * 8 + 4 : 4;
    constexpr int MOST = CACHED ? (KEYS / THREADS + 3) / 8 * 8 + 4 : 4;
    using Mark = typename std::conditional<(MOST > 32), unsigned long long, uint32_t>::type;
    static_assert(MOST <= 64 && MOST * THREADS < 65536, "marks of a thread in a word, counts of a block in 16 bits");
    int2 *const moves = CACHED ? reinterpret_cast<int2 *>(keys) : list_out;
    __syncthreads();
    int turn = 0;
    for (uint32_t base = 0; base < n; base += per * THREADS, turn ^= 1) {
        const uint32_t j0 = base + per * tid;
        uint32_t count = 0;  // holes, fillers << 16
        Mark mark = 0;       // slots of either kind
#pragma unroll
        for (int q = 0; q < MOST / 4; ++q) {
            const uint32_t j = j0 + 4 * q;
            if (4 * q >= per || j >= n) break;
            uint32_t k[4] = {0, 0, 0, 0}, prot = 0;
            if constexpr (CACHED) {
                const uint4 t = *reinterpret_cast<const uint4 *>(keys + j);  // (past n: whatever is there)
                k[0] = t.x, k[1] = t.y, k[2] = t.z, k[3] = t.w;
                prot = bits[j >> 5] >> (j & 31);
            } else {
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    if (j + x < n) k[x] = key_of(w[j + x]), prot |= is_protected(p[j + x]) ? 1u << x : 0u;
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const bool of_class = ((prot >> x & 1) != 0) == in_prot;
                const bool gone = of_class ? k[x] < cut || (k[x] == cut && j + x <= cut_slot) : in_prot;
                const bool below = j + x < keep;
                if (j + x < n && gone == below) mark |= (Mark)1 << (4 * q + x), count += below ? 1u : 1u << 16;
            }
        }
        uint32_t total;
        const uint32_t before = B::scan(count, scratch[turn], total);
        uint32_t hole = holes + (before & 0xFFFF), fill = fills + (before >> 16);
        for (; mark != 0; mark &= mark - 1) {
            const uint32_t slot = j0 + (MOST > 32 ? __ffsll((long long)mark) : __ffs((int)mark)) - 1;
            if (slot < keep) moves[hole++].x = slot;
            else moves[fill++].y = slot;
        }
        holes += total & 0xFFFF;
        fills += total >> 16;
    }
    if (CACHED) {
        __syncthreads();
        for (uint32_t i = tid; i < holes; i += THREADS) list_out[i] = moves[i];
    }
    if (tid == 0) a.count[bh] = (int32_t)holes;
}

template <int THREADS, int KEYS, bool HELD>
cudaError_t launch_select(const EvictArgs &a, cudaStream_t s) {
    auto kern = select_kernel<THREADS, KEYS, HELD>;
    constexpr int smem = (KEYS + KEYS / 32) * 4;
    if (smem > 0) {
        const cudaError_t e = ensure_smem((const void *)kern, smem);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(kern, dim3(a.c.batch * a.c.heads), dim3(THREADS), smem, s, dim3(1), a);
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
    // The ids of a move's two pages; if one is out of range, the move is not made: the hole keeps its token.
    auto pages_of = [&](int2 m, uint32_t &pt, uint32_t &ps, int32_t &to, int32_t &from) {
        pt = page_of(a.c, m.x), ps = page_of(a.c, m.y);
        to = __ldg(table + pt), from = __ldg(table + ps);
        return page_ok(a.c, to) && page_ok(a.c, from);
    };
    uint32_t pt, ps;
    int32_t to, from;
    // (here rather than at the end of the selection, which every head waits for)
    const int64_t meta = (int64_t)bh * a.ld_meta;
    for (int i = part * kMoveThreads + threadIdx.x; i < n; i += per_head * kMoveThreads) {
        const int2 m = list[i];
        if (!pages_of(m, pt, ps, to, from)) continue;
        a.weights_out[meta + m.x] = a.weights[meta + m.y];
        a.positions_out[meta + m.x] = a.positions[meta + m.y];
    }
    const int rows = kMoveThreads / chunks, ch = threadIdx.x % chunks;
    for (int i = part * rows + threadIdx.x / chunks; i < n; i += per_head * rows) {
        const int2 m = list[i];
        if (!pages_of(m, pt, ps, to, from)) {
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
    const int bh = a.c.batch * a.c.heads;
    // more short caches than SMs: small CTAs, of which more share one (the same cache again and
    // again: 256 heads with one slot over 2048 8.0 us, with 512 threads 9.8; 64 heads of 4096 to 2048 23.6 and 20.7)
    cudaError_t e = a.cap <= kSmall && bh > di.sm_count ? launch_select<256, kSmall, true>(a, s)
                    : a.cap <= kMid    ? launch_select<512, kMid, true>(a, s)
                    : a.cap <= kHeld   ? launch_select<1024, kHeld, true>(a, s)
                    : a.cap <= kCached ? launch_select<1024, kCached, false>(a, s)
                                       : launch_select<1024, 0, false>(a, s);
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
