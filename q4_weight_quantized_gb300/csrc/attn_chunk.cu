// Attention of chunks of new tokens over a paged key-value cache, on the tcgen05 tensor cores.
//
// For a row r (token i, head hq of its sequence) that sees the slots [begin_r, end_r):
//     s_j = c q . k_j,  m = max_j s_j,  l = sum_j e^(s_j - m),  o = v_scale sum_j e^(s_j - m) v_j / l
// and parts (m, l, o') over disjoint slots join as in attn_decode.cu.
//
// Bound by the tensor cores for long chunks, by HBM for few rows over long caches.  Hence
//   - The rows of one KV head, token-major (row = token * group + head in group), are cut into units of 256 rows (128
//     for heads of 256): two tiles of 128, MMA M.  A unit's tiles share every key and value that is loaded, so short
//     chunks of grouped heads fill tiles, too.
//   - Per tile of BN slots: S = Q K^T into tensor memory; a thread a row reads its scores, keeps the running maximum and
//     sum, and writes the weights, in 16 bits, over them; O += P V reads them from there (A from tensor memory, V as it
//     lies in the cache: its slots are the K axis, so B is MN-major).  While one tile's warps do the softmax the tensor
//     cores work for the other tile.
//   - The running maximum moves only when a score exceeds it by 2^8; only then is O rescaled, by the softmax's own
//     threads: S of a tile is there only after the O of the tile before.  So a tile's weights are taken by the maximum of
//     the tiles before, in the one pass that finds its own maximum, which counts from the next tile on.  (Heads of 256: one tile of rows, two buffers
//     of S instead; there the rare rescale waits for the product before.)
//   - Work is one list of places (KV head, unit, tile of slots) cut into equal contiguous shares, one per CTA, whatever
//     the lengths are; units that a share does not hold as a whole leave (m, l, o') in the workspace for join_kernel.
//   - Four warps bring keys and values into the swizzled layout the MMAs read.  Where every row sees a whole tile and pages
//     have 8 slots or a multiple, the copy engine does (a box a page's part); else a lane copies 16 bytes at a time and
//     fills what is not there with zeros (any page size, any strides).  An e4m3 cache's tiles are staged one ahead as
//     they are and become f16, exactly, keys and values at once; Q becomes f16 by a power of two a row.
//   - Scores that need more than the scale (a mask's edge, a small call's softcap or a large one, maxima so large that the fused product's
//     rounding counts) are prepared in their place in tensor memory first, so that the pass itself is the same for every tile.
// A slot that some rows of a unit see and others do not may hold values that are not finite: those are taken out of the
// product (0 * infinity would reach every row) and added to the rows that see them at the end.
//
// Measured, heads of 128, 40 of them on 8 KV heads: a prompt of 8192 in 520 us (1320 TFLOP/s), 512 tokens after 65536 in
// 487 us (1416), from an e4m3 cache 622 us; with a softcap 760 TFLOP/s, one above 512 (64 of an e4m3 cache) 465.  Heads of 256, 20 on 4: the same
// chunk in 746 us (925), 966 from an e4m3 cache.  Two tiles of 128 rows and 128 slots take 1.8 us: 1.1 of
// them (2048 cycles of MMAs) is the tensor cores'; softmax -> P V, Q K^T -> softmax of each tile is a chain that two tiles
// cover to that extent.  A unit's end and start cost as much as 5 such places (kExtra; 3: 559 us for the prompt).
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "decode_ops.h"
#include "q4k_ptx.cuh"

namespace q4k {
namespace {

constexpr int kThreads = 512;          // warps 0-3 and 4-7: softmax of a tile of rows each; 8 (9): MMA; 10, 11: queries; 12-15: copies
constexpr int kMmaWarp = 8, kQueryWarp = 10, kCopyWarp = 12, kCopyWarps = 4;
constexpr int kPlanThreads = 1024, kPlanBatch = 2048;  // sequences whose sums lie in shared memory, at most
constexpr int kJoinWarps = 8;
constexpr int kMetaRing = 8;           // tiles whose page masks are kept: more than the ring holds
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;          // how far (log2) a score may exceed the running maximum
constexpr float kFar = 4194304.f;      // maxima (log2) from which on their product's rounding counts
constexpr int kExtra = 5;              // places of the list after a unit's tiles: the time of ending it and beginning the next

template <int D_, bool E4M3_>
struct Cfg {
    static constexpr int D = D_;
    static constexpr bool E4M3 = E4M3_;
    static constexpr int NT = D == 256 ? 1 : 2;        // tiles of 128 rows of a unit
    static constexpr int BN = D == 256 ? 64 : 128;     // slots of a tile
    static constexpr int ROWS = NT * 128;
    static constexpr int SLOT = BN * D * 2;            // bytes of a tile of keys or values in shared memory
    static constexpr int NS = D == 64 ? 8 : E4M3 ? 4 : 5;  // such tiles in the ring, keys and values in turn
    // weights in f16 are kept as 2^7 p, in o' and l alike: at most 2^15, and what lies below 2^-32 of the largest is lost
    static constexpr float LIFT = E4M3 ? 7.f : 0.f;
    // how far (log2) a score may exceed the maximum that its tile's weights are taken by: what f16 holds, and what leaves O room
    // for values up to 2^111
    static constexpr float JUMP = E4M3 ? kSlack : 16.f;
    // Soft caps from which on the short form of c tanh(s / c), off by 3 10^-7 c, adds more to a weight's error than a thirteenth of
    // half a step of its 16 bits.
    static constexpr float LARGE_CAP = E4M3 ? 64.f : 512.f;
    static constexpr int QBYTES = ROWS * D * 2;
    // An e4m3 cache's factors of a unit's rows are written with its queries, once the last scores of the unit before are done, and
    // read with its first scores.  Two tiles of rows: those scores are issued behind the weights of every unit before that one, so
    // one unit's factors at most are unread.  One: scores wait for the products of two tiles before, so the weights may be behind by
    // two whole units of one tile each, besides the one that is written (three, rounded up to a power of two).
    static constexpr uint32_t FACTORS = NT == 2 ? 2 : 4;
    static constexpr int PLAN = 576, MISC = 768 + PLAN + (E4M3 ? (int)FACTORS * ROWS : 0);  // barriers and flags, a small call's list, the
                                                                                            // factors
    static constexpr int RAW = E4M3 ? BN * D : 0;      // bytes of a tile as it lies in an e4m3 cache: one of keys, one of values
    static constexpr int SMEM = QBYTES + NS * SLOT + 2 * RAW + MISC + 1024;  // (+ slack to align the base)
    static constexpr uint32_t S_COL = 0, O_COL = 2 * BN;  // (two tiles of S, whatever NT)
    static constexpr uint32_t COLS = 512;
    // registers of a softmax thread and of the others, together those of the launch: 4 * 128.  (A prompt: 512 us,
    // 517 by 192 and 64; an e4m3 cache, whose copies need more: 689 by 192 and 64, 651 by 176 and 80, 636 by 168 and 88.)
    static constexpr int REGS = E4M3 ? 168 : 176, OTHER_REGS = 256 - REGS;
    static_assert(O_COL + NT * D <= COLS && SMEM <= 227 * 1024, "fits");
};

// What every role needs to know of a unit (ChunkRecord, made by plan_kernel), and of its share's part of it.
struct Unit : ChunkRecord {
    int h, rt;    // KV head, row tile
    int lo, hi;   // the share's tiles of slots
    bool whole;
};

// The list of a small call (few sequences and row tiles), which every CTA makes for itself.
constexpr int kSmall = 32;
struct SmallPlan {
    int64_t places;                       // as ChunkArgs::head
    int units, shares;
    int place_at[kSmall + 1];
    int seq_at[kSmall], len[kSmall], rt_at[kSmall];
};

struct Walk {
    int64_t at, hi, places;
    int h, rt, units, shares;
    const SmallPlan *small;  // or null: the list is in the workspace
};

// row / group for 0 <= row < 2^31
__device__ __forceinline__ int token_of(const ChunkArgs &a, int row) { return (int)(((uint64_t)(uint32_t)row * a.group_mul) >> a.group_shift); }

__device__ __forceinline__ int64_t share_at(int64_t total, int shares, int s) { return total / shares * s + total % shares * s / shares; }

// The row tile of a place: the last of n with place_at <= place, 32 probes at a time.  Whole warps.
__device__ __forceinline__ int find_rt(const ChunkArgs &a, int n, int64_t place) {
    const int lane = threadIdx.x & 31;
    int lo = 0;
    while (n > 1) {
        const int step = (n + 31) / 32, at = lo + lane * step;
        const bool below = lane * step < n && __ldg(a.place_at + at) <= place;
        const int last = 31 - __clz(__ballot_sync(0xFFFFFFFFu, below));
        lo += last * step;
        n = min(step, n - last * step);
    }
    return lo;
}

__device__ __forceinline__ Walk walk_of(const ChunkArgs &a, const SmallPlan *small, int share) {
    Walk w;
    w.small = small;
    w.places = small ? small->places : __ldg(a.head);
    const int shares = w.shares = small ? small->shares : (int)__ldg(a.head + 2);
    const int64_t total = w.places * a.c.heads;
    w.units = small ? small->units : (int)__ldg(a.head + 1);
    w.at = share < shares ? share_at(total, shares, share) : 0;
    w.hi = share < shares ? share_at(total, shares, share + 1) : 0;
    w.h = w.places > 0 ? (int)(w.at / w.places) : 0;
    w.rt = 0;
    if (w.at >= w.hi) return w;
    const int64_t place = w.at - w.h * w.places;
    if (!small) w.rt = find_rt(a, w.units, place);
    else
        while (w.rt + 1 < w.units && small->place_at[w.rt + 1] <= place) ++w.rt;
    return w;
}

__device__ __forceinline__ void load_record(const ChunkArgs &a, int rt, ChunkRecord &r) {
    const int4 *p = reinterpret_cast<const int4 *>(a.records + rt);
    const int4 x = __ldg(p), y = __ldg(p + 1), z = __ldg(p + 2);
    r.b = x.x, r.q0 = x.y, r.e0 = x.z, r.row0 = x.w;
    r.rows = y.x, r.begin = y.y, r.end = y.z, r.base = y.w;
    r.tiles = z.x, r.all_end = z.y, r.all_begin = z.z, r.pad = 0;
}

// A row tile of sequence b, whose n new tokens' rows begin at q0.
template <typename C>
__device__ __forceinline__ void make_record(const ChunkArgs &a, int b, int q0, int n, int len, int tile, ChunkRecord &r) {
    r.b = b, r.q0 = q0, r.e0 = len - n + 1;
    r.row0 = tile * C::ROWS;
    r.rows = min(C::ROWS, n * a.group - r.row0);
    const int first = token_of(a, r.row0), last = token_of(a, r.row0 + r.rows - 1);  // tokens
    auto begin = [&](int tok) { return a.window > 0 && (int64_t)r.e0 + tok > a.window ? (int)(r.e0 + tok - a.window) : 0; };
    r.begin = begin(first), r.end = max(0, r.e0 + last);
    r.all_begin = begin(last), r.all_end = max(0, r.e0 + first);
    r.base = r.begin / C::BN;
    r.tiles = max(1, (int)(((int64_t)r.end + C::BN - 1) / C::BN) - r.base);
    r.pad = 0;
}
template <typename C>
__device__ __forceinline__ void small_record(const ChunkArgs &a, const SmallPlan &p, int rt, ChunkRecord &r) {
    int b = 0;
    for (int i = 1; i < a.c.batch; ++i)
        if (p.rt_at[i] <= rt) b = i;
    make_record<C>(a, b, p.seq_at[b], p.seq_at[b + 1] - p.seq_at[b], p.len[b], rt - p.rt_at[b], r);
}

template <typename C>
__device__ __forceinline__ bool next_unit(const ChunkArgs &a, Walk &w, Unit &u) {
    while (w.at < w.hi) {
        const int64_t first = w.h * w.places + (w.small ? (int64_t)w.small->place_at[w.rt] : __ldg(a.place_at + w.rt));
        if (w.small) small_record<C>(a, *w.small, w.rt, u);
        else load_record(a, w.rt, u);
        u.h = w.h, u.rt = w.rt;
        const int length = u.tiles + kExtra, lo = (int)(w.at - first);
        const int hi = w.hi - first < length ? (int)(w.hi - first) : length;
        w.at += hi - lo;
        if (hi == length && ++w.rt == w.units) w.rt = 0, ++w.h;
        u.lo = lo, u.hi = min(hi, u.tiles);
        u.whole = lo == 0 && u.hi == u.tiles;
        if (u.lo < u.hi) return true;
    }
    return false;
}

// ---------------------------------------------------------------- the list

// As many shares as there are CTAs; for less work one a unit or tile.
__device__ __forceinline__ int shares_of(const ChunkArgs &a, int row_tiles, int64_t places) {
    const int64_t units = (int64_t)row_tiles * a.c.heads, most = max(units, places * a.c.heads - kExtra * units);
    return most < 1 ? 1 : most < a.shares ? (int)most : a.shares;
}

// The list of a small call by one warp; CTA 0's leaves the records for join_kernel.
template <typename C>
__device__ __forceinline__ void small_plan(const ChunkArgs &a, SmallPlan &p) {
    const int lane = threadIdx.x & 31, B = a.c.batch;  // B < 32
    auto sum_before = [&](int v, int &all) {
        int s = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xFFFFFFFFu, s, o);
            if (lane >= o) s += t;
        }
        all = __shfl_sync(0xFFFFFFFFu, s, 31);
        return s - v;
    };
    const int raw = lane <= B ? __ldg(a.starts + lane) : 0, len = lane < B ? __ldg(a.seq_lens + lane) : 0;
    int s = min(max(raw, 0), (int)a.T);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s = max(s, t);
    }
    const bool bad = (lane <= B && s != raw) || (lane < B && len > a.c.capacity);
    const int next = __shfl_down_sync(0xFFFFFFFFu, s, 1), n = lane < B ? next - s : 0;
    int R, all;
    const int first = sum_before((int)(((int64_t)n * a.group + C::ROWS - 1) / C::ROWS), R);
    if (lane <= B) p.seq_at[lane] = s;
    if (lane < B) p.len[lane] = min(max(len, 0), a.c.capacity), p.rt_at[lane] = first;
    __syncwarp();
    ChunkRecord r = {};
    if (lane < R) small_record<C>(a, p, lane, r);
    const int at = sum_before(lane < R ? r.tiles + kExtra : 0, all);
    if (lane < R) p.place_at[lane] = at;
    if (lane == 0) {
        p.place_at[R] = all;
        p.places = all, p.units = R, p.shares = shares_of(a, R, all);
    }
    if (blockIdx.x == 0) {
        if (lane < R) a.records[lane] = r;
        if (bad) atomicOr(a.c.status, kDevIndex);
    }
}

__device__ __forceinline__ int64_t plan_scan(int64_t v, int64_t &total, int64_t *scratch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t sum = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += t;
    }
    if (lane == 31) scratch[warp] = sum;
    __syncthreads();
    int64_t of = scratch[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(0xFFFFFFFFu, of, o);
        if (lane >= o) of += t;
    }
    total = __shfl_sync(0xFFFFFFFFu, of, 31);
    const int64_t before = __shfl_sync(0xFFFFFFFFu, of, warp > 0 ? warp - 1 : 0);
    __syncthreads();
    return sum - v + (warp > 0 ? before : 0);
}

// Largest of the values of earlier threads (0: none).
__device__ __forceinline__ int plan_max(int v, int *scratch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int top = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xFFFFFFFFu, top, o);
        if (lane >= o) top = max(top, t);
    }
    if (lane == 31) scratch[warp] = top;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before = max(before, scratch[w]);
    const int own = __shfl_up_sync(0xFFFFFFFFu, top, 1);
    __syncthreads();
    return max(before, lane > 0 ? own : 0);
}

template <typename C>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const ChunkArgs a) {
    __shared__ int64_t scratch[32];
    __shared__ int first_row[kPlanBatch + 1], first_tile[kPlanBatch + 1];
    pdl_wait();
    pdl_trigger();
    const int B = a.c.batch, tid = threadIdx.x;
    int *const seq_at = B <= kPlanBatch ? first_row : a.seq_at, *const rt_at = B <= kPlanBatch ? first_tile : a.rt_at;
    bool bad = false;
    // chunks: starts, made to not decrease
    const int per = (B + kPlanThreads) / kPlanThreads;  // of batch + 1 values
    const int first = min(tid * per, B + 1), last = min(first + per, B + 1);
    int top = 0;
    auto start = [&](int b) {
        const int s = __ldg(a.starts + b), t = min(max(s, 0), (int)a.T);
        if (s != t || t < top) bad = true;
        return top = max(top, t);
    };
    for (int b = first; b < last; ++b) top = max(top, min(max(__ldg(a.starts + b), 0), (int)a.T));
    top = plan_max(top, reinterpret_cast<int *>(scratch));
    for (int b = first; b < last; ++b) seq_at[b] = start(b);
    __syncthreads();
    int64_t units = 0, all_units;
    auto units_of = [&](int b) {
        const int64_t rows = (int64_t)(seq_at[b + 1] - seq_at[b]) * a.group;
        return (rows + C::ROWS - 1) / C::ROWS;
    };
    for (int b = first; b < min(last, B); ++b) {
        units += units_of(b);
        const int len = __ldg(a.seq_lens + b);
        if (len > a.c.capacity) bad = true;
    }
    units = plan_scan(units, all_units, scratch);
    for (int b = first; b < min(last, B); ++b) {
        rt_at[b] = (int)units;
        units += units_of(b);
    }
    if (tid == 0) rt_at[B] = (int)all_units;
    __syncthreads();
    // places of each unit
    const int R = (int)all_units, per_rt = (R + kPlanThreads - 1) / kPlanThreads;
    const int rt0 = min(tid * per_rt, R), rt1 = min(rt0 + per_rt, R);
    int b = 0;
    if (rt0 < rt1) {  // the sequence of rt0
        int lo = 0, hi = B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (rt_at[mid] <= rt0) lo = mid;
            else hi = mid;
        }
        b = lo;
    }
    auto record = [&](int rt, int &of, ChunkRecord &r) {
        while (rt_at[of + 1] <= rt) ++of;
        make_record<C>(a, of, seq_at[of], seq_at[of + 1] - seq_at[of], min(max(__ldg(a.seq_lens + of), 0), a.c.capacity), rt - rt_at[of], r);
        return r.tiles + kExtra;
    };
    int64_t sum = 0, all;
    int of = b;
    ChunkRecord r;
    for (int rt = rt0; rt < rt1; ++rt) sum += record(rt, of, r);
    sum = plan_scan(sum, all, scratch);
    of = b;
    for (int rt = rt0; rt < rt1; ++rt) {
        a.place_at[rt] = sum;
        sum += record(rt, of, r);
        a.records[rt] = r;
    }
    if (tid == 0) {
        a.place_at[R] = all;
        a.head[0] = all;
        a.head[1] = R;
        a.head[2] = shares_of(a, R, all);
    }
    if (bad) atomicOr(a.c.status, kDevIndex);
}

// ---------------------------------------------------------------- pieces of the main kernel

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)v));
    return r;
}
__device__ __forceinline__ float lo_f32(uint32_t bf16x2) { return __uint_as_float(bf16x2 << 16); }
__device__ __forceinline__ float hi_f32(uint32_t bf16x2) { return __uint_as_float(bf16x2 & 0xFFFF0000u); }

template <int N>
__device__ __forceinline__ void set_regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Instruction descriptor of kind::f16 with fp32 accumulators: [7,10) and [10,13) the operands' format (0 f16, 1 bf16),
// [16] B is MN-major.
__host__ __device__ constexpr uint32_t idesc_of(int M, int N, bool f16, bool b_mn) {
    return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// An MN-major operand with 128-byte swizzle: rows (of K) of 64 values, groups of 8 of them 1024 bytes apart (stride
// offset), blocks of 64 values `block` bytes apart (leading offset).
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t block) {
    return umma_desc_sw128(addr) - ((uint64_t)1 << 16) + ((uint64_t)(block >> 4) << 16);
}

// Does a pair of 16-bit values hold one that is not finite?
template <bool F16>
__device__ __forceinline__ uint32_t not_finite(uint32_t pair) {
    constexpr uint32_t kExp = F16 ? 0x7C00u : 0x7F80u;
    return ((pair & kExp) == kExp ? 0x0000FFFFu : 0u) | ((pair >> 16 & kExp) == kExp ? 0xFFFF0000u : 0u);
}

// Four lanes' four 16-byte values, turned about: lane i of the four gets value i of lane k into w[k].
__device__ __forceinline__ void transpose4(uint4 (&w)[4], int lane) {
    auto swap = [&](uint4 &x, uint4 &y, int bit) {  // lanes without the bit give y and get x's place
        const bool up = lane & bit;
        const uint4 s = up ? x : y;
        uint4 g;
        g.x = __shfl_xor_sync(0xFFFFFFFFu, s.x, bit), g.y = __shfl_xor_sync(0xFFFFFFFFu, s.y, bit);
        g.z = __shfl_xor_sync(0xFFFFFFFFu, s.z, bit), g.w = __shfl_xor_sync(0xFFFFFFFFu, s.w, bit);
        if (up) x = g;
        else y = g;
    };
    swap(w[0], w[1], 1), swap(w[2], w[3], 1);
    swap(w[0], w[2], 2), swap(w[1], w[3], 2);
}

// Takes the values that are not finite out of eight; were there any?
template <bool F16>
__device__ __forceinline__ bool finite_only(uint4 &v) {
    const uint32_t b0 = not_finite<F16>(v.x), b1 = not_finite<F16>(v.y), b2 = not_finite<F16>(v.z), b3 = not_finite<F16>(v.w);
    v.x &= ~b0, v.y &= ~b1, v.z &= ~b2, v.w &= ~b3;
    return b0 | b1 | b2 | b3;
}

struct Bars {
    uint32_t full, empty, s_full, p_full, o_full, q_full, q_free, pv_done, done, raw;
};

// A row of a unit: where it is and what it sees.
struct Row {
    int64_t q_row;        // of q and o
    int head, e, bgn;     // sees the slots [bgn, e)
    bool real;            // (the last tile of a sequence may have fewer rows)
    // row_in: of the unit
    __device__ __forceinline__ void of(const ChunkArgs &a, const Unit &u, int row_in) {
        const int row = u.row0 + row_in;
        real = row_in < u.rows;
        const int tok = real ? token_of(a, row) : 0;
        q_row = (int64_t)u.q0 + tok;
        head = u.h * a.group + (real ? row - tok * a.group : 0);
        e = real ? u.e0 + tok : 0;
        bgn = a.window > 0 && e > a.window ? (int)(e - a.window) : 0;
    }
};

// A tensor copy of box_slots slots of one head into shared memory, counted in bytes on `bar`; slots_at, head: its coordinates.
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap &m, int value, int slot, int head, int page, bool head_first,
                                         uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(&m)), "r"(value), "r"(head_first ? head : slot), "r"(head_first ? slot : head), "r"(page), "r"(bar)
        : "memory");
}

// c tanh(s / c) in units of log2 for a large cap c, s = score * cc / log2(e).  The form by the exponential is off by 3 10^-7 c (the roundings
// of 1 + e^(2 s / c) and of its reciprocal), however small s is: it would lose scores far below the cap.  They have the odd series,
// off by 2^-26 of s up to |s / c| = 1/4; above that 3 10^-7 c is 2^-19 of s.
__device__ __forceinline__ float large_cap(float score, float cc, const ChunkArgs &a) {
    const float t = score * (cc * a.cap_t), t2 = t * t;
    const float series = fmaf(t2, fmaf(t2, fmaf(t2, fmaf(t2, 62.f / 2835.f, -17.f / 315.f), 2.f / 15.f), -1.f / 3.f), 1.f);
    const float far = fmaf(-2.f, rcp_approx(1.f + ex2_approx(t * (2.f * kLog2e))), 1.f) * fminf(a.softcap * kLog2e, 3.4e38f);
    return fabsf(t) < 0.25f ? score * cc * series : far;
}

// SMALL: the CTAs list the work themselves.  CAP: a softcap, taken in the weights' pass (without it a softcap counts as a special
// case, a pass of its own).
template <typename C, bool SMALL, bool CAP>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const ChunkArgs a, const __grid_constant__ CUtensorMap k_map,
                                                            const __grid_constant__ CUtensorMap v_map) {
    constexpr int D = C::D, BN = C::BN, NT = C::NT, NS = C::NS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *const base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t q_smem = smem_u32(base), ring = q_smem + C::QBYTES, raw = ring + NS * C::SLOT, misc = raw + 2 * C::RAW;
    uint8_t *const misc_p = base + C::QBYTES + NS * C::SLOT + 2 * C::RAW;
    Bars bar;
    bar.full = misc, bar.empty = bar.full + 8 * NS, bar.s_full = bar.empty + 8 * NS, bar.p_full = bar.s_full + 16;
    bar.o_full = bar.p_full + 16, bar.q_full = bar.o_full + 16, bar.q_free = bar.q_full + 16, bar.pv_done = bar.q_free + 16, bar.done = bar.pv_done + 16, bar.raw = misc + 256;
    uint32_t *const tmem_holder = reinterpret_cast<uint32_t *>(misc_p + 512);
    volatile int *const abort_flag = reinterpret_cast<volatile int *>(misc_p + 516);
    volatile int *const bad_pages = reinterpret_cast<volatile int *>(misc_p + 524); // a page id was out of range
    // 1 + the last tile of slots walked in which a value that is not finite was taken out (0: none); of an e4m3 cache one for each
    // copying warp (512 tokens after 65536: 624 us, 637 by an atomic maximum of one; a bf16 cache's mixed step: 78 us by that, 81 by four)
    volatile int *const bad_seen = reinterpret_cast<volatile int *>(misc_p + 528);
    volatile uint8_t *const q_factor = misc_p + 768 + C::PLAN;  // [C::FACTORS][C::ROWS]: exponents (biased by 127) of the factors
    volatile uint32_t *const page_mask = reinterpret_cast<volatile uint32_t *>(misc_p + 640);      // [kMetaRing][4]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned int *const status = a.c.status;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(bar.full + 8 * i, kCopyWarps);
            mbar_init(bar.empty + 8 * i, 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(bar.s_full + 8 * t, 1);
            mbar_init(bar.p_full + 8 * t, 4);
            mbar_init(bar.o_full + 8 * t, 1);
            mbar_init(bar.q_full + 8 * t, NT == 2 ? 1 : 2);  // the warps that bring a tile's queries
            mbar_init(bar.q_free + 8 * t, 1);
            mbar_init(bar.pv_done + 8 * t, 1);
        }
        mbar_init(bar.done, NT == 2 ? 1 : 2);
        for (int i = 0; i < 2 * kCopyWarps; ++i) mbar_init(bar.raw + 8 * i, 1);
        *abort_flag = 0;
        for (int i = 0; i < kCopyWarps; ++i) bad_seen[i] = 0;
        *bad_pages = 0;
        fence_mbar_init();
    }
    static_assert(sizeof(SmallPlan) <= C::PLAN, "fits");
    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(tmem_holder), C::COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    pdl_wait();
    pdl_trigger();
    SmallPlan *const small = SMALL ? reinterpret_cast<SmallPlan *>(misc_p + 768) : nullptr;
    if constexpr (SMALL) {
        __builtin_assume(small != nullptr);
        if (warp == 0) small_plan<C>(a, *small);
        __syncthreads();
    }
    Walk walk = walk_of(a, small, blockIdx.x);
    Unit u;

    if (warp < 8) {
        // -------------------------------------------------------- softmax, one row a thread
        set_regs_up<C::REGS>();
        const int t = warp >> 2, row_in = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t o_col = tmem + lanes + C::O_COL + t * D;
        uint32_t s_count = 0, unit_phase = 0;  // tiles and units that this tile of rows has had
        uint32_t tile_count = 0;               // tiles of slots walked (index into the page masks)
        bool ok = true;
        // the next unit that has rows in this tile
        auto advance = [&](Unit &n) {
            while (next_unit<C>(a, walk, n)) {
                if (t * 128 < n.rows) return true;
                tile_count += (uint32_t)(n.hi - n.lo);
            }
            return false;
        };
        Row r;
        uint32_t units = 0;
        if (threadIdx.x == 0) a.joins[blockIdx.x] = make_int4(0, 0, 0, 0);
        for (bool more = t < NT && advance(u); more; more = advance(u), ++units) {
            r.of(a, u, t * 128 + row_in);
            // no row of this warp is there: whatever its scores and weights are (of large calls too few units to look for it: 1 to 2 %)
            const bool none = SMALL && t * 128 + (warp & 3) * 32 >= u.rows;
            // ---- what the tile's rows see
            // every row of the tile sees slots below all_end and from all_begin on
            const int last_tok = token_of(a, min(t * 128 + 127, u.rows - 1) + u.row0);
            const uint32_t all_end = (uint32_t)max(0, u.e0 + token_of(a, u.row0 + t * 128));
            const uint32_t all_begin = a.window > 0 && (int64_t)u.e0 + last_tok > a.window ? (uint32_t)(u.e0 + last_tok - a.window) : 0u;
            float cc = a.scale_log2, f = a.softcap > 0.f ? 1.f : cc;  // a score's factor, to log2
            // neg: -m f, or 0 where there is no maximum yet (rows that are not there have one: 0)
            float m = r.real ? -INFINITY : 0.f, l = 0.f, m_next = m, neg = 0.f;
            // what holds for all rows of the warp: a maximum is to be raised; each has one, and none is far from 0
            bool pending = false, usual = false, far = false;
            // the running maximum becomes m_next; O and l follow
            auto raise = [&](bool has_o) {
                const float neg_new = m_next == -INFINITY ? 0.f : -m_next * f;
                const float fac = m == m_next || m == -INFINITY ? 1.f : ex2_approx(neg_new - neg);
                m = m_next, neg = neg_new;
                far = __any_sync(0xFFFFFFFFu, fabsf(neg) > kFar);
                usual = usual && !far;
                pending = false;
                l *= fac;
                if (!has_o) return true;
                if constexpr (NT == 1) {  // the product before must have ended
                    const uint32_t before = s_count - 2;  // (s_count counts this tile already)
                    if (!__all_sync(0xFFFFFFFFu, mbar_wait(bar.pv_done + 8 * (before & 1), before >> 1 & 1, status))) return false;
                    tc_fence_after();
                }
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld32(o_col + 32 * c, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * fac);
                    tmem_st16(o_col + 32 * c, *reinterpret_cast<uint32_t(*)[16]>(o));
                    tmem_st16(o_col + 32 * c + 16, *reinterpret_cast<uint32_t(*)[16]>(o + 16));
                }
                tmem_st_wait();
                return true;
            };
            for (int i = u.lo; i < u.hi; ++i, ++tile_count) {
                // heads of 256: the two buffers in turn, each with its barriers
                const uint32_t odd = s_count & 1, at = NT == 2 ? (uint32_t)t : odd, phase = NT == 2 ? odd : s_count >> 1 & 1;
                ++s_count;
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(bar.s_full + 8 * at, phase, status))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (none) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar.p_full + 8 * at);
                    continue;
                }
                if constexpr (C::E4M3) {
                    if (i == u.lo) {  // (written before the tile's queries were there)
                        // (not 0, with which a masked score would give NaN)
                        cc = fmaxf(a.scale_log2 * __uint_as_float((uint32_t)q_factor[units % C::FACTORS * C::ROWS + t * 128 + row_in] << 23), 1.17549435e-38f);
                        cc = fminf(cc, a.cc_max);
                        f = a.softcap > 0.f ? 1.f : cc;
                    }
                }
                const uint32_t s_col = tmem + lanes + C::S_COL + at * BN;
                uint32_t s[2][32];
                tmem_ld32(s_col, s[0]);
                const uint32_t j0 = (uint32_t)(u.base + i) * BN;
                const bool pages = *bad_pages != 0, masked = j0 + BN > all_end || j0 < all_begin;
                if (pending && !raise(i > u.lo)) {
                    ok = false;
                    break;
                }
                float2 f2 = make_float2(f, f), n2 = make_float2(neg + C::LIFT, neg + C::LIFT);
                bool prepare = masked || pages || !usual, fresh = true;
                for (;;) {
                    if (prepare) {
                        // ---- a unit's first tile, its edges, a score far above the maximum, soft caps, scales that are not positive,
                        // pages out of range, maxima far from 0: the scores as the weights' pass takes them, 32 slots at a time,
                        // back in their place where they change, and their maximum
                        tmem_ld_wait();
                        const int from = (int)max((int64_t)0, (int64_t)r.bgn - j0), to = (int)min((int64_t)BN, (int64_t)r.e - j0);
                        const float in = a.cap_in * cc, out = a.softcap * kLog2e;
                        uint32_t(&v)[32] = s[0];
                        float mx = -INFINITY;
#pragma unroll 1
                        for (int c = 0; c < BN / 32; ++c) {
                            uint32_t there = 0xFFFFFFFFu;  // a bit for each slot that the row sees
                            if (fresh && (masked || pages)) {
                                if (pages) there = page_mask[(tile_count & (kMetaRing - 1)) * 4 + c];
                                const int lo = from - 32 * c, hi = to - 32 * c;
                                there &= lo <= 0 ? 0xFFFFFFFFu : lo >= 32 ? 0u : 0xFFFFFFFFu << lo;
                                there &= hi >= 32 ? 0xFFFFFFFFu : hi <= 0 ? 0u : (1u << hi) - 1u;
                            }
                            bool changed = __any_sync(0xFFFFFFFFu, there != 0xFFFFFFFFu);
                            if (changed && !__any_sync(0xFFFFFFFFu, there != 0)) {
#pragma unroll
                                for (int k = 0; k < 32; ++k) v[k] = 0xFF800000u;
                            } else {
                                tmem_ld32(s_col + 32 * c, v);
                                tmem_ld_wait();
                                if (fresh && a.odd_scale) {
#pragma unroll
                                    for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * a.score_sign);
                                    changed = true;
                                }
                                if (fresh && a.softcap > 0.f) {
                                    // c tanh(s / c) = c (1 - 2 / (1 + e^(2 s / c))), in units of log2
                                    if (!SMALL && !CAP && a.large_cap) {
#pragma unroll
                                        for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(large_cap(__uint_as_float(v[k]), cc, a));
                                    } else {
#pragma unroll
                                        for (int k = 0; k < 32; ++k)
                                            v[k] = __float_as_uint(fmaf(-2.f * out, rcp_approx(1.f + ex2_approx(__uint_as_float(v[k]) * in)), out));
                                    }
                                    changed = true;
                                }
                                if (__any_sync(0xFFFFFFFFu, there != 0xFFFFFFFFu)) {
#pragma unroll
                                    for (int k = 0; k < 32; ++k) v[k] = there >> k & 1u ? v[k] : 0xFF800000u;
                                }
                                float top[2] = {mx, -INFINITY};
#pragma unroll
                                for (int k = 0; k < 32; k += 2) top[k / 2 & 1] = fmaxf(fmaxf(top[k / 2 & 1], __uint_as_float(v[k])), __uint_as_float(v[k + 1]));
                                mx = fmaxf(top[0], top[1]);
                            }
                            if (changed) {
                                tmem_st16(s_col + 32 * c, *reinterpret_cast<uint32_t(*)[16]>(v));
                                tmem_st16(s_col + 32 * c + 16, *reinterpret_cast<uint32_t(*)[16]>(v + 16));
                            }
                        }
                        tmem_st_wait();
                        if (m == -INFINITY ? mx > -INFINITY : (mx - m) * f > kSlack) m_next = mx;
                        if (__any_sync(0xFFFFFFFFu, m_next != m) && !raise(i > u.lo)) {
                            ok = false;
                            break;
                        }
                        pending = false;
                        usual = (CAP || a.softcap == 0.f) && !a.odd_scale && !far && !__any_sync(0xFFFFFFFFu, m == -INFINITY);
                        n2 = make_float2(neg + C::LIFT, neg + C::LIFT);
                        if (far) {  // the product of the maximum is not to be rounded by itself
                            const float m0 = m == -INFINITY ? 0.f : m;
#pragma unroll 1
                            for (int c = 0; c < BN / 32; ++c) {
                                tmem_ld32(s_col + 32 * c, v);
                                tmem_ld_wait();
#pragma unroll
                                for (int k = 0; k < 32; ++k) v[k] = __float_as_uint((__uint_as_float(v[k]) - m0) * f);
                                tmem_st16(s_col + 32 * c, *reinterpret_cast<uint32_t(*)[16]>(v));
                                tmem_st16(s_col + 32 * c + 16, *reinterpret_cast<uint32_t(*)[16]>(v + 16));
                            }
                            tmem_st_wait();
                            f2 = make_float2(1.f, 1.f), n2 = make_float2(C::LIFT, C::LIFT);
                        }
                        tmem_ld32(s_col, s[0]);
                    }
                    // ---- weights by the maximum so far, in one pass; a larger one counts from the next tile on
                    uint32_t p[BN / 2];
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    float top[2] = {-INFINITY, -INFINITY};
                    tmem_ld_wait();
#pragma unroll
                    for (int c = 0; c < BN / 32; ++c) {
                        if (c + 1 < BN / 32) tmem_ld32(s_col + 32 * (c + 1), s[(c + 1) & 1]);
                        uint32_t (&v)[32] = s[c & 1];
                        if constexpr (CAP) {
                            if (!prepare) {
                                const float2 in2 = make_float2(a.cap_in * cc, a.cap_in * cc), one = make_float2(1.f, 1.f);
                                const float2 out2 = make_float2(a.softcap * kLog2e, a.softcap * kLog2e), less = make_float2(-2.f * out2.x, -2.f * out2.x);
#pragma unroll
                                for (int k = 0; k < 32; k += 2) {
                                    const float2 e = fma2(make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), in2, make_float2(0.f, 0.f));
                                    const float2 d = add2(make_float2(ex2_approx(e.x), ex2_approx(e.y)), one);
                                    const float2 x = fma2(make_float2(rcp_approx(d.x), rcp_approx(d.y)), less, out2);
                                    v[k] = __float_as_uint(x.x), v[k + 1] = __float_as_uint(x.y);
                                }
                            }
                        }
#pragma unroll
                        for (int k = 0; k < 32; k += 2) {
                            const float x = __uint_as_float(v[k]), y = __uint_as_float(v[k + 1]);
                            top[k / 2 & 1] = fmaxf(fmaxf(top[k / 2 & 1], x), y);
                            const float2 z = fma2(make_float2(x, y), f2, n2);
                            const float2 e = make_float2(ex2_approx(z.x), ex2_approx(z.y));
                            sum[k / 2 & 1] = add2(sum[k / 2 & 1], e);
                            p[16 * c + k / 2] = C::E4M3 ? pack_f16(e.x, e.y) : pack_bf16(e.x, e.y);
                        }
                        if (c + 1 < BN / 32) tmem_ld_wait();
                    }
                    const float mx = fmaxf(top[0], top[1]), above = far ? 0.f : (mx - m) * f;
                    pending = __any_sync(0xFFFFFFFFu, above > kSlack);
                    if (pending && __any_sync(0xFFFFFFFFu, above > C::JUMP)) {  // the maximum first, then once more
                        pending = false;
                        fresh = fresh && !prepare;
                        prepare = true;
                        tmem_ld32(s_col, s[0]);
                        continue;
                    }
                    if (above > kSlack) m_next = mx;
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
#pragma unroll
                    for (int c = 0; c < BN / 32; ++c) tmem_st16(s_col + 16 * c, *reinterpret_cast<uint32_t(*)[16]>(p + 16 * c));
                    break;
                }
                if (!ok) break;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar.p_full + 8 * at);
            }
            if (!ok) break;
            // ---- the unit's end
            const int64_t q_row = r.q_row;
            const int head = r.head, e = r.e, bgn = r.bgn;
            const bool real = r.real;
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(bar.o_full + 8 * t, unit_phase, status))) {
                ok = false;
                break;
            }
            unit_phase ^= 1;
            tc_fence_after();
            // in this unit's part, or one of a few that the copies are ahead
            uint32_t mark = (uint32_t)bad_seen[0];
            if constexpr (C::E4M3) {
#pragma unroll
                for (int i = 1; i < kCopyWarps; ++i) mark = max(mark, (uint32_t)bad_seen[i]);
            }
            const bool bad = mark > tile_count - (uint32_t)(u.hi - u.lo);
            // a row that sees slots, all of them -infinity, has no weights: NaN, as 0 / 0 has it
            const float inv = e > bgn ? a.v_scale / l : 0.f;
            const int64_t part_row = (int64_t)(2 * blockIdx.x + (u.lo > 0 ? 0 : 1)) * C::ROWS + t * 128 + row_in;
#pragma unroll 1
            for (int c = none ? D / 32 : 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(o_col + 32 * c, o);
                tmem_ld_wait();
                if (bad && real) {
                    // values that are not finite in tiles that not every row of the unit sees (the copies took them out)
                    for (int i = u.lo; i < u.hi; ++i) {
                        const int64_t j0 = (int64_t)(u.base + i) * BN;
                        if (j0 + BN <= u.all_end && j0 >= u.all_begin) continue;
                        const int64_t to = min((int64_t)e, j0 + BN);
                        for (int64_t j = max((int64_t)bgn, j0); j < to; ++j) {
                            const uint32_t pg = page_of(a.c, (uint32_t)j);
                            const int32_t page = __ldg(a.c.table + u.b * a.c.ld_table + pg);
                            if (!page_ok(a.c, page)) continue;
                            const uint8_t *v = a.c.v + row_bytes_at(a.c, page, u.h, (uint32_t)j - pg * a.c.page_size);
#pragma unroll
                            for (int k = 0; k < 32; ++k) {
                                float x;
                                if constexpr (C::E4M3) x = e4m3_to_f32(v[32 * c + k]);
                                else x = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(v)[32 * c + k] << 16);
                                if (!isfinite(x)) o[k] = __float_as_uint(__uint_as_float(o[k]) + x);
                            }
                        }
                    }
                }
                // a thread has 32 values of its row; four lanes exchange theirs, so that they write four rows one after the
                // other, 64 bytes (or 128) of each at a time instead of 16 bytes of 32 rows
                if (u.whole) {
                    uint4 w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t x[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const float lo = __uint_as_float(o[8 * k + 2 * y]) * inv, hi = __uint_as_float(o[8 * k + 2 * y + 1]) * inv;
                            x[y] = e > bgn ? pack_bf16(lo, hi) : 0u;
                        }
                        w[k] = make_uint4(x[0], x[1], x[2], x[3]);
                    }
                    transpose4(w, lane);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int64_t to = __shfl_sync(0xFFFFFFFFu, real ? q_row * a.ldo + (int64_t)head * D : (int64_t)-1, (lane & ~3) + k);
                        if (to >= 0) reinterpret_cast<uint4 *>(a.o + to + 32 * c)[lane & 3] = w[k];
                    }
                } else {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint4 w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            w[k] = make_uint4(o[16 * half + 4 * k], o[16 * half + 4 * k + 1], o[16 * half + 4 * k + 2], o[16 * half + 4 * k + 3]);
                        transpose4(w, lane);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int row = t * 128 + (row_in & ~3) + k;
                            if (row < u.rows)
                                reinterpret_cast<uint4 *>(a.parts + (part_row - row_in - t * 128 + row) * D + 32 * c + 16 * half)[lane & 3] = w[k];
                        }
                    }
                }
            }
            if (threadIdx.x == 0 && u.lo == 0 && !u.whole) {
                // the share that begins a unit it does not end: join_kernel finds the parts from here
                const int shares = walk.shares;
                const int64_t total = walk.places * a.c.heads;
                const int64_t end = u.h * walk.places + (small ? (int64_t)small->place_at[u.rt] : __ldg(a.place_at + u.rt)) + u.tiles;
                int parts = 2;
                while ((int)blockIdx.x + parts < shares && share_at(total, shares, blockIdx.x + parts) < end) ++parts;
                a.joins[blockIdx.x] = make_int4(u.rt, u.h, parts, 0);
            }
            if (!u.whole && real) a.part_ml[part_row] = make_float2(m == -INFINITY ? -INFINITY : -neg, l);
            tc_fence_before();
        }
        if (!ok && lane == 0) *abort_flag = 1;
    } else if (warp < kCopyWarp) {
        set_regs_down<C::OTHER_REGS>();
        if (warp < kMmaWarp + (NT == 2 ? 1 : 2) && elect_one()) {
            // ---------------------------------------------------- MMA
            // Two tiles of rows: one thread issues a tile's P V and next Q K^T, then the other's, so that while one's run the
            // softmax of the other has the SM's other pipes for itself.  (Issued by two threads they interleave, both end
            // together, and so do the two softmaxes that follow: 4 % slower.)  Heads of
            // 256: a thread for each product.
            constexpr uint32_t kQk = idesc_of(128, BN, C::E4M3, false), kPv = idesc_of(128, D, C::E4M3, true);
            const bool qks = NT == 2 || warp == kMmaWarp, pvs = NT == 2 || warp != kMmaWarp;
            const uint64_t q_desc = umma_desc_sw128(q_smem), k_desc = umma_desc_sw128(ring), v_desc = desc_mn(ring, BN * 128);
            uint32_t slot = 0, full_phase = 0;     // the ring tile that is next
            uint32_t phase = 0, unit_phase = 0;    // of p_full (NT 2), of q_full: a bit for each tile of rows
            uint32_t count = 0;                    // tiles of slots done (NT 1: buffers and their phases go by it)
            bool ok = true;
            auto wait_full = [&] {
                const bool r = mbar_wait(bar.full + 8 * slot, full_phase, status);
                tc_fence_after();
                return r;
            };
            auto next_slot = [&] {
                if (++slot == NS) slot = 0, full_phase ^= 1;
            };
            auto qk = [&](int t, uint32_t buf) {
                const uint64_t kd = k_desc + (uint64_t)(slot * (C::SLOT >> 4)), qd = q_desc + (uint64_t)(t * (128 * D * 2 >> 4));
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    umma_bf16(tmem + C::S_COL + buf * BN, qd + (k / 4) * (128 * 128 >> 4) + 2 * (k % 4),
                              kd + (k / 4) * (BN * 128 >> 4) + 2 * (k % 4), kQk, k != 0);
                umma_commit(bar.s_full + 8 * buf);
            };
            auto pv = [&](int t, uint32_t buf, uint32_t of, bool first) {
                const uint64_t vd = v_desc + (uint64_t)(of * (C::SLOT >> 4));
#pragma unroll
                for (int k = 0; k < BN / 16; ++k)
                    umma_bf16_ts(tmem + C::O_COL + t * D, tmem + C::S_COL + buf * BN + 8 * k, vd + k * (16 * 128 >> 4), kPv, !first || k != 0);
            };
            while (ok && next_unit<C>(a, walk, u)) {
                const int tiles = u.hi - u.lo;
                if (*abort_flag) {
                    ok = false;
                    break;
                }
                if constexpr (NT == 2) {
                    const int nt = u.rows > 128 ? 2 : 1;
                    // the ring holds keys and values in turn: K(0) V(0) K(1) V(1) ...
                    if (!(ok = wait_full())) break;
                    for (int t = 0; t < nt && ok; ++t) {
                        if (!(ok = mbar_wait(bar.q_full + 8 * t, unit_phase >> t & 1, status))) break;
                        unit_phase ^= 1u << t;
                        tc_fence_after();
                        qk(t, t);
                        if (tiles == 1) umma_commit(bar.q_free + 8 * t);
                    }
                    if (!ok) break;
                    umma_commit(bar.empty + 8 * slot);
                    next_slot();
                    for (int i = 0; i < tiles && ok; ++i) {
                        const uint32_t v_slot = slot;
                        const bool last = i + 1 == tiles;
                        for (int t = 0; t < nt; ++t) {
                            if (t == 0 && !(ok = wait_full())) break;
                            if (!(ok = mbar_wait(bar.p_full + 8 * t, phase >> t & 1, status))) break;
                            phase ^= 1u << t;
                            tc_fence_after();
                            pv(t, t, v_slot, i == 0);
                            if (last) {
                                umma_commit(bar.o_full + 8 * t);
                                continue;
                            }
                            if (t == 0) {
                                next_slot();
                                if (!(ok = wait_full())) break;
                            }
                            qk(t, t);
                            if (i + 2 == tiles) umma_commit(bar.q_free + 8 * t);  // the unit's last scores
                        }
                        if (!ok) break;
                        umma_commit(bar.empty + 8 * v_slot);
                        if (!last) umma_commit(bar.empty + 8 * slot);
                        next_slot();
                    }
                } else {
                    if (qks) {
                        if (!(ok = mbar_wait(bar.q_full, unit_phase, status))) break;
                        unit_phase ^= 1;
                    }
                    for (int i = 0; i < tiles; ++i, ++count) {
                        const uint32_t buf = count & 1, of = count >> 1 & 1;
                        if (qks) {
                            if (!(ok = wait_full())) break;
                            // the weights that lay in this buffer have been read
                            if (count >= 2 && !(ok = mbar_wait(bar.pv_done + 8 * buf, of ^ 1, status))) break;
                            tc_fence_after();
                            qk(0, buf);
                            if (i + 1 == tiles) umma_commit(bar.q_free);
                            umma_commit(bar.empty + 8 * slot);
                        }
                        next_slot();
                        if (pvs) {
                            if (!(ok = mbar_wait(bar.p_full + 8 * buf, of, status)) || !(ok = wait_full())) break;
                            pv(0, buf, slot, i == 0);
                            umma_commit(bar.pv_done + 8 * buf);
                            if (i + 1 == tiles) umma_commit(bar.o_full);
                            umma_commit(bar.empty + 8 * slot);
                        }
                        next_slot();
                    }
                }
            }
            if (!ok) *abort_flag = 1;
            umma_commit(bar.done);
        } else if (warp >= kQueryWarp) {
            // ---------------------------------------------------- queries
            // A warp brings a tile's 128 rows (heads of 256: 64 of them each), as soon as the scores of the unit before are done.
            constexpr int LANES = D / 8 < 32 ? D / 8 : 32, AT_ONCE = 32 / LANES;  // of a row, 16 bytes each; rows of an access
            constexpr int ROWS = NT == 2 ? 128 : 64;
            const int t = NT == 2 ? warp - kQueryWarp : 0, row0 = NT == 2 ? 0 : (warp - kQueryWarp) * 64;
            const int c = lane % LANES;
            const uint32_t dst = q_smem + t * (128 * D * 2) + (c / 8) * (128 * 128);
            uint32_t units = 0;
            bool ok = true;
            while (ok && next_unit<C>(a, walk, u)) {
                if (t * 128 >= u.rows) continue;
                if (units > 0 && (!__all_sync(0xFFFFFFFFu, mbar_wait(bar.q_free + 8 * t, (units - 1) & 1, status)) || *abort_flag)) {
                    ok = false;
                    break;
                }
                // (of a small call 32 rows of which none is there are left as they are: their softmax warp does not look at them)
                const int end = SMALL ? min(row0 + ROWS, u.rows - t * 128) : row0 + ROWS;
                for (int r0 = row0; r0 < end; r0 += 32) {
                    Row r;
                    r.of(a, u, t * 128 + r0 + lane);
                    const int64_t at = r.real ? r.q_row * a.ldq + (int64_t)r.head * D : -1;
#pragma unroll 4
                    for (int s = 0; s < 32; s += AT_ONCE) {
                        const int row = r0 + s + lane / LANES;
                        const int64_t from = __shfl_sync(0xFFFFFFFFu, at, s + lane / LANES);
                        const uint4 *src = reinterpret_cast<const uint4 *>(a.q + (from >= 0 ? from : 0)) + c;
                        const uint32_t to = dst + row * 128 + ((c ^ row) & 7) * 16;
                        cp_async16(to, src, from >= 0 ? 16u : 0u);
                    }
                }
                cp_async_commit();
                cp_async_wait<0>();
                if constexpr (C::E4M3) {
                    // to f16 in their place, a lane a row: a power of two takes the row's largest value to [2^14, 2^15)
                    __syncwarp();
                    for (int r0 = row0; r0 < end; r0 += 32) {
                        const int row = r0 + lane;
                        const uint32_t at = q_smem + t * (128 * D * 2) + row * 128;
                        uint32_t top = 0;
#pragma unroll 4
                        for (int x = 0; x < D / 8; ++x) {
                            const uint4 v = lds128(at + (x / 8) * (128 * 128) + ((x ^ row) & 7) * 16);
                            const uint32_t p = max(max(v.x << 16 & 0x7FFFFFFFu, v.x & 0x7FFF0000u), max(v.y << 16 & 0x7FFFFFFFu, v.y & 0x7FFF0000u));
                            top = max(max(top, p), max(max(v.z << 16 & 0x7FFFFFFFu, v.z & 0x7FFF0000u), max(v.w << 16 & 0x7FFFFFFFu, v.w & 0x7FFF0000u)));
                        }
                        const int ex = (int)(top >> 23);
                        // (a row that is not finite gives NaN either way)
                        const int shift = ex == 255 ? 0 : min(127 + 14 - ex, 126);
                        const float f = __uint_as_float((uint32_t)(127 + shift) << 23);
#pragma unroll 4
                        for (int x = 0; x < D / 8; ++x) {
                            const uint32_t to = at + (x / 8) * (128 * 128) + ((x ^ row) & 7) * 16;
                            uint4 v = lds128(to);
                            v.x = pack_f16(lo_f32(v.x) * f, hi_f32(v.x) * f), v.y = pack_f16(lo_f32(v.y) * f, hi_f32(v.y) * f);
                            v.z = pack_f16(lo_f32(v.z) * f, hi_f32(v.z) * f), v.w = pack_f16(lo_f32(v.w) * f, hi_f32(v.w) * f);
                            sts128(to, v);
                        }
                        // the way back, for the row's softmax (which has read those that lay here, see FACTORS)
                        q_factor[units % C::FACTORS * C::ROWS + t * 128 + row] = (uint8_t)(127 - shift);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar.q_full + 8 * t);
                ++units;
            }
            if (!ok && lane == 0) *abort_flag = 1;
        }
    } else {
        // -------------------------------------------------------- copies
        set_regs_down<C::OTHER_REGS>();
        const int w = warp - kCopyWarp;
        // A cached row is copied by as many lanes as 128 bytes of it have 16-byte pieces, block of 64 values after block, so
        // that an access takes whole lines and a row's offset serves several.
        constexpr int E = C::E4M3 ? 1 : 2;               // bytes of a value
        constexpr int LANES = D * E < 128 ? D * E / 16 : 8;  // of a row
        constexpr int PIECES = D * E / (16 * LANES);     // of a row, for a lane
        constexpr int AT_ONCE = 32 / LANES;              // rows of a warp's access
        constexpr int WROWS = BN / kCopyWarps;           // rows of a warp
        constexpr int STEPS = WROWS / AT_ONCE;
        const int sub = lane / LANES, chunk = lane % LANES;
        uint32_t issued = 0, shown = 0;
        uint32_t slot = 0, parity = 1;                   // where the next tile goes; its slot's phase before
        uint32_t show_slot = 0;
        uint32_t tile_count = 0;
        uint32_t edge_bits = 0;  // of the tiles on their way, newest in bit 0: values to be checked?
        // where 16-byte piece c of row r (of this warp's) lies in a tile
        auto place = [&](int r, int c) {
            const int row = w * WROWS + r;
            return (uint32_t)((c / 8) * (BN * 128) + row * 128 + ((c ^ row) & 7) * 16);
        };
        // this warp's part of a tile has landed: checked if need be, and shown to the MMAs
        auto check = [&](uint32_t at) {
            bool any = false;
#pragma unroll 2
            for (int s = 0; s < STEPS; ++s) {
#pragma unroll
                for (int x = 0; x < PIECES; ++x) {
                    const uint32_t p = at + place(s * AT_ONCE + sub, chunk + LANES * x);
                    uint4 v = lds128(p);
                    if (finite_only<false>(v)) {
                        sts128(p, v);
                        any = true;
                    }
                }
            }
            if (any) atomicMax(const_cast<int *>(bad_seen), (int)(shown / 2) + 1);  // (keys and values in turn)
        };
        uint32_t box_bits = 0;   // of the tiles on their way, newest in bit 0: copied by the copy engine?
        auto show = [&](uint32_t upto) {
            while (shown != upto) {
                const uint32_t back = issued - 1 - shown;
                if (!(box_bits >> back & 1u)) {  // (what the copy engine brings counts on the barrier by itself)
                    if (edge_bits >> back & 1u) check(ring + show_slot * C::SLOT);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar.full + 8 * show_slot);
                }
                if (++show_slot == NS) show_slot = 0;
                ++shown;
            }
        };
        // the tile after this one: its page is looked up while this one is copied
        int i = 0, page = 0;
        uint32_t in_page = 0;
        bool seen = false;       // does this lane's row hold a slot that some row of the unit sees?
        auto look_up = [&] {
            const uint32_t j = (uint32_t)(u.base + i) * BN + w * WROWS + lane;
            seen = lane < WROWS && j >= (uint32_t)u.begin && j < (uint32_t)u.end;
            if (seen) {
                const uint32_t pg = page_of(a.c, j);
                in_page = j - pg * a.c.page_size;
                page = __ldg(a.c.table + u.b * a.c.ld_table + pg);
            }
        };
        bool ok = true, more = next_unit<C>(a, walk, u);
        if (more) {
            i = u.lo;
            look_up();
        }
        auto step = [&] {  // to the next tile, whose page is looked up
            if (++i == u.hi) {
                more = next_unit<C>(a, walk, u);
                i = u.lo;
            }
            if (more) look_up();
        };
        if constexpr (C::E4M3) {
            // ---- an e4m3 cache: a tile's bytes come into this warp's part of a buffer of their own, one tile ahead, by the copy
            // engine where the rows are all there, and go from there, as f16, into the ring
            struct Tile {
                int64_t off;
                int page, in, h;
                uint32_t mask;
                bool edge, boxes, first;  // first: of a unit's part
            };
            const uint32_t own = raw + w * (WROWS * D);
            uint32_t raw_phase = 0;
            auto tile_of = [&] {
                Tile n;
                const bool there = !seen || page_ok(a.c, page);
                if (!there) {
                    atomicOr(status, kDevIndex);
                    *bad_pages = 1;
                }
                n.off = seen && there ? row_bytes_at(a.c, page, u.h, in_page) : 1;
                n.page = page, n.in = (int)in_page, n.h = u.h;
                n.first = i == u.lo;
                n.mask = __ballot_sync(0xFFFFFFFFu, there);
                const uint32_t j0 = (uint32_t)(u.base + i) * BN;
                n.edge = j0 + BN > (uint32_t)u.all_end || j0 < (uint32_t)u.all_begin;
                n.boxes = a.box_slots > 0 && __all_sync(0xFFFFFFFFu, lane >= WROWS || (seen && there));
                return n;
            };
            auto fetch = [&](const Tile &n, int kv) {
                const uint32_t to = own + kv * C::RAW;
                if (n.boxes) {
                    const int row = lane * a.box_slots;
                    const int pg = __shfl_sync(0xFFFFFFFFu, n.page, row & 31), in = __shfl_sync(0xFFFFFFFFu, n.in, row & 31);
                    const uint32_t rb = bar.raw + 16 * w + 8 * kv;
                    if (lane == 0) mbar_arrive_expect_tx(rb, WROWS * D);
                    __syncwarp();
                    if (row < WROWS) copy_box(to + row * D, kv == 0 ? k_map : v_map, 0, in, n.h, pg, a.head_first != 0, rb);
                } else {
                    const uint8_t *const pool = (kv == 0 ? a.c.k : a.c.v) + 16 * chunk;
#pragma unroll
                    for (int s = 0; s < STEPS; ++s) {
                        const int64_t o = __shfl_sync(0xFFFFFFFFu, n.off, s * AT_ONCE + sub);
                        const uint32_t bytes = o & 1 ? 0u : 16u;
                        const uint8_t *const src = o & 1 ? pool : pool + o;
#pragma unroll
                        for (int x = 0; x < PIECES; ++x)
                            cp_async16(to + (s * AT_ONCE + sub) * D + 16 * (chunk + LANES * x), src + 16 * LANES * x, bytes);
                    }
                    cp_async_commit();
                }
            };
            Tile now = {}, next = {};
            bool flying = false;  // copies of the copy engine that have not been waited for
            bool any = more;
            if (more) {
                now = tile_of();
                fetch(now, 0), fetch(now, 1);
                flying = now.boxes;
                step();
            }
            for (; any && ok; ++tile_count) {
                const bool follows = more;
                if (follows) {
                    next = tile_of();
                    step();
                }
                if (lane == 0) {
                    if constexpr (WROWS == 32) page_mask[(tile_count & (kMetaRing - 1)) * 4 + w] = now.mask;
                    else reinterpret_cast<volatile uint16_t *>(page_mask)[(tile_count & (kMetaRing - 1)) * 8 + w] = (uint16_t)now.mask;
                }
                // keys and values together: what a wait, a fence or a copy's start costs is paid once (but a unit's first scores
                // do not wait for values)
                const uint32_t slot1 = slot + 1 < NS ? slot + 1 : 0, parity1 = slot + 1 < NS ? parity : parity ^ 1;
                bool here = issued < (uint32_t)NS || (mbar_wait(bar.empty + 8 * slot, parity, status) && mbar_wait(bar.empty + 8 * slot1, parity1, status));
                if (now.boxes) {
                    here = here && mbar_wait(bar.raw + 16 * w, raw_phase, status) && mbar_wait(bar.raw + 16 * w + 8, raw_phase, status);
                } else {
                    cp_async_wait<0>();
                }
                if (!__all_sync(0xFFFFFFFFu, here) || *abort_flag) {
                    ok = false;
                    break;
                }
                if (now.boxes) raw_phase ^= 1, flying = false;
                bool odd = false;
                constexpr int GROUP = STEPS * PIECES < 4 ? STEPS * PIECES : 4;  // pieces read at a time
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const uint32_t from = own + kv * C::RAW + sub * D + 16 * chunk, at = ring + (kv == 0 ? slot : slot1) * C::SLOT;
#pragma unroll
                    for (int g = 0; g < STEPS * PIECES; g += GROUP) {
                        uint4 v[GROUP];
#pragma unroll
                        for (int x = 0; x < GROUP; ++x) v[x] = lds128(from + (g + x) / PIECES * AT_ONCE * D + 16 * LANES * ((g + x) % PIECES));
#pragma unroll
                        for (int x = 0; x < GROUP; ++x) {
                            uint4 lo = make_uint4(e4m3x2_to_f16x2(v[x].x), e4m3x2_to_f16x2(v[x].x >> 16), e4m3x2_to_f16x2(v[x].y), e4m3x2_to_f16x2(v[x].y >> 16));
                            uint4 hi = make_uint4(e4m3x2_to_f16x2(v[x].z), e4m3x2_to_f16x2(v[x].z >> 16), e4m3x2_to_f16x2(v[x].w), e4m3x2_to_f16x2(v[x].w >> 16));
                            if (kv == 1 && now.edge) odd |= finite_only<true>(lo) | finite_only<true>(hi);
                            const int r = (g + x) / PIECES * AT_ONCE + sub, c = 2 * (chunk + LANES * ((g + x) % PIECES));
                            sts128(at + place(r, c), lo);
                            sts128(at + place(r, c + 1), hi);
                        }
                    }
                    if (kv == 0 && now.first) {
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar.full + 8 * slot);
                    }
                }
                if (odd) bad_seen[w] = (int)tile_count + 1;
                fence_proxy_async_smem();  // for the MMAs, and for the copy engine, which may write what has been read
                __syncwarp();
                if (lane == 0 && !now.first) mbar_arrive(bar.full + 8 * slot);
                if (lane == 0) mbar_arrive(bar.full + 8 * slot1);
                issued += 2;
                slot += 2;
                if (slot >= (uint32_t)NS) slot -= NS, parity ^= 1;
                if (follows) {
                    fetch(next, 0), fetch(next, 1);
                    flying = next.boxes;
                }
                now = next;
                any = follows;
            }
            cp_async_wait<0>();
            if (!ok) {
                if (lane == 0) *abort_flag = 1;
                for (int kv = 0; kv < 2 && flying; ++kv) (void)mbar_wait(bar.raw + 16 * w + 8 * kv, raw_phase, status);
            }
        } else {
            for (; more; ++tile_count) {
                const bool there = !seen || page_ok(a.c, page);
                if (!there) {
                    atomicOr(status, kDevIndex);
                    *bad_pages = 1;
                }
                // this lane's row: its offset, or 1 (offsets are multiples of 16) where nothing is to be read
                const int64_t off = seen && there ? row_bytes_at(a.c, page, u.h, in_page) : 1;
                const uint32_t mask = __ballot_sync(0xFFFFFFFFu, there);
                const uint32_t j0 = (uint32_t)(u.base + i) * BN;
                const bool edge = j0 + BN > (uint32_t)u.all_end || j0 < (uint32_t)u.all_begin;
                // rows that are all there come by the copy engine, in boxes within a page (values only where every row sees them)
                const bool boxes = a.box_slots > 0 && __all_sync(0xFFFFFFFFu, lane >= WROWS || (seen && there));
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const uint32_t eb = bar.empty + 8 * slot;
                    if (issued >= (uint32_t)NS && !__all_sync(0xFFFFFFFFu, mbar_test_wait(eb, parity))) {
                        cp_async_wait<0>();  // nothing is held back while this waits
                        show(issued);
                        if (!__all_sync(0xFFFFFFFFu, mbar_wait(eb, parity, status)) || *abort_flag) {
                            ok = false;
                            break;
                        }
                    }
                    if (kv == 0 && lane == 0) {  // (heads of 256: 16 slots a warp, two warps' bits in a word)
                        if constexpr (WROWS == 32) page_mask[(tile_count & (kMetaRing - 1)) * 4 + w] = mask;
                        else reinterpret_cast<volatile uint16_t *>(page_mask)[(tile_count & (kMetaRing - 1)) * 8 + w] = (uint16_t)mask;
                    }
                    const uint8_t *const pool = (kv == 0 ? a.c.k : a.c.v) + 16 * chunk;
                    const uint32_t at = ring + slot * C::SLOT;
                    if (boxes && !(kv == 1 && edge)) {
                        // lane x: block x % (D / 64) of box x / (D / 64)
                        const int row = lane / (D / 64) * a.box_slots, block = lane % (D / 64);
                        const int pg = __shfl_sync(0xFFFFFFFFu, page, row & 31), in = __shfl_sync(0xFFFFFFFFu, (int)in_page, row & 31);
                        if (lane == 0) mbar_arrive_expect_tx(bar.full + 8 * slot, WROWS * D * 2);
                        __syncwarp();
                        if (row < WROWS)
                            copy_box(at + block * (BN * 128) + (w * WROWS + row) * 128, kv == 0 ? k_map : v_map, 64 * block, in, u.h, pg,
                                     a.head_first != 0, bar.full + 8 * slot);
                        cp_async_commit();  // (an empty group: the count of those on their way is that of tiles)
                    } else {
#pragma unroll
                        for (int s = 0; s < STEPS; ++s) {
                            const int64_t o = __shfl_sync(0xFFFFFFFFu, off, s * AT_ONCE + sub);
                            const uint32_t bytes = o & 1 ? 0u : 16u;
                            const uint8_t *const src = o & 1 ? pool : pool + o;
#pragma unroll
                            for (int x = 0; x < PIECES; ++x) cp_async16(at + place(s * AT_ONCE + sub, chunk + LANES * x), src + 16 * LANES * x, bytes);
                        }
                        cp_async_commit();
                    }
                    ++issued;
                    if (++slot == NS) slot = 0, parity ^= 1;
                    edge_bits = edge_bits << 1 | (uint32_t)(kv == 1 && edge);
                    box_bits = box_bits << 1 | (uint32_t)(boxes && !(kv == 1 && edge));
                    constexpr uint32_t kAhead = C::NS - 2;  // tiles on their way
                    if (issued - shown > kAhead) {
                        cp_async_wait<kAhead>();
                        show(issued - kAhead);
                    }
                }
                if (!ok) break;
                step();
            }
            cp_async_wait<0>();
            if (ok) {
                show(issued);
            } else if (lane == 0) {
                *abort_flag = 1;
                // the copy engine's copies land before this CTA leaves (a barrier that others left short of arrivals runs out)
                for (uint32_t n = issued > (uint32_t)NS ? issued - NS : 0; n < issued; ++n)
                    if (box_bits >> (issued - 1 - n) & 1u) (void)mbar_wait_limit(bar.full + 8 * (n % NS), n / NS & 1, status, 10000000ull);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        (void)mbar_wait(bar.done, 0, status);  // no MMA still runs
        tc_fence_after();
        tmem_dealloc(tmem, C::COLS);
    }
}

// ---------------------------------------------------------------- joining

// CTA (s, y): the unit that share s begins and does not end, if there is one; each warp some of its rows.
template <typename C>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const ChunkArgs a) {
    constexpr int D = C::D, PER = D / 32;
    pdl_wait();
    pdl_trigger();
    const int4 what = __ldg(a.joins + blockIdx.x);
    const int s = blockIdx.x, h = what.y, parts = what.z;
    if (parts == 0) return;
    ChunkRecord u;
    load_record(a, what.x, u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int row_in = blockIdx.y * kJoinWarps + warp; row_in < u.rows; row_in += gridDim.y * kJoinWarps) {
        // part k of the row: of share s + k
        auto part = [&](int k) { return (int64_t)(2 * (s + k) + (k == 0 ? 1 : 0)) * C::ROWS + row_in; };
        const float2 nothing = make_float2(-INFINITY, 0.f);
        float2 own = lane < parts ? __ldcg(a.part_ml + part(lane)) : nothing;  // (a lane's first part stays at hand)
        float m = own.x;
        bool number = own.x == own.x;
        for (int k = lane + 32; k < parts; k += 32) {
            const float x = __ldcg(a.part_ml + part(k)).x;
            m = fmaxf(m, x);
            if (x != x) number = false;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        if (!__all_sync(0xFFFFFFFFu, number)) m = __uint_as_float(0x7FC00000u);
        float l = 0.f, o[PER] = {};
        for (int k0 = 0; k0 < parts; k0 += 4) {  // four parts' values on their way at once
            float x[4][PER], w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = k0 + i;
                float2 ml = make_float2(__shfl_sync(0xFFFFFFFFu, own.x, k & 31), __shfl_sync(0xFFFFFFFFu, own.y, k & 31));
                if (k >= 32 && k < parts) ml = __ldcg(a.part_ml + part(k));
                const bool there = k < parts && !(ml.x == -INFINITY && ml.y == 0.f);  // (it saw something)
                w[i] = there ? ex2_approx(ml.x - m) : 0.f;
                if (there) l = fmaf(ml.y, w[i], l);
                const float2 *p = reinterpret_cast<const float2 *>(a.parts + part(there ? k : 0) * D + lane * PER);
#pragma unroll
                for (int y = 0; y < PER; y += 2) {
                    const float2 t = there ? __ldcg(p + y / 2) : make_float2(0.f, 0.f);
                    x[i][y] = t.x, x[i][y + 1] = t.y;
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int y = 0; y < PER; ++y) o[y] = fmaf(x[i][y], w[i], o[y]);
        }
        const int row = u.row0 + row_in, tok = token_of(a, row), e = u.e0 + tok;
        const int bgn = a.window > 0 && e > a.window ? (int)(e - a.window) : 0;
        const float inv = a.v_scale / l;
        uint32_t *dst = reinterpret_cast<uint32_t *>(a.o + ((int64_t)u.q0 + tok) * a.ldo + (int64_t)(h * a.group + row - tok * a.group) * D + lane * PER);
#pragma unroll
        for (int x = 0; x < PER; x += 2) dst[x / 2] = e > bgn ? pack_bf16(o[x] * inv, o[x + 1] * inv) : 0u;
    }
}

template <typename C, bool SMALL, bool CAP>
cudaError_t launch(const DeviceInfo &di, ChunkArgs &a, cudaStream_t s) {
    // setmaxnreg moves registers within what the launch holds: 128 a thread, or the split would wait forever
    static const bool fits = [] {
        cudaFuncAttributes f;
        return cudaFuncGetAttributes(&f, chunk_kernel<C, SMALL, CAP>) == cudaSuccess && 4 * f.numRegs >= 2 * (C::REGS + C::OTHER_REGS);
    }();
    if (!fits) return cudaErrorInvalidConfiguration;
    cudaError_t e = ensure_smem((const void *)chunk_kernel<C, SMALL, CAP>, C::SMEM);
    if (e != cudaSuccess) return e;
    a.shares = di.sm_count < kMaxChunkShares ? di.sm_count : kMaxChunkShares;
    if (!SMALL && (e = launch_pdl(plan_kernel<C>, dim3(1), dim3(kPlanThreads), 0, s, dim3(1), a)) != cudaSuccess) return e;
    // boxes of what divides a page, of 8 (a swizzle atom) to 32 slots (a warp's rows; 16 of heads of 256): blocks of 64 values,
    // or whole rows of an e4m3 cache
    CUtensorMap k_map = {}, v_map = {};
    int box = 1;
    while (box < C::BN / kCopyWarps && a.c.page_size % (2 * box) == 0) box *= 2;
    bool head_first = false;
    const int values = C::E4M3 ? C::D : 64;
    const bool maps = box >= 8 && make_cache_tmap(&k_map, a.c.k, a.c, values, box, !C::E4M3, &head_first) &&
                      make_cache_tmap(&v_map, a.c.v, a.c, values, box, !C::E4M3, &head_first);
    a.box_slots = maps ? box : 0;
    a.head_first = head_first;
    if ((e = launch_pdl(chunk_kernel<C, SMALL, CAP>, dim3(a.shares), dim3(kThreads), C::SMEM, s, dim3(1), a, k_map, v_map)) != cudaSuccess) return e;
    // a warp a row
    const int64_t rows = a.T * a.group;
    const int y = (int)(((rows < C::ROWS ? rows : C::ROWS) + kJoinWarps - 1) / kJoinWarps);
    return launch_pdl(join_kernel<C>, dim3(a.shares, y), dim3(kJoinWarps * 32), 0, s, dim3(1), a);
}


template <typename C>
cudaError_t launch(const DeviceInfo &di, ChunkArgs &a, cudaStream_t s) {
    // Few sequences and row tiles: every CTA lists them itself, a launch less (33 tokens of one sequence: 18.2 us, 20.3 with
    // plan_kernel).  The branch inside one kernel costs the others 1 to 5 %: registers.
    const int64_t units = a.T * a.group / C::ROWS + (a.c.batch < a.T ? a.c.batch : a.T);
    bool small = a.c.batch < kSmall && units <= kSmall;
    // (a factor of infinity would give no number for a score of 0)
    a.cc_max = a.softcap > 0.f ? 3e38f / a.cap_in : INFINITY;
    if (!C::E4M3) a.scale_log2 = a.scale_log2 < a.cc_max ? a.scale_log2 : a.cc_max;
    a.large_cap = a.softcap > C::LARGE_CAP;
    a.cap_t = a.large_cap ? 0.69314718f / a.softcap : 0.f;
    // A large cap is a special case of the kernel for large calls (5.4 us for two tiles of 128 rows and 128 slots): its code in the
    // small calls' kernel costs each of them (512 tokens after 65536 from an e4m3 cache: 638 us instead of 624).
    if (a.large_cap) return launch<C, false, false>(di, a, s);
    if (a.softcap > 0.f) {
        // A soft cap within the weights' pass: 3.4 us for two tiles of 128 rows and 128 slots, 4.4 as a special case (heads of
        // 128).  A small call's kernel has only the latter: where its CTAs may have more than a few tiles each, not that one.
        if (units * a.c.heads * (a.c.capacity / C::BN) > 8 * (int64_t)di.sm_count) small = false;
        if (!small) return launch<C, false, true>(di, a, s);
    }
    return small ? launch<C, true, false>(di, a, s) : launch<C, false, false>(di, a, s);
}

}  // namespace

int chunk_rows(int D) { return D == 256 ? Cfg<256, false>::ROWS : Cfg<128, false>::ROWS; }

cudaError_t launch_attn_chunk(const DeviceInfo &di, ChunkArgs &a, cudaStream_t s) {
    switch (a.c.dim) {
    case 64: return a.c.e4m3 ? launch<Cfg<64, true>>(di, a, s) : launch<Cfg<64, false>>(di, a, s);
    case 128: return a.c.e4m3 ? launch<Cfg<128, true>>(di, a, s) : launch<Cfg<128, false>>(di, a, s);
    default: return a.c.e4m3 ? launch<Cfg<256, true>>(di, a, s) : launch<Cfg<256, false>>(di, a, s);
    }
}

}  // namespace q4k
