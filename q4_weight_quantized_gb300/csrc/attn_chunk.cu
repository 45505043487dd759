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
//     threads: S of a tile is there only after the O of the tile before.  (Heads of 256: one tile of rows, two buffers
//     of S instead; there the rare rescale waits for the product before.)
//   - Work is one list of places (KV head, unit, tile of slots) cut into equal contiguous shares, one per CTA, whatever
//     the lengths are; units that a share does not hold as a whole leave (m, l, o') in the workspace for join_kernel.
//   - Four warps copy keys and values row by row, 16 bytes a lane, into the swizzled layout the MMAs read (any page
//     size, any strides).  An e4m3 cache's values become f16 on the way, exactly, and Q f16 by a power of two a row.
// A slot that some rows of a unit see and others do not may hold values that are not finite: those are taken out of the
// product (0 * infinity would reach every row) and added to the rows that see them at the end.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "decode_ops.h"
#include "q4k_ptx.cuh"

namespace q4k {
namespace {

constexpr int kThreads = 512;          // warps 0-3 and 4-7: softmax of a tile of rows each; 8: MMA; 12-15: copies
constexpr int kMmaWarp = 8, kCopyWarp = 12, kCopyWarps = 4;
constexpr int kSoftmaxRegs = 184, kOtherRegs = 72;  // together those of the launch: 2 * (184 + 72) = 4 * 128
constexpr int kPlanThreads = 1024;
constexpr int kJoinWarps = 8;
constexpr int kMetaRing = 8;           // tiles whose page masks are kept: more than the ring holds
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;          // how far (log2) a score may exceed the running maximum
constexpr int kMinPlaces = 2;          // tiles of a share, at least

template <int D_, bool E4M3_>
struct Cfg {
    static constexpr int D = D_;
    static constexpr bool E4M3 = E4M3_;
    static constexpr int NT = D == 256 ? 1 : 2;        // tiles of 128 rows of a unit
    static constexpr int BN = D == 256 ? 64 : 128;     // slots of a tile
    static constexpr int ROWS = NT * 128;
    static constexpr int SLOT = BN * D * 2;            // bytes of a tile of keys or values in shared memory
    static constexpr int NS = D == 64 ? 8 : 5;         // such tiles in the ring, keys and values in turn
    static constexpr int LAG = NS - 2;                 // of which so many may be on their way
    // weights in f16 are kept as 2^7 p, in o' and l alike: at most 2^15, and what lies below 2^-32 of the largest is lost
    static constexpr float LIFT = E4M3 ? 7.f : 0.f;
    static constexpr int QBYTES = ROWS * D * 2;
    static constexpr int MISC = 1024;
    static constexpr int SMEM = QBYTES + NS * SLOT + MISC + 1024;  // (+ slack to align the base)
    static constexpr uint32_t S_COL = 0, O_COL = NT == 2 ? 2 * BN : 2 * BN;
    static constexpr uint32_t COLS = 512;
    static_assert(O_COL + NT * D <= COLS && SMEM <= 227 * 1024, "fits");
};

// What every role needs to know of a unit and of its share's part of it.
struct Unit {
    int b, h, n, e0;          // sequence, KV head, new tokens, end of token 0's slots
    int64_t q0;               // first row of the sequence in q and o
    int row0, rows;           // rows of the unit within the sequence
    int64_t base;             // its first tile of slots
    int64_t tiles, lo, hi;    // number of them, and the share's
    int end, begin;           // slots that any row sees
    bool whole;
};

struct Walk {
    int64_t at, hi, places;
    int h, rt;
};

__device__ __forceinline__ int64_t share_at(int64_t total, int shares, int s) { return total / shares * s + total % shares * s / shares; }

__device__ __forceinline__ int find_rt(const ChunkArgs &a, int n, int64_t place) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.place_at + mid) <= place) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ Walk walk_of(const ChunkArgs &a, int share) {
    Walk w;
    w.places = __ldg(a.head);
    const int shares = (int)__ldg(a.head + 2);
    const int64_t total = w.places * a.c.heads;
    w.at = share < shares ? share_at(total, shares, share) : 0;
    w.hi = share < shares ? share_at(total, shares, share + 1) : 0;
    w.h = w.places > 0 ? (int)(w.at / w.places) : 0;
    w.rt = w.at < w.hi ? find_rt(a, (int)__ldg(a.head + 1), w.at - w.h * w.places) : 0;
    return w;
}

// The unit of row tile rt: everything but the share's part.
template <typename C>
__device__ __forceinline__ void unit_of(const ChunkArgs &a, int rt, Unit &u) {
    u.b = __ldg(a.rt_seq + rt);
    const int s0 = __ldg(a.seq_at + u.b);
    u.n = __ldg(a.seq_at + u.b + 1) - s0;
    u.q0 = s0;
    const int len = min(max(__ldg(a.seq_lens + u.b), 0), a.c.capacity);
    u.e0 = len - u.n + 1;
    u.row0 = (rt - __ldg(a.rt_at + u.b)) * C::ROWS;
    u.rows = min(C::ROWS, u.n * a.group - u.row0);
    u.end = max(0, u.e0 + (u.row0 + u.rows - 1) / a.group);
    const int64_t begin = (int64_t)u.e0 + u.row0 / a.group - a.window;
    u.begin = a.window > 0 && begin > 0 ? (int)begin : 0;
    u.base = u.begin / C::BN;
    u.tiles = max((int64_t)1, ((int64_t)u.end + C::BN - 1) / C::BN - u.base);
}

template <typename C>
__device__ __forceinline__ bool next_unit(const ChunkArgs &a, Walk &w, Unit &u) {
    if (w.at >= w.hi) return false;
    unit_of<C>(a, w.rt, u);
    u.h = w.h;
    u.lo = w.at - w.h * w.places - __ldg(a.place_at + w.rt);
    u.hi = min(u.tiles, u.lo + (w.hi - w.at));
    u.whole = u.lo == 0 && u.hi == u.tiles;
    w.at += u.hi - u.lo;
    if (u.hi == u.tiles && ++w.rt == (int)__ldg(a.head + 1)) w.rt = 0, ++w.h;
    return true;
}

// ---------------------------------------------------------------- the list

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
    pdl_wait();
    pdl_trigger();
    const int B = a.c.batch, tid = threadIdx.x;
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
    for (int b = first; b < last; ++b) a.seq_at[b] = start(b);
    __syncthreads();
    int64_t units = 0, all_units;
    auto units_of = [&](int b) {
        const int64_t rows = (int64_t)(a.seq_at[b + 1] - a.seq_at[b]) * a.group;
        return (rows + C::ROWS - 1) / C::ROWS;
    };
    for (int b = first; b < min(last, B); ++b) {
        units += units_of(b);
        const int len = __ldg(a.seq_lens + b);
        if (len > a.c.capacity) bad = true;
    }
    units = plan_scan(units, all_units, scratch);
    for (int b = first; b < min(last, B); ++b) {
        a.rt_at[b] = (int)units;
        units += units_of(b);
    }
    if (tid == 0) a.rt_at[B] = (int)all_units;
    __syncthreads();
    // places of each unit
    const int R = (int)all_units, per_rt = (R + kPlanThreads - 1) / kPlanThreads;
    const int rt0 = min(tid * per_rt, R), rt1 = min(rt0 + per_rt, R);
    int b = 0;
    if (rt0 < rt1) {  // the sequence of rt0
        int lo = 0, hi = B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.rt_at[mid] <= rt0) lo = mid;
            else hi = mid;
        }
        b = lo;
    }
    auto places = [&](int rt, int &of) {
        while (a.rt_at[of + 1] <= rt) ++of;
        const int n = a.seq_at[of + 1] - a.seq_at[of], len = min(max(__ldg(a.seq_lens + of), 0), a.c.capacity), e0 = len - n + 1;
        const int row0 = (rt - a.rt_at[of]) * C::ROWS, rows = min(C::ROWS, n * a.group - row0);
        const int end = max(0, e0 + (row0 + rows - 1) / a.group);
        const int64_t begin = (int64_t)e0 + row0 / a.group - a.window;
        return max((int64_t)1, ((int64_t)end + C::BN - 1) / C::BN - (a.window > 0 && begin > 0 ? begin : 0) / C::BN);
    };
    int64_t sum = 0, all;
    int of = b;
    for (int rt = rt0; rt < rt1; ++rt) sum += places(rt, of);
    sum = plan_scan(sum, all, scratch);
    of = b;
    for (int rt = rt0; rt < rt1; ++rt) {
        a.place_at[rt] = sum;
        sum += places(rt, of);
        a.rt_seq[rt] = of;
    }
    if (tid == 0) {
        a.place_at[R] = all;
        a.head[0] = all;
        a.head[1] = R;
        const int64_t most = all * a.c.heads / kMinPlaces;
        a.head[2] = most < 1 ? 1 : most < a.shares ? most : a.shares;
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

struct Bars {
    uint32_t full, empty, s_full, p_full, o_full, q_full, pv_done, done;
};

template <typename C>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const ChunkArgs a) {
    constexpr int D = C::D, BN = C::BN, NT = C::NT, NS = C::NS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *const base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t q_smem = smem_u32(base), ring = q_smem + C::QBYTES, misc = ring + NS * C::SLOT;
    uint8_t *const misc_p = base + C::QBYTES + NS * C::SLOT;
    Bars bar;
    bar.full = misc, bar.empty = bar.full + 8 * NS, bar.s_full = bar.empty + 8 * NS, bar.p_full = bar.s_full + 16;
    bar.o_full = bar.p_full + 16, bar.q_full = bar.o_full + 16, bar.pv_done = bar.q_full + 16, bar.done = bar.pv_done + 8;
    uint32_t *const tmem_holder = reinterpret_cast<uint32_t *>(misc_p + 512);
    volatile int *const abort_flag = reinterpret_cast<volatile int *>(misc_p + 516);
    volatile uint32_t *const bad_unit = reinterpret_cast<volatile uint32_t *>(misc_p + 544);       // [8]
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
            mbar_init(bar.q_full + 8 * t, 4);
        }
        mbar_init(bar.pv_done, 1);
        mbar_init(bar.done, 1);
        *abort_flag = 0;
        for (int i = 0; i < 8; ++i) bad_unit[i] = 0;
        fence_mbar_init();
    }
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
    Walk walk = walk_of(a, blockIdx.x);
    Unit u;

    if (warp < 8) {
        // -------------------------------------------------------- softmax, one row a thread
        set_regs_up<kSoftmaxRegs>();
        const int t = warp >> 2, row_in = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t o_col = tmem + lanes + C::O_COL + t * D;
        uint32_t s_count = 0, unit_phase = 0, seq = 0;  // tiles and units that this tile of rows has had, units walked
        int64_t tile_count = 0;  // tiles of slots walked (index into the page masks)
        bool ok = t < NT;
        for (; ok && next_unit<C>(a, walk, u); ++seq) {
            if (t * 128 >= u.rows) {
                tile_count += u.hi - u.lo;
                continue;
            }
            // ---- the row, and Q into shared memory
            const int row = u.row0 + t * 128 + row_in;
            const bool real = t * 128 + row_in < u.rows;
            const int tok = real ? row / a.group : 0;
            const int64_t q_row = u.q0 + tok;
            const int head = u.h * a.group + (real ? row - tok * a.group : 0);
            const int e = real ? u.e0 + tok : 0;
            const int bgn = a.window > 0 && e > a.window ? (int)(e - a.window) : 0;
            float cc = a.scale_log2;
            {
                const uint4 *src = reinterpret_cast<const uint4 *>(a.q + q_row * a.ldq + (int64_t)head * D);
                const uint32_t dst = q_smem + t * (128 * D * 2) + row_in * 128;
                float up = 1.f;
                if constexpr (C::E4M3) {
                    // f16: a power of two takes the row's largest value to [2^14, 2^15)
                    uint32_t top = 0;
                    if (real)
#pragma unroll 4
                        for (int c = 0; c < D / 8; ++c) {
                            const uint4 v = __ldg(src + c);
                            top = max(top, max(max(v.x << 16 & 0x7FFFFFFFu, v.x & 0x7FFF0000u), max(v.y << 16 & 0x7FFFFFFFu, v.y & 0x7FFF0000u)));
                            top = max(top, max(max(v.z << 16 & 0x7FFFFFFFu, v.z & 0x7FFF0000u), max(v.w << 16 & 0x7FFFFFFFu, v.w & 0x7FFF0000u)));
                        }
                    const int ex = (int)(top >> 23);
                    // (a row that is not finite gives NaN either way)
                    const int shift = ex == 255 ? 0 : min(127 + 14 - ex, 126);
                    up = __uint_as_float((uint32_t)(127 + shift) << 23);
                    cc *= __uint_as_float((uint32_t)(127 - shift) << 23);
                }
#pragma unroll 4
                for (int c = 0; c < D / 8; ++c) {
                    uint4 v = real ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
                    if constexpr (C::E4M3) {
                        const float f = a.q_sign ? -up : up;
                        v.x = pack_f16(lo_f32(v.x) * f, hi_f32(v.x) * f), v.y = pack_f16(lo_f32(v.y) * f, hi_f32(v.y) * f);
                        v.z = pack_f16(lo_f32(v.z) * f, hi_f32(v.z) * f), v.w = pack_f16(lo_f32(v.w) * f, hi_f32(v.w) * f);
                    } else {
                        v.x ^= a.q_sign, v.y ^= a.q_sign, v.z ^= a.q_sign, v.w ^= a.q_sign;
                    }
                    if (a.q_zero) v = make_uint4(0, 0, 0, 0);
                    sts128(dst + (c / 8) * (128 * 128) + ((c % 8) ^ (row_in & 7)) * 16, v);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar.q_full + 8 * t);
            // ---- what the tile's rows see
            const int last_row = min(t * 128 + 127, u.rows - 1) + u.row0;
            const int64_t all_end = (int64_t)u.e0 + (u.row0 + t * 128) / a.group;               // every row sees slots below this ...
            const int64_t all_begin = a.window > 0 ? (int64_t)u.e0 + last_row / a.group - a.window : 0;  // ... and from this on
            float m = -INFINITY, l = 0.f;
            for (int64_t i = u.lo; i < u.hi; ++i, ++tile_count) {
                // heads of 256: the two buffers in turn, each with its barriers
                const uint32_t odd = s_count & 1, at = NT == 2 ? (uint32_t)t : odd, phase = NT == 2 ? odd : s_count >> 1 & 1;
                ++s_count;
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(bar.s_full + 8 * at, phase, status))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t s_col = tmem + lanes + C::S_COL + at * BN;
                float s[BN];
#pragma unroll
                for (int c = 0; c < BN / 32; ++c) tmem_ld32(s_col + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(s + 32 * c));
                tmem_ld_wait();
                const int64_t j0 = (u.base + i) * BN;
                float f = cc;
                if (a.softcap > 0.f) {
                    // c tanh(s / c) = c (1 - 2 / (1 + e^(2 s / c))), in units of log2
                    const float in = a.cap_in * cc, out = a.softcap * kLog2e;
#pragma unroll
                    for (int k = 0; k < BN; ++k) s[k] = fmaf(-2.f * out, rcp_approx(1.f + ex2_approx(s[k] * in)), out);
                    f = 1.f;
                }
                const volatile uint32_t *mask = page_mask + (tile_count & (kMetaRing - 1)) * 4;
                uint32_t pages = 0xFFFFFFFFu;
#pragma unroll
                for (int w = 0; w < BN / 32; ++w) pages &= mask[w];
                if (j0 + BN > all_end || j0 < all_begin || pages != 0xFFFFFFFFu) {
                    const int from = (int)max((int64_t)0, bgn - j0), to = (int)min((int64_t)BN, e - j0);
#pragma unroll
                    for (int w = 0; w < BN / 32; ++w) {
                        const uint32_t there = mask[w];
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (32 * w + k < from || 32 * w + k >= to || !(there >> k & 1u)) s[32 * w + k] = -INFINITY;
                    }
                }
                float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int k = 4; k < BN; ++k) top[k & 3] = fmaxf(top[k & 3], s[k]);
                const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                // a new maximum: rows that had none take theirs, others when it is 2^8 above
                const bool up = m == -INFINITY ? mx > -INFINITY : (mx - m) * f > kSlack;
                if (__any_sync(0xFFFFFFFFu, up)) {
                    const float fac = !up ? 1.f : m == -INFINITY ? 0.f : ex2_approx((m - mx) * f);
                    if (up) m = mx;
                    l *= fac;
                    if (i > u.lo) {
                        if constexpr (NT == 1) {  // the product before must have ended (it is the pv_done phase before this tile's)
                            if (!__all_sync(0xFFFFFFFFu, mbar_wait(bar.pv_done, odd ^ 1, status))) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                        }
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t o[16];
                            asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                                         : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]), "=r"(o[4]), "=r"(o[5]), "=r"(o[6]), "=r"(o[7]),
                                           "=r"(o[8]), "=r"(o[9]), "=r"(o[10]), "=r"(o[11]), "=r"(o[12]), "=r"(o[13]), "=r"(o[14]), "=r"(o[15])
                                         : "r"(o_col + 16 * c)
                                         : "memory");
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * fac);
                            tmem_st16(o_col + 16 * c, o);
                        }
                        tmem_st_wait();
                    }
                }
                const float m0 = m == -INFINITY ? 0.f : m, neg = -m0 * f;
                if (__any_sync(0xFFFFFFFFu, fabsf(neg) > 65536.f)) {  // (m0 f's rounding would count)
#pragma unroll
                    for (int k = 0; k < BN; ++k) s[k] = ex2_approx(fmaf(s[k] - m0, f, C::LIFT));
                } else {
                    const float2 f2 = make_float2(f, f), n2 = make_float2(neg + C::LIFT, neg + C::LIFT);
#pragma unroll
                    for (int k = 0; k < BN; k += 2) {
                        const float2 z = fma2(make_float2(s[k], s[k + 1]), f2, n2);
                        s[k] = ex2_approx(z.x), s[k + 1] = ex2_approx(z.y);
                    }
                }
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < BN / 32; ++c) {
                    uint32_t p[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float x = s[32 * c + 2 * k], y = s[32 * c + 2 * k + 1];
                        sum[k & 1] = add2(sum[k & 1], make_float2(x, y));
                        p[k] = C::E4M3 ? pack_f16(x, y) : pack_bf16(x, y);
                    }
                    tmem_st16(s_col + 16 * c, p);
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar.p_full + 8 * at);
            }
            if (!ok) break;
            // ---- the unit's end
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(bar.o_full + 8 * t, unit_phase, status))) {
                ok = false;
                break;
            }
            unit_phase ^= 1;
            tc_fence_after();
            const bool bad = bad_unit[seq & 7] == seq + 1;
            // a row that sees slots, all of them -infinity, has no weights: NaN, as 0 / 0 has it
            const float inv = e > bgn ? a.v_scale / l : 0.f;
            float *const part = a.parts + ((int64_t)(2 * blockIdx.x + (u.lo > 0 ? 0 : 1)) * C::ROWS + t * 128 + row_in) * D;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(o_col + 32 * c, o);
                tmem_ld_wait();
                if (bad && real) {
                    // values that are not finite in tiles that not every row of the unit sees (the copies took them out)
                    for (int64_t i = u.lo; i < u.hi; ++i) {
                        const int64_t j0 = (u.base + i) * BN;
                        const int64_t unit_end = (int64_t)u.e0 + u.row0 / a.group;
                        const int64_t unit_begin = a.window > 0 ? (int64_t)u.e0 + (u.row0 + u.rows - 1) / a.group - a.window : 0;
                        if (j0 + BN <= unit_end && j0 >= unit_begin) continue;
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
                if (!real) continue;
                if (u.whole) {
                    uint4 *dst = reinterpret_cast<uint4 *>(a.o + q_row * a.ldo + (int64_t)head * D + 32 * c);
#pragma unroll
                    for (int k = 0; k < 32; k += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const float p = __uint_as_float(o[k + 2 * x]) * inv, q = __uint_as_float(o[k + 2 * x + 1]) * inv;
                            w[x] = e > bgn ? pack_bf16(p, q) : 0u;
                        }
                        dst[k / 8] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else {
                    uint4 *dst = reinterpret_cast<uint4 *>(part + 32 * c);
#pragma unroll
                    for (int k = 0; k < 32; k += 4) dst[k / 4] = make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
                }
            }
            if (!u.whole && real)
                a.part_ml[(int64_t)(2 * blockIdx.x + (u.lo > 0 ? 0 : 1)) * C::ROWS + t * 128 + row_in] =
                    make_float2(m == -INFINITY ? -INFINITY : m * (a.softcap > 0.f ? 1.f : cc), l);
            tc_fence_before();
        }
        if (!ok && t < NT && lane == 0) *abort_flag = 1;
    } else if (warp < kCopyWarp) {
        set_regs_down<kOtherRegs>();
        if (warp == kMmaWarp && lane == 0) {
            // ---------------------------------------------------- MMA
            constexpr uint32_t kQk = idesc_of(128, BN, C::E4M3, false), kPv = idesc_of(128, D, C::E4M3, true);
            uint32_t used = 0;               // tiles of the ring consumed or being consumed
            uint32_t p_phase[2] = {0, 0};    // of the tiles of rows, or of the two buffers
            uint32_t count = 0;              // tiles of slots walked
            bool ok = true;
            auto slot_of = [&](uint32_t n) { return n % NS; };
            auto wait_full = [&](uint32_t n) {
                const bool r = mbar_wait(bar.full + 8 * slot_of(n), (n / NS) & 1, status);
                tc_fence_after();
                return r;
            };
            auto qk = [&](int t, uint32_t n, int s_at) {
                const uint64_t qd = umma_desc_sw128(q_smem + t * (128 * D * 2)), kd = umma_desc_sw128(ring + slot_of(n) * C::SLOT);
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    umma_bf16(tmem + C::S_COL + s_at * BN, qd + (k / 4) * (128 * 128 >> 4) + 2 * (k % 4),
                              kd + (k / 4) * (BN * 128 >> 4) + 2 * (k % 4), kQk, k != 0);
            };
            auto pv = [&](int t, uint32_t n, int s_at, bool first) {
                const uint64_t vd = desc_mn(ring + slot_of(n) * C::SLOT, BN * 128);
#pragma unroll
                for (int k = 0; k < BN / 16; ++k)
                    umma_bf16_ts(tmem + C::O_COL + t * D, tmem + C::S_COL + s_at * BN + 8 * k, vd + k * (16 * 128 >> 4), kPv,
                                 !first || k != 0);
            };
            uint32_t q_phase[2] = {0, 0};
            while (ok && next_unit<C>(a, walk, u)) {
                const int nt = u.rows > 128 ? 2 : 1;
                const int64_t tiles = u.hi - u.lo;
                for (int t = 0; t < nt && ok; ++t) {
                    ok = mbar_wait(bar.q_full + 8 * t, q_phase[t], status);
                    q_phase[t] ^= 1;
                }
                if (!ok || !(ok = wait_full(used)) || *abort_flag) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // the ring holds the unit's keys and values in turn: tile i at used + 2 i and used + 2 i + 1
                for (int t = 0; t < nt; ++t) {
                    const int at = NT == 2 ? t : (int)(count & 1);
                    qk(t, used, at);
                    umma_commit(bar.s_full + 8 * at);
                }
                umma_commit(bar.empty + 8 * slot_of(used));
                for (int64_t i = 0; i < tiles && ok; ++i) {
                    const uint32_t kn = used + 2 * (uint32_t)i + 2, vn = used + 2 * (uint32_t)i + 1;
                    const bool more = i + 1 < tiles;
                    if constexpr (NT == 1) {
                        // the next scores into the other buffer, then this tile's product
                        if (more) {
                            if (!(ok = wait_full(kn))) break;
                            const int next = (int)((count + i + 1) & 1);
                            qk(0, kn, next);
                            umma_commit(bar.s_full + 8 * next);
                            umma_commit(bar.empty + 8 * slot_of(kn));
                        }
                        const int at = (int)((count + i) & 1);
                        if (!(ok = mbar_wait(bar.p_full + 8 * at, p_phase[at], status)) || !(ok = wait_full(vn))) break;
                        p_phase[at] ^= 1;
                        pv(0, vn, at, i == 0);
                        umma_commit(bar.pv_done);
                        umma_commit(bar.empty + 8 * slot_of(vn));
                        if (!more) umma_commit(bar.o_full);
                    } else {
                        for (int t = 0; t < nt && ok; ++t) {
                            if (!(ok = mbar_wait(bar.p_full + 8 * t, p_phase[t], status))) break;
                            p_phase[t] ^= 1;
                            if (t == 0 && !(ok = wait_full(vn))) break;
                            tc_fence_after();
                            pv(t, vn, t, i == 0);
                            if (more) {
                                if (t == 0 && !(ok = wait_full(kn))) break;
                                qk(t, kn, t);
                                umma_commit(bar.s_full + 8 * t);
                            } else {
                                umma_commit(bar.o_full + 8 * t);
                            }
                        }
                        if (!ok) break;
                        umma_commit(bar.empty + 8 * slot_of(vn));
                        if (more) umma_commit(bar.empty + 8 * slot_of(kn));
                    }
                }
                used += 2 * (uint32_t)tiles;
                count += (uint32_t)tiles;
            }
            if (!ok) *abort_flag = 1;
            umma_commit(bar.done);
        }
    } else {
        // -------------------------------------------------------- copies
        set_regs_down<kOtherRegs>();
        const int w = warp - kCopyWarp;
        constexpr int RB = D * (C::E4M3 ? 1 : 2);        // bytes of a cached row
        constexpr int PER_ROW = RB / 16;                 // lanes of a row
        constexpr int AT_ONCE = 32 / PER_ROW;            // rows of a warp's access
        constexpr int WROWS = BN / kCopyWarps;           // rows of a warp
        const int sub = lane / PER_ROW, chunk = lane % PER_ROW;
        uint32_t issued = 0, shown = 0, seq = 0;
        int64_t tile_count = 0;
        bool ok = true;
        uint32_t edge_bits = 0;  // of the tiles on their way, newest in bit 0: values to be checked?
        // this warp's part of ring tile n has landed: checked if need be, and shown to the MMAs
        auto check = [&](uint32_t n, uint32_t of) {
            const uint32_t at = ring + (n % NS) * C::SLOT;
            bool any = false;
#pragma unroll 1
            for (int r = 0; r < WROWS; r += AT_ONCE) {
                const int slot = w * WROWS + r + sub;
#pragma unroll
                for (int x = 0; x < (C::E4M3 ? 2 : 1); ++x) {
                    const int c = (C::E4M3 ? 2 : 1) * chunk + x;
                    const uint32_t p = at + (c / 8) * (BN * 128) + slot * 128 + ((c % 8) ^ (slot & 7)) * 16;
                    uint4 v = lds128(p);
                    const uint32_t b0 = not_finite<C::E4M3>(v.x), b1 = not_finite<C::E4M3>(v.y), b2 = not_finite<C::E4M3>(v.z),
                                   b3 = not_finite<C::E4M3>(v.w);
                    if (b0 | b1 | b2 | b3) {
                        v.x &= ~b0, v.y &= ~b1, v.z &= ~b2, v.w &= ~b3;
                        sts128(p, v);
                        any = true;
                    }
                }
            }
            if (any) bad_unit[of & 7] = of + 1;
        };
        uint32_t seq_of[NS];  // unit of each ring tile on its way
#pragma unroll
        for (int i = 0; i < NS; ++i) seq_of[i] = 0;
        auto show = [&](uint32_t upto) {
            while (shown != upto) {
                const uint32_t back = issued - 1 - shown;
                if (edge_bits >> back & 1u) {
                    uint32_t of = 0;
#pragma unroll
                    for (int i = 0; i < NS; ++i)
                        if (i == (int)(shown % NS)) of = seq_of[i];
                    check(shown, of);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar.full + 8 * (shown % NS));
                ++shown;
            }
        };
        for (; ok && next_unit<C>(a, walk, u); ++seq) {
            const int64_t unit_end = (int64_t)u.e0 + u.row0 / a.group;
            const int64_t unit_begin = a.window > 0 ? (int64_t)u.e0 + (u.row0 + u.rows - 1) / a.group - a.window : 0;
            for (int64_t i = u.lo; i < u.hi && ok; ++i, ++tile_count) {
                const int64_t j0 = (u.base + i) * BN;
                // where this lane's slot lies (lanes 0 .. WROWS - 1)
                const int64_t j = j0 + w * WROWS + lane;
                int64_t off = -1;
                bool there = true;
                if (lane < WROWS && j >= u.begin && j < u.end) {
                    const uint32_t pg = page_of(a.c, (uint32_t)j);
                    const int32_t page = __ldg(a.c.table + u.b * a.c.ld_table + pg);
                    there = page_ok(a.c, page);
                    if (there) off = row_bytes_at(a.c, page, u.h, (uint32_t)j - pg * a.c.page_size);
                    else atomicOr(status, kDevIndex);
                }
                const uint32_t mask = __ballot_sync(0xFFFFFFFFu, there);
                const bool edge = j0 + BN > unit_end || j0 < unit_begin;
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const uint32_t n = issued;
                    if (n >= (uint32_t)NS) {
                        const uint32_t eb = bar.empty + 8 * (n % NS), parity = (n / NS - 1) & 1;
                        if (!__all_sync(0xFFFFFFFFu, mbar_test_wait(eb, parity))) {
                            cp_async_wait<0>();  // nothing is held back while this waits
                            show(issued);
                            if (!__all_sync(0xFFFFFFFFu, mbar_wait(eb, parity, status)) || *abort_flag) {
                                ok = false;
                                break;
                            }
                        }
                    }
                    if (kv == 0 && lane == 0) {  // (heads of 256: 16 slots a warp, two warps' bits in a word)
                        if constexpr (WROWS == 32) page_mask[(tile_count & (kMetaRing - 1)) * 4 + w] = mask;
                        else reinterpret_cast<volatile uint16_t *>(page_mask)[(tile_count & (kMetaRing - 1)) * 8 + w] = (uint16_t)mask;
                    }
                    const uint8_t *pool = kv == 0 ? a.c.k : a.c.v;
                    const uint32_t at = ring + (n % NS) * C::SLOT;
                    if constexpr (C::E4M3) {
                        constexpr int STEP = 4;
#pragma unroll 1
                        for (int r = 0; r < WROWS; r += AT_ONCE * STEP) {
                            uint4 v[STEP];
#pragma unroll
                            for (int x = 0; x < STEP; ++x) {
                                const int64_t o = __shfl_sync(0xFFFFFFFFu, off, (r + x * AT_ONCE + sub) & 31);
                                v[x] = o >= 0 && r + x * AT_ONCE < WROWS ? __ldg(reinterpret_cast<const uint4 *>(pool + o) + chunk)
                                                                       : make_uint4(0, 0, 0, 0);
                            }
#pragma unroll
                            for (int x = 0; x < STEP; ++x) {
                                if (r + x * AT_ONCE >= WROWS) continue;
                                const int slot = w * WROWS + r + x * AT_ONCE + sub;
                                const uint32_t row = at + (chunk / 4) * (BN * 128) + slot * 128;
                                const int c = 2 * (chunk % 4);
                                sts128(row + (c ^ (slot & 7)) * 16, make_uint4(e4m3x2_to_f16x2(v[x].x), e4m3x2_to_f16x2(v[x].x >> 16),
                                                                               e4m3x2_to_f16x2(v[x].y), e4m3x2_to_f16x2(v[x].y >> 16)));
                                sts128(row + ((c + 1) ^ (slot & 7)) * 16, make_uint4(e4m3x2_to_f16x2(v[x].z), e4m3x2_to_f16x2(v[x].z >> 16),
                                                                                     e4m3x2_to_f16x2(v[x].w), e4m3x2_to_f16x2(v[x].w >> 16)));
                            }
                        }
                    } else {
#pragma unroll 4
                        for (int r = 0; r < WROWS; r += AT_ONCE) {
                            const int64_t o = __shfl_sync(0xFFFFFFFFu, off, r + sub);
                            const int slot = w * WROWS + r + sub;
                            cp_async16(at + (chunk / 8) * (BN * 128) + slot * 128 + ((chunk % 8) ^ (slot & 7)) * 16,
                                       o >= 0 ? pool + o + chunk * 16 : pool, o >= 0 ? 16 : 0);
                        }
                        cp_async_commit();
                    }
                    ++issued;
                    edge_bits = edge_bits << 1 | (uint32_t)(kv == 1 && edge);
#pragma unroll
                    for (int x = 0; x < NS; ++x)
                        if (x == (int)(n % NS)) seq_of[x] = seq;
                    if constexpr (C::E4M3) {
                        show(issued);
                    } else if (issued - shown > (uint32_t)C::LAG) {
                        cp_async_wait<C::LAG>();
                        show(issued - C::LAG);
                    }
                }
            }
        }
        cp_async_wait<0>();
        if (ok) show(issued);
        else if (lane == 0) *abort_flag = 1;
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

// CTA (s, y): the unit that boundary s between shares is the first to cut, if there is one; each warp some of its rows.
template <typename C>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const ChunkArgs a) {
    constexpr int D = C::D, PER = D / 32;
    pdl_wait();
    pdl_trigger();
    const int64_t places = __ldg(a.head), total = places * a.c.heads;
    const int shares = (int)__ldg(a.head + 2), s = blockIdx.x + 1;
    if (s >= shares) return;
    const int64_t cut = share_at(total, shares, s);
    const int h = (int)(cut / places);
    const int64_t in_head = cut - h * places;
    const int rt = find_rt(a, (int)__ldg(a.head + 1), in_head);
    const int64_t first = __ldg(a.place_at + rt);
    if (first == in_head) return;                                              // the boundary lies between units
    const int64_t start = h * places + first, end = h * places + __ldg(a.place_at + rt + 1);
    if (share_at(total, shares, s - 1) > start) return;                        // an earlier boundary cut it
    Unit u;
    unit_of<C>(a, rt, u);
    int last = s;                                                              // the share that holds its end
    while (last + 1 < shares && share_at(total, shares, last + 1) < end) ++last;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int row_in = blockIdx.y * kJoinWarps + warp; row_in < u.rows; row_in += gridDim.y * kJoinWarps) {
        auto part = [&](int k) { return (int64_t)(2 * k + (k == s - 1 ? 1 : 0)) * C::ROWS + row_in; };
        float m = -INFINITY;
        bool number = true;
        for (int k = s - 1 + lane; k <= last; k += 32) {
            const float x = __ldcg(a.part_ml + part(k)).x;
            m = fmaxf(m, x);
            if (x != x) number = false;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        if (!__all_sync(0xFFFFFFFFu, number)) m = __uint_as_float(0x7FC00000u);
        float l = 0.f, o[PER] = {};
        for (int k = s - 1; k <= last; ++k) {
            const float2 ml = __ldcg(a.part_ml + part(k));
            if (ml.x == -INFINITY && ml.y == 0.f) continue;  // it saw nothing
            const float w = ex2_approx(ml.x - m);
            l = fmaf(ml.y, w, l);
            const float *p = a.parts + part(k) * D + lane * PER;
#pragma unroll
            for (int x = 0; x < PER; ++x) o[x] = fmaf(__ldcg(p + x), w, o[x]);
        }
        const int row = u.row0 + row_in, tok = row / a.group, e = u.e0 + tok;
        const int bgn = a.window > 0 && e > a.window ? (int)(e - a.window) : 0;
        const float inv = a.v_scale / l;
        uint32_t *dst = reinterpret_cast<uint32_t *>(a.o + (u.q0 + tok) * a.ldo + (int64_t)(h * a.group + row - tok * a.group) * D + lane * PER);
#pragma unroll
        for (int x = 0; x < PER; x += 2) dst[x / 2] = e > bgn ? pack_bf16(o[x] * inv, o[x + 1] * inv) : 0u;
    }
}

template <typename C>
cudaError_t launch(const DeviceInfo &di, ChunkArgs &a, cudaStream_t s) {
    // setmaxnreg moves registers within what the launch holds: 128 a thread, or the split would wait forever
    static const bool fits = [] {
        cudaFuncAttributes f;
        return cudaFuncGetAttributes(&f, chunk_kernel<C>) == cudaSuccess && 4 * f.numRegs >= 2 * (kSoftmaxRegs + kOtherRegs);
    }();
    if (!fits) return cudaErrorInvalidConfiguration;
    cudaError_t e = ensure_smem((const void *)chunk_kernel<C>, C::SMEM);
    if (e != cudaSuccess) return e;
    a.shares = di.sm_count < kMaxChunkShares ? di.sm_count : kMaxChunkShares;
    if ((e = launch_pdl(plan_kernel<C>, dim3(1), dim3(kPlanThreads), 0, s, dim3(1), a)) != cudaSuccess) return e;
    if ((e = launch_pdl(chunk_kernel<C>, dim3(a.shares), dim3(kThreads), C::SMEM, s, dim3(1), a)) != cudaSuccess) return e;
    // rows of a unit over 8 CTAs, fewer where the call has few rows
    const int64_t rows = a.T * a.group;
    const int y = rows <= kJoinWarps ? 1 : rows <= 4 * kJoinWarps ? 4 : 8;
    return launch_pdl(join_kernel<C>, dim3(a.shares, y), dim3(kJoinWarps * 32), 0, s, dim3(1), a);
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
