// Attention of a few new tokens over a paged key-value cache, split over the
// cache's length and joined.
//
// For a row r (query token i, head hq) with slots [begin_r, end_r):
//     s_j = c * q . k_j (c = scale * k_scale),  m = max_j s_j,  l = sum_j e^(s_j - m)
//     o   = v_scale * sum_j e^(s_j - m) v_j / l
// and for two disjoint sets of slots A, B with (m, l, o') each (o' not divided by l):
//     M = max(m_A, m_B),  l = l_A e^(m_A - M) + l_B e^(m_B - M),  o' likewise,
// which is what lets warps, CTAs and the joining kernel share one row.
//
// Bound: every cached key and value is read once, so HBM.  Hence
//   - Slots and values are the long sides of the MMAs (m16), the rows of one KV head
//     their short one (n8 tiles): S^T = K Q^T and O^T = V^T P^T.  A group of up to 8 rows
//     costs one n tile, so few rows waste little tensor work and few registers; up to 32
//     rows (16 for D = 256) share one pass over the cache.  The score tile's accumulators
//     are the second product's B operand after one 8 x 8 transpose in registers.
//   - The batch's work is one list of tiles (sequence, head, row tile, 4 steps of
//     slots), cut into equal contiguous shares, one per CTA, whatever the lengths are:
//     a share may end one unit, hold whole units and begin another.  After a unit's
//     tiles the list holds kExtra places that stand for the time of ending one unit and
//     beginning the next.  Whole units are finished in place; parts leave (m, l, o') in
//     the workspace for join_kernel.
//   - Each warp owns a ring of stages in shared memory and fills it with its own steps by
//     16-byte asynchronous copies (any page size, any strides; one address for a step
//     within a page), so no barrier lies in the main loop.  Rows lie RB + 16 bytes
//     apart: eight rows' 16-byte chunks never share banks.  (A bulk copy per row needs
//     fewer instructions, but the copy engine takes 12 to 19 cycles for each: 64 sequences
//     of 2000 to 8192 slots took 320 us.)
//   - The running maximum only moves when a score exceeds it by 2^8: until then no lane
//     needs another's scores and o' is not rescaled.
// Measured (with the join): 8.5 us for 40 heads over 8 KV heads of 128 and 1000 slots, 35 us for 16 sequences of
// 33 to 6001 slots with 4 new tokens, 79 us for 200001 e4m3 slots (5.2 TB/s), 260 us for 64 sequences of 2000 to 8192
// slots with weights (225 us in attn_kernel: 6.2 TB/s with the scores it writes).

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "decode_ops.h"
#include "q4k_ptx.cuh"

namespace q4k {
namespace {

constexpr int kWarps = 4;           // warps of a CTA, each a step of every tile
constexpr int kThreads = kWarps * 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNone = -INFINITY;
constexpr float kSlack = 8.f;       // how far (log2) a score may exceed the running maximum
constexpr int kExtra = 2;           // places of the list after a unit's tiles
constexpr int kWaves = 3, kLong = 40;  // see shares_of
static_assert(kWaves * kMaxAttnResident == kMaxAttnShares, "the workspace holds two parts for each share");

// 16 bytes into shared memory, of which the last 16 - bytes become zeros
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// transpose of an 8 x 8 matrix of 16-bit values held as MMA fragments
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// two e4m3 values (low 16 bits) to two f16 values, exactly
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)v));
    return r;
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
__device__ __forceinline__ float lo_f32(uint32_t bf16x2) { return __uint_as_float(bf16x2 << 16); }
__device__ __forceinline__ float hi_f32(uint32_t bf16x2) { return __uint_as_float(bf16x2 & 0xFFFF0000u); }

// p of an e4m3 cache is kept as 2^7 p, in o' and l alike (see the kernel)
__host__ __device__ constexpr float lift(bool e4m3) { return e4m3 ? 7.f : 0.f; }

// Floats of one part of NR row octets: (m, l) of 8 NR rows, then o' as MMA fragments
// [octet][D / 16][lane][4].
__host__ __device__ constexpr int part_floats(int D, int nr) { return 16 * nr + 8 * nr * D; }

template <int D_, bool E4M3_, int NR_>
struct Cfg {
    static constexpr int D = D_, NR = NR_;                     // values of a head; octets of rows of a unit
    static constexpr bool E4M3 = E4M3_;
    static constexpr int RB = D * (E4M3 ? 1 : 2);              // bytes of a cached row
    static constexpr int PITCH = RB + 16;
    static constexpr int CHUNKS = RB / 16;                     // 16-byte chunks of a row
    static constexpr int TOK = RB <= 128 && (NR < 4 || D == 64) ? 32 : 16;  // slots of a step
    static constexpr int MT = TOK / 16;
    static constexpr int CT = kWarps * TOK;                    // slots of a tile
    static constexpr int STAGE = 2 * TOK * PITCH;              // bytes of a stage: keys, then values
    static constexpr int KS = D / 16;
    static constexpr bool QSMEM = KS * NR >= 32;               // queries in shared memory where registers run out
    static constexpr int QBYTES = QSMEM ? KS * NR * 32 * 8 : 0;
    // a ring of what shared memory holds: two CTAs on an SM, or one where a stage is too large
    static constexpr int HALF = (112 * 1024 - QBYTES) / (kWarps * STAGE), ALL = (222 * 1024 - QBYTES) / (kWarps * STAGE);
    static constexpr int PER_SM = HALF >= 3 ? 2 : 1;
    static constexpr int STAGES = PER_SM == 2 ? (HALF < 6 ? HALF : 6) : (ALL < 6 ? ALL : 6);
    static constexpr int RING = kWarps * STAGES * STAGE;
    static constexpr int SMEM = RING + QBYTES;
    static_assert(STAGES >= 3 && KS * 512 <= STAGE, "a stage holds a warp's fragments of one octet");
};

// Length of sequence b, cut to what table (and weights) can hold, and the slots its rows read.
__device__ __forceinline__ void seq_range(const AttnArgs &a, int b, int &begin, int &len) {
    len = max(0, min(__ldg(a.seq_lens + b), a.cap));
    begin = 0;
    if (a.window > 0) begin = (int)max((int64_t)0, (int64_t)len - a.n_q + 1 - a.window);
}
// Tiles of n slots.  (A sequence has up to 2^31 - 1 slots, and its last tile and chunk may end beyond 2^31: slots that
// are not known to be there are unsigned.)
template <int CT>
__device__ __forceinline__ int tiles_of(int n) {
    return (int)(((uint32_t)n + CT - 1) / CT);
}
// Places of one unit of n slots.
template <int CT>
__device__ __forceinline__ int places(int n) {
    return n > 0 ? tiles_of<CT>(n) + kExtra : 0;
}

// A position in a share: tile `tile` of `tiles` of unit (sequence b, KV head, row tile rt).
struct Pos {
    int b, head, rt, tile, tiles;
    int begin, end;  // slots of the unit: the union of its rows' ranges
    int64_t left;    // places of the share from here on
    // the next sequence with slots, if the share goes on
    template <int CT>
    __device__ __forceinline__ void enter(const AttnArgs &a) {
        for (; left > 0 && b < a.c.batch; ++b) {
            seq_range(a, b, begin, end);
            tiles = end > begin ? tiles_of<CT>(end - begin) : 0;
            if (tiles > 0) return;
        }
        left = 0;
    }
    template <int CT>
    __device__ __forceinline__ void next_unit(const AttnArgs &a) {
        tile = 0;
        if (++rt < a.row_tiles) return;
        rt = 0;
        if (++head < a.c.heads) return;
        head = 0;
        ++b;
        enter<CT>(a);
    }
    template <int CT>
    __device__ __forceinline__ void advance(const AttnArgs &a) {
        --left;
        if (++tile < tiles) return;
        left -= kExtra;
        next_unit<CT>(a);
    }
};

// Slots [begin, end) of row r, of token `tok`, of a sequence of length len.
__device__ __forceinline__ void row_range(const AttnArgs &a, int r, int tok, int len, int &begin, int &end) {
    end = r < a.rows ? max(0, len - a.n_q + 1 + tok) : 0;
    begin = a.window > 0 ? (int)max((int64_t)0, (int64_t)end - a.window) : 0;
}

// The list's `total` places go to a number of shares: share i is [share_begin(i), share_begin(i + 1)).
// One for each resident CTA, so that all run at once; long lists are cut into two or three times as many
// (of kLong places at least), which start as others end and even out how fast the SMs read.  Not into any number
// between: a few more than are resident run on their own at the end (8 sequences of 16384 slots on 344 shares
// took 120 us, on 304 they take 96).
__device__ __forceinline__ int shares_of(int64_t total, int resident) {
    const int64_t waves = min(max(total / ((int64_t)kLong * resident), (int64_t)1), (int64_t)kWaves);
    return (int)min(total, waves * resident);
}
__device__ __forceinline__ int64_t share_begin(int64_t total, int shares, int i) {
    if (i >= shares) return total;
    return total >> 20 ? total * i / shares : (uint32_t)total * (uint32_t)i / (uint32_t)shares;  // (shares <= 2^11)
}
// The share that holds place t: the largest i with floor(total i / shares) <= t.
__device__ __forceinline__ int share_of(int64_t total, int shares, int64_t t) {
    return total >> 20 ? (int)(((t + 1) * shares - 1) / total) : (int)(((uint32_t)(t + 1) * (uint32_t)shares - 1) / (uint32_t)total);
}

// Where this CTA's share begins (left = 0: it is empty); CTA 0 also writes the places before
// each sequence for the joining kernel.
template <int CT>
__device__ __forceinline__ void share_of_list(const AttnArgs &a, Pos &start, int64_t *scratch) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.c.batch + kThreads - 1) / kThreads;  // sequences of a thread
    const int lo = min(tid * per, a.c.batch), hi = min(lo + per, a.c.batch);
    int64_t sum = 0;
    Pos p;  // the last of them; with one a thread, the only one
    p.begin = p.end = 0;
    for (p.b = lo; p.b < hi; ++p.b) {
        seq_range(a, p.b, p.begin, p.end);
        sum += places<CT>(p.end - p.begin);
    }
    sum *= a.unit_heads;
    int64_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) scratch[warp] = inc;
    if (tid == 0) start.left = 0;
    __syncthreads();
    int64_t before = inc - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += scratch[w];
        total += scratch[w];
    }
    const int shares = shares_of(total, a.resident);
    const int64_t t0 = share_begin(total, shares, blockIdx.x), t1 = share_begin(total, shares, blockIdx.x + 1);
    if (t0 < t1 && before <= t0 && t0 < before + sum) {
        // this thread's sequences hold the share's first place
        int64_t at = before;
        int n = places<CT>(p.end - p.begin);
        p.b = lo;
        if (per > 1)
            for (;; ++p.b) {
                seq_range(a, p.b, p.begin, p.end);
                n = places<CT>(p.end - p.begin);
                if (t0 < at + (int64_t)n * a.unit_heads) break;
                at += (int64_t)n * a.unit_heads;
            }
        const int64_t in = t0 - at;
        int hr;
        if (in < 1 << 24) {
            // (the quotient of two floats is off by one at most; whole-number division takes far longer)
            hr = (int)__fdividef((float)in, (float)n);
            const int rest = (int)in - hr * n;
            hr += rest >= n ? 1 : rest < 0 ? -1 : 0;
        } else {
            hr = (int)(in / n);
        }
        p.tile = (int)(in - (int64_t)hr * n);
        p.head = a.row_tiles == 1 ? hr : hr / a.row_tiles;
        p.rt = hr - p.head * a.row_tiles;
        p.tiles = n - kExtra;
        p.left = t1 - t0;
        if (p.tile >= p.tiles) {  // it begins after a unit's tiles
            p.left -= n - p.tile;
            p.next_unit<CT>(a);
        }
        start = p;
    }
    __syncthreads();
    if (blockIdx.x == 0) {
        int64_t at = before;
        for (int b = lo; b < hi; ++b) {
            int begin, len;
            a.prefix[b] = at;
            if (__ldg(a.seq_lens + b) > a.cap) atomicOr(a.c.status, kDevIndex);
            seq_range(a, b, begin, len);
            at += (int64_t)places<CT>(len - begin) * a.unit_heads;
        }
        if (tid == 0) a.prefix[a.c.batch] = total;
    }
}

template <typename C>
__global__ void __launch_bounds__(kThreads, C::PER_SM) attn_kernel(const AttnArgs a) {
    constexpr int D = C::D, TOK = C::TOK, MT = C::MT, KS = C::KS, NR = C::NR;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float sm_m[kWarps][8 * NR], sm_l[kWarps][8 * NR];
    __shared__ float sm_cs[8 * NR];
    __shared__ int64_t sm_scan[kWarps];
    __shared__ uint32_t sm_stage[kWarps];
    __shared__ uint8_t sm_tok[kMaxAttnRows];  // token of a row: rows are token-major
    __shared__ struct {
        int64_t row;
        float inv;
    } sm_out[8 * NR];  // a row's place in o, and v_scale / l
    __shared__ Pos sm_pos;
    __shared__ uint32_t sm_mask[kWarps][C::STAGES];  // slots of a stage that are there
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c4 = lane & 3;
    for (int r = tid; r < a.row_tiles * 8 * NR; r += kThreads) sm_tok[r] = (uint8_t)(min(r, a.rows - 1) / a.group);
    pdl_wait();
    pdl_trigger();
    share_of_list<C::CT>(a, sm_pos, sm_scan);
    Pos cur = sm_pos, nxt = cur;
    if (cur.left <= 0) return;
    bool began = cur.tile == 0;  // the unit begins in this share

    const uint32_t ring = smem_u32(smem) + warp * (C::STAGES * C::STAGE);
    const uint32_t qs = smem_u32(smem) + C::RING;

    // ---- copies.  Lane i holds slot i of a step; the page ids of the step to be copied next are in
    // flight.
    struct Fetched {
        int32_t page, head;
        uint32_t in_page;
        bool in, step;  // step: there is one
    };
    auto fetch_page = [&] {
        Fetched f = {-1, 0, 0, false, nxt.left > 0};
        if (f.step) {
            const uint32_t slot = nxt.begin + (uint32_t)(nxt.tile * kWarps + warp) * TOK + (lane & (TOK - 1));
            const uint32_t pg = page_of(a.c, slot);
            f.in = slot < (uint32_t)nxt.end;
            f.in_page = slot - pg * a.c.page_size;
            f.head = nxt.head;
            if (f.in) f.page = __ldg(a.c.table + nxt.b * a.c.ld_table + pg);
            nxt.advance<C::CT>(a);
        }
        return f;
    };
    auto copy_step = [&](int stage, const Fetched &f) {
        if (f.step) {
            constexpr uint32_t kFull = TOK == 32 ? 0xFFFFFFFFu : (1u << TOK) - 1;
            constexpr int ROWS = 32 / C::CHUNKS;  // rows of a warp's copy instruction
            const bool ok = f.in && page_ok(a.c, f.page);
            if (f.in && !ok) atomicOr(a.c.status, kDevIndex);
            const uint32_t mask = __ballot_sync(0xFFFFFFFFu, ok) & kFull;
            if (lane == 0) sm_mask[warp][stage] = mask;
            const int64_t off = ok ? row_bytes_at(a.c, f.page, f.head, f.in_page) : 0;
            const int r = lane / C::CHUNKS, ch = lane % C::CHUNKS;
            const uint32_t to = ring + stage * C::STAGE + r * C::PITCH + ch * 16;
            if (mask == kFull && __shfl_sync(0xFFFFFFFFu, f.in_page, TOK - 1) - __shfl_sync(0xFFFFFFFFu, f.in_page, 0) == TOK - 1 &&
                __shfl_sync(0xFFFFFFFFu, f.page, TOK - 1) == __shfl_sync(0xFFFFFFFFu, f.page, 0)) {
                // all slots, consecutive rows of one page
                const int64_t first = __shfl_sync(0xFFFFFFFFu, off, 0);
                const uint8_t *k = a.c.k + first + r * a.c.slot_bytes + ch * 16, *v = a.c.v + first + r * a.c.slot_bytes + ch * 16;
#pragma unroll
                for (int i = 0; i < TOK / ROWS; ++i) {
                    cp_async16(to + i * ROWS * C::PITCH, k, 16);
                    cp_async16(to + (TOK + i * ROWS) * C::PITCH, v, 16);
                    k += ROWS * a.c.slot_bytes, v += ROWS * a.c.slot_bytes;
                }
            } else {
#pragma unroll
                for (int i = 0; i < TOK / ROWS; ++i) {
                    const int64_t o = __shfl_sync(0xFFFFFFFFu, off, i * ROWS + r) + ch * 16;
                    const uint32_t n = mask >> (i * ROWS + r) & 1 ? 16 : 0;  // slots that are not there become zeros: 0 * value must be 0
                    cp_async16(to + i * ROWS * C::PITCH, a.c.k + o, n);
                    cp_async16(to + (TOK + i * ROWS) * C::PITCH, a.c.v + o, n);
                }
            }
        }
        cp_async_commit();
    };
    Fetched ahead[C::STAGES];
#pragma unroll
    for (int i = 0; i < C::STAGES; ++i) ahead[i] = fetch_page();

    uint32_t qf[C::QSMEM ? 1 : NR][KS][2];
    float o[NR][KS][4], m[NR][2], l[NR][2], cs[NR][2];
    int in_lo = 0, in_hi = 0;  // slots that every row of the unit reads

    // Queries of a unit as B operands (row n * 8 + g of the unit; values 2 c4, 2 c4 + 1 and 8 on, or for e4m3
    // those that ldmatrix leaves in this lane: 4 c4 .. 4 c4 + 3); e4m3: as f16, scaled by a power of two.
    auto query_octet = [&](const Pos &p, int n, uint32_t (&v)[KS][2]) {
        const int r = p.rt * 8 * NR + n * 8 + g;
        const int tok = sm_tok[r], hq = p.head * a.group + r - tok * a.group;
        const bool there = r < a.rows;
        const uint16_t *row = a.q + ((int64_t)p.b * a.n_q + (there ? tok : 0)) * a.ldq + (int64_t)(there ? hq : 0) * D;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int f = 0; f < 2; ++f)
                v[ks][f] = there ? __ldg(reinterpret_cast<const uint32_t *>(row + ks * 16 + (C::E4M3 ? c4 * 4 + f * 2 : c4 * 2 + f * 8)))
                                 : 0u;
        float up = 1.f;
        if constexpr (C::E4M3) {
            float mx = 0.f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int f = 0; f < 2; ++f) mx = fmaxf(mx, fmaxf(fabsf(lo_f32(v[ks][f])), fabsf(hi_f32(v[ks][f]))));
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
            // 2^(14 - exponent of the largest), at most 2^127: f16 then holds bf16's 8 bits of every value down to 2^-31
            // of the largest, and a smaller one to 2^-39 of it
            const int e = (int)(__float_as_uint(mx) >> 23);
            if (e < 255) up = __uint_as_float((uint32_t)min(127 + 14 + 127 - e, 254) << 23);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int f = 0; f < 2; ++f) v[ks][f] = pack_f16(lo_f32(v[ks][f]) * up, hi_f32(v[ks][f]) * up);
        }
        return a.scale * kLog2e / up;  // the scores' factor of row g
    };
    auto load_queries = [&](const Pos &p) {
        if constexpr (C::QSMEM) {
            __syncthreads();  // the unit before has been read by every warp
            if (warp < NR) {
                uint32_t v[KS][2];
                const float c = query_octet(p, warp, v);
                if (c4 == 0) sm_cs[warp * 8 + g] = c;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
                    asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(qs + ((warp * KS + ks) * 32 + lane) * 8), "r"(v[ks][0]), "r"(v[ks][1])
                                 : "memory");
            }
            __syncthreads();
#pragma unroll
            for (int n = 0; n < NR; ++n) cs[n][0] = sm_cs[n * 8 + 2 * c4], cs[n][1] = sm_cs[n * 8 + 2 * c4 + 1];
        } else {
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                const float c = query_octet(p, n, qf[n]);
                // of rows n * 8 + 2 c4 and + 1, which other lanes hold as row g
                cs[n][0] = __shfl_sync(0xFFFFFFFFu, c, c4 * 8);
                cs[n][1] = __shfl_sync(0xFFFFFFFFu, c, c4 * 8 + 4);
            }
        }
    };
    auto begin_unit = [&](const Pos &p) {
        const int r0 = p.rt * 8 * NR;
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            m[n][0] = m[n][1] = kNone;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int i = 0; i < KS; ++i)
#pragma unroll
                for (int x = 0; x < 4; ++x) o[n][i][x] = 0.f;
        }
        // the first token's rows read the least at the end, the last one's at the begin
        int other;
        const int r1 = min(r0 + 8 * NR, a.rows) - 1;
        row_range(a, r0, sm_tok[r0], p.end, other, in_hi);
        row_range(a, r1, sm_tok[r1], p.end, in_lo, other);
    };
    load_queries(cur);
#pragma unroll
    for (int i = 0; i < C::STAGES - 1; ++i) copy_step(i, ahead[i]);
    Fetched next = ahead[C::STAGES - 1];
    begin_unit(cur);

    int stage = 0;
    while (true) {
        cp_async_wait<C::STAGES - 2>();
        __syncwarp();
        const uint32_t mask = sm_mask[warp][stage];
        // every lane has read the step before, whose stage is filled next
        copy_step(stage == 0 ? C::STAGES - 1 : stage - 1, next);
        next = fetch_page();
        const uint32_t k_at = ring + stage * C::STAGE, v_at = k_at + TOK * C::PITCH;
        const uint32_t j0 = cur.begin + (uint32_t)(cur.tile * kWarps + warp) * TOK;  // first slot of the step
        if (mask) {
            // ---- S^T = K Q^T: slots 16 t + g, + 8 by rows 8 n + 2 c4, + 1
            float s[MT][NR][4];
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int x = 0; x < 4; ++x) s[t][n][x] = 0.f;
            auto query = [&](int n, int ks, uint32_t &b0, uint32_t &b1) {
                if constexpr (C::QSMEM)
                    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(b0), "=r"(b1) : "r"(qs + ((n * KS + ks) * 32 + lane) * 8) : "memory");
                else b0 = qf[n][ks][0], b1 = qf[n][ks][1];
            };
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const uint32_t row = k_at + (t * 16 + (lane & 15)) * C::PITCH + (lane >> 4) * 16;
                if constexpr (!C::E4M3) {
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        uint32_t kf[4];
                        ldsm4(kf, row + ks * 32);
#pragma unroll
                        for (int n = 0; n < NR; ++n) {
                            uint32_t b0, b1;
                            query(n, ks, b0, b1);
                            mma_bf16(s[t][n], kf[0], kf[1], kf[2], kf[3], b0, b1);
                        }
                    }
                } else {
#pragma unroll
                    for (int ks = 0; ks < KS; ks += 2) {
                        uint32_t kf[4];
                        ldsm4(kf, row + ks * 16);
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint32_t a0 = e4m3x2_to_f16x2(kf[2 * x]), a1 = e4m3x2_to_f16x2(kf[2 * x + 1]);
                            const uint32_t a2 = e4m3x2_to_f16x2(kf[2 * x] >> 16), a3 = e4m3x2_to_f16x2(kf[2 * x + 1] >> 16);
#pragma unroll
                            for (int n = 0; n < NR; ++n) {
                                uint32_t b0, b1;
                                query(n, ks + x, b0, b1);
                                mma_f16(s[t][n], a0, a1, a2, a3, b0, b1);
                            }
                        }
                    }
                }
            }
            // ---- scores in units of log2, masked
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int x = 0; x < 4; ++x) s[t][n][x] *= cs[n][x & 1];
            if (a.softcap > 0.f) {
                const float cap = a.softcap * kLog2e;
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int x = 0; x < 4; ++x) s[t][n][x] = cap * tanhf(s[t][n][x] / cap);
            }
            const uint32_t full = TOK == 32 ? 0xFFFFFFFFu : (1u << TOK) - 1;
            const bool inside = j0 >= in_lo && j0 + TOK <= in_hi;
            const int r0 = cur.rt * 8 * NR;
            if (mask != full || !inside) {
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        int begin, end;
                        const int r = r0 + n * 8 + c4 * 2 + e;
                        row_range(a, r, sm_tok[r], cur.end, begin, end);
#pragma unroll
                        for (int t = 0; t < MT; ++t)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int at = t * 16 + h * 8 + g;
                                const uint32_t j = j0 + at;
                                if (!(mask >> at & 1) || j < begin || j >= end) s[t][n][h * 2 + e] = kNone;
                            }
                    }
            }
            if (a.logits) {
                float *at = a.logits + (((int64_t)cur.b * a.c.heads + cur.head) * a.rows + r0 + c4 * 2) * a.ld_logits + j0 + g;
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (r0 + n * 8 + c4 * 2 + e < a.rows) {
#pragma unroll
                            for (int t = 0; t < MT; ++t)
#pragma unroll
                                for (int h = 0; h < 2; ++h)
                                    if (j0 + t * 16 + h * 8 + g < cur.end) at[t * 16 + h * 8] = s[t][n][h * 2 + e];
                        }
                        at += e == 0 ? a.ld_logits : 7 * a.ld_logits;
                    }
            }
            // ---- running maximum (rows 8 n + 2 c4, + 1: the same in all lanes of a column)
            float top[NR][2];
            bool more = false;
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    top[n][e] = kNone;
#pragma unroll
                    for (int t = 0; t < MT; ++t) top[n][e] = fmaxf(top[n][e], fmaxf(s[t][n][e], s[t][n][2 + e]));
                    more |= top[n][e] > m[n][e] + kSlack;
                }
            if (__any_sync(0xFFFFFFFFu, more)) {
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = top[n][e];
                        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
                        x = fmaxf(x, m[n][e]);
                        const float alpha = m[n][e] == kNone ? 0.f : ex2_approx(m[n][e] - x);
                        m[n][e] = x;
                        l[n][e] *= alpha;
#pragma unroll
                        for (int i = 0; i < KS; ++i) {
                            // (o' is 0 while m is -inf)
                            o[n][i][e] *= alpha;
                            o[n][i][2 + e] *= alpha;
                        }
                    }
            }
            // ---- p = 2^(s - m), at most 2^8; e4m3: 2^7 times that, so that f16 holds it between 2^15 and
            // (to 2^-32 in absolute terms) 0
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float base = (m[n][e] == kNone ? 0.f : m[n][e]) - lift(C::E4M3);
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float p = ex2_approx(s[t][n][h * 2 + e] - base);
                            s[t][n][h * 2 + e] = p;
                            l[n][e] += p;
                        }
                }
            // ---- slots that some rows read and others do not (the new tokens themselves, the window's
            // edge): a value there that is not finite must not reach the others as 0 * inf, so it
            // is added row by row and then taken out of the product
            if (!inside && a.n_q > 1) {
                for (int at = 0; at < TOK; ++at) {
                    const uint32_t j = j0 + at;
                    if (!(mask >> at & 1) || (j >= in_lo && j < in_hi)) continue;
                    const uint32_t v_row = v_at + at * C::PITCH;
                    bool odd = false;
                    if (lane * 16 < C::RB) {
                        const uint4 w = lds128(v_row + lane * 16);
                        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            odd |= C::E4M3 ? __vcmpeq4(ws[x] & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0
                                           : __vcmpeq2(ws[x] & 0x7F807F80u, 0x7F807F80u) != 0;
                    }
                    if (!__any_sync(0xFFFFFFFFu, odd)) continue;
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            // (selects: an index into s would move it to memory)
                            float p = 0.f;
#pragma unroll
                            for (int t = 0; t < MT; ++t) {
                                const bool lower = at / 8 == t * 2, upper = at / 8 == t * 2 + 1, mine = (at & 7) == g;
                                p = lower ? s[t][n][e] : upper ? s[t][n][2 + e] : p;
                                s[t][n][e] = lower && mine ? 0.f : s[t][n][e];
                                s[t][n][2 + e] = upper && mine ? 0.f : s[t][n][2 + e];
                            }
                            p = __shfl_sync(0xFFFFFFFFu, p, (at & 7) * 4 + c4);
                            int begin, end;
                            const int r = r0 + n * 8 + c4 * 2 + e;
                            row_range(a, r, sm_tok[r], cur.end, begin, end);
                            if (j >= begin && j < end)
#pragma unroll
                                for (int i = 0; i < KS; ++i)
#pragma unroll
                                    for (int h = 0; h < 2; ++h) {
                                        float v;
                                        if constexpr (C::E4M3) {
                                            uint32_t b;
                                            asm volatile("ld.shared.u8 %0, [%1];" : "=r"(b) : "r"(v_row + i * 16 + 2 * g + h) : "memory");
                                            v = e4m3_to_f32(b);
                                        } else {
                                            uint16_t b;
                                            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(b) : "r"(v_row + (i * 16 + 8 * h + g) * 2) : "memory");
                                            v = __uint_as_float((uint32_t)b << 16);
                                        }
                                        o[n][i][h * 2 + e] = fmaf(p, v, o[n][i][h * 2 + e]);
                                    }
                        }
                    __syncwarp();
                    if (lane * 16 < C::RB) sts128(v_row + lane * 16, make_uint4(0, 0, 0, 0));
                    __syncwarp();
                }
            }
            // ---- O^T += V^T P^T.  p as the sum of two 16-bit values, bf16 or for e4m3 f16: one alone would cost, in bf16,
            // nearly as much as o's own rounding and, in f16, what shows where weights of opposite values nearly cancel
            // (without the second product, e4m3: 78.8 us instead of 79.0 for 200001 slots of 8 heads of 128, 91.6 instead of
            // 96.5 for 64 sequences of 6000 of 64, 45.5 instead of 51.6 for 16 of 6000 with 32 rows of 128)
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                uint32_t ph[NR][2], pl[NR][2];
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float x = s[t][n][h * 2], y = s[t][n][h * 2 + 1];
                        if constexpr (C::E4M3) {
                            const uint32_t hi = pack_f16(x, y);
                            const float2 up = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                            ph[n][h] = transpose8(hi);
                            pl[n][h] = transpose8(pack_f16(x - up.x, y - up.y));
                        } else {
                            const uint32_t hi = pack_bf16(x, y);
                            ph[n][h] = transpose8(hi);
                            pl[n][h] = transpose8(pack_bf16(x - lo_f32(hi), y - hi_f32(hi)));
                        }
                    }
                const uint32_t row = v_at + (t * 16 + (lane & 7) + (C::E4M3 ? lane & 8 : (lane >> 4) * 8)) * C::PITCH +
                                     (C::E4M3 ? lane >> 4 : lane >> 3 & 1) * 16;
                if constexpr (!C::E4M3) {
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        uint32_t vf[4];
                        ldsm4_trans(vf, row + i * 32);
#pragma unroll
                        for (int n = 0; n < NR; ++n) {
                            mma_bf16(o[n][i], vf[0], vf[1], vf[2], vf[3], ph[n][0], ph[n][1]);
                            mma_bf16(o[n][i], vf[0], vf[1], vf[2], vf[3], pl[n][0], pl[n][1]);
                        }
                    }
                } else {
                    // a transposed 8 x 8 matrix of byte pairs: a register holds values d, d + 1 of two slots;
                    // the tile's rows g take the even d, rows g + 8 the odd ones
#pragma unroll
                    for (int i = 0; i < KS; i += 2) {
                        uint32_t vf[4];
                        ldsm4_trans(vf, row + i * 16);
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint32_t a0 = e4m3x2_to_f16x2(prmt(vf[2 * x], 0, 0x20u)), a1 = e4m3x2_to_f16x2(prmt(vf[2 * x], 0, 0x31u));
                            const uint32_t a2 = e4m3x2_to_f16x2(prmt(vf[2 * x + 1], 0, 0x20u)), a3 = e4m3x2_to_f16x2(prmt(vf[2 * x + 1], 0, 0x31u));
#pragma unroll
                            for (int n = 0; n < NR; ++n) {
                                mma_f16(o[n][i + x], a0, a1, a2, a3, ph[n][0], ph[n][1]);
                                mma_f16(o[n][i + x], a0, a1, a2, a3, pl[n][0], pl[n][1]);
                            }
                        }
                    }
                }
            }
        } else if (a.logits) {
            // none of the step's slots is there: no row has a score for them
            const int r0 = cur.rt * 8 * NR, rows = min(8 * NR, a.rows - r0);
            float *at = a.logits + (((int64_t)cur.b * a.c.heads + cur.head) * a.rows + r0) * a.ld_logits + j0 + lane;
            if (lane < TOK && j0 + lane < cur.end)
#pragma unroll 1
                for (int r = 0; r < rows; ++r, at += a.ld_logits) *at = kNone;
        }
        __syncwarp();
        const uint32_t read_stage = ring + stage * C::STAGE;  // free until the next step
        stage = stage + 1 == C::STAGES ? 0 : stage + 1;

        const bool ends = cur.tile + 1 == cur.tiles;
        if (!ends && cur.left > 1) {
            --cur.left;
            ++cur.tile;
            continue;
        }
        // ---- the unit or the share ends: join the warps
        const Pos was = cur;
        cur.advance<C::CT>(a);
        const bool more_units = cur.left > 0;
        if (!C::QSMEM && more_units) load_queries(cur);  // (on their way during what follows; cs is not needed any more)
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, l[n][e], 4);
                l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, l[n][e], 8);
                l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, l[n][e], 16);
                if (g == 0) sm_m[warp][n * 8 + c4 * 2 + e] = m[n][e], sm_l[warp][n * 8 + c4 * 2 + e] = l[n][e];
            }
        if (lane == 0) sm_stage[warp] = read_stage;
        __syncthreads();
        // of its share's parts, a CTA leaves that of a unit begun before it in slot 0 and that of a unit
        // that goes on after it in slot 1
        const bool whole = began && ends;
        float *part = a.parts + (2 * (int64_t)blockIdx.x + began) * part_floats(D, NR);
        // thread r joins (m, l) of row r, for everybody
        if (tid < 8 * NR) {
            float mt = kNone, lt = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mt = fmaxf(mt, sm_m[w][tid]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = sm_m[w][tid] == kNone ? 0.f : ex2_approx(sm_m[w][tid] - mt);
                lt = fmaf(f, sm_l[w][tid], lt);
                sm_l[w][tid] = f;
            }
            const int r = was.rt * 8 * NR + tid, tok = sm_tok[r];
            sm_out[tid].row = ((int64_t)was.b * a.n_q + tok) * a.ldo + (int64_t)(was.head * a.group + r - tok * a.group) * D;
            sm_out[tid].inv = lt > 0.f || lt != lt ? a.v_scale / lt : 0.f;
            if (!whole) *reinterpret_cast<float2 *>(part + 2 * tid) = make_float2(mt, lt);
            else if (a.unit_ml) a.unit_ml[((int64_t)was.b * a.unit_heads + was.head * a.row_tiles) * 8 * NR + r] = make_float2(mt, lt);
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float f = sm_l[warp][n * 8 + c4 * 2 + e];
#pragma unroll
                for (int i = 0; i < KS; ++i) o[n][i][e] *= f, o[n][i][2 + e] *= f;
            }
        // o' of an octet from one warp to another through the stage that the first has just read
        auto put = [&](const float (&f)[KS][4]) {
#pragma unroll
            for (int i = 0; i < KS; ++i)
                sts128(read_stage + lane * 16 + i * 512,
                       make_uint4(__float_as_uint(f[i][0]), __float_as_uint(f[i][1]), __float_as_uint(f[i][2]), __float_as_uint(f[i][3])));
        };
        auto add = [&](int from, float (&f)[KS][4]) {
            const uint32_t at = sm_stage[from] + lane * 16;
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                const uint4 t = lds128(at + i * 512);
                f[i][0] += __uint_as_float(t.x), f[i][1] += __uint_as_float(t.y);
                f[i][2] += __uint_as_float(t.z), f[i][3] += __uint_as_float(t.w);
            }
        };
        auto write_out = [&](int n, const float (&f)[KS][4]) {
            if (whole) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = n * 8 + c4 * 2 + e;
                    if (was.rt * 8 * NR + r >= a.rows) continue;
                    uint16_t *out = a.o + sm_out[r].row;
                    const float inv = sm_out[r].inv;
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        const uint32_t t = pack_bf16(f[i][e] * inv, f[i][2 + e] * inv);
                        if constexpr (C::E4M3) {
                            *reinterpret_cast<uint32_t *>(out + i * 16 + 2 * g) = t;
                        } else {
                            out[i * 16 + g] = (uint16_t)t;
                            out[i * 16 + 8 + g] = (uint16_t)(t >> 16);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < KS; ++i)
                    *reinterpret_cast<float4 *>(part + 16 * NR + ((n * KS + i) * 32 + lane) * 4) = make_float4(f[i][0], f[i][1], f[i][2], f[i][3]);
            }
        };
        if constexpr (NR == 1) {
            // warps 2 and 3 to 0 and 1, then 1 to 0
            if (warp >= 2) put(o[0]);
            __syncthreads();
            if (warp < 2) add(warp + 2, o[0]);
            if (warp == 1) put(o[0]);
            __syncthreads();
            if (warp == 0) {
                add(1, o[0]);
                write_out(0, o[0]);
            }
        } else {
            // warp n collects octet n: in round k from warp n + k
#pragma unroll 1
            for (int k = 1; k < kWarps; ++k) {
                const int to = (warp - k) & (kWarps - 1);
#pragma unroll
                for (int n = 0; n < NR; ++n)
                    if (n == to) put(o[n]);
                __syncthreads();
#pragma unroll
                for (int n = 0; n < NR; ++n)
                    if (n == warp) add((warp + k) & (kWarps - 1), o[n]);
                __syncthreads();
            }
#pragma unroll
            for (int n = 0; n < NR; ++n)
                if (n == warp) write_out(n, o[n]);
        }
        __syncthreads();
        if (!more_units) break;
        if (C::QSMEM) load_queries(cur);
        begin_unit(cur);
        began = true;
    }
    cp_async_wait<0>();
}

// The parts of a unit: those of CTAs [first, last], none if the unit has no slots; one
// CTA alone has finished the unit (whole).
struct Parts {
    int first, last;
    bool empty, whole;
};
__device__ __forceinline__ Parts parts_of(const AttnArgs &a, int b, int hr) {
    const int64_t p0 = __ldg(a.prefix + b), p1 = __ldg(a.prefix + b + 1), total = __ldg(a.prefix + a.c.batch);
    Parts r = {0, 0, p0 == p1, false};
    if (!r.empty) {
        const int64_t all = p1 - p0;
        const int64_t n = all >> 31 ? all / a.unit_heads : (uint32_t)all / (uint32_t)a.unit_heads, t = p0 + hr * n;
        const int shares = shares_of(total, a.resident);
        r.first = share_of(total, shares, t);
        r.last = share_of(total, shares, t + n - kExtra - 1);
        r.whole = r.first == r.last;
    }
    return r;
}
__device__ __forceinline__ const float *part_at(const AttnArgs &a, const Parts &p, int i) {
    return a.parts + (int64_t)(2 * i + (i == p.first)) * a.part_floats;
}
constexpr int kJoinWarps = 16;  // of a block, at most

// (m, l) of row lane % 8 of octet n over the unit's parts x / 8, x = first, first + step, ... (multiples of 32 and
// the lane), joined over the lanes of the row.  kAhead: loads on their way at once.
template <int kAhead>
__device__ __forceinline__ float2 join_parts(const AttnArgs &a, const Parts &p, int n, int first, int step) {
    const int parts = p.last - p.first + 1;
    float top = kNone, sum = 0.f;
    for (int x0 = first; x0 < parts * 8; x0 += kAhead * step) {
        float2 ml[kAhead];
#pragma unroll
        for (int y = 0; y < kAhead; ++y) {
            const int x = x0 + y * step;
            ml[y] = x < parts * 8 ? *reinterpret_cast<const float2 *>(part_at(a, p, p.first + x / 8) + 2 * (n * 8 + x % 8)) : make_float2(kNone, 0.f);
        }
#pragma unroll
        for (int y = 0; y < kAhead; ++y) {
            if (ml[y].x == kNone) {
                sum += ml[y].y;  // 0, or NaN where every score is
                continue;
            }
            const float m = fmaxf(top, ml[y].x);
            sum = sum * ex2_approx(top - m) + ml[y].y * ex2_approx(ml[y].x - m);
            top = m;
        }
    }
    float m = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 8));
    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
    if (top != kNone) sum *= ex2_approx(top - m);
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 8);
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 16);
    return make_float2(m, sum);
}
// That of row `row` over warps w0, w0 + step, ... < w1, from scratch ([2][kJoinWarps][8]).
__device__ __forceinline__ float2 join_warps(const float (*scratch)[kJoinWarps][8], int row, int w0, int w1, int step) {
    float mt = kNone, lt = 0.f;
    for (int w = w0; w < w1; w += step) mt = fmaxf(mt, scratch[0][w][row]);
    for (int w = w0; w < w1; w += step) {
        const float mw = scratch[0][w][row];
        lt += scratch[1][w][row] * (mw == kNone ? 1.f : ex2_approx(mw - mt));
    }
    return make_float2(mt, lt);
}
// (m, l) of the 8 rows of octet n over all parts; every thread of the block calls it.  Row lane % 8's come back
// to every lane.
template <int kAhead>
__device__ __forceinline__ float2 join_ml(const AttnArgs &a, const Parts &p, int n, float (*scratch)[kJoinWarps][8]) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const float2 own = join_parts<kAhead>(a, p, n, tid, blockDim.x);
    __syncthreads();  // (what the scratch held has been read)
    if (lane < 8) scratch[0][warp][lane] = own.x, scratch[1][warp][lane] = own.y;
    __syncthreads();
    return join_warps(scratch, lane & 7, 0, warps, 1);
}

// Weights w of slots lo .. hi - 1 from the rows' scores z.  GROUPS: a chunk is fewer slots than the block takes at a
// time, and its rows are dealt to groups of threads, whose sums are added in red.
template <bool GROUPS, int kAt>
__device__ __forceinline__ void add_up(const AttnArgs &a, float *w, const float *z, uint32_t begin, uint32_t lo, uint32_t hi, int chunk, const float *sm_m,
                                       const float *sm_r, float *red) {
    constexpr int kRowsAhead = 4;  // rows whose scores are on their way at once
    const int groups = GROUPS ? kAt * blockDim.x / chunk : 1, per = blockDim.x / groups;
    const int group = GROUPS ? threadIdx.x / per : 0, t = threadIdx.x - group * per;
    for (uint32_t j0 = lo + t; GROUPS || j0 < hi; j0 += kAt * per) {
        float sum[kAt], old[kAt];
#pragma unroll
        for (int x = 0; x < kAt; ++x) {
            sum[x] = 0.f;
            if (group == 0 && j0 + x * per < hi) old[x] = w[j0 + x * per];
        }
        for (int r0 = group * kRowsAhead; r0 < a.rows; r0 += groups * kRowsAhead) {
            float s[kRowsAhead][kAt];
#pragma unroll
            for (int y = 0; y < kRowsAhead; ++y)
#pragma unroll
                for (int x = 0; x < kAt; ++x) {
                    const uint32_t j = j0 + x * per;
                    s[y][x] = r0 + y < a.rows && j >= begin && j < hi ? __ldg(z + (r0 + y) * a.ld_logits + j) : kNone;
                }
#pragma unroll
            for (int y = 0; y < kRowsAhead; ++y) {
                if (r0 + y >= a.rows) break;
                const float m = sm_m[r0 + y], f = sm_r[r0 + y];
#pragma unroll
                for (int x = 0; x < kAt; ++x) sum[x] = s[y][x] == kNone ? sum[x] : fmaf(ex2_approx(s[y][x] - m), f, sum[x]);
            }
        }
        if constexpr (GROUPS) {
            if (group > 0)
#pragma unroll
                for (int x = 0; x < kAt; ++x) red[(group - 1) * chunk + x * per + t] = sum[x];
            __syncthreads();
            if (group > 0) return;
            for (int g = 0; g < groups - 1; ++g)
#pragma unroll
                for (int x = 0; x < kAt; ++x) sum[x] += red[g * chunk + x * per + t];
        }
#pragma unroll
        for (int x = 0; x < kAt; ++x)
            if (j0 + x * per < hi) w[j0 + x * per] = fmaf(old[x], a.decay, sum[x]);
        if (GROUPS) return;  // (one turn covers the chunk)
    }
}

// A chunk of slots of one KV head's weights: weights <- decay * weights + sum of the rows' 2^(s - m) / l.
__device__ __forceinline__ void weigh(const AttnArgs &a, uint32_t id, int chunks, int chunk, float *sm_m, float *sm_r,
                                      float (*scratch)[kJoinWarps][8], float *red) {
    const uint32_t bh = id / (uint32_t)chunks;
    const int b = (int)(bh / (uint32_t)a.c.heads), h = (int)(bh - (uint32_t)b * (uint32_t)a.c.heads);
    int begin, len;
    seq_range(a, b, begin, len);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x, warps = threads >> 5;
    const int lo = (int)(id - bh * (uint32_t)chunks) * chunk;
    if (lo >= len) return;
    const int hi = lo + min(chunk, len - lo);
    if (hi > begin) {
        // the octets' (m, l): `at_once` octets at a time, a team of warps each
        const int octets = a.row_tiles * a.tile_rows / 8, at_once = min(octets, warps), team = warps / at_once;
        for (int o0 = 0; o0 < octets; o0 += at_once) {
            const int q = warp % at_once, o = o0 + q, mate = warp / at_once;
            float2 ml = make_float2(kNone, 0.f);
            if (o < octets && mate < team) {
                const int rt = o * 8 / a.tile_rows, n = o - rt * (a.tile_rows / 8);
                const Parts p = parts_of(a, b, h * a.row_tiles + rt);
                if (!p.whole) ml = join_parts<4>(a, p, n, mate * 32 + lane, team * 32);
                else if (mate == 0) ml = a.unit_ml[((int64_t)b * a.unit_heads + h * a.row_tiles) * a.tile_rows + o * 8 + (lane & 7)];
            }
            if (lane < 8) scratch[0][warp][lane] = ml.x, scratch[1][warp][lane] = ml.y;
            __syncthreads();
            const int r = o0 * 8 + tid;
            if (tid < at_once * 8 && r < a.rows) {
                const float2 all = join_warps(scratch, tid & 7, tid >> 3, team * at_once, at_once);
                sm_m[r] = all.x == kNone ? 0.f : all.x;
                sm_r[r] = all.y > 0.f || all.y != all.y ? ex2_approx(lift(a.c.e4m3 != 0)) / all.y : 0.f;
            }
            __syncthreads();
        }
    }
    float *w = a.weights + (int64_t)bh * a.ld_weights;
    const float *z = a.logits + (int64_t)bh * a.rows * a.ld_logits;
    constexpr int kAt = 4;  // slots of a thread at a time
    if (kAt * threads > chunk) add_up<true, kAt>(a, w, z, begin, lo, hi, chunk, sm_m, sm_r, red);
    else add_up<false, kAt>(a, w, z, begin, lo, hi, chunk, sm_m, sm_r, red);
}

// The first join_blocks blocks: units in several parts, and zeros for units without slots, `blocks` blocks a unit.
// A block joins 16 values of the 8 rows of an octet at a time (one fragment: 32 lanes of float4), its warps
// taking turns at the parts.  The others add up weights; they join (m, l) for themselves, which costs less than
// waiting for a kernel of its own.
template <bool WEIGH>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const AttnArgs a, int blocks, uint32_t join_blocks, int chunks, int chunk) {
    __shared__ float4 sm[kJoinWarps][32];
    __shared__ float scratch[2][kJoinWarps][8];
    const int warps = blockDim.x >> 5;
    pdl_wait();
    pdl_trigger();
    if constexpr (WEIGH) {
        __shared__ float sm_m[kMaxAttnRows], sm_r[kMaxAttnRows];
        if (blockIdx.x >= join_blocks) {
            weigh(a, blockIdx.x - join_blocks, chunks, chunk, sm_m, sm_r, scratch, reinterpret_cast<float *>(sm));
            return;
        }
    }
    const int D = a.c.dim, ks = D / 16, fragments = a.tile_rows / 8 * ks;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c4 = lane & 3;
    const uint32_t unit = blockIdx.x / (uint32_t)blocks, block = blockIdx.x - unit * (uint32_t)blocks;
    const int b = (int)(unit / (uint32_t)a.unit_heads), hr = (int)(unit - (uint32_t)b * (uint32_t)a.unit_heads);
    const Parts p = parts_of(a, b, hr);
    if (p.whole) return;
    const int head = hr / a.row_tiles, parts = p.last - p.first + 1;
    for (int fragment = (int)block; fragment < fragments; fragment += blocks) {
        const int n = fragment / ks, i = fragment - n * ks, r0 = (hr - head * a.row_tiles) * a.tile_rows + n * 8;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        float l[2] = {0.f, 0.f};
        if (!p.empty) {
            // the fragments of this warp's first parts are on their way during the join of (m, l)
            constexpr int kAhead = 4;
            float4 t[kAhead];
            const int64_t at = 2 * a.tile_rows + (fragment * 32 + lane) * 4, at_ml = 2 * (n * 8 + c4 * 2);
#pragma unroll
            for (int y = 0; y < kAhead; ++y)
                if (warp + y * warps < parts) t[y] = *reinterpret_cast<const float4 *>(part_at(a, p, p.first + warp + y * warps) + at);
            const float2 own = join_ml<WEIGH ? 4 : 1>(a, p, n, scratch);  // (with WEIGH, the code that weigh has)
            float mt[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) mt[e] = __shfl_sync(0xFFFFFFFFu, own.x, c4 * 2 + e), l[e] = __shfl_sync(0xFFFFFFFFu, own.y, c4 * 2 + e);
            for (int x0 = warp; x0 < parts; x0 += kAhead * warps) {
#pragma unroll
                for (int y = 0; y < kAhead; ++y) {
                    const int x = x0 + y * warps;
                    if (x < parts) {
                        const float4 ml = *reinterpret_cast<const float4 *>(part_at(a, p, p.first + x) + at_ml);
                        const float f0 = ml.x == kNone ? 0.f : ex2_approx(ml.x - mt[0]), f1 = ml.z == kNone ? 0.f : ex2_approx(ml.z - mt[1]);
                        v.x = fmaf(f0, t[y].x, v.x), v.y = fmaf(f1, t[y].y, v.y);
                        v.z = fmaf(f0, t[y].z, v.z), v.w = fmaf(f1, t[y].w, v.w);
                        if (x + kAhead * warps < parts)
                            t[y] = *reinterpret_cast<const float4 *>(part_at(a, p, p.first + x + kAhead * warps) + at);
                    }
                }
            }
            sm[warp][lane] = v;
            __syncthreads();
            if (warp > 0) continue;
            for (int w = 1; w < warps; ++w) {
                const float4 x = sm[w][lane];
                v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
            }
        } else if (warp > 0) {
            continue;
        }
        const float lo[2] = {v.x, v.y}, hi[2] = {v.z, v.w};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = r0 + c4 * 2 + e;
            if (r >= a.rows) continue;
            uint16_t *out = a.o + ((int64_t)b * a.n_q + r / a.group) * a.ldo + (int64_t)(head * a.group + r % a.group) * D + i * 16;
            const float inv = l[e] > 0.f || l[e] != l[e] ? a.v_scale / l[e] : 0.f;
            const uint32_t t = pack_bf16(lo[e] * inv, hi[e] * inv);
            if (a.c.e4m3) {
                *reinterpret_cast<uint32_t *>(out + 2 * g) = t;
            } else {
                out[g] = (uint16_t)t;
                out[8 + g] = (uint16_t)(t >> 16);
            }
        }
    }
}

template <int D, bool E4M3, int NR>
cudaError_t launch(AttnArgs &a, const DeviceInfo &di, cudaStream_t s) {
    using C = Cfg<D, E4M3, NR>;
    auto kern = attn_kernel<C>;
    cudaError_t e = ensure_smem((const void *)kern, C::SMEM);
    if (e != cudaSuccess) return e;
    // as many CTAs as are resident at once
    a.resident = di.sm_count * C::PER_SM < kMaxAttnResident ? di.sm_count * C::PER_SM : kMaxAttnResident;
    a.part_floats = part_floats(D, NR);
    const int64_t units = (int64_t)a.c.batch * a.unit_heads;
    // no more CTAs than the list has places, were every length the largest
    int64_t slots = a.cap;
    if (a.window > 0 && a.window + a.n_q < slots) slots = a.window + a.n_q;
    const int64_t most = units * ((slots + C::CT - 1) / C::CT + kExtra);
    const int64_t ctas = most < (int64_t)a.resident * kWaves ? most : (int64_t)a.resident * kWaves;
    e = launch_pdl(kern, dim3((unsigned)ctas), dim3(kThreads), C::SMEM, s, dim3(1), a);
    if (e != cudaSuccess) return e;
    // a block a fragment where units are few; fewer where most units are whole and their blocks only find that out
    const int64_t fragments = NR * (D / 16);
    int64_t blocks = (16 * di.sm_count + units - 1) / units;
    if (blocks > fragments) blocks = fragments;
    // a few units may be in hundreds of parts each
    const int join_threads = units * 64 <= a.resident ? kJoinWarps * 32 : kThreads;
    // weights: chunks of 2048 slots, which make the start of a block little work beside the rest, unless that leaves SMs
    // idle; at the least 512, or 256 and 128 where more than 16 and 32 rows lengthen the rest (64 heads of one row over 32000
    // slots: 37 us with 256 and 35 with 512; 112 rows of 41 sequences of 45 to 91 slots: 36 with 512, 34 with 256, 31
    // with 128)
    const int64_t heads = (int64_t)a.c.batch * a.c.heads;
    int chunk = 2048, chunks = 0;
    if (a.weights) {
        const int least = a.rows > 32 ? 128 : a.rows > 16 ? 256 : 512;
        while (chunk > least && heads * ((slots + chunk - 1) / chunk) < 4 * di.sm_count) chunk /= 2;  // (of slots in the window)
        chunks = (int)(((int64_t)a.cap + chunk - 1) / chunk);
    }
    return launch_pdl(a.weights ? join_kernel<true> : join_kernel<false>, dim3((unsigned)(units * blocks + heads * chunks)), dim3(join_threads), 0, s, dim3(1), a, (int)blocks,
                      (uint32_t)(units * blocks), chunks > 0 ? chunks : 1, chunk);
}

template <int D, bool E4M3>
cudaError_t launch_rows(AttnArgs &a, const DeviceInfo &di, cudaStream_t s) {
    switch (a.tile_rows) {
        case 8: return launch<D, E4M3, 1>(a, di, s);
        case 16: return launch<D, E4M3, 2>(a, di, s);
        default:
            if constexpr (D <= 128) return launch<D, E4M3, 4>(a, di, s);
            return cudaErrorInvalidValue;
    }
}

}  // namespace

// One octet of rows where they fit; otherwise as few row tiles of up to 32 rows (16 for D =
// 256, whose accumulators fill the registers) as hold them.
int attn_tile_rows(int D, int rows) { return rows <= 8 ? 8 : rows <= 16 || D == 256 ? 16 : 32; }
int attn_part_floats(int D, int tile_rows) { return part_floats(D, tile_rows / 8); }

cudaError_t launch_attn_decode(const DeviceInfo &di, AttnArgs &a, cudaStream_t s) {
    if (a.c.e4m3) return a.c.dim == 64 ? launch_rows<64, true>(a, di, s) : a.c.dim == 128 ? launch_rows<128, true>(a, di, s) : launch_rows<256, true>(a, di, s);
    return a.c.dim == 64 ? launch_rows<64, false>(a, di, s) : a.c.dim == 128 ? launch_rows<128, false>(a, di, s) : launch_rows<256, false>(a, di, s);
}

}  // namespace q4k
