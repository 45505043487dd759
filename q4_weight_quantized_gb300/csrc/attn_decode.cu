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
// Bound: every cached key and value is read once, so HBM; with up to 16 rows per KV
// head (group x new tokens) the tensor work is the same for any row count.  Hence
//   - The rows of one KV head are the 16 rows of mma.m16n8k16 (more rows: further row
//     tiles, which find the cache in L2); keys and values go through the MMA straight
//     from the ring, the two score tiles of a step turn in registers into the
//     A operand of the second product, and nothing but the cache is ever re-read.
//   - The batch's work is one list of tiles (sequence, head, row tile, 4 steps of
//     slots), cut into equal contiguous shares, one per CTA, whatever the lengths are:
//     a share may end one unit, hold whole units and begin another.  Whole units are
//     finished in place; parts leave (m, l, o') in the workspace for join_kernel.
//   - Each warp owns a ring of stages in shared memory which it fills with 16-byte
//     asynchronous copies of its own steps, so no barrier lies in the main loop; page
//     ids are loaded one step before the copies that need them.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "decode_ops.h"
#include "q4k_ptx.cuh"

namespace q4k {
namespace {

constexpr int kWarps = 4;           // warps of a CTA, each a step of every tile
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;           // rows of a row tile (mma m)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNone = -INFINITY;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
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
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
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

// floats of one part: (m, l) of 16 rows, then o' [16][D]
__host__ __device__ constexpr int part_floats(int D) { return 2 * kRows + kRows * D; }
// p of an e4m3 cache is kept as 2^15 p, in o' and l alike (see the kernel)
__host__ __device__ constexpr float lift(bool e4m3) { return e4m3 ? 15.f : 0.f; }

template <int D_, bool E4M3_>
struct Cfg {
    static constexpr int D = D_;
    static constexpr bool E4M3 = E4M3_;
    static constexpr int RB = D * (E4M3 ? 1 : 2);              // bytes of a cached row
    static constexpr int TOK = RB <= 128 ? 32 : 16;            // slots of a step
    static constexpr int CT = kWarps * TOK;                    // slots of a tile
    static constexpr int CHUNKS = RB / 16;                     // 16-byte chunks of a row
    static constexpr int STAGE = 2 * TOK * RB;                 // bytes of a stage: keys, then values
    static constexpr int STAGES = STAGE <= 4096 ? 4 : 3;
    static constexpr bool QSMEM = D > 128;                     // queries in shared memory: no registers left for them
    static constexpr int KS = D / 16;                          // k steps of the first product
    static constexpr int RING = kWarps * STAGES * STAGE;
    static constexpr int MERGE = kRows * D * 4;                // o' of the CTA
    static constexpr int QBYTES = QSMEM ? KS * 32 * 16 : 0;
    static constexpr int SMEM = RING + MERGE + QBYTES;
    // rows alternate over the 128-byte bank lines so that eight rows' chunks (bf16,
    // ldmatrix) or two neighbouring rows' four chunks (e4m3 keys) never share banks
    static __device__ __forceinline__ uint32_t chunk_at(uint32_t row, uint32_t chunk) {
        if constexpr (E4M3) {
            if constexpr (RB == 64) return row * RB + (chunk ^ ((row >> 1) & 3)) * 16;
            return row * RB + (chunk ^ (((row & 1) << 2) | ((row >> 1) & 3))) * 16;
        }
        return row * RB + (chunk ^ (row & 7)) * 16;
    }
};

// A position in the list of tiles: tile `tile` of `tiles` of unit (b, hr = head * row
// tiles + row tile).
struct Pos {
    int b, hr, tile, tiles;
    int begin, end;  // slots of the unit: the union of its rows' ranges
};

// Length of sequence b, cut to what table (and weights) can hold, and the slots its rows read.
__device__ __forceinline__ void seq_range(const AttnArgs &a, int b, int &begin, int &len) {
    len = max(0, min(__ldg(a.seq_lens + b), a.cap));
    begin = 0;
    if (a.window > 0) begin = (int)max((int64_t)0, (int64_t)len - a.n_q + 1 - a.window);
}
__device__ __forceinline__ void enter(const AttnArgs &a, Pos &p, int ct) {
    // the next sequence with slots; the list ends at a.c.batch
    for (; p.b < a.c.batch; ++p.b) {
        seq_range(a, p.b, p.begin, p.end);
        p.tiles = (p.end - p.begin + ct - 1) / ct;
        if (p.tiles > 0) return;
    }
}
__device__ __forceinline__ void advance(const AttnArgs &a, Pos &p, int ct) {
    if (++p.tile < p.tiles) return;
    p.tile = 0;
    if (++p.hr < a.unit_heads) return;
    p.hr = 0;
    ++p.b;
    enter(a, p, ct);
}

// Slots [begin, end) of row r (token-major: token r / group) of a sequence of length len.
__device__ __forceinline__ void row_range(const AttnArgs &a, int r, int len, int &begin, int &end) {
    if (r >= a.rows) {
        begin = end = 0;
        return;
    }
    end = max(0, len - a.n_q + 1 + r / a.group);
    begin = a.window > 0 ? (int)max((int64_t)0, (int64_t)end - a.window) : 0;
}

template <typename C>
__global__ void __launch_bounds__(kThreads, C::D == 256 && !C::E4M3 ? 1 : 2) attn_kernel(const AttnArgs a) {
    constexpr int D = C::D, TOK = C::TOK, NT = TOK / 8, KS = C::KS;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ float sm_m[kWarps][kRows], sm_l[kWarps][kRows];
    __shared__ uint32_t sm_mask[kWarps][C::STAGES];
    __shared__ int64_t sm_scan[kWarps + 2];
    __shared__ Pos sm_pos;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c4 = lane & 3;
    pdl_wait();
    pdl_trigger();

    // ---- this CTA's share of the list: tiles [t0, t1)
    int64_t t0, t1;
    {
        const int per = (a.c.batch + kThreads - 1) / kThreads;
        const int lo = min(tid * per, a.c.batch), hi = min(lo + per, a.c.batch);
        int64_t sum = 0;
        for (int b = lo; b < hi; ++b) {
            int begin, len;
            const int raw = __ldg(a.seq_lens + b);
            if (raw > a.cap && blockIdx.x == 0) atomicOr(a.c.status, kDevIndex);
            seq_range(a, b, begin, len);
            sum += (len - begin + C::CT - 1) / C::CT;
        }
        sum *= a.unit_heads;
        int64_t inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) sm_scan[warp] = inc;
        __syncthreads();
        int64_t before = inc - sum, total = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += sm_scan[w];
            total += sm_scan[w];
        }
        const int64_t shares = min((int64_t)a.ctas, total);  // none of them empty
        t0 = blockIdx.x < shares ? total * blockIdx.x / shares : total;
        t1 = blockIdx.x < shares ? total * (blockIdx.x + 1) / shares : total;
        if (t0 < t1 && before <= t0 && t0 < before + sum) {
            // this thread's sequences hold the share's first tile
            Pos p;
            int64_t at = before;
            for (p.b = lo;; ++p.b) {
                seq_range(a, p.b, p.begin, p.end);
                p.tiles = (p.end - p.begin + C::CT - 1) / C::CT;
                if (t0 < at + (int64_t)p.tiles * a.unit_heads) break;
                at += (int64_t)p.tiles * a.unit_heads;
            }
            p.hr = (int)((t0 - at) / p.tiles);
            p.tile = (int)((t0 - at) % p.tiles);
            sm_pos = p;
        }
        if (blockIdx.x == 0) {
            int64_t at = before;
            for (int b = lo; b < hi; ++b) {
                int begin, len;
                a.prefix[b] = at;
                seq_range(a, b, begin, len);
                at += (int64_t)((len - begin + C::CT - 1) / C::CT) * a.unit_heads;
            }
            if (tid == 0) a.prefix[a.c.batch] = total;
        }
        if (t0 >= t1) return;
        __syncthreads();
    }
    Pos cur = sm_pos, nxt = cur;

    const uint32_t ring = smem_u32(smem) + warp * (C::STAGES * C::STAGE);
    float *merge = reinterpret_cast<float *>(smem + C::RING);
    uint4 *qs = reinterpret_cast<uint4 *>(smem + C::RING + C::MERGE);

    // ---- copies: the page id of this lane's slot of the next step to be copied is in flight
    int64_t to_copy = t1 - t0;  // tiles whose copies are still to be issued
    int32_t page = -1;
    int slot = 0;
    bool in = false;
    auto fetch_page = [&] {
        if (to_copy > 0) {
            slot = nxt.begin + (nxt.tile * kWarps + warp) * TOK + lane;
            in = lane < TOK && slot < nxt.end;
            page = in ? __ldg(a.c.table + nxt.b * a.c.ld_table + page_of(a.c, slot)) : -1;
        }
    };
    auto copy_step = [&](int stage) {
        if (to_copy > 0) {
            const bool ok = in && page_ok(a.c, page);
            if (in && !ok) atomicOr(a.c.status, kDevIndex);
            const uint32_t mask = __ballot_sync(0xFFFFFFFFu, ok);
            if (lane == 0) sm_mask[warp][stage] = mask;
            const int64_t off =
                ok ? row_bytes_at(a.c, page, nxt.hr / a.row_tiles, (uint32_t)slot - page_of(a.c, slot) * a.c.page_size) : 0;
            const uint32_t dst = ring + stage * C::STAGE;
#pragma unroll
            for (int i = 0; i < TOK * C::CHUNKS / 32; ++i) {
                const int row = (i * 32 + lane) / C::CHUNKS, ch = lane % C::CHUNKS;
                const int64_t o = __shfl_sync(0xFFFFFFFFu, off, row) + ch * 16;
                const uint32_t n = (mask >> row & 1) * 16;  // slots that are not there become zeros
                cp_async16(dst + C::chunk_at(row, ch), a.c.k + o, n);
                cp_async16(dst + TOK * C::RB + C::chunk_at(row, ch), a.c.v + o, n);
            }
            --to_copy;
            advance(a, nxt, C::CT);
        }
        cp_async_commit();
        fetch_page();
    };
    fetch_page();
#pragma unroll
    for (int s = 0; s < C::STAGES - 1; ++s) copy_step(s);

    uint32_t qf[C::QSMEM ? 1 : KS][4];
    float o[D / 8][4], m[2], l[2], cs[2];
    int rb[2], re[2];        // slot ranges of rows g and g + 8
    int in_lo = 0, in_hi = 0;  // slots that every row of the tile reads
    bool fresh = true;       // the next step begins a unit (or the share)
    int stage = 0;

    for (int64_t left = t1 - t0; left > 0; --left) {
        const int head = cur.hr / a.row_tiles, r0 = (cur.hr % a.row_tiles) * kRows;
        if (fresh) {
            // queries of rows g, g + 8 as the A operand; e4m3: as f16 scaled by a power of two
            float mx[2] = {0.f, 0.f};
            const uint16_t *qrow[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = r0 + g + 8 * h;
                const int tok = r / a.group, hq = head * a.group + r % a.group;
                qrow[h] = r < a.rows ? a.q + ((int64_t)cur.b * a.n_q + tok) * a.ldq + (int64_t)hq * D : nullptr;
                row_range(a, r, cur.end, rb[h], re[h]);
                m[h] = kNone;
                l[h] = 0.f;
            }
            auto q_at = [&](int h, int ks, int half) -> uint32_t {
                // the pair of query values that meets key values (k = 2 c4, 2 c4 + 1 | + 8) of k step ks
                const int d = C::E4M3 ? (ks / 4) * 64 + c4 * 16 + (ks % 4) * 4 + half * 2 : ks * 16 + c4 * 2 + half * 8;
                return qrow[h] ? __ldg(reinterpret_cast<const uint32_t *>(qrow[h] + d)) : 0u;
            };
            float up[2] = {1.f, 1.f};
            if constexpr (C::E4M3) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    for (int ks = 0; ks < KS; ++ks)
                        for (int f = 0; f < 2; ++f) {
                            const uint32_t v = q_at(h, ks, f);
                            mx[h] = fmaxf(mx[h], fmaxf(fabsf(lo_f32(v)), fabsf(hi_f32(v))));
                        }
                    mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xFFFFFFFFu, mx[h], 1));
                    mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xFFFFFFFFu, mx[h], 2));
                    // 2^(14 - exponent of the largest): f16 then holds bf16's 8 bits of every value
                    // down to 2^-30 of the largest (exponents are kept where 2^(14 - e) is a float)
                    const int e = (int)(__float_as_uint(mx[h]) >> 23);
                    if (e > 14 && e < 255) up[h] = __uint_as_float((uint32_t)(min(127 + 14 + 127 - e, 254)) << 23);
                }
            }
            auto q_frag = [&](int ks, uint32_t (&f)[4]) {
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t v = q_at(h, ks, half);
                        f[half * 2 + h] = C::E4M3 ? pack_f16(lo_f32(v) * up[h], hi_f32(v) * up[h]) : v;
                    }
            };
            if constexpr (C::QSMEM) {
                __syncthreads();  // the unit before has been read by every warp
                for (int ks = warp; ks < KS; ks += kWarps) {
                    uint32_t f[4];
                    q_frag(ks, f);
                    qs[ks * 32 + lane] = make_uint4(f[0], f[1], f[2], f[3]);
                }
                __syncthreads();
            } else {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) q_frag(ks, qf[ks]);
            }
            cs[0] = a.scale / up[0];
            cs[1] = a.scale / up[1];
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
            // rows of this tile: first and last token decide what all of them read
            const int r_last = min(r0 + kRows, a.rows) - 1;
            int b_, e_;
            row_range(a, r0, cur.end, b_, in_hi);
            row_range(a, r_last, cur.end, in_lo, e_);
            fresh = false;
        }

        cp_async_wait<C::STAGES - 2>();
        __syncwarp();
        copy_step((stage + C::STAGES - 1) % C::STAGES);

        const uint32_t ks_addr = ring + stage * C::STAGE, vs_addr = ks_addr + TOK * C::RB;
        const uint32_t mask = sm_mask[warp][stage];
        const int j0 = cur.begin + (cur.tile * kWarps + warp) * TOK;  // first slot of the step
        if (mask) {
            // ---- s = q k^T
            float s[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
            if constexpr (!C::E4M3) {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t qa[4];
                    if constexpr (C::QSMEM) {
                        const uint4 t = qs[ks * 32 + lane];
                        qa[0] = t.x, qa[1] = t.y, qa[2] = t.z, qa[3] = t.w;
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) qa[i] = qf[ks][i];
                    }
#pragma unroll
                    for (int n = 0; n < NT; n += 2) {
                        uint32_t kb[4];
                        ldsm4(kb, ks_addr + C::chunk_at(n * 8 + (lane & 7) + ((lane >> 4) << 3), 2 * ks + ((lane >> 3) & 1)));
                        mma_bf16_16816(s[n], qa, kb[0], kb[1], s[n]);
                        mma_bf16_16816(s[n + 1], qa, kb[2], kb[3], s[n + 1]);
                    }
                }
            } else {
#pragma unroll
                for (int kq = 0; kq < KS / 4; ++kq) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint4 w = lds128(ks_addr + C::chunk_at(n * 8 + g, 4 * kq + c4));
                        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t qa[4];
                            if constexpr (C::QSMEM) {
                                const uint4 t = qs[(kq * 4 + i) * 32 + lane];
                                qa[0] = t.x, qa[1] = t.y, qa[2] = t.z, qa[3] = t.w;
                            } else {
#pragma unroll
                                for (int x = 0; x < 4; ++x) qa[x] = qf[kq * 4 + i][x];
                            }
                            mma_f16_16816(s[n], qa, e4m3x2_to_f16x2(ww[i]), e4m3x2_to_f16x2(ww[i] >> 16), s[n]);
                        }
                    }
                }
            }
            // ---- scores in units of log2, masked
            if (a.softcap > 0.f) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s[n][i] = a.softcap * kLog2e * tanhf(s[n][i] * cs[i >> 1] / a.softcap);
            } else {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[n][i] *= cs[i >> 1] * kLog2e;
            }
            const uint32_t full = TOK == 32 ? 0xFFFFFFFFu : (1u << TOK) - 1;
            const bool inside = j0 >= in_lo && j0 + TOK <= in_hi;
            if (mask != full || !inside) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int t = n * 8 + c4 * 2 + (i & 1), j = j0 + t, h = i >> 1;
                        if (!(mask >> t & 1) || j < rb[h] || j >= re[h]) s[n][i] = kNone;
                    }
            }
            if (a.logits) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = r0 + g + 8 * h;
                    if (r < a.rows) {
                        float *row = a.logits + (((int64_t)cur.b * a.c.heads + head) * a.rows + r) * a.ld_logits;
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int j = j0 + n * 8 + c4 * 2 + i;
                                if (j < cur.end) row[j] = s[n][h * 2 + i];
                            }
                    }
                }
            }
            // ---- running maximum and sum; e4m3: p is 2^15 times itself, in o' and l alike, so that
            // f16 holds p down to 2^-39
            constexpr float kLift = lift(C::E4M3);
            float alpha[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float t = kNone;
#pragma unroll
                for (int n = 0; n < NT; ++n) t = fmaxf(t, fmaxf(s[n][h * 2], s[n][h * 2 + 1]));
                t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 1));
                t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 2));
                const float mn = fmaxf(m[h], t);
                const float base = mn == kNone ? 0.f : mn;
                alpha[h] = ex2_approx(m[h] - base);
                m[h] = mn;
                float sum = 0.f;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float p = ex2_approx(s[n][h * 2 + i] - base + kLift);
                        s[n][h * 2 + i] = p;
                        sum += p;
                    }
                l[h] = l[h] * alpha[h] + sum;
            }
            if (__any_sync(0xFFFFFFFFu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    o[n][0] *= alpha[0], o[n][1] *= alpha[0];
                    o[n][2] *= alpha[1], o[n][3] *= alpha[1];
                }
            }
            // ---- slots that some rows read and others do not (the new tokens themselves, the window's
            // edge): 0 * inf must not reach the others, so these are added row by row and then
            // taken out of the product
            if (!inside && a.n_q > 1) {
                for (int t = 0; t < TOK; ++t) {
                    const int j = j0 + t;
                    if (!(mask >> t & 1) || (j >= in_lo && j < in_hi)) continue;
                    float p0 = 0.f, p1 = 0.f;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        if (n == t / 8) {
                            p0 = t & 1 ? s[n][1] : s[n][0], p1 = t & 1 ? s[n][3] : s[n][2];
                            if (c4 == (t & 7) / 2) {
                                if (t & 1) s[n][1] = s[n][3] = 0.f;
                                else s[n][0] = s[n][2] = 0.f;
                            }
                        }
                    p0 = __shfl_sync(0xFFFFFFFFu, p0, (lane & ~3) | (t & 7) / 2);
                    p1 = __shfl_sync(0xFFFFFFFFu, p1, (lane & ~3) | (t & 7) / 2);
                    const bool on0 = j >= rb[0] && j < re[0], on1 = j >= rb[1] && j < re[1];
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        float v0, v1;
                        if constexpr (C::E4M3) {
                            const int d = (n / 2) * 16 + c4 * 4 + (n & 1);
                            const uint32_t at = vs_addr + C::chunk_at(t, d / 16) + d % 16;
                            uint32_t b0, b1;
                            asm volatile("ld.shared.u8 %0, [%1];" : "=r"(b0) : "r"(at) : "memory");
                            asm volatile("ld.shared.u8 %0, [%1];" : "=r"(b1) : "r"(at + 2) : "memory");
                            v0 = e4m3_to_f32(b0), v1 = e4m3_to_f32(b1);
                        } else {
                            const int d = n * 8 + c4 * 2;
                            uint32_t v;
                            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(vs_addr + C::chunk_at(t, d / 8) + (d % 8) * 2) : "memory");
                            v0 = lo_f32(v), v1 = hi_f32(v);
                        }
                        if (on0) o[n][0] = fmaf(p0, v0, o[n][0]), o[n][1] = fmaf(p0, v1, o[n][1]);
                        if (on1) o[n][2] = fmaf(p1, v0, o[n][2]), o[n][3] = fmaf(p1, v1, o[n][3]);
                    }
                    __syncwarp();
                    if (lane < C::CHUNKS)
                        asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(vs_addr + C::chunk_at(t, lane)), "r"(0) : "memory");
                    __syncwarp();
                }
            }
            // ---- o' += p v, p as the sum of two 16-bit values (one alone would cost as much as o's own
            // rounding)
#pragma unroll
            for (int kk = 0; kk < TOK / 16; ++kk) {
                uint32_t ph[4], pl[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = s[kk * 2 + (i >> 1)][(i & 1) * 2], y = s[kk * 2 + (i >> 1)][(i & 1) * 2 + 1];
                    if constexpr (C::E4M3) {
                        ph[i] = pack_f16(x, y);
                        const float2 b = __half22float2(*reinterpret_cast<__half2 *>(&ph[i]));
                        pl[i] = pack_f16(x - b.x, y - b.y);
                    } else {
                        ph[i] = pack_bf16(x, y);
                        pl[i] = pack_bf16(x - lo_f32(ph[i]), y - hi_f32(ph[i]));
                    }
                }
                if constexpr (!C::E4M3) {
#pragma unroll
                    for (int n = 0; n < D / 8; n += 2) {
                        uint32_t vb[4];
                        ldsm4_trans(vb, vs_addr + C::chunk_at(kk * 16 + (lane & 15), n + (lane >> 4)));
                        mma_bf16_16816(o[n], ph, vb[0], vb[1], o[n]);
                        mma_bf16_16816(o[n + 1], ph, vb[2], vb[3], o[n + 1]);
                        mma_bf16_16816(o[n], pl, vb[0], vb[1], o[n]);
                        mma_bf16_16816(o[n + 1], pl, vb[2], vb[3], o[n + 1]);
                    }
                } else {
                    // a transposed 8 x 8 matrix of byte pairs: each register holds values d, d + 1 of two
                    // slots; tile 2i takes the even d, tile 2i + 1 the odd ones
#pragma unroll
                    for (int n = 0; n < D / 8; n += 4) {
                        uint32_t vb[4];
                        ldsm4_trans(vb, vs_addr + C::chunk_at(kk * 16 + (lane & 15), n / 2 + (lane >> 4)));
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const uint32_t sel = x & 1 ? 0x31u : 0x20u;
                            const uint32_t b0 = e4m3x2_to_f16x2(prmt(vb[(x >> 1) * 2], 0, sel));
                            const uint32_t b1 = e4m3x2_to_f16x2(prmt(vb[(x >> 1) * 2 + 1], 0, sel));
                            mma_f16_16816(o[n + x], ph, b0, b1, o[n + x]);
                            mma_f16_16816(o[n + x], pl, b0, b1, o[n + x]);
                        }
                    }
                }
            }
        }
        __syncwarp();
        stage = (stage + 1) % C::STAGES;

        // ---- the unit or the share ends: join the warps
        if (cur.tile + 1 == cur.tiles || left == 1) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 1);
                l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 2);
                if (c4 == 0) sm_m[warp][g + 8 * h] = m[h], sm_l[warp][g + 8 * h] = l[h];
            }
            __syncthreads();
            float f[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float top = kNone;
                for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm_m[w][g + 8 * h]);
                f[h] = m[h] == kNone ? 0.f : ex2_approx(m[h] - top);
            }
            for (int w = 0; w < kWarps; ++w) {
                if (w == warp) {
#pragma unroll
                    for (int n = 0; n < D / 8; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int d = C::E4M3 ? (n / 2) * 16 + c4 * 4 + (n & 1) + (i & 1) * 2 : n * 8 + c4 * 2 + (i & 1);
                            float *at = merge + (g + 8 * (i >> 1)) * D + d;
                            const float v = f[i >> 1] == 0.f ? 0.f : o[n][i] * f[i >> 1];
                            *at = w == 0 ? v : *at + v;
                        }
                }
                __syncthreads();
            }
            const int rows = min(kRows, a.rows - r0);
            // of its share's parts, a CTA leaves that of a unit begun before it in slot 0 and that of a
            // unit that goes on after it in slot 1
            const bool began = cur.tile <= t1 - t0 - left;
            const bool whole = began && cur.tile + 1 == cur.tiles;
            const int64_t unit = (int64_t)cur.b * a.unit_heads + cur.hr;
            float *part = a.parts + (2 * (int64_t)blockIdx.x + began) * part_floats(D);
            for (int r = warp; r < rows; r += kWarps) {
                float top = kNone, sum = 0.f;
                for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm_m[w][r]);
                for (int w = 0; w < kWarps; ++w)
                    if (sm_m[w][r] != kNone) sum += sm_l[w][r] * ex2_approx(sm_m[w][r] - top);
                if (whole) {
                    const int rr = r0 + r;
                    uint16_t *out = a.o + ((int64_t)cur.b * a.n_q + rr / a.group) * a.ldo +
                                    (int64_t)(head * a.group + rr % a.group) * D;
                    const float inv = sum > 0.f || sum != sum ? a.v_scale / sum : 0.f;
                    for (int d = lane * 2; d < D; d += 64)
                        *reinterpret_cast<uint32_t *>(out + d) = pack_bf16(merge[r * D + d] * inv, merge[r * D + d + 1] * inv);
                    if (lane == 0) a.unit_ml[unit * kRows + r] = make_float2(top, sum);
                } else {
                    for (int d = lane * 4; d < D; d += 128)
                        *reinterpret_cast<float4 *>(part + 2 * kRows + r * D + d) = *reinterpret_cast<const float4 *>(merge + r * D + d);
                    if (lane == 0) part[2 * r] = top, part[2 * r + 1] = sum;
                }
            }
            __syncthreads();
            fresh = true;
        }
        advance(a, cur, C::CT);
    }
    cp_async_wait<0>();
}

// The parts of a unit: those of CTAs [first, last], none if the unit has no slots; one
// CTA alone has finished the unit (whole).
struct Parts {
    int64_t first, last;
    bool empty, whole;
};
__device__ __forceinline__ Parts parts_of(const AttnArgs &a, int64_t unit) {
    const int64_t b = unit / a.unit_heads, hr = unit % a.unit_heads;
    const int64_t p0 = a.prefix[b], p1 = a.prefix[b + 1], total = a.prefix[a.c.batch];
    const int64_t tiles = (p1 - p0) / a.unit_heads, t = p0 + hr * tiles;
    Parts r = {0, 0, tiles == 0, false};
    if (!r.empty) {
        // share i holds the tiles [total i / shares, total (i + 1) / shares)
        const int64_t shares = min((int64_t)a.ctas, total);
        r.first = ((t + 1) * shares - 1) / total;
        r.last = ((t + tiles) * shares - 1) / total;
        r.whole = r.first == r.last;
    }
    return r;
}
__device__ __forceinline__ const float *part_at(const AttnArgs &a, const Parts &p, int64_t i) {
    return a.parts + (2 * i + (i == p.first)) * part_floats(a.c.dim);
}
// (m, l) of one row over all its parts; every lane of the warp calls it and gets it.
__device__ __forceinline__ float2 join_ml(const AttnArgs &a, const Parts &p, int64_t unit, int row) {
    if (p.empty) return make_float2(kNone, 0.f);
    if (p.whole) return a.unit_ml[unit * kRows + row];
    const int lane = threadIdx.x & 31;
    float m = kNone, l = 0.f;
    for (int64_t i = p.first + lane; i <= p.last; i += 32) {
        const float2 ml = *reinterpret_cast<const float2 *>(part_at(a, p, i) + 2 * row);
        if (ml.x == kNone) continue;
        const float top = fmaxf(m, ml.x);
        l = l * ex2_approx(m - top) + ml.y * ex2_approx(ml.x - top);
        m = top;
    }
    float top = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if (m != kNone) l *= ex2_approx(m - top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
    return make_float2(top, l);
}

constexpr int kChunk = 2048;  // slots of a block that adds up weights

// Blocks [0, join_blocks): the rows of units in several parts (a warp a row), and zeros
// for units without slots.  The others: a chunk of slots of one KV head's weights.
__global__ void __launch_bounds__(kThreads) join_kernel(const AttnArgs a, int join_blocks, int chunks) {
    __shared__ float sm_m[kMaxAttnRows], sm_r[kMaxAttnRows];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = a.c.dim;
    if ((int)blockIdx.x < join_blocks) {
        const int64_t unit = blockIdx.x / (kRows / kWarps);
        const int row = (blockIdx.x % (kRows / kWarps)) * kWarps + warp;
        const int b = (int)(unit / a.unit_heads), hr = (int)(unit % a.unit_heads);
        const int r = (hr % a.row_tiles) * kRows + row;
        if (r >= a.rows) return;
        const Parts p = parts_of(a, unit);
        if (p.whole) return;
        uint16_t *out = a.o + ((int64_t)b * a.n_q + r / a.group) * a.ldo +
                        (int64_t)(hr / a.row_tiles * a.group + r % a.group) * D;
        const float2 ml = join_ml(a, p, unit, row);
        const float inv = ml.y > 0.f || ml.y != ml.y ? a.v_scale / ml.y : 0.f;
        for (int d = lane * 2; d < D; d += 64) {
            float x = 0.f, y = 0.f;
            if (!p.empty) {
#pragma unroll 8
                for (int64_t i = p.first; i <= p.last; ++i) {
                    const float *part = part_at(a, p, i);
                    const float mi = part[2 * row];
                    const float2 v = *reinterpret_cast<const float2 *>(part + 2 * kRows + row * D + d);
                    const float f = mi == kNone ? 0.f : ex2_approx(mi - ml.x);
                    x = fmaf(f, v.x, x), y = fmaf(f, v.y, y);
                }
            }
            *reinterpret_cast<uint32_t *>(out + d) = pack_bf16(x * inv, y * inv);
        }
        return;
    }
    const int64_t id = blockIdx.x - join_blocks;
    const int64_t bh = id / chunks;
    const int b = (int)(bh / a.c.heads), h = (int)(bh % a.c.heads);
    int begin, len;
    seq_range(a, b, begin, len);
    const int lo = (int)(id % chunks) * kChunk, hi = min(lo + kChunk, len);
    if (lo >= len) return;
    if (hi > begin)
        for (int rt = 0; rt < a.row_tiles; ++rt) {
            const int64_t unit = (int64_t)b * a.unit_heads + h * a.row_tiles + rt;
            const Parts p = parts_of(a, unit);
            for (int row = warp; row < kRows && rt * kRows + row < a.rows; row += kWarps) {
                const float2 ml = join_ml(a, p, unit, row);
                if (lane == 0) {
                    sm_m[rt * kRows + row] = ml.x == kNone ? 0.f : ml.x;
                    sm_r[rt * kRows + row] = ml.y > 0.f || ml.y != ml.y ? ex2_approx(lift(a.c.e4m3 != 0)) / ml.y : 0.f;
                }
            }
        }
    __syncthreads();
    float *w = a.weights + bh * a.ld_weights;
    const float *z = a.logits + bh * a.rows * a.ld_logits;
    for (int j = lo + threadIdx.x; j < hi; j += kThreads) {
        float sum = 0.f;
        if (j >= begin)
            for (int r = 0; r < a.rows; ++r) {
                const float s = z[r * a.ld_logits + j];
                if (s != kNone) sum = fmaf(ex2_approx(s - sm_m[r]), sm_r[r], sum);
            }
        w[j] = fmaf(w[j], a.decay, sum);
    }
}

template <int D, bool E4M3>
cudaError_t launch(AttnArgs &a, const DeviceInfo &di, cudaStream_t s) {
    using C = Cfg<D, E4M3>;
    auto kern = attn_kernel<C>;
    cudaError_t e = ensure_smem((const void *)kern, C::SMEM);
    if (e != cudaSuccess) return e;
    // as many CTAs as are resident at once
    const int per_sm = C::SMEM <= 112 * 1024 ? 2 : 1;
    a.ctas = di.sm_count * per_sm < kMaxAttnCtas ? di.sm_count * per_sm : kMaxAttnCtas;
    e = launch_pdl(kern, dim3(a.ctas), dim3(kThreads), C::SMEM, s, dim3(1), a);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)a.c.batch * a.unit_heads;
    const int64_t join_blocks = units * (kRows / kWarps);
    const int chunks = a.weights ? (a.cap + kChunk - 1) / kChunk : 0;
    return launch_pdl(join_kernel, dim3((unsigned)(join_blocks + (int64_t)a.c.batch * a.c.heads * chunks)), dim3(kThreads), 0, s,
                      dim3(1), a, (int)join_blocks, chunks > 0 ? chunks : 1);
}

}  // namespace

int attn_part_floats(int D) { return part_floats(D); }

cudaError_t launch_attn_decode(const DeviceInfo &di, AttnArgs &a, cudaStream_t s) {
    if (a.c.e4m3) return a.c.dim == 64 ? launch<64, true>(a, di, s) : a.c.dim == 128 ? launch<128, true>(a, di, s) : launch<256, true>(a, di, s);
    return a.c.dim == 64 ? launch<64, false>(a, di, s) : a.c.dim == 128 ? launch<128, false>(a, di, s) : launch<256, false>(a, di, s);
}

}  // namespace q4k
