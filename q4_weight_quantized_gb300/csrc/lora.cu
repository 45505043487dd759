// Low-rank adapters of many requests beside a shared projection:
//     y[t] += c_a B_a (A_a x[t]),  a = ids[t].
//
// Two products over the tokens of one adapter at a time (a tile: an adapter and at most 192 of its tokens), the
// inner sums v[t] = c_a A_a x[t] between them in the workspace:
//   shrink   v: m16n8k16 MMAs, 16 tokens by R.  The K axis is split over the warps of a CTA and the CTAs of a cluster (few
//            tiles must fill the GPU), whose sums are added in their order through each other's shared memory.  Any
//            pairing of k positions gives the same sum, so a lane's eight consecutive values of a row are its share of two
//            MMA steps: operands come straight from global memory, 16 bytes at a time.
//   expand   y: the fp32 inner sums are split into three bf16 pieces of 8 significant bits each (exact), so that the
//            second product has exact products, too.  Columns are dealt to MMA tiles so that a lane owns four
//            consecutive ones: y is read and written 16 bytes at a time.  Warps share nothing; a warp keeps its columns
//            of B in registers and walks the tile's tokens, 16 at a time, the next ones' y on its way.
// More than 192 tokens are sorted by adapter first (the experts' counting sort), then the two kernels run.  Up to 192 find their
// tiles themselves, and clusters of CTAs do both products in one launch, the inner sums staying in shared memory; meanwhile a
// CTA's part of B comes into L2.  Where few adapters have tokens the clusters that the GPU holds are shared out to them: groups
// of 16 tokens first, then columns, for which each makes the first product again.
// What is not finite in B is no part of the second product (a piece may be 0, and 0 * infinity is no number); it adds its own.
// Bound by HBM: of many tokens by y, read and written once, of few by the adapters' matrices and by latency.
// Measured: 32 tokens, 24 adapters of rank 16, 5120 x 5120 10 us (11.1 as two launches); 64 tokens, 16 adapters of rank up
// to 64, 5120 -> 17408 22 us (45 as two launches); 83 tokens of one adapter of rank 16, 768 -> 6526 14 us (54 by one cluster);
// 4096 tokens, 4 adapters of rank 16, 5120 -> 17408 122 us: 5.0 TB/s, of which expand_kernel about 100 (5.7 TB/s); 6944 tokens of
// rank 128, 408 -> 5120 111 us (118 with 32 columns a warp, 148 with 16), the issue of three products for one (302 with each warp splitting the inner sums for itself).
#include <cuda_runtime.h>

#include <atomic>

#include "decode_ops.h"
#include "q4k_ptx.cuh"

namespace q4k {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;  // of expand_kernel
constexpr int kMaxCluster = 8;  // tile_kernel's clusters are of that many
constexpr int kTileTokens = kMoeTileItems;
static_assert(kLoraSmall <= kTileTokens, "the tokens of a small call fit in one tile");

struct Tile {
    int adapter, count, rank;
};

// Tile `k` of the sorted tokens, these in list[]; count 0: nothing to do.  Every thread of THREADS calls it.
template <int THREADS>
__device__ __forceinline__ Tile tile_of(const LoraArgs &a, int k, int *list) {
    Tile t = {-1, 0, 0};
    if (k >= __ldg(a.n_tiles)) return t;
    const int4 r = __ldg(a.tiles + k);
    t.adapter = r.x, t.count = r.z;
    for (int i = threadIdx.x; i < r.z; i += THREADS) list[i] = __ldg(a.perm + r.y + i);
    __syncthreads();
    t.rank = a.ranks ? min(max(__ldg(a.ranks + t.adapter), 0), a.R) : a.R;
    return t;
}

// What cluster blockIdx.y of a small call does: an adapter's tokens (those with adapters at all, by their first token, have the
// clusters dealt out to them evenly), of these every `stride`-th 16 from first_token on, and part `part` of `parts` of the columns.
// first_at, one for each adapter, is kLoraSmall.
struct Small : Tile {
    int first_token, stride, part, parts;
};
template <int THREADS>
__device__ __forceinline__ Small small_tile(const LoraArgs &a, int *list, uint32_t (*masks)[THREADS / 32], int *first_at) {
    static_assert(kLoraSmall <= THREADS, "a token a thread");
    constexpr int WARPS = THREADS / 32;
    const int tid = threadIdx.x, warp = tid >> 5;
    const uint32_t below = (1u << (tid & 31)) - 1u;
    Small t = {};
    const int id = tid < a.T ? __ldg(a.ids + tid) : -1;
    const bool in = id >= 0 && id < a.n_adapters;
    if (id >= a.n_adapters && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(a.status, kDevIndex);
    if (in) atomicMin(first_at + id, tid);
    __syncthreads();
    const uint32_t first = __ballot_sync(0xFFFFFFFFu, in && first_at[id] == tid);
    if ((tid & 31) == 0) masks[0][warp] = first;
    __syncthreads();
    int active = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) active += __popc(masks[0][w]);
    if (active == 0) return t;
    const int each = max(1, (int)gridDim.y / active), k = blockIdx.y / each;
    if (k >= active) return t;
    int left = k, at = 0;  // the k-th first token
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        const uint32_t m = masks[0][w], it = __ballot_sync(0xFFFFFFFFu, (m >> (tid & 31) & 1u) && __popc(m & below) == left);
        if (it) at = 32 * w + __ffs(it) - 1;
        left -= __popc(m);
    }
    t.adapter = __ldg(a.ids + at);
    const uint32_t mine = __ballot_sync(0xFFFFFFFFu, id == t.adapter);
    if ((tid & 31) == 0) masks[1][warp] = mine;
    __syncthreads();
    int before = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += __popc(masks[1][w]);
        t.count += __popc(masks[1][w]);
    }
    if (id == t.adapter) list[before + __popc(mine & below)] = tid;
    __syncthreads();
    t.rank = a.ranks ? min(max(__ldg(a.ranks + t.adapter), 0), a.R) : a.R;
    // tokens first; columns as long as what each cluster does of them is not small beside the first product, which every one makes
    const int share = blockIdx.y - k * each, groups = (t.count + 15) / 16;
    t.stride = min(each, groups);
    // (N, K <= 2^21)
    t.parts = max(1, min(each / t.stride, (int)(8 * (uint32_t)a.N / (uint32_t)a.K)));
    t.part = share / t.stride, t.first_token = share - t.part * t.stride;
    if (t.part >= t.parts) t.count = 0;
    return t;
}

__device__ __forceinline__ uint4 ldg16(const uint16_t *p) { return __ldg(reinterpret_cast<const uint4 *>(p)); }

// The sums of tokens m0 .. m0 + 15 over this CTA's K chunk into red[0] (its warps' added), whole CTA.  U: steps of 32 k whose
// loads are in flight.
template <int NT, int U, int W>
__device__ __forceinline__ void inner_sums(const LoraArgs &a, const Tile &tile, const int *list, int m0, float (*red)[16][NT * 8 + 1]) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
    const int k_end = (int)min((int64_t)(blockIdx.x + 1) * a.k_chunk, a.K);
    const uint16_t *rows = a.a + (int64_t)tile.adapter * a.R * a.K;
    const uint16_t *x0 = m0 + g < tile.count ? a.x + list[m0 + g] * a.ldx : nullptr;
    const uint16_t *x1 = m0 + g + 8 < tile.count ? a.x + list[m0 + g + 8] * a.ldx : nullptr;
    float acc[NT][4] = {};
    for (int k = blockIdx.x * a.k_chunk + 32 * warp + 8 * tq; k - 8 * tq < k_end; k += 32 * W * U) {
        uint4 xa[U], xb[U], w[U][NT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = k + 32 * W * u;
            const bool in = at < k_end;
            const uint4 zero = make_uint4(0, 0, 0, 0);
            xa[u] = in && x0 ? ldg16(x0 + at) : zero;
            xb[u] = in && x1 ? ldg16(x1 + at) : zero;
#pragma unroll
            for (int n = 0; n < NT; ++n) w[u][n] = in && 8 * n + g < tile.rank ? ldg16(rows + (int64_t)(8 * n + g) * a.K + at) : zero;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t lo[4] = {xa[u].x, xb[u].x, xa[u].y, xb[u].y}, hi[4] = {xa[u].z, xb[u].z, xa[u].w, xb[u].w};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma_bf16_16816(acc[n], lo, w[u][n].x, w[u][n].y, acc[n]);
                mma_bf16_16816(acc[n], hi, w[u][n].z, w[u][n].w, acc[n]);
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        red[warp][g][8 * n + 2 * tq] = acc[n][0], red[warp][g][8 * n + 2 * tq + 1] = acc[n][1];
        red[warp][g + 8][8 * n + 2 * tq] = acc[n][2], red[warp][g + 8][8 * n + 2 * tq + 1] = acc[n][3];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * a.R; i += W * 32) {
        const int row = i / a.R, r = i - row * a.R;
        float s = red[0][row][r];
#pragma unroll
        for (int w = 1; w < W; ++w) s += red[w][row][r];
        red[0][row][r] = s;
    }
}

// What the CTAs of the cluster have in `mine`, added in their order.
__device__ __forceinline__ float cluster_total(const float *mine) {
    float s = 0.f;
    for (uint32_t c = 0; c < gridDim.x; ++c) s += ld_shared_cluster_f32(map_shared_rank(smem_u32(mine), c));
    return s;
}

template <int NT, int U, int W>
__global__ void __launch_bounds__(W * 32) shrink_kernel(const LoraArgs a) {
    pdl_wait();
    pdl_trigger();
    __shared__ int list[kTileTokens];
    __shared__ float red[W][16][NT * 8 + 1];
    const int64_t cta = ((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
    for (int64_t t = cta * (W * 32) + threadIdx.x; t < a.T; t += (int64_t)gridDim.x * gridDim.y * gridDim.z * (W * 32))
        if (__ldg(a.ids + t) >= a.n_adapters) atomicOr(a.status, kDevIndex);
    const Tile tile = tile_of<W * 32>(a, blockIdx.y, list);
    const float scale = a.scales && tile.count > 0 ? __ldg(a.scales + tile.adapter) : 1.f;
    // (the CTAs of a cluster have the same tile and tokens)
    for (int m0 = 16 * blockIdx.z; m0 < tile.count; m0 += 16 * gridDim.z) {
        inner_sums<NT, U, W>(a, tile, list, m0, red);
        if (gridDim.x > 1) cluster_sync();
        else __syncthreads();
        for (int i = threadIdx.x; i < 16 * a.R; i += W * 32) {
            const int row = i / a.R, r = i - row * a.R;
            if (row % gridDim.x != blockIdx.x || m0 + row >= tile.count) continue;
            const float s = gridDim.x > 1 ? cluster_total(&red[0][row][r]) : red[0][row][r];
            a.v[(int64_t)list[m0 + row] * a.R + r] = r < tile.rank ? s * scale : 0.f;
        }
        if (gridDim.x > 1) cluster_sync();  // the others have read this CTA's sums
        else __syncthreads();
    }
}

// v as three values of bf16's 8 significant bits, exactly (what is not finite stays in the first)
__device__ __forceinline__ void split3(float v, uint32_t (&piece)[3]) {
    const uint32_t bits = __float_as_uint(v);
    if ((bits & 0x7F800000u) == 0x7F800000u) {
        piece[0] = (bits & 0x007FFFFFu) ? 0x7FC0u : bits >> 16;
        piece[1] = piece[2] = 0;
        return;
    }
    piece[0] = bits >> 16;
    const float r = v - __uint_as_float(bits & 0xFFFF0000u);
    piece[1] = __float_as_uint(r) >> 16;
    piece[2] = __float_as_uint(r - __uint_as_float(__float_as_uint(r) & 0xFFFF0000u)) >> 16;
}

// KS steps of the first operand from 16 tokens' inner values: lane's rows g and g + 8 (null: no token), from value 4 tq on;
// values beyond the rank are 0, those beyond R are not there.
template <int KS>
__device__ __forceinline__ void split_rows(const float4 (&t)[KS][2], uint32_t (&frag)[KS][3][4]) {
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t p0[3], p1[3], p2[3], p3[3];
            split3(t[s][h].x, p0), split3(t[s][h].y, p1), split3(t[s][h].z, p2), split3(t[s][h].w, p3);
#pragma unroll
            for (int k = 0; k < 3; ++k) frag[s][k][h] = p0[k] | p1[k] << 16, frag[s][k][2 + h] = p2[k] | p3[k] << 16;
        }
}

// A lane's part of B's rows: inner values 16 s + 4 tq .. + 3, what lies beyond the rank taken out.  In a group of 16 columns,
// column 2 j + e of MMA tile i is the group's column 4 j + 2 i + e.
template <int KS>
struct Columns {
    const uint16_t *row;  // the lane's first column of group 0
    int64_t left;         // columns from there on
    int in;               // steps of which something lies within the rank
    uint32_t mask[KS][2];
    __device__ __forceinline__ Columns(const LoraArgs &a, const Tile &tile) {
        const int lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3, first = 4 * (g >> 1) + (g & 1);
        row = a.b + ((int64_t)tile.adapter * a.N + first) * a.R + 4 * tq;
        left = a.N - first;
        in = (tile.rank - 4 * tq + 15) >> 4;  // (not positive: none)
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int n = tile.rank - (16 * s + 4 * tq);
            mask[s][0] = n >= 2 ? 0xFFFFFFFFu : n == 1 ? 0x0000FFFFu : 0u;
            mask[s][1] = n >= 4 ? 0xFFFFFFFFu : n == 3 ? 0x0000FFFFu : 0u;
        }
    }
    // the group that begins at column n (none: n beyond N)
    __device__ __forceinline__ void load(int R, int64_t n, uint32_t (&b)[2][KS][2]) const {
        const uint16_t *p = row + n * R;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const uint2 w = n + 2 * i < left && s < in ? __ldg(reinterpret_cast<const uint2 *>(p + 2 * i * R + 16 * s)) : make_uint2(0, 0);
                b[i][s][0] = w.x, b[i][s][1] = w.y;
            }
    }
    // (is any of the lane's values not finite?  0 times it is no number)
    __device__ __forceinline__ bool cut(uint32_t (&b)[2][KS][2]) const {
        uint32_t sum = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    b[i][s][x] &= mask[s][x];
                    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"(b[i][s][x]), "r"(0u));
                }
        return (sum & 0x7FFF7FFFu) != 0;
    }
    // in place of each such value 1 with its sign: what it adds has the sign of what the value itself adds later (an infinite inner
    // value times 0 would be no number)
    __device__ __forceinline__ void finite_only(uint32_t (&b)[2][KS][2]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint32_t &p = b[i][s][x];
                    if ((p & 0x7F80u) == 0x7F80u) p = (p & 0xFFFF8000u) | 0x3F80u;
                    if ((p & 0x7F800000u) == 0x7F800000u) p = (p & 0x8000FFFFu) | 0x3F800000u;
                }
    }
};
// Four values of a row of y from column n on (row null: none)
template <bool VEC>
__device__ __forceinline__ float4 load_y(const LoraArgs &a, const float *row, int64_t n) {
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    const int64_t left = row ? a.N - n : 0;
    if (VEC) {
        if (left > 0) y = *reinterpret_cast<const float4 *>(row + n);
    } else {
        if (left > 0) y.x = row[n];
        if (left > 1) y.y = row[n + 1];
        if (left > 2) y.z = row[n + 2];
        if (left > 3) y.w = row[n + 3];
    }
    return y;
}
template <bool VEC>
__device__ __forceinline__ void store_y(const LoraArgs &a, float *row, int64_t n, float4 y) {
    const int64_t left = row ? a.N - n : 0;
    if (VEC) {
        if (left > 0) *reinterpret_cast<float4 *>(row + n) = y;
    } else {
        if (left > 0) row[n] = y.x;
        if (left > 1) row[n + 1] = y.y;
        if (left > 2) row[n + 2] = y.z;
        if (left > 3) row[n + 3] = y.w;
    }
}
// acc += the group's products with step s of the tokens, the smallest pieces first
template <int KS>
__device__ __forceinline__ void multiply(float (&acc)[2][4], const uint32_t (&frag)[3][4], const uint32_t (&b)[2][KS][2], int s) {
#pragma unroll
    for (int k = 2; k >= 0; --k)
#pragma unroll
        for (int i = 0; i < 2; ++i) mma_bf16_16816(acc[i], frag[k], b[i][s][0], b[i][s][1], acc[i]);
}
// Values of B that are not finite are no part of the product: a piece of an inner value may be 0 where the value is not, and 0 *
// infinity is no number.  What they add to columns n .. n + columns - 1 of rows list[begin .. end - 1], whose inner values v() gives,
// by the warp that adds the product to them.
template <typename V>
__device__ __forceinline__ void add_infinite(const LoraArgs &a, const Tile &tile, int64_t n, int columns, const int *list, int begin, int end, V &&v) {
    __syncwarp();
#pragma unroll 1
    for (int i = threadIdx.x & 31; i < columns && n + i < a.N; i += 32) {
        const uint16_t *b = a.b + ((int64_t)tile.adapter * a.N + n + i) * a.R;
#pragma unroll 1
        for (int r = 0; r < tile.rank; ++r) {
            const float x = __uint_as_float((uint32_t)__ldg(b + r) << 16);
            if (isfinite(x)) continue;
#pragma unroll 1
            for (int m = begin; m < end; ++m) a.y[list[m] * a.ldy + n + i] += x * v(m, r);
        }
    }
    __syncwarp();
}
__device__ __forceinline__ float4 plus(float4 y, const float (&acc)[2][4], int h) {
    return make_float4(y.x + acc[0][2 * h], y.y + acc[0][2 * h + 1], y.z + acc[1][2 * h], y.w + acc[1][2 * h + 1]);
}

// KS: MMA steps over the inner values (R / 16, or the next power of two); CG: groups of 16 columns a warp
template <int KS, int CG, bool VEC>
__global__ void __launch_bounds__(kThreads) expand_kernel(const LoraArgs a) {
    __shared__ int list[kTileTokens];
    // before the previous kernel has ended: what it does not write (it has itself waited for the writer of y and of the list)
    const Tile tile = tile_of<kThreads>(a, blockIdx.y, list);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
    const int64_t n0 = ((int64_t)blockIdx.x * kWarps + warp) * (16 * CG);
    // this CTA's tokens of the tile
    const int some = kTileTokens / gridDim.z, begin = some * blockIdx.z, end = min(begin + some, tile.count);
    if (begin >= end) {
        pdl_wait();
        return;
    }
    const Columns<KS> columns(a, tile);
    uint32_t b[CG][2][KS][2];
#pragma unroll
    for (int c = 0; c < CG; ++c) columns.load(a.R, n0 + 16 * c, b[c]);
    // y's values of rows m0 + g and m0 + g + 8 on their way
    struct Rows {
        float *at[2];
        float4 y[CG][2];
    };
    auto load = [&](int m0, Rows &r) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            r.at[h] = m0 + g + 8 * h < end ? a.y + list[m0 + g + 8 * h] * a.ldy : nullptr;
#pragma unroll
            for (int c = 0; c < CG; ++c) r.y[c][h] = load_y<VEC>(a, r.at[h], n0 + 16 * c + 4 * tq);
        }
    };
    // one step of 16 tokens' inner values, from value 16 s + 4 tq on
    auto load_v = [&](int m0, int s, float4 (&t)[1][2]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float *v = m0 + g + 8 * h < end ? a.v + (int64_t)list[m0 + g + 8 * h] * a.R + 4 * tq : nullptr;
            t[0][h] = v && 16 * s + 4 * tq < a.R ? __ldcg(reinterpret_cast<const float4 *>(v + 16 * s)) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    auto store = [&](const Rows &r, const float (&acc)[CG][2][4]) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < CG; ++c) store_y<VEC>(a, r.at[h], n0 + 16 * c + 4 * tq, plus(r.y[c][h], acc[c], h));
    };
    // two sets in turn (copied from one to the other they would be waited for)
    Rows even, odd;
    load(begin, even);
    pdl_wait();
    pdl_trigger();
    // values of B that are not finite: what they add comes first, then the products without them
    auto cut = [&] {
        bool infinite = false;
#pragma unroll
        for (int c = 0; c < CG; ++c) infinite |= columns.cut(b[c]);
        if (!__any_sync(0xFFFFFFFFu, infinite)) return;
#pragma unroll
        for (int c = 0; c < CG; ++c) columns.finite_only(b[c]);
        add_infinite(a, tile, n0, 16 * CG, list, begin, end, [&](int m, int r) { return __ldcg(a.v + (int64_t)list[m] * a.R + r); });
        load(begin, even);
        if (KS == 1 && begin + 16 < end) load(begin + 16, odd);
    };
    if constexpr (KS == 1) {
        auto finish = [&](const float4 (&t)[1][2], const Rows &r) {
            float acc[CG][2][4] = {};
            uint32_t frag[1][3][4];
            split_rows<1>(t, frag);
#pragma unroll
            for (int c = 0; c < CG; ++c) multiply<KS>(acc[c], frag[0], b[c], 0);
            store(r, acc);
        };
        auto rest = [&](int m0, const Rows &r) {
            float4 t[1][2];
            load_v(m0, 0, t);
            finish(t, r);
        };
        {
            float4 t[1][2];
            if (begin + 16 < end) load(begin + 16, odd);
            load_v(begin, 0, t);
            cut();
            finish(t, even);
        }
        for (int m0 = begin + 16; m0 < end; m0 += 32) {
            if (m0 + 16 < end) load(m0 + 16, even);
            rest(m0, odd);
            if (m0 + 16 >= end) break;
            if (m0 + 32 < end) load(m0 + 32, odd);
            rest(m0 + 16, even);
        }
    } else {
        // higher ranks: the warps split the 16 tokens' inner values once for all of them, a step or more each, one group ahead
        __shared__ __align__(16) uint4 pieces[2][KS][3][32];
        constexpr int OWN = (KS + kWarps - 1) / kWarps;
        float4 t[OWN][1][2];
        auto fetch = [&](int m0) {
#pragma unroll
            for (int o = 0; o < OWN; ++o)
                if (kWarps * o + warp < KS) load_v(m0, kWarps * o + warp, t[o]);
        };
        auto split = [&](int buf) {
#pragma unroll
            for (int o = 0; o < OWN; ++o) {
                uint32_t frag[1][3][4];
                split_rows<1>(t[o], frag);
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    if (kWarps * o + warp < KS)
                        pieces[buf][kWarps * o + warp][k][lane] = make_uint4(frag[0][k][0], frag[0][k][1], frag[0][k][2], frag[0][k][3]);
            }
        };
        auto finish = [&](int buf, const Rows &r) {
            float acc[CG][2][4] = {};
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                uint32_t frag[3][4];
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    const uint4 f = pieces[buf][s][k][lane];
                    frag[k][0] = f.x, frag[k][1] = f.y, frag[k][2] = f.z, frag[k][3] = f.w;
                }
#pragma unroll
                for (int c = 0; c < CG; ++c) multiply<KS>(acc[c], frag, b[c], s);
            }
            store(r, acc);
        };
        fetch(begin);
        cut();
        split(0);
        __syncthreads();
        for (int m0 = begin; m0 < end; m0 += 32) {
            if (m0 + 16 < end) load(m0 + 16, odd), fetch(m0 + 16);
            finish(0, even);
            if (m0 + 16 >= end) break;
            split(1);
            __syncthreads();
            if (m0 + 32 < end) load(m0 + 32, even), fetch(m0 + 32);
            finish(1, odd);
            if (m0 + 32 < end) split(0);
            __syncthreads();
        }
    }
}

// Both products of a tile by one cluster: K and the columns are dealt to its CTAs.  G: groups of 16 columns on their way at once.
template <int NT, int U, int W, int G, bool VEC>
__global__ void __launch_bounds__(W * 32, NT <= 4 ? 2 : 1) tile_kernel(const LoraArgs a) {
    constexpr int KS = NT == 1 ? 1 : NT / 2;
    __shared__ int list[kTileTokens];
    __shared__ uint32_t masks[2][W];
    extern __shared__ float red_smem[];
    int *const first_at = reinterpret_cast<int *>(red_smem);
    for (int i = threadIdx.x; i < a.n_adapters; i += W * 32) first_at[i] = kLoraSmall;
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    float (*const red)[16][NT * 8 + 1] = reinterpret_cast<float (*)[16][NT * 8 + 1]>(red_smem);  // [W]
    __shared__ __align__(16) float v[16][KS * 16 + 4];
    const Small tile = small_tile<W * 32>(a, list, masks, first_at);
    if (tile.count == 0) return;  // (so does the whole cluster)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
    const float scale = a.scales ? __ldg(a.scales + tile.adapter) : 1.f;
    // this CTA's columns, whole groups
    const int ctas = kMaxCluster * tile.parts, per = ((uint32_t)(a.N + ctas - 1) / (uint32_t)ctas + 15) / 16 * 16;
    const int64_t first = min((int64_t)per * (tile.part * kMaxCluster + blockIdx.x), a.N), last = min(first + per, a.N);
    if (threadIdx.x == 0 && last > first && 4 * tile.rank >= 3 * a.R) {  // (of lower ranks too much would not be read)
        const uint16_t *from = a.b + ((int64_t)tile.adapter * a.N + first) * a.R;
        const int64_t bytes = (last - first) * a.R * 2;
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"((uint32_t)(bytes < (1 << 19) ? bytes : 1 << 19)) : "memory");
    }
    for (int i = threadIdx.x; i < 16 * (KS * 16 + 4); i += W * 32) (&v[0][0])[i] = 0.f;  // (what lies beyond R)
    const Columns<KS> columns(a, tile);
    struct Batch {
        uint32_t b[G][2][KS][2];
        float4 y[G][2];
    };
    for (int m0 = 16 * tile.first_token; m0 < tile.count; m0 += 16 * tile.stride) {
        float *rows[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) rows[h] = m0 + g + 8 * h < tile.count ? a.y + list[m0 + g + 8 * h] * a.ldy : nullptr;
        auto load = [&](int64_t n, Batch &t) {
#pragma unroll
            for (int c = 0; c < G; ++c) {
                const int64_t at = n + 16 * W * c;
                columns.load(a.R, at < last ? at : a.N, t.b[c]);
#pragma unroll
                for (int h = 0; h < 2; ++h) t.y[c][h] = load_y<VEC>(a, at < last ? rows[h] : nullptr, at + 4 * tq);
            }
        };
        // (the first columns are on their way during the first product, the next ones always)
        Batch even, odd;
        load(first + 16 * warp, even);
        inner_sums<NT, U, W>(a, tile, list, m0, red);
        cluster_sync();
        // each CTA adds up some of the tokens' sums, for all
        for (int i = threadIdx.x; i < 16 * a.R; i += W * 32) {
            const int row = i / a.R, r = i - row * a.R;
            if (row % kMaxCluster != blockIdx.x) continue;
            float part[kMaxCluster], s = 0.f;
#pragma unroll
            for (int c = 0; c < kMaxCluster; ++c) part[c] = ld_shared_cluster_f32(map_shared_rank(smem_u32(&red[0][row][r]), c));
#pragma unroll
            for (int c = 0; c < kMaxCluster; ++c) s += part[c];
            s = r < tile.rank ? s * scale : 0.f;
#pragma unroll
            for (int c = 0; c < kMaxCluster; ++c) st_shared_cluster_f32(map_shared_rank(smem_u32(&v[row][r]), c), s);
        }
        cluster_sync();
        float4 t[KS][2];
        uint32_t frag[KS][3][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int s = 0; s < KS; ++s) t[s][h] = *reinterpret_cast<const float4 *>(&v[g + 8 * h][16 * s + 4 * tq]);
        split_rows<KS>(t, frag);
        auto finish = [&](int64_t n, Batch &t) {
#pragma unroll
            for (int c = 0; c < G; ++c) {
                const int64_t at = n + 16 * W * c;
                const bool infinite = __any_sync(0xFFFFFFFFu, columns.cut(t.b[c]));
                if (infinite) columns.finite_only(t.b[c]);
                float acc[2][4] = {};
#pragma unroll
                for (int s = 0; s < KS; ++s) multiply<KS>(acc, frag[s], t.b[c], s);
#pragma unroll
                for (int h = 0; h < 2; ++h) store_y<VEC>(a, at < last ? rows[h] : nullptr, at + 4 * tq, plus(t.y[c][h], acc, h));
                if (infinite) add_infinite(a, tile, at, 16, list, m0, min(m0 + 16, tile.count), [&](int m, int r) { return v[m - m0][r]; });
            }
        };
        constexpr int64_t STEP = 16 * W * G;
        for (int64_t n = first + 16 * warp; n < last; n += 2 * STEP) {
            if (n + STEP < last) load(n + STEP, odd);
            finish(n, even);
            if (n + STEP >= last) break;
            if (n + 2 * STEP < last) load(n + 2 * STEP, even);
            finish(n + STEP, odd);
        }
        // (v is written again only behind the next cluster barrier, which every warp reaches after it has read v)
    }
}

template <int KS, int CG>
cudaError_t launch_expand(const DeviceInfo &di, const LoraArgs &a, bool vec, unsigned tiles, cudaStream_t s) {
    // (a tile's tokens over 2, 3 or 4 CTAs where that fills four an SM)
    const int64_t columns = kWarps * 16 * CG, x = (a.N + columns - 1) / columns, z = 4 * di.sm_count / (x * (a.T / kTileTokens + 1));
    return launch_pdl(vec ? expand_kernel<KS, CG, true> : expand_kernel<KS, CG, false>,
                      dim3((unsigned)x, tiles, z < 1 ? 1 : z < 4 ? (unsigned)z : 4), dim3(kThreads), 0, s, dim3(1), a);
}

// K over `splits` CTAs, in whole steps of a CTA's warps; returns how many have something to do
unsigned split_k(LoraArgs &a, int64_t splits, int64_t unit) {
    if (splits > kMaxCluster) splits = kMaxCluster;
    if (splits > (a.K + unit - 1) / unit) splits = (a.K + unit - 1) / unit;
    a.k_chunk = (int32_t)(((a.K + splits - 1) / splits + unit - 1) / unit * unit);
    return (unsigned)((a.K + a.k_chunk - 1) / a.k_chunk);
}

template <int NT, int U, int W>
cudaError_t launch_shrink(const DeviceInfo &di, LoraArgs &a, unsigned tiles, cudaStream_t s) {
    // 16 tokens a CTA (the tokens of a tile over several); K over as many CTAs as an SM holds of them, each with a full round of
    // loads at least (1028 tokens, 17408 -> 515, rank 8: 30 us, 48 by two; 955 tokens, 2048 -> 5120, rank 64: 29 us, 37 by eight)
    const int64_t ctas = (NT <= 2 ? 4 : 2) * di.sm_count;
    const unsigned z = kTileTokens / 16;
    const int64_t groups = a.T / 16 + (a.n_adapters < a.T ? a.n_adapters : a.T);  // of 16 tokens, at most
    int64_t splits = ctas / groups, most = a.K / (32 * W * U);
    if (splits > most) splits = most;
    const unsigned n = split_k(a, splits > 1 ? splits : 1, 32 * W);
    return launch_pdl(shrink_kernel<NT, U, W>, dim3(n, tiles, z), dim3(W * 32), 0, s, dim3(n), a);
}

// Clusters of tile_kernel that the device holds at a time, asked once for each kernel and device (1, and asked again, if that fails).
template <int NT, int U, int W, int G, bool VEC>
unsigned resident_clusters(int device, int smem) {
    constexpr int kDevices = 64;
    static std::atomic<unsigned> kept[kDevices];
    std::atomic<unsigned> *const at = device < kDevices ? &kept[device] : nullptr;
    if (at && *at) return *at;
    cudaLaunchAttribute of[1] = {};
    of[0].id = cudaLaunchAttributeClusterDimension;
    of[0].val.clusterDim = {kMaxCluster, 1, 1};
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(kMaxCluster), c.blockDim = dim3(W * 32), c.dynamicSmemBytes = smem, c.attrs = of, c.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, tile_kernel<NT, U, W, G, VEC>, &c) != cudaSuccess) (void)cudaGetLastError();
    if (n < 1) return 1u;
    if (at) *at = (unsigned)n;
    return (unsigned)n;
}

template <int NT, int U, int W, int G, bool VEC>
cudaError_t launch_tile(const DeviceInfo &di, const LoraArgs &a, unsigned tiles, cudaStream_t s) {
    constexpr int smem = W * 16 * (NT * 8 + 1) * 4;  // (the adapters' first tokens lie there first: 4 bytes for each of 1024)
    static_assert(smem >= 4 * 1024, "fits");
    auto kern = tile_kernel<NT, U, W, G, VEC>;
    const cudaError_t e = smem > 32 * 1024 ? ensure_smem((const void *)kern, smem) : cudaSuccess;
    if (e != cudaSuccess) return e;
    // clusters: one an adapter (a token, if there are fewer), and as many as the GPU holds, where few adapters can share them
    const unsigned resident = resident_clusters<NT, U, W, G, VEC>(di.device, smem), clusters = tiles > resident ? tiles : resident;
    return launch_pdl(kern, dim3(kMaxCluster, clusters), dim3(W * 32), smem, s, dim3(kMaxCluster), a);
}
template <int NT, int U, int W, int G>
cudaError_t launch_tile(const DeviceInfo &di, LoraArgs &a, bool vec, unsigned tiles, cudaStream_t s) {
    a.k_chunk = (int32_t)(((a.K + kMaxCluster - 1) / kMaxCluster + 31) / 32 * 32);
    return vec ? launch_tile<NT, U, W, G, true>(di, a, tiles, s) : launch_tile<NT, U, W, G, false>(di, a, tiles, s);
}

}  // namespace

cudaError_t launch_lora_add(const DeviceInfo &di, LoraArgs &a, cudaStream_t s) {
    const bool vec = (reinterpret_cast<uintptr_t>(a.y) & 15) == 0 && a.ldy % 4 == 0 && a.N % 4 == 0;
    if (!a.tiles) {
        const unsigned tiles = (unsigned)(a.n_adapters < a.T ? a.n_adapters : a.T);
        return a.R <= 8 ? launch_tile<1, 4, 8, 2>(di, a, vec, tiles, s) : a.R <= 16 ? launch_tile<2, 4, 8, 2>(di, a, vec, tiles, s)
             : a.R <= 32 ? launch_tile<4, 2, 8, 1>(di, a, vec, tiles, s) : a.R <= 64 ? launch_tile<8, 2, 8, 2>(di, a, vec, tiles, s)
                         : launch_tile<16, 1, 8, 1>(di, a, vec, tiles, s);
    }
    cudaError_t e = launch_moe_route(a.ids, a.T, a.n_adapters, a.offsets, a.perm, false, a.tiles, a.n_tiles, s);
    if (e != cudaSuccess) return e;
    const unsigned tiles = (unsigned)moe_max_tiles(a.n_adapters, a.T);
    e = a.R <= 8 ? launch_shrink<1, 4, 8>(di, a, tiles, s) : a.R <= 16 ? launch_shrink<2, 2, 8>(di, a, tiles, s)
      : a.R <= 32 ? launch_shrink<4, 2, 8>(di, a, tiles, s) : a.R <= 64 ? launch_shrink<8, 2, 8>(di, a, tiles, s)
                  : launch_shrink<16, 1, 4>(di, a, tiles, s);
    if (e != cudaSuccess) return e;
    return a.R <= 16 ? launch_expand<1, 2>(di, a, vec, tiles, s) : a.R <= 32 ? launch_expand<2, 3>(di, a, vec, tiles, s)
         : a.R <= 64 ? launch_expand<4, 2>(di, a, vec, tiles, s) : launch_expand<8, 3>(di, a, vec, tiles, s);
}

}  // namespace q4k
