// Low-rank adapters of many requests beside a shared projection:
//     y[t] += c_a B_a (A_a x[t]),  a = ids[t].
//
// Two products over the tokens of one adapter at a time (a tile: an adapter and at most 192 of its tokens), the
// inner sums v[t] = A_a x[t] between them in the workspace:
//   shrink   v: m16n8k16 MMAs, 16 tokens by R, the K axis split over CTAs (few tiles must fill the GPU) and over the
//            warps of a CTA.  Any pairing of k positions gives the same sum, so a lane's eight consecutive values of a
//            row are its share of two MMA steps: operands come straight from global memory, 16 bytes at a time.
//   expand   y: adds up the K parts in their order, multiplies by the adapter's scale, and splits the fp32 value into
//            three bf16 pieces of 8 significant bits each (exact), so that the second product has exact products, too.
//            Columns are dealt to MMA tiles so that a lane owns four consecutive ones: y is read and written 16 bytes
//            at a time, the reads on their way before the inner sums are there.
// Up to 192 tokens find their tile themselves: the CTA of a token that is its adapter's first gathers the
// others.  More are sorted by adapter first (the experts' counting sort).
// Bound by HBM: of many tokens by y, read and written once, of few by the adapters' matrices and by latency.
#include <cuda_runtime.h>

#include "decode_ops.h"
#include "q4k_ptx.cuh"

namespace q4k {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kTileTokens = kMoeTileItems;
static_assert(kLoraSmall <= kTileTokens, "the tokens of a small call fit in one tile");

struct Tile {
    int adapter, count, rank;
};

// The tile of CTA row `k`, its tokens in list[]; count 0: nothing to do.  Every thread calls it.
__device__ __forceinline__ Tile tile_of(const LoraArgs &a, int k, int *list, uint32_t *masks) {
    Tile t = {-1, 0, 0};
    if (a.tiles) {
        if (k >= __ldg(a.n_tiles)) return t;
        const int4 r = __ldg(a.tiles + k);
        t.adapter = r.x, t.count = r.z;
        for (int i = threadIdx.x; i < r.z; i += kThreads) list[i] = __ldg(a.perm + r.y + i);
        __syncthreads();
    } else {
        const int id = __ldg(a.ids + k), warp = threadIdx.x >> 5;
        if (id < 0) return t;
        if (id >= a.n_adapters) {
            if (threadIdx.x == 0) atomicOr(a.status, kDevIndex);
            return t;
        }
        bool mine[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int at = i * kThreads + threadIdx.x;
            mine[i] = at < a.T && __ldg(a.ids + at) == id;
            const uint32_t m = __ballot_sync(0xFFFFFFFFu, mine[i]);
            if ((threadIdx.x & 31) == 0) masks[i * kWarps + warp] = m;
        }
        __syncthreads();
        int first = -1, before[2] = {0, 0};
#pragma unroll
        for (int w = 0; w < 2 * kWarps; ++w) {
            if (first < 0 && masks[w]) first = 32 * w + __ffs(masks[w]) - 1;
            if (w < warp) before[0] += __popc(masks[w]);
            if (w < kWarps + warp) before[1] += __popc(masks[w]);
            t.count += __popc(masks[w]);
        }
        if (first != k) {
            t.count = 0;
            return t;
        }
        t.adapter = id;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (mine[i])
                list[before[i] + __popc(masks[i * kWarps + warp] & ((1u << (threadIdx.x & 31)) - 1u))] = i * kThreads + threadIdx.x;
        __syncthreads();
    }
    t.rank = a.ranks ? min(max(__ldg(a.ranks + t.adapter), 0), a.R) : a.R;
    return t;
}

__device__ __forceinline__ uint4 ldg16(const uint16_t *p) { return __ldg(reinterpret_cast<const uint4 *>(p)); }

// NT: groups of eight inner values (R / 8, or the next power of two); U: steps of 32 k whose loads are in flight
template <int NT, int U>
__global__ void __launch_bounds__(kThreads) shrink_kernel(const LoraArgs a) {
    pdl_wait();
    pdl_trigger();
    __shared__ int list[kTileTokens];
    __shared__ uint32_t masks[2 * kWarps];
    __shared__ float red[kWarps][16][NT * 8 + 1];
    if (a.tiles) {  // (a small call's CTAs see the ids themselves)
        const int64_t cta = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
        for (int64_t t = cta * kThreads + threadIdx.x; t < a.T; t += (int64_t)gridDim.x * gridDim.y * kThreads)
            if (__ldg(a.ids + t) >= a.n_adapters) atomicOr(a.status, kDevIndex);
    }
    const Tile tile = tile_of(a, blockIdx.y, list, masks);
    if (tile.count == 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
    const int k_end = (int)min((int64_t)(blockIdx.x + 1) * a.k_chunk, a.K);
    const uint16_t *rows = a.a + (int64_t)tile.adapter * a.R * a.K;
    for (int m0 = 0; m0 < tile.count; m0 += 16) {
        const uint16_t *x0 = m0 + g < tile.count ? a.x + list[m0 + g] * a.ldx : nullptr;
        const uint16_t *x1 = m0 + g + 8 < tile.count ? a.x + list[m0 + g + 8] * a.ldx : nullptr;
        float acc[NT][4] = {};
        for (int k = blockIdx.x * a.k_chunk + 32 * warp + 8 * tq; k - 8 * tq < k_end; k += 32 * kWarps * U) {
            uint4 xa[U], xb[U], w[U][NT];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int at = k + 32 * kWarps * u;
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
        for (int i = threadIdx.x; i < 16 * a.R; i += kThreads) {
            const int row = i / a.R, r = i - row * a.R;
            if (m0 + row < tile.count)
                a.part[((int64_t)blockIdx.x * a.T + list[m0 + row]) * a.R + r] =
                    (red[0][row][r] + red[1][row][r]) + (red[2][row][r] + red[3][row][r]);
        }
        __syncthreads();
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

// KS: MMA steps over the inner values (R / 16, or the next power of two); CG: groups of 16 columns a warp
template <int KS, int CG, bool VEC>
__global__ void __launch_bounds__(kThreads) expand_kernel(const LoraArgs a) {
    __shared__ int list[kTileTokens];
    __shared__ uint32_t masks[2 * kWarps];
    __shared__ __align__(16) float v[16][KS * 16 + 4];
    // before the previous kernel has ended: what it does not write (it has itself waited for the writer of y and of the list)
    const Tile tile = tile_of(a, blockIdx.y, list, masks);
    if (tile.count == 0) {
        pdl_wait();
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
    const int64_t n0 = ((int64_t)blockIdx.x * kWarps + warp) * (16 * CG) + 4 * tq;
    const float scale = a.scales ? __ldg(a.scales + tile.adapter) : 1.f;
    // B: column 2 j + e of MMA tile i of a group is the group's column 4 j + 2 i + e; inner values 16 s + 4 tq .. + 3
    uint32_t b[CG][2][KS][2];
#pragma unroll
    for (int c = 0; c < CG; ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t n = n0 - 4 * tq + 16 * c + 4 * (g >> 1) + 2 * i + (g & 1);
            const uint16_t *row = a.b + ((int64_t)tile.adapter * a.N + n) * a.R + 4 * tq;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const int left = tile.rank - (16 * s + 4 * tq);  // values within the rank
                uint2 w = n < a.N && left > 0 ? __ldg(reinterpret_cast<const uint2 *>(row + 16 * s)) : make_uint2(0, 0);
                if (left < 4) w.y &= left == 3 ? 0x0000FFFFu : 0u;
                if (left < 2) w.x &= 0x0000FFFFu;
                b[c][i][s][0] = w.x, b[c][i][s][1] = w.y;
            }
        }
    bool waited = false;
    for (int m0 = 0; m0 < tile.count; m0 += 16) {
        // y's values of rows g and g + 8
        float4 y[CG][2];
        float *rows[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            rows[h] = m0 + g + 8 * h < tile.count ? a.y + list[m0 + g + 8 * h] * a.ldy + n0 : nullptr;
#pragma unroll
            for (int c = 0; c < CG; ++c) {
                y[c][h] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (rows[h]) {
                    const int64_t left = a.N - (n0 + 16 * c);
                    const float *p = rows[h] + 16 * c;
                    if (VEC) {
                        if (left > 0) y[c][h] = *reinterpret_cast<const float4 *>(p);
                    } else {
                        if (left > 0) y[c][h].x = p[0];
                        if (left > 1) y[c][h].y = p[1];
                        if (left > 2) y[c][h].z = p[2];
                        if (left > 3) y[c][h].w = p[3];
                    }
                }
            }
        }
        if (!waited) {
            pdl_wait();
            pdl_trigger();
        }
        waited = true;
        for (int i = threadIdx.x; i < 16 * KS * 16; i += kThreads) {
            const int row = i / (KS * 16), r = i % (KS * 16);
            float sum = 0.f;
            if (m0 + row < tile.count && r < tile.rank) {
                const float *p = a.part + (int64_t)list[m0 + row] * a.R + r;
                for (int s = 0; s < a.splits; ++s) sum += __ldcg(p + (int64_t)s * a.T * a.R);
            }
            v[row][r] = sum * scale;
        }
        __syncthreads();
        float acc[CG][2][4] = {};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            uint32_t frag[3][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4 t = *reinterpret_cast<const float4 *>(&v[g + 8 * h][16 * s + 4 * tq]);
                uint32_t p0[3], p1[3], p2[3], p3[3];
                split3(t.x, p0), split3(t.y, p1), split3(t.z, p2), split3(t.w, p3);
#pragma unroll
                for (int k = 0; k < 3; ++k) frag[k][h] = p0[k] | p1[k] << 16, frag[k][2 + h] = p2[k] | p3[k] << 16;
            }
#pragma unroll
            for (int k = 2; k >= 0; --k)
#pragma unroll
                for (int c = 0; c < CG; ++c)
#pragma unroll
                    for (int i = 0; i < 2; ++i) mma_bf16_16816(acc[c][i], frag[k], b[c][i][s][0], b[c][i][s][1], acc[c][i]);
        }
        __syncthreads();  // v is free
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (!rows[h]) continue;
#pragma unroll
            for (int c = 0; c < CG; ++c) {
                const int64_t left = a.N - (n0 + 16 * c);
                float *p = rows[h] + 16 * c;
                const float4 t = make_float4(y[c][h].x + acc[c][0][2 * h], y[c][h].y + acc[c][0][2 * h + 1],
                                             y[c][h].z + acc[c][1][2 * h], y[c][h].w + acc[c][1][2 * h + 1]);
                if (VEC) {
                    if (left > 0) *reinterpret_cast<float4 *>(p) = t;
                } else {
                    if (left > 0) p[0] = t.x;
                    if (left > 1) p[1] = t.y;
                    if (left > 2) p[2] = t.z;
                    if (left > 3) p[3] = t.w;
                }
            }
        }
    }
}

template <int KS, int CG>
cudaError_t launch_expand(const LoraArgs &a, bool vec, unsigned tiles, cudaStream_t s) {
    const int64_t columns = kWarps * 16 * CG;
    return launch_pdl(vec ? expand_kernel<KS, CG, true> : expand_kernel<KS, CG, false>,
                      dim3((unsigned)((a.N + columns - 1) / columns), tiles), dim3(kThreads), 0, s, dim3(1), a);
}

}  // namespace

// (of sizes alone: the workspace is laid out by it)
LoraSplit lora_split(int64_t K, int64_t T, int n_adapters) {
    constexpr int kCtas = 4 * 152;  // four an SM, were every tile there
    const int64_t tiles = T <= kLoraSmall ? T : moe_max_tiles(n_adapters, T);
    int64_t splits = (kCtas + tiles - 1) / tiles;
    const int64_t most = (K + 32 * kWarps - 1) / (32 * kWarps);
    if (splits > most) splits = most;
    LoraSplit r;
    const int64_t unit = 32 * kWarps;
    r.k_chunk = ((K + splits - 1) / splits + unit - 1) / unit * unit;
    r.splits = (int)((K + r.k_chunk - 1) / r.k_chunk);
    return r;
}

cudaError_t launch_lora_add(const DeviceInfo &di, const LoraArgs &a, cudaStream_t s) {
    unsigned tiles = (unsigned)a.T;
    if (a.tiles) {
        const cudaError_t e = launch_moe_route(a.ids, a.T, a.n_adapters, a.offsets, a.perm, false, a.tiles, a.n_tiles, s);
        if (e != cudaSuccess) return e;
        tiles = (unsigned)moe_max_tiles(a.n_adapters, a.T);
    }
    auto shrink = a.R <= 8 ? shrink_kernel<1, 4> : a.R <= 16 ? shrink_kernel<2, 4> : a.R <= 32 ? shrink_kernel<4, 2>
                : a.R <= 64 ? shrink_kernel<8, 1> : shrink_kernel<16, 1>;
    const cudaError_t e = launch_pdl(shrink, dim3((unsigned)a.splits, tiles), dim3(kThreads), 0, s, dim3(1), a);
    if (e != cudaSuccess) return e;
    const bool vec = (reinterpret_cast<uintptr_t>(a.y) & 15) == 0 && a.ldy % 4 == 0 && a.N % 4 == 0;
    return a.R <= 16 ? launch_expand<1, 4>(a, vec, tiles, s) : a.R <= 32 ? launch_expand<2, 4>(a, vec, tiles, s)
         : a.R <= 64 ? launch_expand<4, 2>(a, vec, tiles, s) : launch_expand<8, 1>(a, vec, tiles, s);
}

}  // namespace q4k
