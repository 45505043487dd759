// The end of one block and the start of the next in one pass:
//     h = r + scale * gate * post(y),  r' = h,  x = bf16(pre(h))
// post and pre being RMS or layer norms over a row; x may (also) be 8 bits a value, with a scale for each 32.
//
// Bound by HBM for many rows (a row of y and r read, of r' and x written, each once)
// and by latency for few.  A CTA holds a whole row in registers between the two norms,
// up to 16384 values; only longer rows are read again.  A mean is
// taken off before the squares are summed (E[x^2] - E[x]^2 would cancel): within a warp by
// two sums over registers, over the warps by their means and squares, with one barrier.
// Everything is fp32 until the two outputs.
// Measured: 2.9 us for a row of 5120; 36 us for 4096 rows of 5120 (RMS, a gate, 16-bit residual:
// 5.9 TB/s), 41 with two layer norms and biases.  With 8-bit output instead of bf16 40 us (two RMS norms, 16-bit
// residual: 4.8 TB/s), the issue of its arithmetic: 58 with a division a value.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "decode_ops.h"
#include "q4k_ptx.cuh"

namespace q4k {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kNone = 0, kLayer = 2;  // Q4K_NORM_NONE, Q4K_NORM_LAYER

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
// Sum over the CTA with one barrier, in the same order on every call: two scratch arrays in turn.
__device__ __forceinline__ float turn_sum(float v, float2 (*scratch)[32], int &turn) {
    v = warp_sum(v);
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warps == 1) return v;
    if (lane == 0) scratch[turn][warp].x = v;
    __syncthreads();
    v = lane < warps ? scratch[turn][lane].x : 0.f;
    turn ^= 1;
    return warp_sum(v);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// v in 8 bits at the scale s = a / 127, a being the largest |v| of its block (so small that s is 0: 0)
__device__ __forceinline__ int in_eight(float v, float s) {
    return s > 0.f ? (int)copysignf(fminf(rintf(fabsf(v) / s), 127.f), v) : 0;
}
// Four of them as bytes, and s, for a of usual size; false where this may not be the rule's rounding.  s is a times the reciprocal
// of 127, corrected by its remainder (Markstein's division: the nearest value), and v / s is v times the reciprocal of s, off by
// 2^-22 of it, 2^-15 at most: added to 3 * 2^22 it is rounded to a whole number whose low byte lies in the sum's; not to be relied on
// where it lies within 5 10^-5 of the middle between two.  (A division for every value: 57.8 us for 4096 rows of 5120.)
__device__ __forceinline__ bool four_in_eight(const float *v, float a, float &s, uint32_t &word) {
    constexpr float kInv = 1.0f / 127.0f, kMagic = 12582912.0f;
    s = a * kInv;
    s = fmaf(fmaf(-127.0f, s, a), kInv, s);
    const float inv = rcp_approx(s);
    const float2 i2 = make_float2(inv, inv), m2 = make_float2(kMagic, kMagic), none = make_float2(-1.f, -1.f);
    const float2 x = make_float2(v[0], v[1]), y = make_float2(v[2], v[3]);
    const float2 u = fma2(x, i2, m2), w = fma2(y, i2, m2);
    const float2 du = fma2(x, i2, fma2(u, none, m2)), dw = fma2(y, i2, fma2(w, none, m2));
    word = prmt(prmt(__float_as_uint(u.x), __float_as_uint(u.y), 0x0040u), prmt(__float_as_uint(w.x), __float_as_uint(w.y), 0x0040u), 0x5410u);
    return fmaxf(fmaxf(fabsf(du.x), fabsf(du.y)), fmaxf(fabsf(dw.x), fabsf(dw.y))) < 0.49995f && a > 1e-30f && a < 1e38f;
}

// A row of D values over a CTA: thread t holds group i (of NV) of four values, elements
// 4 (i threads + t) .. + 3 (VEC: 16-byte accesses), or i * 4 + x -> (4 i + x) threads + t.
// Values past D are 0; FULL: there are none.
template <int NV, bool VEC, bool FULL = false>
struct Slice {
    int D, tid, threads;
    __device__ __forceinline__ bool in(int i, int x) const { return FULL || at(i, x) < D; }
    __device__ __forceinline__ int at(int i, int x) const { return VEC ? 4 * (i * threads + tid) + x : (4 * i + x) * threads + tid; }
    __device__ __forceinline__ void load(const float *p, float (&v)[4 * NV]) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if constexpr (VEC) {
                const float4 t = in(i, 0) ? __ldg(reinterpret_cast<const float4 *>(p + at(i, 0))) : make_float4(0.f, 0.f, 0.f, 0.f);
                v[4 * i] = t.x, v[4 * i + 1] = t.y, v[4 * i + 2] = t.z, v[4 * i + 3] = t.w;
            } else {
#pragma unroll
                for (int x = 0; x < 4; ++x) v[4 * i + x] = in(i, x) ? __ldg(p + at(i, x)) : 0.f;
            }
        }
    }
    __device__ __forceinline__ void load(const uint16_t *p, float (&v)[4 * NV]) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if constexpr (VEC) {
                const uint2 t = in(i, 0) ? __ldg(reinterpret_cast<const uint2 *>(p + at(i, 0))) : make_uint2(0, 0);
                v[4 * i] = __uint_as_float(t.x << 16), v[4 * i + 1] = __uint_as_float(t.x & 0xFFFF0000u);
                v[4 * i + 2] = __uint_as_float(t.y << 16), v[4 * i + 3] = __uint_as_float(t.y & 0xFFFF0000u);
            } else {
#pragma unroll
                for (int x = 0; x < 4; ++x) v[4 * i + x] = in(i, x) ? __uint_as_float((uint32_t)__ldg(p + at(i, x)) << 16) : 0.f;
            }
        }
    }
    __device__ __forceinline__ void store(float *p, const float (&v)[4 * NV]) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if constexpr (VEC) {
                if (in(i, 0)) *reinterpret_cast<float4 *>(p + at(i, 0)) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            } else {
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    if (in(i, x)) p[at(i, x)] = v[4 * i + x];
            }
        }
    }
    __device__ __forceinline__ void store(uint16_t *p, const float (&v)[4 * NV]) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint2 t = make_uint2(pack_bf16(v[4 * i], v[4 * i + 1]), pack_bf16(v[4 * i + 2], v[4 * i + 3]));
            if constexpr (VEC) {
                if (in(i, 0)) *reinterpret_cast<uint2 *>(p + at(i, 0)) = t;
            } else {
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    if (in(i, x)) p[at(i, x)] = (uint16_t)((x < 2 ? t.x : t.y) >> (x & 1) * 16);
            }
        }
    }
    // 8 bits a value, with a scale for each 32 consecutive ones (D % 32 == 0: a block lies in eight neighbouring threads'
    // groups of four, VEC, or in a warp's single values, and is there as a whole or not at all):
    //     s = max |v| / 127, q = rint(v / s), at most 127 in magnitude (so is an infinity's); 0 for a block of zeros or
    // with a NaN
    __device__ __forceinline__ void store8(int8_t *q, float *scale, const float (&v)[4 * NV]) const {
        // |v| orders like its bits: the largest as whole numbers
        if constexpr (VEC) {
            uint32_t top[NV], word[NV];
            float s[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const uint32_t m01 = max(__float_as_uint(fabsf(v[4 * i])), __float_as_uint(fabsf(v[4 * i + 1])));
                const uint32_t m23 = max(__float_as_uint(fabsf(v[4 * i + 2])), __float_as_uint(fabsf(v[4 * i + 3])));
                top[i] = max(m01, m23);
            }
#pragma unroll
            for (int o = 4; o > 0; o >>= 1)
#pragma unroll
                for (int i = 0; i < NV; ++i) top[i] = max(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], o));
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const float a = __uint_as_float(top[i]);
                if (four_in_eight(v + 4 * i, a, s[i], word[i])) continue;
                s[i] = a / 127.0f;
                word[i] = 0;
#pragma unroll 1
                for (int x = 0; x < 4; ++x)
                    word[i] |= ((uint32_t)in_eight(x == 0 ? v[4 * i] : x == 1 ? v[4 * i + 1] : x == 2 ? v[4 * i + 2] : v[4 * i + 3], s[i]) & 0xFFu) << (8 * x);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!in(i, 0)) continue;
                *reinterpret_cast<uint32_t *>(q + at(i, 0)) = word[i];
                if ((tid & 7) == 0) scale[at(i, 0) / 32] = s[i];
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if constexpr (!VEC) {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float a = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fabsf(v[4 * i + x]))));
                    const float s = a / 127.0f;
                    if (!in(i, x)) continue;
                    q[at(i, x)] = (int8_t)in_eight(v[4 * i + x], s);
                    if ((tid & 31) == 0) scale[at(i, x) / 32] = s;
                }
            }
        }
    }
    // number of the row's values in warp w
    __device__ __forceinline__ float values_of_warp(int w) const {
        int n = 0;
#pragma unroll
        for (int i = 0; i < NV * (VEC ? 1 : 4); ++i) n += min(max((VEC ? (D + 3) / 4 : D) - i * threads - 32 * w, 0), 32);
        return (float)(VEC ? 4 * n : n);
    }
    __device__ __forceinline__ float inverse_of_warp() const { return 1.f / fmaxf(values_of_warp(tid >> 5), 1.f); }
    // Takes the mean off (kind kLayer) and returns 1 / the norm.  Each warp knows the mean of its values and the
    // squares about it before the one barrier; with n values each,
    //     sum (v - mean)^2 = sum over warps of (squares + n (warp's mean - mean)^2).
    // in_warp, in_lane: inverse_of_warp() and values_of_warp(lane).
    __device__ __forceinline__ float scale_of(float (&v)[4 * NV], int kind, float eps, float inv, float in_warp, float in_lane,
                                              float2 (*scratch)[32], int &turn) const {
        float sum = 0.f;
        if (kind != kLayer) {
#pragma unroll
            for (int k = 0; k < 4 * NV; ++k) sum = fmaf(v[k], v[k], sum);
            return 1.f / sqrtf(turn_sum(sum, scratch, turn) * inv + eps);
        }
#pragma unroll
        for (int k = 0; k < 4 * NV; ++k) sum += v[k];
        float mean = warp_sum(sum) * in_warp, square = 0.f;
#pragma unroll
        for (int k = 0; k < 4 * NV; ++k) {
            const float d = v[k] - mean;
            if (in(k / 4, VEC ? 0 : k & 3)) square = fmaf(d, d, square);
        }
        square = warp_sum(square);
        const int warps = threads >> 5, lane = tid & 31;
        if (warps > 1) {
            if (lane == 0) scratch[turn][tid >> 5] = make_float2(mean, square);
            __syncthreads();
            const float2 of = lane < warps ? scratch[turn][lane] : make_float2(0.f, 0.f);
            turn ^= 1;
            const float n = lane < warps ? in_lane : 0.f;
            mean = warp_sum(n * of.x) * inv;
            const float d = of.x - mean;
            square = warp_sum(lane < warps ? fmaf(n * d, d, of.y) : 0.f);
        }
#pragma unroll
        for (int k = 0; k < 4 * NV; ++k) v[k] = in(k / 4, VEC ? 0 : k & 3) ? v[k] - mean : 0.f;
        return 1.f / sqrtf(square * inv + eps);
    }
    // v <- norm(v)
    __device__ __forceinline__ void norm(float (&v)[4 * NV], int kind, const float *w, const float *b, float eps, float2 (*scratch)[32],
                                         int &turn) const {
        float t[4 * NV];
        if (w) load(w, t);  // (on its way during the sums)
        const float f = scale_of(v, kind, eps, 1.f / (float)D, inverse_of_warp(), values_of_warp(tid & 31), scratch, turn);
#pragma unroll
        for (int k = 0; k < 4 * NV; ++k) v[k] *= f;
        if (w) {
#pragma unroll
            for (int k = 0; k < 4 * NV; ++k) v[k] *= t[k];
        }
        if (b) {
            load(b, t);
#pragma unroll
            for (int k = 0; k < 4 * NV; ++k) v[k] += t[k];
        }
    }
};

template <int NV, bool VEC, bool BF16, bool X8>
__global__ void __launch_bounds__(kMaxThreads) norm_kernel(const NormArgs a) {
    using Res = typename std::conditional<BF16, uint16_t, float>::type;
    __shared__ float2 scratch[2][32];
    int turn = 0;
    pdl_wait();
    pdl_trigger();
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;  // (several rows a CTA: a warp each, without barriers)
    if (row >= a.M) return;
    const Slice<NV, VEC> s = {(int)a.D, (int)threadIdx.x, (int)blockDim.x};
    float h[4 * NV];
    s.load(static_cast<const Res *>(a.r_in) + row * a.ldr, h);  // (on its way during the first norm)
    if (a.y) {
        float y[4 * NV], t[4 * NV];
        s.load(a.y + row * a.ldy, y);
        if (a.gate) s.load(a.gate + row * a.ld_gate, t);
        if (a.post != kNone) s.norm(y, a.post, a.post_w, a.post_b, a.post_eps, scratch, turn);
        if (a.gate) {
#pragma unroll
            for (int k = 0; k < 4 * NV; ++k) y[k] *= t[k];
        }
#pragma unroll
        for (int k = 0; k < 4 * NV; ++k) h[k] = fmaf(a.scale, y[k], h[k]);
    }
    if (a.r_out) s.store(static_cast<Res *>(a.r_out) + row * a.ldr, h);
    if (!X8 && !a.x) return;
    if (a.pre != kNone) s.norm(h, a.pre, a.pre_w, a.pre_b, a.pre_eps, scratch, turn);
    if (!X8 || a.x) s.store(a.x + row * a.ldx, h);
    if constexpr (X8) s.store8(a.q + row * a.D, a.q_scale + row * (a.D / 32), h);
}

// Many rows: a few CTAs an SM walk them, one row in registers while the next ones are copied into a ring in
// shared memory, whole rows at a time.  What is the same for every row stays in registers and shared memory; a CTA
// a row reads it from L2 each time, as much again as the row itself (4096 x 5120: 51 us against 36).
constexpr int kRing = 8;  // rows of the ring, at most (8192 x 768: 15.7 us, with 4 18.0)

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}

// (640: 96 registers a thread, so that two CTAs of up to 320 threads share an SM)
template <int NV, bool BF16, bool FULL, bool X8>
__global__ void __launch_bounds__(640) norm_rows_kernel(const NormArgs a, int stages, uint32_t ring_bytes) {
    using Res = typename std::conditional<BF16, uint16_t, float>::type;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(8) uint64_t bars[kRing];
    __shared__ float2 scratch[2][32];
    const int D = (int)a.D, tid = threadIdx.x;
    const Slice<NV, true, FULL> s = {D, tid, (int)blockDim.x};
    const bool gate_rows = a.y && a.gate && a.ld_gate != 0;
    const uint32_t y_bytes = a.y ? 4u * D : 0u, r_bytes = (uint32_t)sizeof(Res) * D, g_bytes = gate_rows ? 4u * D : 0u;
    const uint32_t stage_bytes = y_bytes + r_bytes + g_bytes;
    if (tid < stages) mbar_init(smem_u32(&bars[tid]), 1);
    fence_mbar_init();
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    // row: of the ring's stage, in the order of the walk
    auto copy = [&](int64_t row, int stage) {
        const uint32_t bar = smem_u32(&bars[stage]), at = smem_u32(ring) + stage * stage_bytes;
        mbar_arrive_expect_tx(bar, stage_bytes);
        if (a.y) bulk_copy(at, a.y + row * a.ldy, y_bytes, bar);
        bulk_copy(at + y_bytes, static_cast<const Res *>(a.r_in) + row * a.ldr, r_bytes, bar);
        if (gate_rows) bulk_copy(at + y_bytes + r_bytes, a.gate + row * a.ld_gate, g_bytes, bar);
    };
    if (tid == 0)
        for (int i = 0; i < stages; ++i)
            if (blockIdx.x + (int64_t)i * gridDim.x < a.M) copy(blockIdx.x + (int64_t)i * gridDim.x, i);
    // a limit that only tests a copy (q4k_set_gemv_wait_limit_ns) tests the first row's here, where it is on its way for certain:
    // behind the weights' loads a short row has mostly landed
    const bool soon = a.wait_ns >= 1000ull || mbar_wait_limit(smem_u32(&bars[0]), 0, a.status, a.wait_ns);
    // scale * gate * post_w and pre_w
    float wy[4 * NV], wx[4 * NV];
#pragma unroll
    for (int k = 0; k < 4 * NV; ++k) wy[k] = a.scale, wx[k] = 1.f;
    auto times = [&](float (&w)[4 * NV], const float *p) {
        float t[4 * NV];
        s.load(p, t);
#pragma unroll
        for (int k = 0; k < 4 * NV; ++k) w[k] *= t[k];
    };
    if (a.y && a.post != kNone && a.post_w) times(wy, a.post_w);
    if (a.y && a.gate && !gate_rows) times(wy, a.gate);
    const bool out = X8 || a.x;  // is pre(h) wanted
    if (out && a.pre != kNone && a.pre_w) times(wx, a.pre_w);
    // and scale * gate * post_b and pre_b, in shared memory behind the ring (registers are short): each thread's own
    const bool post_b = a.y && a.post != kNone && a.post_b, pre_b = out && a.pre != kNone && a.pre_b;
    float *const by = reinterpret_cast<float *>(ring + ring_bytes), *const bx = by + (post_b ? D : 0);
    if (post_b) {
        float t[4 * NV];
#pragma unroll
        for (int k = 0; k < 4 * NV; ++k) t[k] = a.scale;
        times(t, a.post_b);
        if (a.gate && !gate_rows) times(t, a.gate);
        s.store(by, t);
    }
    if (pre_b) {
        float t[4 * NV];
        s.load(a.pre_b, t);
        s.store(bx, t);
    }
    // four values of one of them
    auto four = [&](const float *p, int i) {
        return s.in(i, 0) ? *reinterpret_cast<const float4 *>(p + s.at(i, 0)) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    const float inv = 1.f / (float)D, in_warp = s.inverse_of_warp(), in_lane = s.values_of_warp(tid & 31);
    int turn = 0, stage = 0;
    uint32_t parity = 0;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
        const bool landed = soon && mbar_wait_limit(smem_u32(&bars[stage]), parity, a.status, a.wait_ns);
        const uint8_t *at = ring + stage * stage_bytes;
        float v[4 * NV], h[4 * NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = s.at(i, 0);
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f), r = y;
            if (s.in(i, 0)) {
                if (a.y) y = *reinterpret_cast<const float4 *>(at + 4 * e);
                if constexpr (BF16) {
                    const uint2 t = *reinterpret_cast<const uint2 *>(at + y_bytes + 2 * e);
                    r = make_float4(__uint_as_float(t.x << 16), __uint_as_float(t.x & 0xFFFF0000u), __uint_as_float(t.y << 16),
                                    __uint_as_float(t.y & 0xFFFF0000u));
                } else {
                    r = *reinterpret_cast<const float4 *>(at + y_bytes + 4 * e);
                }
            }
            v[4 * i] = y.x, v[4 * i + 1] = y.y, v[4 * i + 2] = y.z, v[4 * i + 3] = y.w;
            h[4 * i] = r.x, h[4 * i + 1] = r.y, h[4 * i + 2] = r.z, h[4 * i + 3] = r.w;
        }
        if (a.y) {
            if (a.post != kNone) {
                const float f = s.scale_of(v, a.post, a.post_eps, inv, in_warp, in_lane, scratch, turn);
#pragma unroll
                for (int k = 0; k < 4 * NV; ++k) v[k] *= f;
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const float4 b = post_b ? four(by, i) : make_float4(0.f, 0.f, 0.f, 0.f);
                const float b4[4] = {b.x, b.y, b.z, b.w};
                if (gate_rows) {
                    const float4 t = four(reinterpret_cast<const float *>(at + y_bytes + r_bytes), i);
                    const float t4[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
                    for (int x = 0; x < 4; ++x) h[4 * i + x] = fmaf(t4[x], fmaf(v[4 * i + x], wy[4 * i + x], b4[x]), h[4 * i + x]);
                } else {
#pragma unroll
                    for (int x = 0; x < 4; ++x) h[4 * i + x] = fmaf(v[4 * i + x], wy[4 * i + x], h[4 * i + x]) + b4[x];
                }
            }
        }
        // the stage has been read; or some thread gave up on it, and all leave (one may give up on what another has seen land)
        if (__syncthreads_or(!landed)) {
            // thread 0 has issued the copies of this row and of the next stages - 1
            for (int i = 0; tid == 0 && i < stages && row + (int64_t)i * gridDim.x < a.M; ++i) {
                const int of = stage + i < stages ? stage + i : stage + i - stages;
                mbar_wait(smem_u32(&bars[of]), of < stage ? parity ^ 1 : parity, a.status);
            }
            return;
        }
        if (tid == 0 && row + (int64_t)stages * gridDim.x < a.M) copy(row + (int64_t)stages * gridDim.x, stage);
        if (++stage == stages) stage = 0, parity ^= 1;
        if (a.r_out) s.store(static_cast<Res *>(a.r_out) + row * a.ldr, h);
        if (!out) continue;
        if (a.pre != kNone) {
            const float f = s.scale_of(h, a.pre, a.pre_eps, inv, in_warp, in_lane, scratch, turn);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const float4 b = pre_b ? four(bx, i) : make_float4(0.f, 0.f, 0.f, 0.f);
                const float b4[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int x = 0; x < 4; ++x) h[4 * i + x] = fmaf(h[4 * i + x] * f, wx[4 * i + x], b4[x]);
            }
        }
        if (!X8 || a.x) s.store(a.x + row * a.ldx, h);
        if constexpr (X8) s.store8(a.q + row * D, a.q_scale + row * (D / 32), h);
    }
}

// Rows too long for registers: every pass reads the row again and forms h anew; r_out
// (which may be r_in) is written in the last one.
__global__ void __launch_bounds__(kMaxThreads) norm_long_kernel(const NormArgs a) {
    __shared__ float2 scratch[2][32];
    int turn = 0;
    pdl_wait();
    pdl_trigger();
    const int64_t row = blockIdx.x, D = a.D;
    const float *y = a.y ? a.y + row * a.ldy : nullptr;
    const float *gate = a.gate ? a.gate + row * a.ld_gate : nullptr;
    const float n = (float)D;
    auto total = [&](auto &&value) {
        float s = 0.f;
        for (int64_t e = threadIdx.x; e < D; e += blockDim.x) s += value(e);
        return turn_sum(s, scratch, turn);
    };
    float y_mean = 0.f, y_f = 1.f;
    if (y && a.post != kNone) {
        if (a.post == kLayer) y_mean = total([&](int64_t e) { return __ldg(y + e); }) / n;
        y_f = 1.f / sqrtf(total([&](int64_t e) { const float d = __ldg(y + e) - y_mean; return d * d; }) / n + a.post_eps);
    }
    auto h_at = [&](int64_t e) {
        const float r = a.bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(a.r_in)[row * a.ldr + e] << 16)
                               : static_cast<const float *>(a.r_in)[row * a.ldr + e];
        if (!y) return r;
        float v = __ldg(y + e);
        if (a.post != kNone) {
            v = (v - y_mean) * y_f;
            if (a.post_w) v *= __ldg(a.post_w + e);
            if (a.post_b) v += __ldg(a.post_b + e);
        }
        if (gate) v *= __ldg(gate + e);
        return fmaf(a.scale, v, r);
    };
    float h_mean = 0.f, h_f = 1.f;
    if ((a.x || a.q) && a.pre != kNone) {
        if (a.pre == kLayer) h_mean = total(h_at) / n;
        h_f = 1.f / sqrtf(total([&](int64_t e) { const float d = h_at(e) - h_mean; return d * d; }) / n + a.pre_eps);
    }
    for (int64_t e = threadIdx.x; e < D; e += blockDim.x) {
        const float h = h_at(e);
        if (a.r_out) {
            if (a.bf16) static_cast<uint16_t *>(a.r_out)[row * a.ldr + e] = __bfloat16_as_ushort(__float2bfloat16_rn(h));
            else static_cast<float *>(a.r_out)[row * a.ldr + e] = h;
        }
        if (a.x || a.q) {
            float v = h;
            if (a.pre != kNone) {
                v = (h - h_mean) * h_f;
                if (a.pre_w) v *= __ldg(a.pre_w + e);
                if (a.pre_b) v += __ldg(a.pre_b + e);
            }
            if (a.x) a.x[row * a.ldx + e] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
            if (a.q) {  // (D % 32 == 0: whole warps)
                const float top = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fabsf(v)))), s = top / 127.0f;
                a.q[row * D + e] = (int8_t)in_eight(v, s);
                if ((threadIdx.x & 31) == 0) a.q_scale[row * (D / 32) + e / 32] = s;
            }
        }
    }
}

template <int NV>
cudaError_t launch(const NormArgs &a, bool vec, int threads, cudaStream_t s) {
    auto kern = a.q ? (a.bf16 ? (vec ? norm_kernel<NV, true, true, true> : norm_kernel<NV, false, true, true>)
                              : (vec ? norm_kernel<NV, true, false, true> : norm_kernel<NV, false, false, true>))
                    : (a.bf16 ? (vec ? norm_kernel<NV, true, true, false> : norm_kernel<NV, false, true, false>)
                              : (vec ? norm_kernel<NV, true, false, false> : norm_kernel<NV, false, false, false>));
    // rows of one warp: eight to a CTA where they are many (8038 x 65: 8.5 us with one, 5 with eight)
    const int rows = threads == 32 && a.M >= 2048 ? 8 : 1;
    return launch_pdl(kern, dim3((unsigned)((a.M + rows - 1) / rows)), dim3(threads, rows), 0, s, dim3(1), a);
}

template <int NV>
cudaError_t launch_rows(const NormArgs &a, int stages, int ring, int smem, int per_sm, int threads, int sm_count, cudaStream_t s) {
    const bool full = a.D == 4 * NV * threads;
    auto kern = a.q ? (full ? (a.bf16 ? norm_rows_kernel<NV, true, true, true> : norm_rows_kernel<NV, false, true, true>)
                            : (a.bf16 ? norm_rows_kernel<NV, true, false, true> : norm_rows_kernel<NV, false, false, true>))
                    : (full ? (a.bf16 ? norm_rows_kernel<NV, true, true, false> : norm_rows_kernel<NV, false, true, false>)
                            : (a.bf16 ? norm_rows_kernel<NV, true, false, false> : norm_rows_kernel<NV, false, false, false>));
    cudaError_t e = ensure_smem((const void *)kern, smem);
    if (e != cudaSuccess) return e;
    const int64_t grid = a.M < (int64_t)sm_count * per_sm ? a.M : (int64_t)sm_count * per_sm;
    return launch_pdl(kern, dim3((unsigned)grid), dim3(threads), smem, s, dim3(1), a, stages, (uint32_t)ring);
}

}  // namespace

cudaError_t launch_norm_residual(const DeviceInfo &di, const NormArgs &a, cudaStream_t s) {
    auto al = [](const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
    const uintptr_t rb = a.bf16 ? 8 : 16;
    const bool vec = a.D % 4 == 0 && a.ldr % 4 == 0 && al(a.r_in, rb) && al(a.r_out, rb) &&
                     (!a.y || (al(a.y, 16) && a.ldy % 4 == 0)) && (!a.gate || (al(a.gate, 16) && a.ld_gate % 4 == 0)) &&
                     (!a.x || (al(a.x, 8) && a.ldx % 4 == 0)) && al(a.post_w, 16) && al(a.post_b, 16) && al(a.pre_w, 16) &&
                     al(a.pre_b, 16);
    const int64_t quads = (a.D + 3) / 4;  // groups of four values
    // many rows that can be copied whole: a ring of at least two rows a CTA (577 x 5120: 5.9 us, a CTA a row 9.5); those of
    // one warp go to a warp each below (8038 x 64: 7.6 us with the ring).  The two forms round in another order, so where a
    // row's bits must not depend on M the ring takes few rows, too (one of 5120: 3.0 us, a CTA a row 2.9; the other way
    // about, 4096 of them take 87 instead of 37)
    const int64_t row_bytes = a.D * ((a.y ? 4 : 0) + (a.bf16 ? 2 : 4) + (a.y && a.gate && a.ld_gate != 0 ? 4 : 0));
    const bool bulk = vec && a.D % 8 == 0 && al(a.r_in, 16) && (a.bf16 ? a.ldr % 8 == 0 : true);
    // values of a thread: as many as leave no thread without any (8192 x 768 with 16 a thread of two warps, a quarter of
    // them idle: 19.3 us, with 8 of three: 17.8)
    int nv = quads > 128 ? 4 : quads > 64 ? 2 : 1;
    while (nv > 1 && quads % (32 * nv) != 0 && quads % 32 == 0 && quads <= 640 * (nv / 2)) nv /= 2;
    const int threads_many = (int)(((quads + nv - 1) / nv + 31) / 32 * 32);
    if (bulk && threads_many > 32 && threads_many <= 640 && (a.M >= di.sm_count || a.invariant)) {
        const int64_t biases = 4 * a.D * ((a.y && a.post != kNone && a.post_b ? 1 : 0) + ((a.x || a.q) && a.pre != kNone && a.pre_b ? 1 : 0));
        int per_sm = (nv == 4 ? 640 : 960) / threads_many;  // (as many as the registers allow)
        if (per_sm > 10) per_sm = 10;
        while (per_sm > 1 && (220 * 1024) / per_sm < 2 * row_bytes + biases + 1024) --per_sm;
        int64_t stages = ((220 * 1024) / per_sm - 1024 - biases) / row_bytes;
        if (stages > kRing) stages = kRing;
        if (stages >= 2) {
            const int ring = (int)(stages * row_bytes), smem = (int)(ring + biases);
            return nv == 4   ? launch_rows<4>(a, (int)stages, ring, smem, per_sm, threads_many, di.sm_count, s)
                   : nv == 2 ? launch_rows<2>(a, (int)stages, ring, smem, per_sm, threads_many, di.sm_count, s)
                             : launch_rows<1>(a, (int)stages, ring, smem, per_sm, threads_many, di.sm_count, s);
        }
    }
    // a CTA a row, values in registers: eight a thread, which leave registers for the loads ahead, up to 8192
    // (2000 x 12375, which spills: 125 us; with 32 values of half as many threads 174)
    if (quads > 4 * kMaxThreads) return launch_pdl(norm_long_kernel, dim3((unsigned)a.M), dim3(kMaxThreads), 0, s, dim3(1), a);
    const int of_thread = quads > 2 * kMaxThreads ? 4 : quads > kMaxThreads / 2 ? 2 : 1;
    const int threads = (int)(((quads + of_thread - 1) / of_thread + 31) / 32 * 32);
    return of_thread == 4 ? launch<4>(a, vec, threads, s) : of_thread == 2 ? launch<2>(a, vec, threads, s) : launch<1>(a, vec, threads, s);
}

}  // namespace q4k
