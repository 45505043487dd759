// The end of one block and the start of the next in one pass:
//     h = r + scale * gate * post(y),  r' = h,  x = bf16(pre(h))
// post and pre being RMS or layer norms over a row.
//
// Bound by HBM for many rows (a row of y and r read, of r' and x written, each once)
// and by latency for few.  A CTA holds a whole row in registers between the two norms,
// up to kMaxThreads * 16 values; only longer rows are read again.  A mean is
// taken off before the squares are summed (two reductions over registers cost little,
// and E[x^2] - E[x]^2 would cancel).  Everything is fp32 until the two outputs.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "decode_ops.h"
#include "q4k_ptx.cuh"

namespace q4k {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kNone = 0, kLayer = 2;  // Q4K_NORM_NONE, Q4K_NORM_LAYER

// Sum over the CTA, in the same order on every call; scratch holds 33 floats.
__device__ __forceinline__ float block_sum(float v, float *scratch) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warps == 1) return v;
    __syncthreads();  // the sum before has been read
    if (lane == 0) scratch[warp] = v;
    __syncthreads();
    v = lane < warps ? scratch[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

__device__ __forceinline__ float bf16_at(const uint16_t *p) { return __uint_as_float((uint32_t)__ldg(p) << 16); }

// Thread t's value k (0 <= k < 4 NV) is element (k / 4 * threads + t) * 4 + k % 4 of the
// row (VEC: 16-byte accesses) or k * threads + t.
template <bool VEC>
__device__ __forceinline__ int64_t element(int k) {
    return VEC ? ((int64_t)(k / 4) * blockDim.x + threadIdx.x) * 4 + (k & 3) : (int64_t)k * blockDim.x + threadIdx.x;
}

template <int NV, bool VEC>
__device__ __forceinline__ void load_f32(const float *p, int64_t D, float (&v)[4 * NV]) {
#pragma unroll
    for (int k = 0; k < 4 * NV; k += VEC ? 4 : 1) {
        const int64_t e = element<VEC>(k);
        if constexpr (VEC) {
            const float4 t = e < D ? __ldg(reinterpret_cast<const float4 *>(p + e)) : make_float4(0.f, 0.f, 0.f, 0.f);
            v[k] = t.x, v[k + 1] = t.y, v[k + 2] = t.z, v[k + 3] = t.w;
        } else {
            v[k] = e < D ? __ldg(p + e) : 0.f;
        }
    }
}

// v <- norm(v); values past D are left alone
template <int NV, bool VEC>
__device__ __forceinline__ void norm_row(float (&v)[4 * NV], int64_t D, int kind, const float *w, const float *b, float eps,
                                         float *scratch) {
    float sum = 0.f;
    if (kind == kLayer) {
#pragma unroll
        for (int k = 0; k < 4 * NV; ++k)
            if (element<VEC>(k) < D) sum += v[k];
        const float mean = block_sum(sum, scratch) / (float)D;
#pragma unroll
        for (int k = 0; k < 4 * NV; ++k) v[k] -= mean;
    }
    sum = 0.f;
#pragma unroll
    for (int k = 0; k < 4 * NV; ++k)
        if (element<VEC>(k) < D) sum = fmaf(v[k], v[k], sum);
    const float f = 1.f / sqrtf(block_sum(sum, scratch) / (float)D + eps);
    float t[4 * NV];
    if (w) {
        load_f32<NV, VEC>(w, D, t);
#pragma unroll
        for (int k = 0; k < 4 * NV; ++k) v[k] = v[k] * f * t[k];
    } else {
#pragma unroll
        for (int k = 0; k < 4 * NV; ++k) v[k] *= f;
    }
    if (b) {
        load_f32<NV, VEC>(b, D, t);
#pragma unroll
        for (int k = 0; k < 4 * NV; ++k) v[k] += t[k];
    }
}

template <int NV, bool VEC>
__global__ void __launch_bounds__(kMaxThreads) norm_kernel(const NormArgs a) {
    __shared__ float scratch[33];
    pdl_wait();
    pdl_trigger();
    const int64_t row = blockIdx.x, D = a.D;
    float h[4 * NV];
    // the residual row: loaded before the first norm waits for its sums
    if (a.bf16) {
        const uint16_t *r = static_cast<const uint16_t *>(a.r_in) + row * a.ldr;
#pragma unroll
        for (int k = 0; k < 4 * NV; k += VEC ? 4 : 1) {
            const int64_t e = element<VEC>(k);
            if constexpr (VEC) {
                const uint2 t = e < D ? __ldg(reinterpret_cast<const uint2 *>(r + e)) : make_uint2(0, 0);
                h[k] = __uint_as_float(t.x << 16), h[k + 1] = __uint_as_float(t.x & 0xFFFF0000u);
                h[k + 2] = __uint_as_float(t.y << 16), h[k + 3] = __uint_as_float(t.y & 0xFFFF0000u);
            } else {
                h[k] = e < D ? bf16_at(r + e) : 0.f;
            }
        }
    } else {
        load_f32<NV, VEC>(static_cast<const float *>(a.r_in) + row * a.ldr, D, h);
    }
    if (a.y) {
        float y[4 * NV];
        load_f32<NV, VEC>(a.y + row * a.ldy, D, y);
        if (a.post != kNone) norm_row<NV, VEC>(y, D, a.post, a.post_w, a.post_b, a.post_eps, scratch);
        if (a.gate) {
            float t[4 * NV];
            load_f32<NV, VEC>(a.gate + row * a.ld_gate, D, t);
#pragma unroll
            for (int k = 0; k < 4 * NV; ++k) y[k] *= t[k];
        }
#pragma unroll
        for (int k = 0; k < 4 * NV; ++k) h[k] = fmaf(a.scale, y[k], h[k]);
    }
    if (a.r_out) {
#pragma unroll
        for (int k = 0; k < 4 * NV; k += VEC ? 4 : 1) {
            const int64_t e = element<VEC>(k);
            if (e >= D) continue;
            if (a.bf16) {
                uint16_t *r = static_cast<uint16_t *>(a.r_out) + row * a.ldr;
                if constexpr (VEC)
                    *reinterpret_cast<uint2 *>(r + e) =
                        make_uint2(__bfloat16_as_ushort(__float2bfloat16_rn(h[k])) | (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(h[k + 1])) << 16,
                                   __bfloat16_as_ushort(__float2bfloat16_rn(h[k + 2])) | (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(h[k + 3])) << 16);
                else r[e] = __bfloat16_as_ushort(__float2bfloat16_rn(h[k]));
            } else {
                float *r = static_cast<float *>(a.r_out) + row * a.ldr;
                if constexpr (VEC) *reinterpret_cast<float4 *>(r + e) = make_float4(h[k], h[k + 1], h[k + 2], h[k + 3]);
                else r[e] = h[k];
            }
        }
    }
    if (!a.x) return;
    if (a.pre != kNone) norm_row<NV, VEC>(h, D, a.pre, a.pre_w, a.pre_b, a.pre_eps, scratch);
    uint16_t *x = a.x + row * a.ldx;
#pragma unroll
    for (int k = 0; k < 4 * NV; k += VEC ? 4 : 1) {
        const int64_t e = element<VEC>(k);
        if (e >= D) continue;
        if constexpr (VEC)
            *reinterpret_cast<uint2 *>(x + e) =
                make_uint2(__bfloat16_as_ushort(__float2bfloat16_rn(h[k])) | (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(h[k + 1])) << 16,
                           __bfloat16_as_ushort(__float2bfloat16_rn(h[k + 2])) | (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(h[k + 3])) << 16);
        else x[e] = __bfloat16_as_ushort(__float2bfloat16_rn(h[k]));
    }
}

// Rows too long for registers: every pass reads the row again and forms h anew; r_out
// (which may be r_in) is written in the last one.
__global__ void __launch_bounds__(kMaxThreads) norm_long_kernel(const NormArgs a) {
    __shared__ float scratch[33];
    pdl_wait();
    pdl_trigger();
    const int64_t row = blockIdx.x, D = a.D;
    const float *y = a.y ? a.y + row * a.ldy : nullptr;
    const float *gate = a.gate ? a.gate + row * a.ld_gate : nullptr;
    const float n = (float)D;
    auto total = [&](auto &&value) {
        float s = 0.f;
        for (int64_t e = threadIdx.x; e < D; e += blockDim.x) s += value(e);
        return block_sum(s, scratch);
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
    if (a.x && a.pre != kNone) {
        if (a.pre == kLayer) h_mean = total(h_at) / n;
        h_f = 1.f / sqrtf(total([&](int64_t e) { const float d = h_at(e) - h_mean; return d * d; }) / n + a.pre_eps);
    }
    for (int64_t e = threadIdx.x; e < D; e += blockDim.x) {
        const float h = h_at(e);
        if (a.r_out) {
            if (a.bf16) static_cast<uint16_t *>(a.r_out)[row * a.ldr + e] = __bfloat16_as_ushort(__float2bfloat16_rn(h));
            else static_cast<float *>(a.r_out)[row * a.ldr + e] = h;
        }
        if (a.x) {
            float v = h;
            if (a.pre != kNone) {
                v = (h - h_mean) * h_f;
                if (a.pre_w) v *= __ldg(a.pre_w + e);
                if (a.pre_b) v += __ldg(a.pre_b + e);
            }
            a.x[row * a.ldx + e] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
        }
    }
}

template <int NV>
cudaError_t launch(const NormArgs &a, bool vec, int threads, cudaStream_t s) {
    return launch_pdl(vec ? norm_kernel<NV, true> : norm_kernel<NV, false>, dim3((unsigned)a.M), dim3(threads), 0, s, dim3(1), a);
}

}  // namespace

cudaError_t launch_norm_residual(const DeviceInfo &di, const NormArgs &a, cudaStream_t s) {
    (void)di;
    auto al = [](const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
    const uintptr_t rb = a.bf16 ? 8 : 16;
    const bool vec = a.D % 4 == 0 && a.ldr % 4 == 0 && al(a.r_in, rb) && al(a.r_out, rb) &&
                     (!a.y || (al(a.y, 16) && a.ldy % 4 == 0)) && (!a.gate || (al(a.gate, 16) && a.ld_gate % 4 == 0)) &&
                     (!a.x || (al(a.x, 8) && a.ldx % 4 == 0)) && al(a.post_w, 16) && al(a.post_b, 16) && al(a.pre_w, 16) &&
                     al(a.pre_b, 16);
    const int64_t quads = (a.D + 3) / 4;  // groups of four values
    if (quads > 4 * kMaxThreads) return launch_pdl(norm_long_kernel, dim3((unsigned)a.M), dim3(kMaxThreads), 0, s, dim3(1), a);
    const int nv = quads > 2 * kMaxThreads ? 4 : quads > kMaxThreads / 2 ? 2 : 1;
    const int threads = (int)(((quads + nv - 1) / nv + 31) / 32 * 32);
    return nv == 4 ? launch<4>(a, vec, threads, s) : nv == 2 ? launch<2>(a, vec, threads, s) : launch<1>(a, vec, threads, s);
}

}  // namespace q4k
