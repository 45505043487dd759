// The end of one block and the start of the next in one pass:
//     h = r + scale * gate * post(y),  r' = h,  x = bf16(pre(h))
// post and pre being RMS or layer norms over a row.
//
// Bound by HBM for many rows (a row of y and r read, of r' and x written, each once)
// and by latency for few.  A CTA holds a whole row in registers between the two norms,
// up to 16384 values; only longer rows are read again.  A mean is
// taken off before the squares are summed (two reductions over registers cost little,
// and E[x^2] - E[x]^2 would cancel).  Everything is fp32 until the two outputs.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

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

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// A row of D values over a CTA: thread t holds group i (of NV) of four values, elements
// 4 (i threads + t) .. + 3 (VEC: 16-byte accesses), or i * 4 + x -> (4 i + x) threads + t.
// Values past D are 0.
template <int NV, bool VEC>
struct Slice {
    int D, tid, threads;
    __device__ __forceinline__ int at(int i, int x) const { return VEC ? 4 * (i * threads + tid) + x : (4 * i + x) * threads + tid; }
    __device__ __forceinline__ void load(const float *p, float (&v)[4 * NV]) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if constexpr (VEC) {
                const float4 t = at(i, 0) < D ? __ldg(reinterpret_cast<const float4 *>(p + at(i, 0))) : make_float4(0.f, 0.f, 0.f, 0.f);
                v[4 * i] = t.x, v[4 * i + 1] = t.y, v[4 * i + 2] = t.z, v[4 * i + 3] = t.w;
            } else {
#pragma unroll
                for (int x = 0; x < 4; ++x) v[4 * i + x] = at(i, x) < D ? __ldg(p + at(i, x)) : 0.f;
            }
        }
    }
    __device__ __forceinline__ void load(const uint16_t *p, float (&v)[4 * NV]) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if constexpr (VEC) {
                const uint2 t = at(i, 0) < D ? __ldg(reinterpret_cast<const uint2 *>(p + at(i, 0))) : make_uint2(0, 0);
                v[4 * i] = __uint_as_float(t.x << 16), v[4 * i + 1] = __uint_as_float(t.x & 0xFFFF0000u);
                v[4 * i + 2] = __uint_as_float(t.y << 16), v[4 * i + 3] = __uint_as_float(t.y & 0xFFFF0000u);
            } else {
#pragma unroll
                for (int x = 0; x < 4; ++x) v[4 * i + x] = at(i, x) < D ? __uint_as_float((uint32_t)__ldg(p + at(i, x)) << 16) : 0.f;
            }
        }
    }
    __device__ __forceinline__ void store(float *p, const float (&v)[4 * NV]) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if constexpr (VEC) {
                if (at(i, 0) < D) *reinterpret_cast<float4 *>(p + at(i, 0)) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            } else {
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    if (at(i, x) < D) p[at(i, x)] = v[4 * i + x];
            }
        }
    }
    __device__ __forceinline__ void store(uint16_t *p, const float (&v)[4 * NV]) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint2 t = make_uint2(pack_bf16(v[4 * i], v[4 * i + 1]), pack_bf16(v[4 * i + 2], v[4 * i + 3]));
            if constexpr (VEC) {
                if (at(i, 0) < D) *reinterpret_cast<uint2 *>(p + at(i, 0)) = t;
            } else {
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    if (at(i, x) < D) p[at(i, x)] = (uint16_t)((x < 2 ? t.x : t.y) >> (x & 1) * 16);
            }
        }
    }
    // v <- norm(v)
    __device__ __forceinline__ void norm(float (&v)[4 * NV], int kind, const float *w, const float *b, float eps, float *scratch) const {
        float t[4 * NV];
        if (w) load(w, t);  // (on its way during the sums)
        const float inv = 1.f / (float)D;
        float sum = 0.f;
        if (kind == kLayer) {
#pragma unroll
            for (int k = 0; k < 4 * NV; ++k) sum += v[k];
            const float mean = block_sum(sum, scratch) * inv;
#pragma unroll
            for (int k = 0; k < 4 * NV; ++k) v[k] = at(k / 4, VEC ? 0 : k & 3) < D ? v[k] - mean : 0.f;
            sum = 0.f;
        }
#pragma unroll
        for (int k = 0; k < 4 * NV; ++k) sum = fmaf(v[k], v[k], sum);
        const float f = 1.f / sqrtf(block_sum(sum, scratch) * inv + eps);
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

template <int NV, bool VEC, bool BF16>
__global__ void __launch_bounds__(NV <= 2 ? kMaxThreads : 512) norm_kernel(const NormArgs a) {
    using Res = typename std::conditional<BF16, uint16_t, float>::type;
    __shared__ float scratch[33];
    pdl_wait();
    pdl_trigger();
    const int64_t row = blockIdx.x;
    const Slice<NV, VEC> s = {(int)a.D, (int)threadIdx.x, (int)blockDim.x};
    float h[4 * NV];
    s.load(static_cast<const Res *>(a.r_in) + row * a.ldr, h);  // (on its way during the first norm)
    if (a.y) {
        float y[4 * NV], t[4 * NV];
        s.load(a.y + row * a.ldy, y);
        if (a.gate) s.load(a.gate + row * a.ld_gate, t);
        if (a.post != kNone) s.norm(y, a.post, a.post_w, a.post_b, a.post_eps, scratch);
        if (a.gate) {
#pragma unroll
            for (int k = 0; k < 4 * NV; ++k) y[k] *= t[k];
        }
#pragma unroll
        for (int k = 0; k < 4 * NV; ++k) h[k] = fmaf(a.scale, y[k], h[k]);
    }
    if (a.r_out) s.store(static_cast<Res *>(a.r_out) + row * a.ldr, h);
    if (!a.x) return;
    if (a.pre != kNone) s.norm(h, a.pre, a.pre_w, a.pre_b, a.pre_eps, scratch);
    s.store(a.x + row * a.ldx, h);
}

// Many rows: two CTAs an SM walk them, one row in registers while the next ones are copied into a ring in
// shared memory, whole rows at a time.  What is the same for every row stays in registers; a CTA a row reads
// it from L2 each time, as much again as the row itself.
constexpr int kRing = 4;  // rows of the ring, at most

// Sum over the CTA with one barrier: two scratch arrays in turn.
__device__ __forceinline__ float turn_sum(float v, float (*scratch)[32], int &turn) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warps == 1) return v;
    if (lane == 0) scratch[turn][warp] = v;
    __syncthreads();
    v = lane < warps ? scratch[turn][lane] : 0.f;
    turn ^= 1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}

// (640: 96 registers a thread, so that two CTAs of up to 320 threads share an SM)
template <int NV, bool BF16>
__global__ void __launch_bounds__(640) norm_rows_kernel(const NormArgs a, int stages) {
    using Res = typename std::conditional<BF16, uint16_t, float>::type;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(8) uint64_t bars[kRing];
    __shared__ float scratch[2][32];
    const int D = (int)a.D, tid = threadIdx.x;
    const Slice<NV, true> s = {D, tid, (int)blockDim.x};
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
    const float *post_b = a.post != kNone ? a.post_b : nullptr, *pre_b = a.pre != kNone ? a.pre_b : nullptr;
    if (a.y && a.post != kNone && a.post_w && !post_b) times(wy, a.post_w);
    if (a.y && a.gate && !gate_rows) times(wy, a.gate);
    if (a.x && a.pre != kNone && a.pre_w) times(wx, a.pre_w);
    const float inv = 1.f / (float)D;
    int turn = 0, stage = 0;
    uint32_t parity = 0;
    auto scale_of = [&](float (&v)[4 * NV], int kind, float eps) {  // takes the mean off, returns 1 / the norm
        float sum = 0.f;
        if (kind == kLayer) {
#pragma unroll
            for (int k = 0; k < 4 * NV; ++k) sum += v[k];
            const float mean = turn_sum(sum, scratch, turn) * inv;
#pragma unroll
            for (int k = 0; k < 4 * NV; ++k) v[k] = s.at(k / 4, 0) < D ? v[k] - mean : 0.f;
            sum = 0.f;
        }
#pragma unroll
        for (int k = 0; k < 4 * NV; ++k) sum = fmaf(v[k], v[k], sum);
        return 1.f / sqrtf(turn_sum(sum, scratch, turn) * inv + eps);
    };
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
        if (!mbar_wait(smem_u32(&bars[stage]), parity, a.status)) {
            mbar_wait(smem_u32(&bars[stage]), parity, a.status);  // the copies may still land
            return;  // (every thread waits for the same phase and gives up alike)
        }
        const uint8_t *at = ring + stage * stage_bytes;
        float v[4 * NV], h[4 * NV];
        const bool gate_on = gate_rows;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = s.at(i, 0);
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f), r = y;
            if (e < D) {
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
                const float f = scale_of(v, a.post, a.post_eps);
#pragma unroll
                for (int k = 0; k < 4 * NV; ++k) v[k] *= f;
                if (post_b) {  // (then post_w is not among wy)
                    float t[4 * NV];
                    if (a.post_w) {
                        s.load(a.post_w, t);
#pragma unroll
                        for (int k = 0; k < 4 * NV; ++k) v[k] *= t[k];
                    }
                    s.load(post_b, t);
#pragma unroll
                    for (int k = 0; k < 4 * NV; ++k) v[k] += t[k];
                }
            }
            if (gate_on) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (s.at(i, 0) < D) {
                        const float4 t = *reinterpret_cast<const float4 *>(at + y_bytes + r_bytes + 4 * s.at(i, 0));
                        v[4 * i] *= t.x, v[4 * i + 1] *= t.y, v[4 * i + 2] *= t.z, v[4 * i + 3] *= t.w;
                    }
            }
#pragma unroll
            for (int k = 0; k < 4 * NV; ++k) h[k] = fmaf(v[k], wy[k], h[k]);
        }
        __syncthreads();  // the stage has been read
        if (tid == 0 && row + (int64_t)stages * gridDim.x < a.M) copy(row + (int64_t)stages * gridDim.x, stage);
        if (++stage == stages) stage = 0, parity ^= 1;
        if (a.r_out) s.store(static_cast<Res *>(a.r_out) + row * a.ldr, h);
        if (!a.x) continue;
        if (a.pre != kNone) {
            const float f = scale_of(h, a.pre, a.pre_eps);
#pragma unroll
            for (int k = 0; k < 4 * NV; ++k) h[k] = h[k] * f * wx[k];
            if (pre_b) {
                float t[4 * NV];
                s.load(pre_b, t);
#pragma unroll
                for (int k = 0; k < 4 * NV; ++k) h[k] += t[k];
            }
        }
        s.store(a.x + row * a.ldx, h);
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
    auto kern = a.bf16 ? (vec ? norm_kernel<NV, true, true> : norm_kernel<NV, false, true>)
                       : (vec ? norm_kernel<NV, true, false> : norm_kernel<NV, false, false>);
    return launch_pdl(kern, dim3((unsigned)a.M), dim3(threads), 0, s, dim3(1), a);
}

template <int NV>
cudaError_t launch_rows(const NormArgs &a, int stages, int smem, int per_sm, int threads, int sm_count, cudaStream_t s) {
    auto kern = a.bf16 ? norm_rows_kernel<NV, true> : norm_rows_kernel<NV, false>;
    cudaError_t e = ensure_smem((const void *)kern, smem);
    if (e != cudaSuccess) return e;
    const int64_t grid = a.M < (int64_t)sm_count * per_sm ? a.M : (int64_t)sm_count * per_sm;
    return launch_pdl(kern, dim3((unsigned)grid), dim3(threads), smem, s, dim3(1), a, stages);
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
    if (quads > 2 * kMaxThreads) {
        if (quads > 8 * 512) return launch_pdl(norm_long_kernel, dim3((unsigned)a.M), dim3(kMaxThreads), 0, s, dim3(1), a);
        const int threads = (int)(((quads + 7) / 8 + 31) / 32 * 32);
        return launch<8>(a, vec, threads, s);
    }
    // many rows that can be copied whole: a ring of at least two rows a CTA (device time of one CTA a row
    // against the ring at 4096 x 5120: 51 and 36 us)
    const int64_t row_bytes = a.D * ((a.y ? 4 : 0) + (a.bf16 ? 2 : 4) + (a.y && a.gate && a.ld_gate != 0 ? 4 : 0));
    const bool bulk = vec && a.D % 8 == 0 && al(a.r_in, 16) && (a.bf16 ? a.ldr % 8 == 0 : true);
    const int nv = quads > 128 ? 4 : quads > 64 ? 2 : 1;
    const int threads_many = (int)(((quads + nv - 1) / nv + 31) / 32 * 32);
    if (bulk && threads_many <= 640 && a.M >= 4 * di.sm_count) {
        int per_sm = 640 / threads_many;
        if (per_sm > 8) per_sm = 8;
        while (per_sm > 1 && (220 * 1024) / per_sm < 2 * row_bytes + 1024) --per_sm;
        int64_t stages = ((220 * 1024) / per_sm - 1024) / row_bytes;
        if (stages > kRing) stages = kRing;
        if (stages >= 2) {
            const int smem = (int)(stages * row_bytes);
            return nv == 4   ? launch_rows<4>(a, (int)stages, smem, per_sm, threads_many, di.sm_count, s)
                   : nv == 2 ? launch_rows<2>(a, (int)stages, smem, per_sm, threads_many, di.sm_count, s)
                             : launch_rows<1>(a, (int)stages, smem, per_sm, threads_many, di.sm_count, s);
        }
    }
    const int few = quads > kMaxThreads / 2 ? 2 : 1;
    const int threads = (int)(((quads + few - 1) / few + 31) / 32 * 32);
    return few == 2 ? launch<2>(a, vec, threads, s) : launch<1>(a, vec, threads, s);
}

}  // namespace q4k
