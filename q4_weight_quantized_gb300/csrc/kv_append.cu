// Rotary embedding of new queries and keys, and the write of new keys and values into
// the paged cache.
//
// A pair (a, b) at angle theta becomes (a cos - b sin, b cos + a sin), each product and
// sum rounded to fp32 (no contraction, so the stored 8- and 16-bit values do not hang
// on how the compiler fuses).  Bound by HBM for prompts (4 bytes read and 1 or 2
// written per value) and by latency for a decode step.  One thread takes a unit of
// eight values: for half pairing four values and their partners half the rotary width
// on, so every access is 16 bytes (8 or 4 for the outputs) and neighbouring threads
// touch neighbouring bytes; pointers, strides or widths that do not allow that take a
// value (or pair) per thread.
// Measured: 2.0 us for 16 tokens of 40 and 8 heads of 128; 43.5 us for 8191 tokens of 32 and 4 heads into an e4m3
// cache, half the width rotated (245 MB at 5.6 TB/s).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "decode_ops.h"
#include "q4k_ptx.cuh"

namespace q4k {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// nearest e4m3 of two values, beyond +-448 to +-448, NaN to NaN
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Four consecutive values of a row, in the output's type.
__device__ __forceinline__ void store4(void *row, int at, const float *x, bool e4m3) {
    if (e4m3) reinterpret_cast<uint32_t *>(row)[at / 4] = pack_e4m3(x[0], x[1]) | pack_e4m3(x[2], x[3]) << 16;
    else reinterpret_cast<uint2 *>(row)[at / 4] = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
}
__device__ __forceinline__ void store1(void *row, int at, float x, bool e4m3) {
    if (e4m3) static_cast<uint8_t *>(row)[at] = (uint8_t)pack_e4m3(x, 0.f);
    else static_cast<uint16_t *>(row)[at] = (uint16_t)pack_bf16(x, 0.f);
}

__device__ __forceinline__ void rotate(float &a, float &b, float c, float s) {
    const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = x;
}

// Units of a head: VEC: eight values each; otherwise the rotary pairs, then single values.
// n = id / per_token by one multiplication (id < 2^31, see KvView).
template <bool VEC>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendArgs a, int64_t t0, uint32_t all, uint32_t per_token, uint32_t mul,
                                                          uint32_t shift, uint32_t units, float k_inv, float v_inv) {
    pdl_wait();
    pdl_trigger();
    const int D = a.c.dim, half = a.rope_dim / 2;
    const int q_heads = a.q ? a.n_heads : 0;
    for (uint32_t id = blockIdx.x * kThreads + threadIdx.x; id < all; id += gridDim.x * kThreads) {
        const uint32_t nth = (uint32_t)(((uint64_t)id * mul) >> shift), in_token = id - nth * per_token;
        const int64_t t = t0 + nth;
        int head = (int)(VEC ? in_token >> (31 - __clz(units)) : in_token / units);  // (VEC: units is a power of two)
        const int u = (int)(in_token - (uint32_t)head * units);
        const int kind = head < q_heads ? 0 : head < q_heads + a.c.heads ? 1 : 2;  // query, key, value
        if (kind) head -= q_heads + (kind == 2 ? a.c.heads : 0);
        // ---- where the token goes
        const int seq = __ldg(a.seq + t), slot = __ldg(a.slot + t), pos = __ldg(a.pos + t);
        bool ok = seq >= 0 && seq < a.c.batch && slot >= 0 && slot < a.c.capacity &&
                  (a.rope_dim == 0 || (pos >= 0 && pos < a.n_pos)) && (!(a.weights || a.positions) || slot < a.ld_meta);
        int32_t page = -1;
        if (ok) page = __ldg(a.c.table + seq * a.c.ld_table + page_of(a.c, slot));
        ok = ok && page_ok(a.c, page);
        if (!ok) {
            atomicOr(a.c.status, kDevIndex);
            if (kind) continue;
        }
        const float *src;
        void *dst;
        bool e4m3 = false;
        float scale = 1.f;
        if (kind == 0) {
            src = a.q + t * a.ldq + (int64_t)head * D;
            dst = a.q_out + t * a.ldqo + (int64_t)head * D;
        } else {
            src = (kind == 1 ? a.k + t * a.ldk : a.v + t * a.ldv) + (int64_t)head * D;
            dst = (kind == 1 ? a.c.k : a.c.v) + row_bytes_at(a.c, page, head, (uint32_t)slot - page_of(a.c, slot) * a.c.page_size);
            e4m3 = a.c.e4m3 != 0;
            scale = kind == 1 ? k_inv : v_inv;
            if (kind == 1 && u == 0) {
                const int64_t at = ((int64_t)seq * a.c.heads + head) * a.ld_meta + slot;
                if (a.weights) a.weights[at] = 0.f;
                if (a.positions) a.positions[at] = pos;
            }
        }
        const bool turn = kind < 2 && ok;
        const float *cs = a.rope + (int64_t)pos * a.rope_dim;
        if constexpr (VEC) {
            alignas(16) float x[8];
            const bool in_rope = u < a.rope_dim / 8;
            const bool split = in_rope && !a.pairs;  // four values and their partners
            const int at0 = split ? 4 * u : 8 * u, at1 = split ? half + 4 * u : 8 * u + 4;
            *reinterpret_cast<float4 *>(x) = __ldg(reinterpret_cast<const float4 *>(src + at0));
            *reinterpret_cast<float4 *>(x + 4) = __ldg(reinterpret_cast<const float4 *>(src + at1));
            if (in_rope && turn) {
                // pairs 4 u .. 4 u + 3 either way
                const float4 c = __ldg(reinterpret_cast<const float4 *>(cs + 4 * u));
                const float4 s = __ldg(reinterpret_cast<const float4 *>(cs + half + 4 * u));
                if (split) {
                    rotate(x[0], x[4], c.x, s.x), rotate(x[1], x[5], c.y, s.y);
                    rotate(x[2], x[6], c.z, s.z), rotate(x[3], x[7], c.w, s.w);
                } else {
                    rotate(x[0], x[1], c.x, s.x), rotate(x[2], x[3], c.y, s.y);
                    rotate(x[4], x[5], c.z, s.z), rotate(x[6], x[7], c.w, s.w);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = ok ? x[i] * scale : 0.f;
            store4(dst, at0, x, e4m3);
            store4(dst, at1, x + 4, e4m3);
        } else {
            if (u < half) {
                const int i = a.pairs ? 2 * u : u, j = a.pairs ? 2 * u + 1 : u + half;
                float x = __ldg(src + i), y = __ldg(src + j);
                if (turn) rotate(x, y, __ldg(cs + u), __ldg(cs + half + u));
                store1(dst, i, ok ? x * scale : 0.f, e4m3);
                store1(dst, j, ok ? y * scale : 0.f, e4m3);
            } else {
                const int i = u + half;
                store1(dst, i, ok ? __ldg(src + i) * scale : 0.f, e4m3);
            }
        }
    }
}

bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

cudaError_t launch_kv_append(const DeviceInfo &di, const AppendArgs &a, cudaStream_t s) {
    const bool vec = (!a.q || (al16(a.q) && a.ldq % 4 == 0 && al16(a.q_out) && a.ldqo % 8 == 0)) && al16(a.k) &&
                     a.ldk % 4 == 0 && al16(a.v) && a.ldv % 4 == 0 && a.rope_dim % 8 == 0 && (a.rope_dim == 0 || al16(a.rope));
    const int D = a.c.dim, units = vec ? D / 8 : a.rope_dim / 2 + (D - a.rope_dim);
    const int64_t per_token = ((a.q ? a.n_heads : 0) + 2 * a.c.heads) * (int64_t)units;
    uint32_t l = 0;
    while (((int64_t)1 << l) < per_token) ++l;
    const uint32_t shift = 31 + l, mul = (uint32_t)((((uint64_t)1 << shift) + per_token - 1) / per_token);
    const float k_inv = 1.0f / a.c.k_scale, v_inv = 1.0f / a.c.v_scale;
    // tokens of a launch: fewer than 2^31 units (a call of that size takes several)
    const int64_t most = ((int64_t)1 << 30) / per_token;
    for (int64_t t0 = 0; t0 < a.T; t0 += most) {
        const int64_t all = (a.T - t0 < most ? a.T - t0 : most) * per_token;
        int64_t blocks = (all + kThreads - 1) / kThreads;
        const int64_t cap = (int64_t)di.sm_count * 64;
        if (blocks > cap) blocks = cap;
        const cudaError_t e = launch_pdl(vec ? append_kernel<true> : append_kernel<false>, dim3((unsigned)blocks), dim3(kThreads), 0, s, dim3(1),
                                         a, t0, (uint32_t)all, (uint32_t)per_token, mul, shift, (uint32_t)units, k_inv, v_inv);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace q4k
