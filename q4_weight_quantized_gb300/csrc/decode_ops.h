// Arguments and launchers of the operators between a decode step's weight products
// (attn_decode.cu, kv_append.cu, kv_evict.cu, norm.cu, sample.cu).  The C-ABI layer
// (decode_api.cu) has validated them.
#pragma once

#include "kv_cache.h"
#include "q4k_internal.h"

namespace q4k {

constexpr int kMaxAttnResident = 512;  // CTAs of an attention call that run at once, at most
constexpr int kMaxAttnShares = 3 * kMaxAttnResident;  // shares of its work (the workspace holds two parts for each)
constexpr int kMaxAttnRows = 1024;  // query rows of one KV head: n_q * group

struct AttnArgs {
    KvView c;
    const int32_t *seq_lens;
    const uint16_t *q;
    int64_t ldq;
    uint16_t *o;
    int64_t ldo;
    int32_t n_q, group, rows;        // rows = n_q * group, token-major
    int32_t tile_rows, row_tiles;    // rows of a row tile (attn_tile_rows), row tiles per KV head
    int32_t unit_heads;              // units per sequence = heads * row_tiles
    int32_t cap;                     // largest length: of the table, and of the weights if kept
    int64_t window;
    float scale, softcap;            // scale * k_scale
    float v_scale, decay;
    float *weights;
    int64_t ld_weights;
    // workspace
    float *logits;                   // [batch * heads][rows][ld_logits], with weights only
    int64_t ld_logits;
    float *parts;                    // [2 * shares] parts
    int32_t part_floats;
    float2 *unit_ml;                 // [batch * unit_heads][tile_rows]: (m, l) of units finished by one CTA; with weights only
    int64_t *prefix;                 // [batch + 1]: places of the list before each sequence
    int32_t resident;
};
int attn_tile_rows(int D, int rows);
int attn_part_floats(int D, int tile_rows);
cudaError_t launch_attn_decode(const DeviceInfo &di, AttnArgs &a, cudaStream_t s);

struct AppendArgs {
    KvView c;
    int64_t T;
    const float *q, *k, *v;
    int64_t ldq, ldk, ldv;
    const int32_t *seq, *slot, *pos;
    const float *rope;
    int64_t n_pos;
    int32_t n_heads, rope_dim, pairs;
    uint16_t *q_out;
    int64_t ldqo;
    float *weights;
    int32_t *positions;
    int64_t ld_meta;
};
cudaError_t launch_kv_append(const DeviceInfo &di, const AppendArgs &a, cudaStream_t s);

struct EvictArgs {
    KvView c;
    const int32_t *seq_lens;
    int32_t *new_lens;
    int32_t budget, sinks, recent, cap;
    const float *weights;
    const int32_t *positions;
    float *weights_out;
    int32_t *positions_out;
    int64_t ld_meta;
    // workspace
    int32_t *count;  // [batch * heads]: moves of each head
    int2 *moves;     // [batch * heads][max_moves]: slot to, slot from
    int64_t max_moves;
};
cudaError_t launch_kv_evict(const DeviceInfo &di, const EvictArgs &a, cudaStream_t s);

struct NormArgs {
    int64_t M, D;
    const float *y;
    int64_t ldy;
    int post;
    const float *post_w, *post_b;
    float post_eps;
    const float *gate;
    int64_t ld_gate;
    float scale;
    const void *r_in;
    void *r_out;
    int64_t ldr;
    int bf16;
    int pre;
    const float *pre_w, *pre_b;
    float pre_eps;
    uint16_t *x;
    int64_t ldx;
    int invariant;  // a row's bits must not depend on M
    unsigned long long wait_ns;  // limit of the ring's waits
    unsigned int *status;
};
cudaError_t launch_norm_residual(const DeviceInfo &di, const NormArgs &a, cudaStream_t s);

struct SampleArgs {
    const float *logits;
    int64_t M, ldl;
    int32_t V, ctas;  // ctas of a row: chosen by the launcher
    float one;        // 1: what no compiler knows (see the kernel)
    const float *temperature;
    const int32_t *top_k;
    const float *top_p, *min_p, *u;
    int32_t *token;
    float *prob;
};
cudaError_t launch_sample(const DeviceInfo &di, const SampleArgs &a, cudaStream_t s);

}  // namespace q4k
