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
    int8_t *q;     // 8-bit output with its scales, or null
    float *q_scale;
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

struct PlanArgs {
    KvView c;
    int32_t *table;  // c.table, to write
    const int32_t *seq_lens, *n_new, *first_pos, *held, *free_count;
    int32_t *held_out, *free_pages, *count_out;
    int64_t T;
    int32_t *after_lens, *starts, *seq, *slot, *pos;
    // workspace
    int32_t *back_at, *take_at;  // [batch + 1]: pages returned and taken before each request
    int32_t *list;               // [2]: length of the free list before the call, and with the pages returned
};
cudaError_t launch_batch_plan(const DeviceInfo &di, const PlanArgs &a, cudaStream_t s);

constexpr int kMaxChunkShares = 160;  // CTAs of an attention call over chunks, at most (the workspace holds two parts for each)
// (api.cu; made anew on each call, none is kept)
bool make_cache_tmap(CUtensorMap *m, const void *pool, const KvView &c, int box_values, int box_slots, bool swizzle, bool *head_first);

// A unit of rows (chunk_rows() of them at most) of a sequence, the same for every KV head.
struct alignas(16) ChunkRecord {
    int32_t b, q0, e0;          // sequence, its first row in q and o, the end of its first new token's slots
    int32_t row0, rows;         // rows within the sequence
    int32_t begin, end;         // slots that any row sees: [begin, end)
    int32_t base, tiles;        // its tiles of slots: the first, their number
    int32_t all_end, all_begin; // every row sees slots below all_end, and from all_begin on
    int32_t pad;
};
struct ChunkArgs {
    KvView c;
    const int32_t *starts, *seq_lens;
    const uint16_t *q;
    int64_t T, ldq;
    uint16_t *o;
    int64_t ldo;
    int32_t group;
    int64_t window;
    float scale_log2;             // |scale| * k_scale * log2(e)
    int32_t odd_scale;            // a scale that is not positive: scores times score_sign first
    float score_sign;
    uint32_t group_mul, group_shift;  // row / group for 0 <= row < 2^31 (see KvView)
    float softcap, cap_in;        // and 2 / softcap
    float cc_max;                 // a score's factor, at most: cap_in times it is finite
    int32_t large_cap;            // a cap beside which scores may be very small,
    float cap_t;                  // and ln 2 / softcap
    float v_scale;
    int32_t shares;
    int32_t box_slots;            // slots of a tensor copy's box: what divides a page, up to 32; 0: none can be made
    int32_t head_first;           // see make_cache_tmap
    // workspace
    int32_t *seq_at, *rt_at;      // [batch + 1]: first row of each sequence, row tiles before it (of many sequences)
    ChunkRecord *records;         // [row tiles]
    int64_t *place_at;            // [row tiles + 1]: places of the list before each row tile, of one KV head
    int64_t *head;                // places, row tiles, shares
    int4 *joins;                  // [shares]: row tile, KV head and number of parts of the unit that a share begins and does not end
    float *parts;                 // [2 * shares][rows][D]
    float2 *part_ml;              // [2 * shares][rows]
};
int chunk_rows(int D);            // rows of a row tile
cudaError_t launch_attn_chunk(const DeviceInfo &di, ChunkArgs &a, cudaStream_t s);

constexpr int kLoraSmall = 192;  // tokens of a call whose CTAs find their adapters' tokens themselves
struct LoraArgs {
    int32_t n_adapters, R;
    int64_t N, K;
    const uint16_t *a, *b;
    const int32_t *ranks;
    const float *scales;
    const int32_t *ids;
    const uint16_t *x;
    int64_t T, ldx;
    float *y;
    int64_t ldy;
    unsigned int *status;
    int32_t k_chunk;             // of the K axis, a CTA's
    // workspace
    float *v;                    // [T][R]: the inner sums
    int32_t *offsets, *perm;     // more than kLoraSmall tokens: sorted by adapter (else null)
    int4 *tiles;
    int *n_tiles;
};
cudaError_t launch_lora_add(const DeviceInfo &di, LoraArgs &a, cudaStream_t s);

}  // namespace q4k
