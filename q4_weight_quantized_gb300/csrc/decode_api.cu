// C-ABI of the operators between a decode step's weight products: argument
// validation, workspace layout and dispatch.  Their contract is in include/q4k.h.
#include <cuda_runtime.h>

#include <cstring>
#include <type_traits>
#include <utility>

#include <cmath>

#include "decode_ops.h"
#include "q4k_api.h"

using namespace q4k;

namespace {

constexpr int64_t kInt31 = (int64_t)1 << 31;
size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }
bool scale_ok(float v) { return v > 0.f && std::isfinite(v); }

// The cache descriptor's sizes (no pointer is looked at).
bool cache_shape_ok(const q4k_kv_cache *c) {
    if (c->dtype != Q4K_KV_BF16 && c->dtype != Q4K_KV_E4M3) return false;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return false;
    if (c->batch < 1 || c->batch > 65535 || c->n_kv_heads < 1 || c->n_kv_heads > 1024 ||
        (int64_t)c->batch * c->n_kv_heads > (1 << 24))
        return false;
    if (c->page_size < 1 || c->max_pages < 1 || (int64_t)c->page_size * c->max_pages >= kInt31) return false;
    if (c->n_pages < 1 || c->n_pages >= kInt31 || c->ld_table < c->max_pages) return false;
    if (c->page_stride < 1 || c->head_stride < 1 || c->slot_stride < c->head_dim) return false;
    // the last value's byte must be addressable
    const double last = (double)c->n_pages * c->page_stride + (double)c->n_kv_heads * c->head_stride +
                        (double)c->page_size * c->slot_stride;
    return last < 4e18 && scale_ok(c->k_scale) && scale_ok(c->v_scale);
}

q4k_status cache_check(const q4k_kv_cache *c) {
    if (!c || !c->k || !c->v || !c->page_table) return Q4K_ERR_NULL;
    if (!cache_shape_ok(c)) return Q4K_ERR_SHAPE;
    const int64_t unit = c->dtype == Q4K_KV_E4M3 ? 16 : 8;  // elements of 16 bytes
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->page_table, 4) || c->page_stride % unit ||
        c->head_stride % unit || c->slot_stride % unit)
        return Q4K_ERR_ALIGN;
    return Q4K_OK;
}

KvView view(const q4k_kv_cache *c, const DeviceInfo &di) {
    const int64_t e = c->dtype == Q4K_KV_E4M3 ? 1 : 2;
    KvView v = {};
    v.k = static_cast<uint8_t *>(c->k);
    v.v = static_cast<uint8_t *>(c->v);
    v.table = c->page_table;
    v.ld_table = c->ld_table;
    v.page_bytes = c->page_stride * e;
    v.head_bytes = c->head_stride * e;
    v.slot_bytes = c->slot_stride * e;
    v.n_pages = c->n_pages;
    v.batch = c->batch;
    v.max_pages = c->max_pages;
    v.page_size = c->page_size;
    v.heads = c->n_kv_heads;
    v.capacity = c->max_pages * c->page_size;
    uint32_t l = 0;
    while (((uint64_t)1 << l) < (uint64_t)c->page_size) ++l;
    v.div_shift = 31 + l;
    v.div_mul = (uint32_t)((((uint64_t)1 << v.div_shift) + c->page_size - 1) / c->page_size);
    v.dim = c->head_dim;
    v.e4m3 = c->dtype == Q4K_KV_E4M3;
    v.k_scale = c->k_scale;
    v.v_scale = c->v_scale;
    v.status = di.status;
    return v;
}

// Argument of type T from 8 bytes.
template <typename T>
T argument(const char *slot) {
    if constexpr (std::is_floating_point<T>::value) {
        double v;
        std::memcpy(&v, slot, 8);
        return (T)v;
    } else {
        int64_t v;
        std::memcpy(&v, slot, 8);
        if constexpr (std::is_pointer<T>::value) return reinterpret_cast<T>(v);
        else return static_cast<T>(v);
    }
}
template <typename... Args, size_t... I>
q4k_status call_each(q4k_status (*f)(Args...), const char *slots, std::index_sequence<I...>) {
    return f(argument<Args>(slots + 8 * I)...);
}
template <typename... Args>
q4k_status call(q4k_status (*f)(Args...), const void *slots) {
    if (!slots) return Q4K_ERR_NULL;
    return call_each(f, static_cast<const char *>(slots), std::index_sequence_for<Args...>{});
}

q4k_status finish(cudaError_t e) { return e == cudaSuccess ? Q4K_OK : cuda_fail(e); }

bool attn_shape_ok(const q4k_kv_cache *c, int32_t n_heads, int32_t n_q, int64_t ld_weights) {
    if (!cache_shape_ok(c) || n_heads < 1 || n_heads % c->n_kv_heads || n_q < 1 || n_q > 64) return false;
    const int64_t rows = (int64_t)n_q * (n_heads / c->n_kv_heads);
    if (rows > kMaxAttnRows) return false;
    // the scores' bytes in the workspace
    if ((double)c->batch * c->n_kv_heads * (double)rows * (double)ld_weights * 4 > 4e18) return false;
    const int tile = attn_tile_rows(c->head_dim, (int)rows);
    const int64_t units = (int64_t)c->batch * c->n_kv_heads * ((rows + tile - 1) / tile);
    // blocks of the joining kernel; tiles times shares in 64 bits
    return units * (tile / 8) * (c->head_dim / 16) < kInt31;
}

struct AttnLayout {
    size_t parts, unit_ml, prefix, logits, total;
};
AttnLayout attn_layout(const q4k_kv_cache *c, int32_t n_heads, int32_t n_q, int64_t ld_weights) {
    const size_t rows = (size_t)n_q * (n_heads / c->n_kv_heads);
    const size_t tile = (size_t)attn_tile_rows(c->head_dim, (int)rows), units = (size_t)c->batch * c->n_kv_heads * ((rows + tile - 1) / tile);
    AttnLayout l;
    size_t at = 0;
    l.parts = at;
    at += align256((size_t)2 * kMaxAttnShares * attn_part_floats(c->head_dim, (int)tile) * 4);
    l.unit_ml = at;
    if (ld_weights > 0) at += align256(units * tile * sizeof(float2));
    l.prefix = at;
    at += align256(((size_t)c->batch + 1) * 8);
    l.logits = at;
    at += align256((size_t)c->batch * c->n_kv_heads * rows * (size_t)ld_weights * 4);
    l.total = at;
    return l;
}

// moves of a head: what is filled lies below budget, what fills it at or above
int64_t evict_max_moves(int64_t cap, int64_t budget) {
    const int64_t m = cap - budget < budget ? cap - budget : budget;
    return m > 0 ? m : 1;
}
int64_t evict_cap(const q4k_kv_cache *c, int64_t ld_meta) {
    const int64_t table = (int64_t)c->max_pages * c->page_size;
    return ld_meta < table ? ld_meta : table;
}

}  // namespace

extern "C" {

q4k_status q4k_kv_append(const q4k_kv_cache *cache, int64_t T, int32_t n_heads, const float *q, int64_t ldq,
                         const float *k, int64_t ldk, const float *v, int64_t ldv, const int32_t *seq,
                         const int32_t *slot, const int32_t *pos, const float *rope, int64_t n_pos, int32_t rope_dim,
                         int rope_mode, uint16_t *q_out, int64_t ldqo, float *weights, int32_t *positions,
                         int64_t ld_meta, void *stream) {
    q4k_status st = cache_check(cache);
    if (st != Q4K_OK) return st;
    if (!k || !v || !seq || !slot || !pos || (q != nullptr) != (q_out != nullptr) || (rope_dim > 0 && !rope))
        return Q4K_ERR_NULL;
    const int64_t row = (int64_t)cache->n_kv_heads * cache->head_dim;
    if (T < 1 || T >= kInt31 || ldk < row || ldv < row || rope_dim < 0 || rope_dim > cache->head_dim || rope_dim % 2 ||
        (rope_dim > 0 && (n_pos < 1 || n_pos > kInt31)) || (rope_mode != Q4K_ROPE_HALF && rope_mode != Q4K_ROPE_PAIRS))
        return Q4K_ERR_SHAPE;
    if (q && (n_heads < 1 || n_heads > 65536 || ldq < (int64_t)n_heads * cache->head_dim || ldqo < (int64_t)n_heads * cache->head_dim))
        return Q4K_ERR_SHAPE;
    if ((weights || positions) && ld_meta < 1) return Q4K_ERR_SHAPE;
    if (!aligned(q, 4) || !aligned(k, 4) || !aligned(v, 4) || !aligned(seq, 4) || !aligned(slot, 4) || !aligned(pos, 4) ||
        !aligned(rope, 4) || !aligned(q_out, 2) || !aligned(weights, 4) || !aligned(positions, 4))
        return Q4K_ERR_ALIGN;
    DeviceInfo di;
    if ((st = check_device(&di)) != Q4K_OK) return st;
    AppendArgs a = {};
    a.c = view(cache, di);
    a.T = T;
    a.q = q, a.k = k, a.v = v;
    a.ldq = ldq, a.ldk = ldk, a.ldv = ldv;
    a.seq = seq, a.slot = slot, a.pos = pos;
    a.rope = rope;
    a.n_pos = n_pos;
    a.n_heads = n_heads;
    a.rope_dim = rope_dim;
    a.pairs = rope_mode == Q4K_ROPE_PAIRS;
    a.q_out = q_out;
    a.ldqo = ldqo;
    a.weights = weights;
    a.positions = positions;
    a.ld_meta = ld_meta;
    return finish(launch_kv_append(di, a, static_cast<cudaStream_t>(stream)));
}

size_t q4k_attn_decode_workspace_size(const q4k_kv_cache *cache, int32_t n_heads, int32_t n_q, int64_t ld_weights) {
    if (!cache || ld_weights < 0 || ld_weights >= kInt31 || !attn_shape_ok(cache, n_heads, n_q, ld_weights)) return 0;
    return attn_layout(cache, n_heads, n_q, ld_weights).total;
}

q4k_status q4k_attn_decode(const q4k_kv_cache *cache, const int32_t *seq_lens, const uint16_t *q, int64_t ldq,
                           int32_t n_heads, int32_t n_q, float scale, float softcap, int64_t window, uint16_t *o,
                           int64_t ldo, float *weights, int64_t ld_weights, float decay, void *ws, size_t ws_bytes,
                           void *stream) {
    q4k_status st = cache_check(cache);
    if (st != Q4K_OK) return st;
    if (!seq_lens || !q || !o || !ws) return Q4K_ERR_NULL;
    if (!attn_shape_ok(cache, n_heads, n_q, weights ? ld_weights : 0) || ldq < (int64_t)n_heads * cache->head_dim ||
        ldo < (int64_t)n_heads * cache->head_dim || window < 0 || !std::isfinite(scale) || !(softcap >= 0.f) ||
        !std::isfinite(softcap))
        return Q4K_ERR_SHAPE;
    if (weights && (ld_weights < 1 || ld_weights >= kInt31 || !std::isfinite(decay))) return Q4K_ERR_SHAPE;
    if (!aligned(seq_lens, 4) || !aligned(q, 16) || !aligned(o, 16) || ldq % 8 || ldo % 8 || !aligned(weights, 4) ||
        !aligned(ws, 256))
        return Q4K_ERR_ALIGN;
    const AttnLayout l = attn_layout(cache, n_heads, n_q, weights ? ld_weights : 0);
    if (ws_bytes < l.total) return Q4K_ERR_WORKSPACE;
    DeviceInfo di;
    if ((st = check_device(&di)) != Q4K_OK) return st;
    uint8_t *base = static_cast<uint8_t *>(ws);
    AttnArgs a = {};
    a.c = view(cache, di);
    a.seq_lens = seq_lens;
    a.q = q, a.ldq = ldq, a.o = o, a.ldo = ldo;
    a.n_q = n_q;
    a.group = n_heads / cache->n_kv_heads;
    a.rows = n_q * a.group;
    a.tile_rows = attn_tile_rows(cache->head_dim, a.rows);
    a.row_tiles = (a.rows + a.tile_rows - 1) / a.tile_rows;
    a.unit_heads = cache->n_kv_heads * a.row_tiles;
    a.cap = weights && ld_weights < a.c.capacity ? (int32_t)ld_weights : a.c.capacity;
    a.window = window < kInt31 ? window : 0;  // no sequence is that long
    a.scale = scale * cache->k_scale;
    a.softcap = softcap;
    a.v_scale = cache->v_scale;
    a.decay = decay;
    a.weights = weights;
    a.ld_weights = ld_weights;
    a.logits = weights ? reinterpret_cast<float *>(base + l.logits) : nullptr;
    a.ld_logits = ld_weights;
    a.parts = reinterpret_cast<float *>(base + l.parts);
    a.unit_ml = weights ? reinterpret_cast<float2 *>(base + l.unit_ml) : nullptr;
    a.prefix = reinterpret_cast<int64_t *>(base + l.prefix);
    return finish(launch_attn_decode(di, a, static_cast<cudaStream_t>(stream)));
}

size_t q4k_kv_evict_workspace_size(const q4k_kv_cache *cache, int64_t ld_meta) {
    if (!cache || ld_meta < 1 || ld_meta >= kInt31 || !cache_shape_ok(cache)) return 0;
    const size_t bh = (size_t)cache->batch * cache->n_kv_heads;
    // whatever the budget: at most half of the slots move
    return align256(bh * 4) + align256(bh * ((size_t)evict_cap(cache, ld_meta) / 2 + 1) * sizeof(int2));
}

q4k_status q4k_kv_evict(const q4k_kv_cache *cache, const int32_t *seq_lens, int32_t *new_lens, int64_t budget,
                        int64_t sinks, int64_t recent, const float *weights, const int32_t *positions,
                        float *weights_out, int32_t *positions_out, int64_t ld_meta, void *ws, size_t ws_bytes,
                        void *stream) {
    q4k_status st = cache_check(cache);
    if (st != Q4K_OK) return st;
    if (!seq_lens || !new_lens || !weights || !positions || !weights_out || !positions_out || !ws) return Q4K_ERR_NULL;
    if (ld_meta < 1 || ld_meta >= kInt31 || budget < 1 || budget >= kInt31 || sinks < 0 || recent < 0 || sinks > budget ||
        recent > budget - sinks)
        return Q4K_ERR_SHAPE;
    if (!aligned(seq_lens, 4) || !aligned(new_lens, 4) || !aligned(weights, 4) || !aligned(positions, 4) ||
        !aligned(weights_out, 4) || !aligned(positions_out, 4) || !aligned(ws, 256))
        return Q4K_ERR_ALIGN;
    if (ws_bytes < q4k_kv_evict_workspace_size(cache, ld_meta)) return Q4K_ERR_WORKSPACE;
    DeviceInfo di;
    if ((st = check_device(&di)) != Q4K_OK) return st;
    EvictArgs a = {};
    a.c = view(cache, di);
    a.seq_lens = seq_lens;
    a.new_lens = new_lens;
    a.budget = (int32_t)budget;
    a.sinks = (int32_t)sinks;
    a.recent = (int32_t)recent;
    a.cap = (int32_t)evict_cap(cache, ld_meta);
    a.weights = weights;
    a.positions = positions;
    a.weights_out = weights_out;
    a.positions_out = positions_out;
    a.ld_meta = ld_meta;
    const size_t bh = (size_t)cache->batch * cache->n_kv_heads;
    a.count = static_cast<int32_t *>(ws);
    a.moves = reinterpret_cast<int2 *>(static_cast<uint8_t *>(ws) + align256(bh * 4));
    a.max_moves = evict_max_moves(a.cap, budget);
    return finish(launch_kv_evict(di, a, static_cast<cudaStream_t>(stream)));
}

q4k_status q4k_norm_residual(int64_t M, int64_t D, const float *y, int64_t ldy, int post, const float *post_w,
                             const float *post_b, float post_eps, const float *gate, int64_t ld_gate, float scale,
                             const void *r_in, void *r_out, int64_t ldr, int r_dtype, int pre, const float *pre_w,
                             const float *pre_b, float pre_eps, uint16_t *x, int64_t ldx, void *stream) {
    if (!r_in || (!r_out && !x)) return Q4K_ERR_NULL;
    auto kind_ok = [](int k) { return k == Q4K_NORM_NONE || k == Q4K_NORM_RMS || k == Q4K_NORM_LAYER; };
    if (M < 1 || M >= kInt31 || D < 1 || D > (1 << 20) || (y && ldy < D) || ldr < D || (x && ldx < D) ||
        (gate && ld_gate != 0 && ld_gate < D) || !kind_ok(post) || !kind_ok(pre) ||
        (r_dtype != Q4K_RES_FP32 && r_dtype != Q4K_RES_BF16) || !(post_eps >= 0.f) || !(pre_eps >= 0.f))
        return Q4K_ERR_SHAPE;
    const uintptr_t ra = r_dtype == Q4K_RES_FP32 ? 4 : 2;
    if (!aligned(y, 4) || !aligned(post_w, 4) || !aligned(post_b, 4) || !aligned(gate, 4) || !aligned(r_in, ra) ||
        !aligned(r_out, ra) || !aligned(pre_w, 4) || !aligned(pre_b, 4) || !aligned(x, 2))
        return Q4K_ERR_ALIGN;
    DeviceInfo di;
    q4k_status st = check_device(&di);
    if (st != Q4K_OK) return st;
    NormArgs a = {};
    a.M = M, a.D = D;
    a.y = y, a.ldy = ldy;
    a.post = post, a.post_w = post_w, a.post_b = post_b, a.post_eps = post_eps;
    a.gate = gate, a.ld_gate = ld_gate, a.scale = scale;
    a.r_in = r_in, a.r_out = r_out, a.ldr = ldr, a.bf16 = r_dtype == Q4K_RES_BF16;
    a.pre = pre, a.pre_w = pre_w, a.pre_b = pre_b, a.pre_eps = pre_eps;
    a.x = x, a.ldx = ldx;
    a.invariant = batch_invariant();
    a.wait_ns = wait_limit_ns();
    a.status = di.status;
    return finish(launch_norm_residual(di, a, static_cast<cudaStream_t>(stream)));
}

q4k_status q4k_sample(const float *logits, int64_t M, int64_t V, int64_t ldl, const float *temperature,
                      const int32_t *top_k, const float *top_p, const float *min_p, const float *u, int32_t *token,
                      float *prob, void *stream) {
    if (!logits || !u || !token) return Q4K_ERR_NULL;
    if (M < 1 || M > (1 << 24) || V < 1 || V > (1 << 22) || ldl < V) return Q4K_ERR_SHAPE;
    if (!aligned(logits, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) || !aligned(top_p, 4) || !aligned(min_p, 4) ||
        !aligned(u, 4) || !aligned(token, 4) || !aligned(prob, 4))
        return Q4K_ERR_ALIGN;
    DeviceInfo di;
    q4k_status st = check_device(&di);
    if (st != Q4K_OK) return st;
    SampleArgs a = {};
    a.logits = logits;
    a.M = M, a.ldl = ldl;
    a.V = (int32_t)V;
    a.temperature = temperature, a.top_k = top_k, a.top_p = top_p, a.min_p = min_p, a.u = u;
    a.token = token, a.prob = prob;
    return finish(launch_sample(di, a, static_cast<cudaStream_t>(stream)));
}

// What the Python package calls.
q4k_status q4k_kv_append_slots(const void *slots) { return call(q4k_kv_append, slots); }
q4k_status q4k_attn_decode_slots(const void *slots) { return call(q4k_attn_decode, slots); }
q4k_status q4k_kv_evict_slots(const void *slots) { return call(q4k_kv_evict, slots); }
q4k_status q4k_norm_residual_slots(const void *slots) { return call(q4k_norm_residual, slots); }
q4k_status q4k_sample_slots(const void *slots) { return call(q4k_sample, slots); }

}  // extern "C"
