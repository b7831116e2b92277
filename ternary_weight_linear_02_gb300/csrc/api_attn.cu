// api_attn.cu -- the C ABI of the rotary, cache and attention calls (declared in
// include/ternary_linear.h): argument validation, then one launch function each.
#include <cmath>

#include "kernels.h"
#include "ternary_linear.h"

namespace {

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

tl_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return TL_OK;
    cudaGetLastError();
    return TL_ERR_CUDA;
}

// A strided [tokens, heads, D] tensor (or its leading axes): element alignment is
// required, and `rows16` reports whether every row starts on a 16-byte boundary.
// Offsets stay far inside 63 bits: |stride| < 2^40, axis < 2^31 in any use.
bool stride_ok(int64_t s) { return s > -((int64_t)1 << 40) && s < ((int64_t)1 << 40); }
bool rows16(const void *p, int64_t s0, int64_t s1, int size) {
    return aligned(p, 16) && (s0 * size) % 16 == 0 && (s1 * size) % 16 == 0;
}

tl_status check_cache(const tl_kv_cache *c, tl::KvCache *out) {
    if (c == nullptr) return TL_ERR_NULL;
    if (c->format != TL_KV_INT8 && c->format != TL_KV_FP8 && c->format != TL_KV_INT4) return TL_ERR_DTYPE;
    if (c->head_dim != 64 && c->head_dim != 128) return TL_ERR_SHAPE;
    if (c->page_size < 16 || c->page_size % 16 != 0 || c->page_size > (1 << 20)) return TL_ERR_SHAPE;
    if (c->kv_heads < 1 || c->kv_heads > (1 << 16)) return TL_ERR_SHAPE;
    if (c->pages < 1 || c->pages >= ((int64_t)1 << 31)) return TL_ERR_SHAPE;
    // groups of 16 places are counted in 32 bits (2^36 places: beyond any memory)
    if (c->pages > ((int64_t)1 << 32) / ((int64_t)c->kv_heads * (c->page_size / 16))) return TL_ERR_SHAPE;
    if (!c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale) return TL_ERR_NULL;
    if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scale, 16) ||
        !aligned(c->v_scale, 16))
        return TL_ERR_ALIGN;
    out->kc = static_cast<uint8_t *>(c->k_codes);
    out->vc = static_cast<uint8_t *>(c->v_codes);
    out->ks = c->k_scale;
    out->vs = c->v_scale;
    out->pages = c->pages;
    out->P = c->page_size;
    out->Hk = c->kv_heads;
    out->D = c->head_dim;
    out->fmt = c->format;
    return TL_OK;
}

constexpr int64_t kMaxTokens = (int64_t)1 << 31;
// keys of a sequence: counts of whole tiles (up to 128 keys) and places in them fit 31 bits
constexpr int64_t kMaxKeys = kMaxTokens - 256;

}  // namespace

extern "C" {

tl_status ternary_rope_table(float *table, int64_t positions, int32_t rotary_dim, double base,
                             double factor, double original_len, double ramp_lo, double ramp_hi,
                             double magnitude, void *stream) {
    if (positions < 0 || positions >= kMaxTokens) return TL_ERR_SHAPE;
    if (rotary_dim < 2 || rotary_dim % 2 != 0 || rotary_dim > 1024) return TL_ERR_SHAPE;
    if (!(base > 0) || !(factor > 0) || !std::isfinite(base) || !std::isfinite(factor) ||
        !std::isfinite(original_len) || !std::isfinite(ramp_lo) || !std::isfinite(ramp_hi) ||
        !std::isfinite(magnitude))
        return TL_ERR_VALUE;
    if (positions == 0) return TL_OK;
    if (table == nullptr) return TL_ERR_NULL;
    if (!aligned(table, 16)) return TL_ERR_ALIGN;
    tl::CallDevice d;
    if (const int s = tl::begin_call(&d)) return (tl_status)s;
    tl::RopeTableArgs a{table, positions, rotary_dim, base, factor, original_len, ramp_lo, ramp_hi, magnitude};
    return from_cuda(tl::launch_rope_table(a, reinterpret_cast<cudaStream_t>(stream)));
}

tl_status ternary_rope(const void *x, int64_t x_token_stride, int64_t x_head_stride, void *out,
                       int64_t out_token_stride, int64_t out_head_stride, int32_t dtype,
                       int64_t tokens, int32_t heads, int32_t head_dim, const int64_t *positions,
                       const float *table, int64_t table_rows, int32_t rotary_dim, uint32_t flags,
                       void *stream) {
    if (dtype != TL_F16 && dtype != TL_BF16 && dtype != TL_F32) return TL_ERR_DTYPE;
    if (flags & ~(uint32_t)(TL_ROPE_INTERLEAVED | TL_ROPE_INVERSE)) return TL_ERR_DTYPE;
    if (tokens < 0 || tokens >= kMaxTokens || heads < 0 || heads > (1 << 16)) return TL_ERR_SHAPE;
    if (head_dim < 2 || head_dim > 1024) return TL_ERR_SHAPE;
    if (rotary_dim < 2 || rotary_dim % 2 != 0 || rotary_dim > head_dim) return TL_ERR_SHAPE;
    if (table_rows < 0) return TL_ERR_SHAPE;
    if (!stride_ok(x_token_stride) || !stride_ok(x_head_stride) || !stride_ok(out_token_stride) ||
        !stride_ok(out_head_stride))
        return TL_ERR_SHAPE;
    if (tokens == 0 || heads == 0) return TL_OK;
    if (!x || !out || !positions || !table) return TL_ERR_NULL;
    const int size = dtype == TL_F32 ? 4 : 2;
    if (!aligned(x, size) || !aligned(out, size) || !aligned(positions, 8) || !aligned(table, 16))
        return TL_ERR_ALIGN;
    tl::CallDevice d;
    if (const int s = tl::begin_call(&d)) return (tl_status)s;
    tl::RopeArgs a{};
    a.x = x;
    a.out = out;
    a.xt = x_token_stride;
    a.xh = x_head_stride;
    a.ot = out_token_stride;
    a.oh = out_head_stride;
    a.positions = positions;
    a.table = table;
    a.table_rows = table_rows;
    a.tokens = tokens;
    a.heads = heads;
    a.D = head_dim;
    a.R = rotary_dim;
    a.inverse = (flags & TL_ROPE_INVERSE) ? 1 : 0;
    a.status = d.status;
    const bool vec = head_dim % 16 == 0 && rotary_dim % 16 == 0 && rows16(x, x_token_stride, x_head_stride, size) &&
                     rows16(out, out_token_stride, out_head_stride, size);
    return from_cuda(tl::launch_rope(a, dtype, (flags & TL_ROPE_INTERLEAVED) != 0, vec, d.sm_count,
                                     reinterpret_cast<cudaStream_t>(stream)));
}

tl_status ternary_kv_append(const tl_kv_cache *cache, const void *k, int64_t k_token_stride,
                            int64_t k_head_stride, const void *v, int64_t v_token_stride,
                            int64_t v_head_stride, int32_t dtype, int64_t tokens,
                            const int64_t *slots, const void *q, int64_t q_token_stride,
                            int64_t q_head_stride, void *q_out, int64_t q_out_token_stride,
                            int64_t q_out_head_stride, int32_t q_heads, const int64_t *positions,
                            const float *table, int64_t table_rows, int32_t rotary_dim,
                            uint32_t flags, void *stream) {
    tl::KvAppendArgs a{};
    if (const tl_status s = check_cache(cache, &a.c)) return s;
    if (dtype != TL_F16 && dtype != TL_BF16) return TL_ERR_DTYPE;
    if (flags & ~(uint32_t)TL_ROPE_INTERLEAVED) return TL_ERR_DTYPE;
    if (tokens < 0 || tokens >= kMaxTokens || q_heads < 0 || q_heads > (1 << 16)) return TL_ERR_SHAPE;
    if (table && (rotary_dim < 16 || rotary_dim % 16 != 0 || rotary_dim > a.c.D || table_rows < 0))
        return TL_ERR_SHAPE;
    if (!table && flags) return TL_ERR_DTYPE;
    if (!stride_ok(k_token_stride) || !stride_ok(k_head_stride) || !stride_ok(v_token_stride) ||
        !stride_ok(v_head_stride))
        return TL_ERR_SHAPE;
    const bool has_q = q != nullptr && q_heads > 0;
    if (has_q && (!stride_ok(q_token_stride) || !stride_ok(q_head_stride) || !stride_ok(q_out_token_stride) ||
                  !stride_ok(q_out_head_stride)))
        return TL_ERR_SHAPE;
    if (tokens == 0) return TL_OK;
    if (!k || !v || !slots) return TL_ERR_NULL;
    if (table && !positions) return TL_ERR_NULL;
    if (has_q && (!q_out || !table)) return TL_ERR_NULL;
    if (!aligned(k, 2) || !aligned(v, 2) || !aligned(slots, 8)) return TL_ERR_ALIGN;
    if (has_q && (!aligned(q, 2) || !aligned(q_out, 2))) return TL_ERR_ALIGN;
    if (table && (!aligned(table, 16) || !aligned(positions, 8))) return TL_ERR_ALIGN;
    tl::CallDevice d;
    if (const int s = tl::begin_call(&d)) return (tl_status)s;
    a.k = k;
    a.v = v;
    a.kt = k_token_stride;
    a.kh = k_head_stride;
    a.vt = v_token_stride;
    a.vh = v_head_stride;
    a.slots = slots;
    a.tokens = tokens;
    a.status = d.status;
    bool vec = rows16(k, k_token_stride, k_head_stride, 2) && rows16(v, v_token_stride, v_head_stride, 2);
    if (has_q) {
        a.q = q;
        a.qo = q_out;
        a.qt = q_token_stride;
        a.qh = q_head_stride;
        a.qot = q_out_token_stride;
        a.qoh = q_out_head_stride;
        a.Hq = q_heads;
        vec = vec && rows16(q, q_token_stride, q_head_stride, 2) &&
              rows16(q_out, q_out_token_stride, q_out_head_stride, 2);
    }
    if (table) {
        a.positions = positions;
        a.table = table;
        a.table_rows = table_rows;
        a.R = rotary_dim;
    }
    return from_cuda(tl::launch_kv_append(a, dtype == TL_BF16, (flags & TL_ROPE_INTERLEAVED) != 0, vec,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

tl_status ternary_kv_read(const tl_kv_cache *cache, const int64_t *slots, int64_t tokens, void *k,
                          void *v, int32_t out_dtype, void *stream) {
    tl::KvReadArgs a{};
    if (const tl_status s = check_cache(cache, &a.c)) return s;
    if (out_dtype != TL_F16 && out_dtype != TL_BF16 && out_dtype != TL_F32) return TL_ERR_DTYPE;
    if (tokens < 0 || tokens >= kMaxTokens) return TL_ERR_SHAPE;
    if (tokens == 0 || (!k && !v)) return TL_OK;
    if (!slots) return TL_ERR_NULL;
    if (!aligned(slots, 8) || !aligned(k, 16) || !aligned(v, 16)) return TL_ERR_ALIGN;
    tl::CallDevice d;
    if (const int s = tl::begin_call(&d)) return (tl_status)s;
    a.slots = slots;
    a.tokens = tokens;
    a.k = k;
    a.v = v;
    a.status = d.status;
    return from_cuda(tl::launch_kv_read(a, out_dtype, reinterpret_cast<cudaStream_t>(stream)));
}

static bool attention_sizes(int64_t batch, int64_t draft, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
    if (batch < 0 || batch > (1 << 16) || draft < 0 || draft > (1 << 16)) return false;
    if (kv_heads < 1 || kv_heads > (1 << 16) || q_heads < 1 || q_heads > (1 << 16) || q_heads % kv_heads != 0)
        return false;
    if (head_dim != 64 && head_dim != 128) return false;
    // rows, rounded up to whole row blocks, are counted in 31 bits
    return batch * kv_heads * (draft * (q_heads / kv_heads) + 128) < kMaxTokens;
}

int64_t ternary_tree_attention_workspace(int64_t batch, int64_t draft, int32_t q_heads,
                                         int32_t kv_heads, int32_t head_dim, int64_t max_keys) {
    if (!attention_sizes(batch, draft, q_heads, kv_heads, head_dim) || max_keys < 0 || max_keys > kMaxKeys) return -1;
    if (batch == 0 || draft == 0) return 0;
    return tl::tree_attention_workspace(batch, draft, q_heads, kv_heads, head_dim, max_keys);
}

tl_status ternary_tree_attention(const void *q, int64_t q_batch_stride, int64_t q_token_stride,
                                 int64_t q_head_stride, int32_t dtype, int64_t batch,
                                 int64_t draft, int32_t q_heads, const tl_kv_cache *cache,
                                 const int32_t *page_table, int64_t page_table_stride,
                                 int64_t max_pages, const int32_t *context_len,
                                 const uint8_t *tree, int64_t tree_batch_stride,
                                 int64_t tree_row_stride, float scale, void *out, float *lse,
                                 void *workspace, int64_t workspace_bytes, void *stream) {
    tl::AttnArgs a{};
    if (const tl_status s = check_cache(cache, &a.c)) return s;
    if (dtype != TL_F16 && dtype != TL_BF16) return TL_ERR_DTYPE;
    if (!attention_sizes(batch, draft, q_heads, a.c.Hk, a.c.D)) return TL_ERR_SHAPE;
    if (!(scale > 0.f) || !std::isfinite(scale)) return TL_ERR_VALUE;
    if (!stride_ok(q_batch_stride) || !stride_ok(q_token_stride) || !stride_ok(q_head_stride) ||
        !stride_ok(page_table_stride) || !stride_ok(tree_batch_stride) || !stride_ok(tree_row_stride))
        return TL_ERR_SHAPE;
    // a sequence's page-table row holds the new tokens at least (below)
    if (max_pages < 0 || max_pages > kMaxKeys / a.c.P) return TL_ERR_SHAPE;
    if (batch == 0 || draft == 0) return TL_OK;
    if (max_pages * a.c.P < draft) return TL_ERR_SHAPE;
    if (!q || !page_table || !context_len || !out) return TL_ERR_NULL;
    if (!aligned(q, 2) || !aligned(out, 16) || !aligned(page_table, 4) || !aligned(context_len, 4) ||
        !aligned(lse, 4))
        return TL_ERR_ALIGN;
    const int64_t need = tl::tree_attention_workspace(batch, draft, q_heads, a.c.Hk, a.c.D, max_pages * a.c.P);
    if (need > 0 && !workspace) return TL_ERR_NULL;
    if (!aligned(workspace, 16)) return TL_ERR_ALIGN;
    if (workspace_bytes < need) return TL_ERR_SHAPE;
    tl::CallDevice d;
    if (const int s = tl::begin_call(&d)) return (tl_status)s;
    a.q = q;
    a.qb = q_batch_stride;
    a.qt = q_token_stride;
    a.qh = q_head_stride;
    a.pages = page_table;
    a.pages_stride = page_table_stride;
    a.max_keys = max_pages * a.c.P;
    a.ctx = context_len;
    a.tree = tree;
    a.tree_b = tree_batch_stride;
    a.tree_r = tree_row_stride;
    a.scale = scale;
    a.out = out;
    a.lse = lse;
    a.ws = static_cast<float *>(workspace);
    a.B = (int)batch;
    a.T = (int)draft;
    a.Hq = q_heads;
    a.G = q_heads / a.c.Hk;
    a.q_vec = rows16(q, q_token_stride, q_head_stride, 2) && (q_batch_stride * 2) % 16 == 0;
    a.status = d.status;
    a.wait_limit = d.wait_limit;
    a.stall = d.stall;
    a.bf = dtype == TL_BF16;
    return from_cuda(tl::launch_tree_attention(a, d.sm_count, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
