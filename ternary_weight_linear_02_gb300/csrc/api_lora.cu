// api_lora.cu -- the C ABI of the low-rank adapters (declared in include/ternary_linear.h):
// argument validation, then the launch.
#include "api_util.h"

namespace {

using tl::aligned;

constexpr int64_t kMaxTokens = (int64_t)1 << 30, kMaxAdapters = 2048;

// The arguments checked and put in order.  *done: nothing is left to do.
tl_status args_of(const void *x, int64_t x_stride, const tl_adapters *ad, const int32_t *which, const void *y, int64_t y_stride,
                  void *out, int64_t out_stride, int32_t out_dtype, int64_t tokens, bool gated, tl::LoraArgs *to, bool *done) {
    *done = false;
    if (ad == nullptr) return TL_ERR_NULL;
    if (ad->dtype != TL_F16 && ad->dtype != TL_BF16) return TL_ERR_DTYPE;
    if (out_dtype != TL_F32 && out_dtype != ad->dtype) return TL_ERR_DTYPE;
    if (ad->adapters < 1 || ad->adapters > kMaxAdapters || ad->shards < 1 || ad->shards > tl::kMaxShards) return TL_ERR_SHAPE;
    if (ad->rank < 8 || ad->rank > 128 || ad->rank % 8 != 0) return TL_ERR_SHAPE;
    if (ad->inputs < 1 || ad->inputs > ((int64_t)1 << 24)) return TL_ERR_SHAPE;
    if (tokens < 0 || tokens >= kMaxTokens) return TL_ERR_SHAPE;
    if (!tl::stride_ok(x_stride) || !tl::stride_ok(y_stride) || !tl::stride_ok(out_stride)) return TL_ERR_SHAPE;
    tl::LoraArgs &a = *to;
    a = tl::LoraArgs{};
    const int size = out_dtype == TL_F32 ? 4 : 2;
    bool columns8 = true;  // threads' columns start on 16 bytes: 8 columns of 2 bytes, 4 of 4 (gated: 4)
    for (int i = 0; i < ad->shards; ++i) {
        const int64_t n = ad->shard_rows[i];
        if (n < 0 || n > ((int64_t)1 << 24)) return TL_ERR_SHAPE;
        columns8 = columns8 && n % 8 == 0;
        a.shard[i] = n;
        a.N += n;
    }
    if (gated && (ad->shards != 2 || a.shard[0] != a.shard[1])) return TL_ERR_SHAPE;
    *done = tokens == 0 || a.N == 0;
    if (*done) return TL_OK;
    if (!x || !ad->a || !ad->b || !which || !y || !out) return TL_ERR_NULL;
    if (!aligned(x, 2) || !aligned(ad->a, 16) || !aligned(ad->b, 16) || !aligned(ad->scale, 4) || !aligned(which, 4) ||
        !aligned(y, size) || !aligned(out, size))
        return TL_ERR_ALIGN;
    if (out == y && (gated || out_stride != y_stride)) return TL_ERR_VALUE;
    a.x = x;
    a.a = ad->a;
    a.b = ad->b;
    a.y = y;
    a.out = out;
    a.scale = ad->scale;
    a.which = which;
    a.xs = x_stride;
    a.ys = y_stride;
    a.os = out_stride;
    a.M = tokens;
    a.K = ad->inputs;
    a.S = ad->shards;
    a.R = ad->rank;
    a.adapters = ad->adapters;
    a.gated = gated;
    a.vec_x = a.K % 8 == 0 && aligned(x, 16) && x_stride % 8 == 0;
    a.vec_y = columns8 && aligned(y, 16) && aligned(out, 16) && y_stride * size % 16 == 0 && out_stride * size % 16 == 0;
    a.ranks = a.S * a.R;
    return TL_OK;
}

tl_status run(const void *x, int64_t x_stride, const tl_adapters *ad, const int32_t *which, const void *y, int64_t y_stride,
              void *out, int64_t out_stride, int32_t out_dtype, int64_t tokens, void *workspace, int64_t workspace_bytes,
              bool gated, void *stream) {
    tl::LoraArgs a;
    bool done;
    const tl_status s = args_of(x, x_stride, ad, which, y, y_stride, out, out_stride, out_dtype, tokens, gated, &a, &done);
    if (s != TL_OK || done) return s;
    if (!aligned(workspace, 16)) return TL_ERR_ALIGN;
    const int64_t need = tl::lora_workspace(tokens, ad->adapters);
    if (need > 0 && !workspace) return TL_ERR_NULL;
    if (workspace_bytes < need) return TL_ERR_SHAPE;
    tl::CallDevice d;
    if (const int e = tl::begin_call(&d)) return (tl_status)e;
    a.wait_limit = d.wait_limit;
    a.stall = d.stall;
    a.status = d.status;
    return tl::from_cuda(tl::launch_lora(a, ad->dtype, out_dtype == TL_F32, workspace, d.sm_count, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int64_t ternary_lora_workspace(int64_t tokens, int64_t adapters) {
    if (tokens < 0 || tokens >= kMaxTokens || adapters < 1 || adapters > kMaxAdapters) return -1;
    return tl::lora_workspace(tokens, adapters);
}

tl_status ternary_lora_add(const void *x, int64_t x_stride, const tl_adapters *adapters, const int32_t *which, const void *y,
                           int64_t y_stride, void *out, int64_t out_stride, int32_t out_dtype, int64_t tokens, void *workspace,
                           int64_t workspace_bytes, void *stream) {
    return run(x, x_stride, adapters, which, y, y_stride, out, out_stride, out_dtype, tokens, workspace, workspace_bytes, false,
               stream);
}

tl_status ternary_lora_silu_mul(const void *x, int64_t x_stride, const tl_adapters *adapters, const int32_t *which, const void *y,
                                int64_t y_stride, void *out, int64_t out_stride, int32_t out_dtype, int64_t tokens, void *workspace,
                                int64_t workspace_bytes, void *stream) {
    return run(x, x_stride, adapters, which, y, y_stride, out, out_stride, out_dtype, tokens, workspace, workspace_bytes, true,
               stream);
}

int32_t ternary_test_lora_tile(const void *x, int64_t x_stride, const tl_adapters *adapters, const int32_t *which, const void *y,
                               int64_t y_stride, void *out, int64_t out_stride, int32_t out_dtype, int64_t tokens, int32_t gated) {
    tl::LoraArgs a;
    bool done;
    if (args_of(x, x_stride, adapters, which, y, y_stride, out, out_stride, out_dtype, tokens, gated != 0, &a, &done) != TL_OK) return -1;
    return done ? 0 : tl::lora_tile(a, out_dtype == TL_F32);
}

}  // extern "C"
