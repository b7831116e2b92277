// api_verify.cu -- the C ABI of the verification of drafted tokens (declared in
// include/ternary_linear.h): argument validation, then the launch.
#include "api_util.h"

extern "C" tl_status ternary_verify_drafts(const void *target, int64_t target_batch_stride,
                                           int64_t target_node_stride, const void *draft_probs,
                                           int64_t draft_batch_stride, int64_t draft_node_stride,
                                           int32_t dtype, const int64_t *tokens, int64_t tokens_stride,
                                           const int32_t *parent, int64_t parent_stride,
                                           const float *uniform, int64_t uniform_stride, int64_t batch,
                                           int64_t draft, int64_t vocab, int32_t *path, int32_t *count,
                                           int64_t *out_tokens, void *stream) {
    using tl::aligned;
    if (dtype != TL_F16 && dtype != TL_BF16 && dtype != TL_F32) return TL_ERR_DTYPE;
    if (batch < 0 || batch > (1 << 16) || draft < 0 || draft > tl::kMaxDraft) return TL_ERR_SHAPE;
    // a block's run of tokens is rounded up to 256 in 31 bits
    if (vocab < 1 || vocab > ((int64_t)1 << 31) - (1 << 12)) return TL_ERR_SHAPE;
    for (const int64_t s : {target_batch_stride, target_node_stride, draft_batch_stride, draft_node_stride, tokens_stride,
                            parent_stride, uniform_stride})
        if (!tl::stride_ok(s)) return TL_ERR_SHAPE;
    if (batch == 0) return TL_OK;
    if (!target || !uniform || !count || !out_tokens) return TL_ERR_NULL;
    if (draft > 0 && (!tokens || !path)) return TL_ERR_NULL;
    const int size = dtype == TL_F32 ? 4 : 2;
    if (!aligned(target, size) || !aligned(draft_probs, size) || !aligned(tokens, 8) || !aligned(parent, 4) ||
        !aligned(uniform, 4) || !aligned(path, 4) || !aligned(count, 4) || !aligned(out_tokens, 8))
        return TL_ERR_ALIGN;
    tl::CallDevice d;
    if (const int s = tl::begin_call(&d)) return (tl_status)s;
    tl::VerifyArgs a{};
    a.target = target;
    a.target_b = target_batch_stride;
    a.target_n = target_node_stride;
    a.draft = draft > 0 ? draft_probs : nullptr;
    a.draft_b = draft_batch_stride;
    a.draft_n = draft_node_stride;
    a.tokens = tokens;
    a.tokens_b = tokens_stride;
    a.parent = parent;
    a.parent_b = parent_stride;
    a.uniform = uniform;
    a.uniform_b = uniform_stride;
    a.path = path;
    a.count = count;
    a.out = out_tokens;
    a.B = batch;
    a.T = (int)draft;
    a.V = (int)vocab;
    a.status = d.status;
    const auto rows16 = [&](const void *p, int64_t s0, int64_t s1) {
        return aligned(p, 16) && s0 * size % 16 == 0 && s1 * size % 16 == 0;
    };
    const bool vec = rows16(target, target_batch_stride, target_node_stride) &&
                     (!a.draft || rows16(draft_probs, draft_batch_stride, draft_node_stride));
    return tl::from_cuda(tl::launch_verify(a, dtype, vec, d.sm_count, reinterpret_cast<cudaStream_t>(stream)));
}
