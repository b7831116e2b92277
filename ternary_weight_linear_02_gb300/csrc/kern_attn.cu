// kern_attn.cu -- attention of new tokens (one, a chain or a tree of drafts) over the
// quantised paged cache: which kernel serves a call, and its workspace.
#include "kernels.h"

namespace tl {

namespace {

// Rows of a kv head (new tokens x query heads that share it): up to 16 the streaming kernel,
// whose warp MMAs keep up with the cache's bytes (6 sequences of up to 4099 keys, 32 heads,
// int4: 78 us at 16 rows against 106 us); above, it would need more registers than a
// thread has or read the cache twice, and the tcgen05 kernel takes 128 rows at a time
// (106 us at 25 rows, against 125 us of a three-block streaming form at 24).
constexpr int64_t kStreamMaxRows = 16;
bool use_tile(int64_t rows) { return rows > kStreamMaxRows; }

}  // namespace

// Two slots per block (attn_sched.cuh): rows of D, a maximum and a sum each.
int64_t tree_attention_workspace(int64_t, int64_t T, int Hq, int Hk, int D) {
    const int64_t rows = T * (Hq / Hk);
    const int64_t blocks = use_tile(rows) ? 2 : 3, slot = use_tile(rows) ? 128 : rows <= 8 ? 8 : 16;
    return kMaxSms * blocks * 2 * slot * (D + 2) * 4;
}

cudaError_t launch_tree_attention(const AttnArgs &a, int sm_count, cudaStream_t st) {
    const int sms = sm_count < kMaxSms ? sm_count : kMaxSms;
    const bool tile = use_tile((int64_t)a.T * a.G);
    switch (a.c.fmt) {
    case 0: return launch_attn_int8(a, tile, sms, st);
    case 1: return launch_attn_fp8(a, tile, sms, st);
    default: return launch_attn_int4(a, tile, sms, st);
    }
}

}  // namespace tl
