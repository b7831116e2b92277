// kern_attn.cu -- attention of new tokens (one, a chain or a tree of drafts) over the
// quantised paged cache: which kernel serves a call, and its workspace.
#include "kernels.h"

namespace tl {

namespace {

// blocks resident per SM of the streaming kernel (its launch bounds and shared memory)
constexpr int kStreamBlocks = 3;

}  // namespace

int64_t tree_attention_workspace(int64_t, int64_t, int, int, int D) {
    // two slots per block: 16 rows of D, a maximum and a sum each
    return (int64_t)kMaxSms * kStreamBlocks * 2 * 16 * (D + 2) * 4;
}

cudaError_t launch_tree_attention(const AttnArgs &a, bool bf, int sm_count, cudaStream_t st) {
    const int nc = (sm_count < kMaxSms ? sm_count : kMaxSms) * kStreamBlocks;
    switch (a.c.fmt) {
    case 0: return launch_stream_int8(a, bf, nc, st);
    case 1: return launch_stream_fp8(a, bf, nc, st);
    default: return launch_stream_int4(a, bf, nc, st);
    }
}

}  // namespace tl
