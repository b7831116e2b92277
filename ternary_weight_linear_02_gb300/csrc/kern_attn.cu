// kern_attn.cu -- attention of new tokens (one, a chain or a tree of drafts) over the
// quantised paged cache: which kernel serves a call, and its workspace.
#include "kernels.h"

namespace tl {

namespace {

// Rows of a kv head (new tokens x query heads that share it): up to 16 the streaming kernel,
// whose warp MMAs keep up with the cache's bytes.  Streaming against tcgen05, 32 heads, int4:
// 6 sequences of up to 4099 keys, 9 rows 69 / 72 us, 16 rows 73 / 74; one, 13 rows 26 / 30;
// 32 of up to 300 keys, 12 rows 47 / 67.  Above, it would need more registers than a thread
// has or read the cache twice (24 rows in three blocks of 8: 125 us), and the tcgen05 kernel
// takes 128 rows at a time (24 rows: 75 us).
constexpr int64_t kStreamMaxRows = 16;
bool use_tile(int64_t rows) { return rows > kStreamMaxRows; }

// A block per unit, or runs of tiles dealt to as many blocks as fit the GPU?  Times in us,
// fitted to both forms over contexts of 50 to 20000 keys: beginning and ending a unit,
// a tile (with the blocks per SM that run at once), and what dealing costs beside (finding
// the run, partial results, the join and its launch).  The lengths are not known here: the
// page table's width stands for them.  A unit per block against dealt, in us:
//   one token, 28 heads on 4, fp8: 32 sequences of 100 keys 6.5 / 10.4, of 1000 17.5 / 18.3;
//   one of 1000 16.5 / 9.3, of 20000 205 / 19; int8, 64 of up to 8192 118 / 91, and with 28
//   kv heads 527 / 547;
//   trees: 8 of 64, 500 keys, 28 on 4 34 / 47; 6 of 23, 32 heads, int4, 500 keys 27 / 31,
//   4099 keys 122 / 74.
bool use_direct(int64_t B, int64_t T, int Hq, int Hk, int64_t max_keys) {
    const int64_t rows = T * (Hq / Hk);
    const bool tile = use_tile(rows);
    const int64_t keys = tile ? 64 : rows <= 8 ? 128 : 64, rtiles = tile ? (rows + 127) / 128 : 1;
    const double tiles = (double)((max_keys + keys - 1) / keys), units = (double)(B * Hk * rtiles);
    const double slots = 152.0 * (tile ? 2 : 3), ends = tile ? 7.0 : 4.0, step = tile ? 1.5 : keys == 128 ? 1.3 : 1.1;
    const double waves = (double)(int64_t)((units + slots - 1) / slots);
    const double whole = waves * (ends + step * tiles);
    const double dealt = (units * tiles < slots ? step : units * tiles / slots * step) + units / slots * ends + (tile ? 14.0 : 9.0);
    return whole <= dealt;
}

}  // namespace

// Two slots per block (attn_sched.cuh): rows of D, a maximum and a sum each.
int64_t tree_attention_workspace(int64_t B, int64_t T, int Hq, int Hk, int D, int64_t max_keys) {
    if (use_direct(B, T, Hq, Hk, max_keys)) return 0;
    const int64_t rows = T * (Hq / Hk);
    const int64_t blocks = use_tile(rows) ? 2 : 3, slot = use_tile(rows) ? 128 : rows <= 8 ? 8 : 16;
    return kMaxSms * blocks * 2 * slot * (D + 2) * 4;
}

cudaError_t launch_tree_attention(const AttnArgs &args, int sm_count, cudaStream_t st) {
    AttnArgs a = args;
    a.direct = use_direct(a.B, a.T, a.Hq, a.c.Hk, a.max_keys);
    const int sms = sm_count < kMaxSms ? sm_count : kMaxSms;
    const bool tile = use_tile((int64_t)a.T * a.G);
    switch (a.c.fmt) {
    case 0: return launch_attn_int8(a, tile, sms, st);
    case 1: return launch_attn_fp8(a, tile, sms, st);
    default: return launch_attn_int4(a, tile, sms, st);
    }
}

}  // namespace tl
