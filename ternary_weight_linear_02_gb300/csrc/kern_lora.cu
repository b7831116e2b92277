// kern_lora.cu -- low-rank adapters: which tiles, and how they are dealt (the kernel is in
// kern_lora.cuh).
#include <climits>

#include "kern_lora.cuh"

namespace tl {

namespace {

// Lanes of one key count together, since runs of tokens would queue up at one address: the lanes of this lane's
// key, and the count of the key before this lane's (negative keys are not counted).
__device__ __forceinline__ uint32_t same_key(int key) { return __match_any_sync(0xffffffffu, key); }
__device__ __forceinline__ int count_key(int *counts, int key, uint32_t same) {
    const int lane = threadIdx.x & 31, leader = __ffs(same) - 1;
    int base = 0;
    if (lane == leader && key >= 0) base = atomicAdd(&counts[key], __popc(same));
    return __shfl_sync(0xffffffffu, base, leader) + __popc(same & ((1u << lane) - 1u));
}

// Tokens sorted by adapter and cut into tiles of TM, for more tokens or adapters than each block
// looks through by itself.  plan: [0] tiles, from 4 on (adapter, first, tokens) of each, then the
// sorted tokens.  Where a token lies within its adapter's run hangs on the order of atomics,
// what is computed for it does not: rows of a tile do not meet.
__global__ void __launch_bounds__(1024) lora_plan_kernel(LoraArgs a, int TM, int *plan) {
    extern __shared__ int sh[];
    __shared__ int wsum[32], wtile[32];
    constexpr int N = 8;  // tokens of a thread looked up together (kept, where these are all)
    const int keys = a.adapters + 1, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int *const cursor = sh, *const first = sh + keys + 1, *const tile = first + keys + 1;
    pdl_launch_dependents();
    pdl_wait();
    int key[N];
    uint32_t same[N];
    const auto look = [&](int64_t t0, bool report) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int64_t t = t0 + i * 1024 + tid;
            key[i] = t < a.M ? a.which[t] : INT_MIN;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (report && key[i] >= a.adapters) flag_value(a.status);
            key[i] = key[i] == INT_MIN && t0 + i * 1024 + tid >= a.M ? -1 : key[i] >= 0 && key[i] < a.adapters ? key[i] : a.adapters;
        }
    };
    for (int i = tid; i < keys; i += 1024) cursor[i] = 0;
    __syncthreads();
    for (int64_t t0 = 0; t0 < a.M; t0 += N * 1024) {
        look(t0, true);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            same[i] = same_key(key[i]);
            count_key(cursor, key[i], same[i]);
        }
    }
    __syncthreads();
    // running sums of tokens and of tiles over the adapters
    const int each = (keys + 1023) / 1024;
    int n = 0, m = 0;
    for (int i = 0; i < each; ++i) {
        const int k = tid * each + i;
        if (k < keys) n += cursor[k], m += (cursor[k] + TM - 1) / TM;
    }
    int un = n, um = m;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, un, o), w = __shfl_up_sync(0xffffffffu, um, o);
        if (lane >= o) un += u, um += w;
    }
    if (lane == 31) wsum[warp] = un, wtile[warp] = um;
    __syncthreads();
    int bn = un - n, bm = um - m;
    for (int i = 0; i < warp; ++i) bn += wsum[i], bm += wtile[i];
    for (int i = 0; i < each; ++i) {
        const int k = tid * each + i;
        if (k < keys) {
            const int c = cursor[k];
            first[k] = cursor[k] = bn;
            tile[k] = bm;
            bn += c;
            bm += (c + TM - 1) / TM;
            if (k == keys - 1) first[keys] = bn, tile[keys] = bm;
        }
    }
    __syncthreads();
    int *const order = plan + 4 + 3 * a.max_tiles;
    for (int64_t t0 = 0; t0 < a.M; t0 += N * 1024) {
        const bool again = a.M > N * 1024;
        if (again) look(t0, false);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (again) same[i] = same_key(key[i]);
            const int at = count_key(cursor, key[i], same[i]);
            // (a place beyond the tokens: `which` changed since they were counted)
            if (key[i] >= 0 && at < a.M) order[at] = (int)(t0 + i * 1024 + tid);
        }
    }
    const int tiles = tile[keys];
    if (tid == 0) plan[0] = tiles;
    for (int u = tid; u < tiles; u += 1024) {
        int x = 0, y = keys - 1;  // the last adapter whose tiles begin at or before u: it has some
        while (x < y) {
            const int mid = (x + y + 1) >> 1;
            if (tile[mid] <= u) x = mid;
            else y = mid - 1;
        }
        const int at = first[x] + (u - tile[x]) * TM;
        int *const p = plan + 4 + 3 * u;
        p[0] = x;
        p[1] = at;
        p[2] = min(TM, first[x + 1] - at);
    }
}

// Tiles of 128 tokens where tiles of 16 would read the adapters again and again: from 32 ranks on, 2048 tokens and 120 an
// adapter that can be there on average; below, 256 tokens an adapter and 70 MB of the adapters read again (B a quarter: the
// expand gains least).  Rows and columns (eights) start on 16 bytes; up to 64 ranks, which h's tiles of shared memory
// hold; the ranks of one launch's shards, each rounded up to 16, take up to 128 columns of tensor memory, and more shards
// are more launches.  Measured (us, tiles of 16 / 128; tokens x adapters, 3584 to 3584 columns): rank 16, 2048 x 2: 24 / 28;
// 4096 x 6: 34 / 35; 8192 x 32: 66 / 78; 8192 x 6: 60 / 51; 4096 x 4 to 18944: 76 / 87; from 18944: 84 / 56; rank 24, 4096 x 4: 46 /
// 37; rank 32, 2048 x 16: 38 / 38; 8192 x 48: 102 / 88; 8192 x 16: 98 / 58; rank 64, 1024 x 4: 25 / 31; 2048 x 8: 48 / 46; 8192 x 6:
// 137 / 60; from 18944: 340 / 103; to 18944, rank 32, 2048 x 4: 66 / 79.  Gated layers, whose columns are many, keep to tiles of 16.
// fp32 outputs, whose blocks of columns are half as wide: 256 tokens an adapter and 110 MB of A read again.  Rank 16, 8192 x 6:
// 94 / 102; from 18944: 232 / 167; rank 32, 2048 x 4: 43 / 56; 8192 x 16: 118 / 109; rank 48, 4096 x 4: 65 / 81; rank 64, 2048 x 8:
// 55 / 70; 8192 x 6: 157 / 116; from 18944: 362 / 181.
constexpr int kBigRanks = 128;
bool big_tiles(const LoraArgs &a, bool f32) {
    if (!a.vec_x || !a.vec_y || a.gated || a.R > 64) return false;
    const int64_t present = a.adapters + 1 < a.M ? a.adapters + 1 : a.M;
    const double ranks = (double)a.M / 16 * a.R * 2, again = ranks * a.S * a.K;
    if (f32) return a.M >= 256 * present && again >= 110e6;
    if (a.R >= 32) return a.M >= 2048 && a.M >= 120 * present;
    return a.M >= 256 * present && again + ranks * a.N / 4 >= 70e6;
}

int64_t tiles_bound(int64_t M, int64_t adapters, int TM) {
    const int64_t present = adapters + 1 < M ? adapters + 1 : M;
    return (M + present * (TM - 1)) / TM;
}

}  // namespace

int64_t lora_workspace(int64_t M, int64_t adapters) {
    if (M <= kLoraFind && adapters <= kLoraFind) return 0;
    return 4 * (4 + 3 * tiles_bound(M, adapters, 16) + M);
}

int lora_tile(const LoraArgs &a, bool f32) { return big_tiles(a, f32) ? 128 : 16; }

cudaError_t launch_lora(const LoraArgs &args, int dtype, bool f32, void *workspace, int sm_count, cudaStream_t st) {
    LoraArgs a = args;
    const int TM = lora_tile(a, f32);
    const bool big = TM == 128;
    const int units = (int)tiles_bound(a.M, a.adapters, TM);
    // Blocks a tile: 8, 6, 4, 2 or 1, as many as make two blocks an SM (gated, where three fit: 2.7) of the tiles that tokens
    // spread evenly over the adapters would give.  (Of all that there could be, a third more, blocks would be too
    // few.)  Measured (us, C = 2, 4, 6, 8; tokens x adapters, rank 16, 3584 columns in): gated 2 x 18944, 333 x 40: 86 / 53 / 42 / 41;
    // 512 x 64: 82 / 56 / 52 / 62; 1024 x 4: 97 / 61 / 57 / 69; 1000 x 200: 119 / 114 / 118 / 124; plain 18944, 333 x 40: 40 / 28 /
    // 24 / 33; 3584, 64 x 64: 15 / 12 / 13 / 16; 1024 x 8: 19 / 16 / 26 / 23; 1024 x 100: 22 / 27 / 37 / 37; tiles of 128, rank 32, 8192 x
    // 16: 79 / 69 / 81 / 80; rank 64, 18944 to 3584, 8192 x 6: 157 / 132 / 164 / 156.  7 is worse than 6 and 8 throughout.
    const double present = (double)(a.adapters + 1 < a.M ? a.adapters + 1 : a.M), even = (double)a.M / TM + present / 2;
    const double most = (a.gated ? 2.7 : 2.0) * sm_count / (even > present ? even : present);
    a.C = most >= 8 ? 8 : most >= 6 ? 6 : most >= 4 ? 4 : most >= 2 ? 2 : 1;
    a.plan = nullptr;
    if (lora_workspace(a.M, a.adapters) > 0) {
        a.max_tiles = units;
        int *const plan = static_cast<int *>(workspace);
        const cudaError_t e = launch_chained(lora_plan_kernel, 1, 1024, 3 * (a.adapters + 2) * sizeof(int), 0, st, a, TM, plan);
        if (e != cudaSuccess) return e;
        a.plan = plan;
    }
    const int shards = a.S, most_shards = kBigRanks / ((a.R + 15) / 16 * 16),
              at_once = big && most_shards < shards ? most_shards : shards;
    for (int s0 = 0; s0 < shards; s0 += at_once) {
        LoraArgs b = a;
        b.S = shards - s0 < at_once ? shards - s0 : at_once;
        b.rank0 = s0 * a.R;
        for (int i = 0; i < s0; ++i) b.col0 += a.shard[i];
        for (int i = 0; i < b.S; ++i) b.shard[i] = a.shard[s0 + i];
        const cudaError_t e = dtype == 1 ? launch_lora_bf16(b, f32, big, units, st) : launch_lora_f16(b, f32, big, units, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace tl
