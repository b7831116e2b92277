// attn_sched.cuh -- how the attention kernels divide their work, and the partial
// results that join blocks of one unit.
//
// A unit is one block of rows of one (sequence, kv head); it has ceil(L / KT) tiles of
// KT keys, L = context + new tokens.  The tiles of all units, unit after unit, are
// dealt to the blocks in equal consecutive runs: block c of nc takes tiles
// [c N / nc, (c + 1) N / nc).  Lengths live on the device, so every block computes N
// and its first unit itself.  Ragged batches and single long sequences both fill the
// GPU, and the division -- and with it the order of every sum -- depends on the
// sizes alone.
//
// A block that runs through a whole unit writes its output.  Otherwise it leaves a
// partial result (unnormalised rows, running maximum, running sum): in its slot 0
// if the unit is the first of its run, else in slot 1 (it is then the last).
#pragma once

#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace tl {

constexpr float kAttnLow = -3e38f;  // a running maximum before any key (finite: no inf - inf)
// f16 weights: 2^kAttnUp times their ratio to the running maximum, which lags the true one
// by at most 2^kAttnSlack; times a value scale of at most half the reference: below 2^15
constexpr float kAttnUp = 14.f, kAttnSlack = 2.f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Keys of sequence b, clamped to its page-table row.
__device__ __forceinline__ int attn_context(const AttnArgs &a, int b) {
    const int c = a.ctx[b], most = (int)(a.max_keys - a.T);
    if (c < 0 || c > most) {
        flag_value(a.status);
        return c < 0 ? 0 : most;
    }
    return c;
}

// Place of a block's run: N tiles in all, and the sequence b in which tile `x` lies, with
// the number of tiles before b.
struct AttnPlace {
    int64_t N;       // tiles of the whole call
    int64_t before;  // tiles of the sequences before b
    int b;
};

// Number of tiles of sequence b over all its units.
template <int KT>
__device__ __forceinline__ int64_t attn_tiles(const AttnArgs &a, int b, int units) {
    return (int64_t)((attn_context(a, b) + a.T + KT - 1) / KT) * units;
}

// Executed by the whole block (NTHR threads); sh: NTHR / 32 + 2 64-bit words of shared
// memory.  pick(N) gives the tile that is looked for.
template <int KT, int NTHR, typename Pick>
__device__ __forceinline__ AttnPlace attn_place(const AttnArgs &a, int units, int64_t *sh, Pick pick) {
    constexpr int NW = NTHR / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // inclusive sums over one chunk of NTHR sequences; `total` of the chunk in sh[NW]
    auto scan = [&](int b0) -> int64_t {
        const int64_t own = b0 + tid < a.B ? attn_tiles<KT>(a, b0 + tid, units) : 0;
        int64_t v = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        if (lane == 31) sh[warp] = v;
        __syncthreads();
        int64_t pre = 0;
        for (int w = 0; w < warp; ++w) pre += sh[w];
        if (tid == NTHR - 1) sh[NW] = pre + v;
        return pre + v - own;  // exclusive
    };
    AttnPlace r{0, 0, 0};
    int64_t first = 0;  // this thread's exclusive sum in the first chunk
    for (int b0 = 0; b0 < a.B; b0 += NTHR) {
        const int64_t e = scan(b0);
        if (b0 == 0) first = e;
        __syncthreads();
        r.N += sh[NW];
        __syncthreads();
    }
    const int64_t x = pick(r.N);
    int64_t base = 0;
    for (int b0 = 0; b0 < a.B; b0 += NTHR) {
        int64_t e = first;
        if (b0 > 0) {
            e = scan(b0);
            __syncthreads();
            base += sh[NW + 1];
        }
        const int64_t own = b0 + tid < a.B ? attn_tiles<KT>(a, b0 + tid, units) : 0;
        if (tid == 0) sh[0] = -1;
        __syncthreads();
        if (x >= base + e && x < base + e + own) {
            sh[0] = b0 + tid;
            sh[1] = base + e;
        }
        if (tid == NTHR - 1) sh[NW + 1] = e + own;  // the chunk's total, for the next one
        __syncthreads();
        if (sh[0] >= 0) {
            r.b = (int)sh[0];
            r.before = sh[1];
            break;
        }
        __syncthreads();
    }
    __syncthreads();
    return r;
}

// The block that holds tile x.
__device__ __forceinline__ int attn_block_of(int64_t x, int64_t N, int nc) {
    return (int)(((x + 1) * nc - 1) / N);
}
__device__ __forceinline__ int64_t attn_first_tile(int c, int64_t N, int nc) { return c * N / nc; }

// A slot of partial results: ROWS rows of D, then their maxima, then their sums.
template <int ROWS, int D>
struct AttnSlot {
    static constexpr int64_t floats = (int64_t)ROWS * (D + 2);
    static __device__ __forceinline__ float *at(float *ws, int c, int which) {
        return ws + (2ll * c + which) * floats;
    }
};

// A walk over a block's run of tiles.
struct AttnWalk {
    int b, unit, tile, tiles, ctx;  // unit: index within the sequence
    template <int KT>
    __device__ __forceinline__ void start(const AttnArgs &a, const AttnPlace &p, int64_t x) {
        b = p.b;
        ctx = attn_context(a, b);
        tiles = (ctx + a.T + KT - 1) / KT;
        const int64_t r = x - p.before;
        unit = (int)(r / tiles);
        tile = (int)(r - (int64_t)unit * tiles);
    }
    // to the next tile (not past the last of the call)
    template <int KT>
    __device__ __forceinline__ void next(const AttnArgs &a, int units) {
        if (++tile < tiles) return;
        tile = 0;
        if (++unit < units) return;
        unit = 0;
        if (++b < a.B) {
            ctx = attn_context(a, b);
            tiles = (ctx + a.T + KT - 1) / KT;
        }
    }
};

// Page of a key, checked.
__device__ __forceinline__ int attn_page(const AttnArgs &a, int b, int key) {
    int p = __ldg(a.pages + b * a.pages_stride + (unsigned)key / (unsigned)a.c.P);
    if ((unsigned)p >= (unsigned)a.c.pages) {
        flag_value(a.status);
        p = 0;
    }
    return p;
}

// Joins the partial results of each unit that more than one block worked on: one block
// per (unit, row), its four warps sharing the partial results, sums in block order.
// Launched as a dependent of the main kernel, so it computes its place meanwhile.
template <bool BF, int KT, int ROWS, int D>
__global__ void __launch_bounds__(128) attn_join_kernel(AttnArgs a, int rtiles, int nc) {
    __shared__ int64_t sh[8];
    __shared__ float sm[4], sl[4], so[4][D];
    constexpr int E = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int R = a.T * a.G, units = a.c.Hk * rtiles;
    const int row = blockIdx.x % ROWS;
    const int64_t u = blockIdx.x / ROWS;
    const int b = (int)(u / units), unit = (int)(u % units), hk = unit / rtiles, rt = unit % rtiles;
    const int grow = rt * ROWS + row;  // row of the (sequence, kv head)
    // tiles before sequence b, and all of them
    int64_t pre = 0, all = 0;
    for (int i = threadIdx.x; i < a.B; i += 128) {
        const int64_t n = attn_tiles<KT>(a, i, units);
        all += n;
        if (i < b) pre += n;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        pre += __shfl_xor_sync(0xffffffffu, pre, o);
        all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    if (lane == 0) sh[warp] = pre, sh[4 + warp] = all;
    __syncthreads();
    pre = sh[0] + sh[1] + sh[2] + sh[3];
    const int64_t N = sh[4] + sh[5] + sh[6] + sh[7];
    const int64_t tiles = attn_tiles<KT>(a, b, 1);
    const int64_t s = pre + unit * tiles;
    const int c0 = attn_block_of(s, N, nc), c1 = attn_block_of(s + tiles - 1, N, nc);
    pdl_wait();
    if (c0 == c1 || grow >= R) return;
    using Slot = AttnSlot<ROWS, D>;
    const int first = attn_first_tile(c0, N, nc) == s ? 0 : 1;  // slot of the unit in its first block
    float m = kAttnLow, l = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    // blocks with no tile (N < nc) lie between: they hold nothing of the unit
    for (int c = c0 + warp; c <= c1; c += 4) {
        if (attn_first_tile(c, N, nc) == attn_first_tile(c + 1, N, nc)) continue;
        const float *p = Slot::at(a.ws, c, c == c0 ? first : 0);
        const float pm = p[ROWS * D + row], pl = p[ROWS * (D + 1) + row];
        float v[E];
        if constexpr (E == 4) {
            const float4 x = reinterpret_cast<const float4 *>(p + row * D)[lane];
            v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
        } else {
            const float2 x = reinterpret_cast<const float2 *>(p + row * D)[lane];
            v[0] = x.x, v[1] = x.y;
        }
        const float mn = fmaxf(m, pm), f = ex2(m - mn), g = ex2(pm - mn);
        m = mn;
        l = l * f + pl * g;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * f + v[e] * g;
    }
    if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = o[e];
    __syncthreads();
    const float M = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    float L = 0.f, x = 0.f;
    const int d = threadIdx.x;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const float g = ex2(sm[w] - M);
        L += sl[w] * g;
        if (d < D) x += so[w][d] * g;
    }
    const int64_t out_row = ((int64_t)b * a.T + grow / a.G) * a.Hq + hk * a.G + grow % a.G;
    if (d < D) OutStore<BF ? 1 : 0>::st(a.out, out_row * D + d, L == 0.f ? 0.f : x / L);
    if (a.lse && d == 0) a.lse[out_row] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

}  // namespace tl
