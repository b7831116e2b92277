// attn_sched.cuh -- how the attention kernels divide their work, and the partial
// results that join blocks of one unit.
//
// A unit is one block of rows of one (sequence, kv head); it has ceil(L / KT) tiles of
// KT keys, L = context + new tokens.  The tiles of all units, unit after unit, are
// dealt to the blocks in equal consecutive runs: block c of nc takes tiles
// [c N / nc, (c + 1) N / nc), nc being the blocks launched or N if that is less.  Lengths
// live on the device, so every block computes N and its first unit itself.  Ragged batches
// and single long sequences both fill the GPU, and the division -- and with it the order of
// every sum -- depends on the sizes alone.
//
// In that count each unit has OV more tiles than it has keys for, before its own: they
// stand for the cost of beginning and ending a unit (queries, joins), without which a
// block given a run of short units would be the last to end by far.  Nothing is done in
// them, and a block whose run ends within them does not touch the unit.  (6 trees of 23,
// 32 heads, up to 4099 keys, int4: with the margin below, 249 us without these tiles and
// that margin, 125 us with both, as the kernel was then; 74 us now.)
//
// Where contexts can only be short (by the page table's width), or units are many, a block
// takes one whole unit instead (AttnArgs::direct): nothing to find, nothing to join.
//
// A block that runs through a whole unit writes its output.  Otherwise it leaves a
// partial result (unnormalised rows, running maximum, running sum): in its slot 0
// if the unit is the first of its run, else in slot 1 (it is then the last).
#pragma once

#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "rope.cuh"

namespace tl {

constexpr float kAttnLow = -3e38f;  // a running maximum before any key (finite: no inf - inf)
// f16 weights, each with its value scale: products e sv.  In powers of two, with score z_j and
// size x_j = max(log2 |sv_j|, kAttnSmall), a row's reference r follows the largest z_j + x_j
// among the keys that this row sees:
//   e_j = 2^(z_j - r),  product_j = e_j (sv_j 2^-kAttnBias).
// r moves only when some z_j + x_j exceeds it by kAttnFull (so products stay below 2^15), and
// then to kAttnRoom below: the largest lies between 2^10 and 2^15, products down to 2^-24 of
// it keep all 11 bits of f16, whatever scales other keys or other rows have.  (The tcgen05
// kernel may take a bound that is up to kAttnSpread higher: 2^6, 2^-20.)  The sum of the
// weights counts e_j, whose range in fp32 the bias centres: for scales of up to 2^128 terms
// down to 2^-24 of the largest weight count, and with scales of 2^kAttnSmall and less (rows
// of zeros) 2^25 equal weights fit.  A row whose largest product is far below 2^kAttnSmall of its
// largest weight leaves f16 at the lower end: it loses bits from 2^-94 on.
// Differences z_j - r are exact where they matter, sums z_j + x_j are not: beyond kAttnCoarse a
// reference taken from a sum is held against the differences that it leaves, and raised where one
// exceeds kAttnFull.  So scores up to 2^29 give their answer; beyond, where fp32 has steps
// larger than the room that f16 leaves, all weights of a row may vanish.
// With scores of a standard deviation of 2.6 (3.7 in powers of two) and no margin, half the
// 64-key tiles moved some row of a warp, which cost more than the tile itself (8 trees of 64
// over 16384 keys: 382 us against 265 with the margin, as the kernel was then; 205 us now).
constexpr float kAttnBias = 16.f, kAttnRoom = 10.f + kAttnBias, kAttnFull = 15.f + kAttnBias, kAttnSpread = 4.f, kAttnSmall = -72.f;
constexpr float kAttnCoarse = 1048576.f;
constexpr float kAttnUnbias = 1.f / 65536.f, kAttnRebias = 65536.f;  // 2^-kAttnBias, 2^kAttnBias
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// at least the sum of two terms that is y after its rounding and this one
__device__ __forceinline__ float attn_above(float y) { return fmaf(fabsf(y), 0x1p-23f, y); }
// x_j of a value scale; finite for every bit pattern
__device__ __forceinline__ float attn_size(float sv) { return fminf(fmaxf(lg2(fabsf(sv)), kAttnSmall), 128.f); }

// Allows a kernel `bytes` of dynamic shared memory on the current device.  `done`, one per kernel,
// remembers the devices where that has succeeded (the call costs a microsecond of the host's time).
template <typename K>
cudaError_t attn_allow_smem(std::atomic<uint64_t> &done, K *kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// bf16 queries enter the product as f16, a row scaled by the power of two that takes its largest
// element to [2^15, 2^16): exact for elements down to 2^-32 of it (a bf16 has 8 bits), below that
// rounded at 2^-40 of it.  `e`: biased exponent of the largest, 255 for a row with an infinity or a
// NaN, which stays as it is.  Rows below 2^-95 take the scale of those at 2^-95; f16 holds all
// their bits.
struct QueryScale {
    float down, up;
    __device__ __forceinline__ explicit QueryScale(uint32_t e) {
        const uint32_t c = max(e, 32u);
        down = e == 255u ? 1.f : __uint_as_float((269u - c) << 23);
        up = e == 255u ? 1.f : __uint_as_float((c - 15u) << 23);
    }
};

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
    int b, ctx;      // ctx: b's context
};

// Keys per tile, and tiles counted beside a unit's own.
template <int KEYS, int BESIDE>
struct AttnTiling {
    static constexpr int KT = KEYS, OV = BESIDE;
    // own tiles of a unit of a sequence with ctx committed keys
    static __device__ __forceinline__ int tiles(const AttnArgs &a, int ctx) { return (ctx + a.T + KT - 1) / KT; }
};

// Tiles counted for sequence b.
template <typename TL>
__device__ __forceinline__ int64_t attn_tiles(const AttnArgs &a, int b, int units) {
    return (int64_t)(TL::tiles(a, attn_context(a, b)) + TL::OV) * units;
}

// Up to kPlaceFast sequences: every warp on its own, one load per 32 sequences and no barrier.
constexpr int kPlaceFast = 128;
template <typename TL, typename Pick>
__device__ __forceinline__ AttnPlace attn_place_warp(const AttnArgs &a, int units, Pick pick) {
    constexpr int CH = kPlaceFast / 32;
    const int lane = threadIdx.x & 31;
    int ctx[CH], incl[CH];  // tiles of one unit per sequence fit 32 bits, and so do 32 of them
    int64_t N = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int b = c * 32 + lane;
        ctx[c] = b < a.B ? attn_context(a, b) : 0;
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        int v = c * 32 + lane < a.B ? TL::tiles(a, ctx[c]) + TL::OV : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        incl[c] = v;
        N += __shfl_sync(0xffffffffu, v, 31);
    }
    AttnPlace r{N * units, 0, 0, 0};
    int64_t x = pick(r.N), base = 0;
    bool found = false;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const uint32_t beyond = __ballot_sync(0xffffffffu, (base + incl[c]) * units > x);
        if (!found && beyond) {
            const int l = __ffs(beyond) - 1;
            found = true;
            r.b = c * 32 + l;
            r.ctx = __shfl_sync(0xffffffffu, ctx[c], l);
            const int upto = __shfl_sync(0xffffffffu, incl[c], l > 0 ? l - 1 : 0);
            r.before = (base + (l > 0 ? upto : 0)) * units;
        }
        base += __shfl_sync(0xffffffffu, incl[c], 31);
    }
    return r;
}

// Executed by the whole block (NTHR threads); sh: NTHR / 32 + 2 64-bit words of shared
// memory.  pick(N) gives the tile that is looked for.
template <typename TL, int NTHR, typename Pick>
__device__ __forceinline__ AttnPlace attn_place(const AttnArgs &a, int units, int64_t *sh, Pick pick) {
    if (a.B <= kPlaceFast) return attn_place_warp<TL>(a, units, pick);
    constexpr int NW = NTHR / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // inclusive sums over one chunk of NTHR sequences; `total` of the chunk in sh[NW]
    auto scan = [&](int b0) -> int64_t {
        const int64_t own = b0 + tid < a.B ? attn_tiles<TL>(a, b0 + tid, units) : 0;
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
    AttnPlace r{0, 0, 0, 0};
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
        const int64_t own = b0 + tid < a.B ? attn_tiles<TL>(a, b0 + tid, units) : 0;
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
    r.ctx = attn_context(a, r.b);
    return r;
}

// The block that holds tile x.
__device__ __forceinline__ int attn_block_of(int64_t x, int64_t N, int nc) {
    const int64_t n = (x + 1) * nc - 1;
    return (n >> 32) || (N >> 32) ? (int)(n / N) : (int)((uint32_t)n / (uint32_t)N);
}
__device__ __forceinline__ int64_t attn_first_tile(int c, int64_t N, int nc) {
    const int64_t n = c * N;
    return n >> 32 ? n / nc : (uint32_t)n / (uint32_t)nc;
}

// A slot of partial results: ROWS rows of D, then their maxima, then their sums.
template <int ROWS, int D>
struct AttnSlot {
    static constexpr int64_t floats = (int64_t)ROWS * (D + 2);
    static __device__ __forceinline__ float *at(float *ws, int c, int which) {
        return ws + (2ll * c + which) * floats;
    }
};

// A walk over a block's run of tiles: sequence b, kv head hk, row block rt, tile of the unit.
struct AttnWalk {
    int b, hk, rt, tile, tiles, ctx;
    int at, end;  // counted tiles from the run's start on; at < end: the walk is inside the run
    template <typename TL>
    __device__ __forceinline__ void start(const AttnArgs &a, const AttnPlace &p, int64_t x0, int64_t x1, int rtiles) {
        b = p.b;
        ctx = p.ctx;
        tiles = TL::tiles(a, ctx);
        const int64_t r = x0 - p.before;
        // a sequence's tiles fit 32 bits in any cache that fits memory; wider division otherwise
        const int all = tiles + TL::OV;
        const int unit = r < (1ll << 31) ? (int)((unsigned)r / (unsigned)all) : (int)(r / all);
        const int v = (int)(r - (int64_t)unit * all) - TL::OV;
        tile = v < 0 ? 0 : v;
        at = tile - v;
        end = (int)(x1 - x0);
        hk = rtiles == 1 ? unit : unit / rtiles;
        rt = unit - hk * rtiles;
    }
    // one whole unit, the `index`-th of the call
    template <typename TL>
    __device__ __forceinline__ void start_unit(const AttnArgs &a, int index, int rtiles) {
        const int units = a.c.Hk * rtiles, unit = index % units;
        b = index / units;
        hk = rtiles == 1 ? unit : unit / rtiles;
        rt = unit - hk * rtiles;
        ctx = attn_context(a, b);
        tile = at = 0;
        tiles = end = TL::tiles(a, ctx);
    }
    // a block's run, or its unit; false: the block has none
    template <typename TL, int NTHR>
    __device__ __forceinline__ bool start_block(const AttnArgs &a, int rtiles, int64_t *sh) {
        if (a.direct) {
            start_unit<TL>(a, blockIdx.x, rtiles);
            return true;
        }
        int nc = gridDim.x;
        const AttnPlace place = attn_place<TL, NTHR>(a, a.c.Hk * rtiles, sh, [&](int64_t N) {
            if (N < nc) nc = (int)N;  // no block without a tile
            return attn_first_tile(blockIdx.x, N, nc);
        });
        if ((int)blockIdx.x >= nc) return false;
        start<TL>(a, place, attn_first_tile(blockIdx.x, place.N, nc), attn_first_tile(blockIdx.x + 1, place.N, nc), rtiles);
        return inside();
    }
    __device__ __forceinline__ bool inside() const { return at < end; }
    __device__ __forceinline__ bool last_of_unit() const { return tile + 1 == tiles; }
    // whether the next tile is inside the run too
    template <typename TL>
    __device__ __forceinline__ bool more() const { return at + 1 + (last_of_unit() ? TL::OV : 0) < end; }
    // to the next tile; whether a unit begins there
    template <typename TL>
    __device__ __forceinline__ bool next(const AttnArgs &a, int rtiles) {
        ++at;
        if (++tile < tiles) return false;
        at += TL::OV;
        tile = 0;
        if (++rt < rtiles) return true;
        rt = 0;
        if (++hk < a.c.Hk) return true;
        hk = 0;
        if (++b < a.B) {
            ctx = attn_context(a, b);
            tiles = TL::tiles(a, ctx);
        }
        return true;
    }
};

// Pages of the keys of a unit's tiles: page index pi in the sequence's row of
// the page table, place off in the page; moved along without a division.
struct AttnPages {
    int pi, off, last;  // last: page index of the unit's last key
    __device__ __forceinline__ void start(const AttnArgs &a, const AttnWalk &w, int key) {
        pi = (int)((unsigned)key / (unsigned)a.c.P);
        off = key - pi * a.c.P;
        last = (int)((unsigned)(w.ctx + a.T - 1) / (unsigned)a.c.P);
    }
    __device__ __forceinline__ void next(const AttnArgs &a, int keys) {
        off += keys;
        while (off >= a.c.P) off -= a.c.P, ++pi;
    }
    // the page (unchecked) that holds the key, or for a place beyond the last key that key's
    __device__ __forceinline__ int fetch(const AttnArgs &a, int b) const {
        return __ldg(a.pages + b * a.pages_stride + min(pi, last));
    }
};

// A group is 16 places of one (page, kv head); its index fits 32 bits (checked by the call).
__device__ __forceinline__ uint32_t attn_group(const AttnArgs &a, int page, int hk, int off) {
    if ((unsigned)page >= (unsigned)a.c.pages) {
        flag_value(a.status);
        page = 0;
    }
    return ((uint32_t)page * (uint32_t)a.c.Hk + (uint32_t)hk) * (uint32_t)(a.c.P >> 4) + (uint32_t)(off >> 4);
}

// e4m3 caches: writes NaN over the elements d0 .. d0 + n - 1 of a new token's result (16-bit, or
// fp32 where it is a part of one; written before by the same thread) where a new token that it
// sees has a NaN code.  The products take such codes as finite, since other rows do not see them.
// Called, and so not inlined, only where one was met.
template <int D>
__device__ __noinline__ void attn_put_nans(const uint8_t *codes, const int *pages, int npages, int P, int Hk, int hk, const uint8_t *tree,
                                           int T, int tok, int ctx, int d0, int n, uint16_t *out, float *part) {
    for (int i = 0; i < T; ++i) {
        if (!(tree ? tree[i] != 0 : i <= tok)) continue;
        const int pi = (ctx + i) / P, off = ctx + i - pi * P, page = pages[pi];
        const int64_t in = (unsigned)page < (unsigned)npages ? page : 0;
        const uint8_t *c = codes + ((in * Hk + hk) * P + off) * D;
        for (int e = d0; e < d0 + n; ++e) {
            if ((c[e] & 0x7F) != 0x7F) continue;
            if (out) out[e] = 0x7FFF;  // (of either type)
            else part[e] = __uint_as_float(0x7FC00000u);
        }
    }
}
template <int D>
__device__ __forceinline__ void attn_put_nans(const AttnArgs &a, const AttnWalk &w, int tok, int d0, int n, void *out, float *part) {
    attn_put_nans<D>(a.c.vc, a.pages + w.b * a.pages_stride, (int)a.c.pages, a.c.P, a.c.Hk, w.hk,
                     a.tree ? a.tree + w.b * a.tree_b + tok * a.tree_r : nullptr, a.T, tok, w.ctx, d0, n, static_cast<uint16_t *>(out), part);
}

// 16-bit values of the call's dtype
__device__ __forceinline__ uint32_t attn_pack(const AttnArgs &a, float lo, float hi) {
    return a.bf ? pack2(__nv_bfloat16(), lo, hi) : pack2(__half(), lo, hi);
}
__device__ __forceinline__ float2 attn_unpack(const AttnArgs &a, uint32_t w) {
    return a.bf ? unpack2(__nv_bfloat16(), w) : unpack2(__half(), w);
}
__device__ __forceinline__ void attn_store(const AttnArgs &a, int64_t i, float v) {
    if (a.bf) OutStore<1>::st(a.out, i, v);
    else OutStore<0>::st(a.out, i, v);
}

// Where a unit's partial results lie: blocks c0 .. c1 (c0 == c1: none, its one block wrote
// the output), the first of them in slot `first`.  Executed by a whole block of NW warps;
// sh: 2 NW 64-bit words.
struct AttnParts {
    int c0, c1, first;
};
template <typename TL, int NW>
__device__ __forceinline__ AttnParts attn_parts(const AttnArgs &a, int b, int unit, int units, int nc, int64_t *sh) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t pre = 0, all = 0;  // tiles before sequence b, and of the call
    for (int i = threadIdx.x; i < a.B; i += NW * 32) {
        const int64_t n = attn_tiles<TL>(a, i, units);
        all += n;
        if (i < b) pre += n;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        pre += __shfl_xor_sync(0xffffffffu, pre, o);
        all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    if (lane == 0) sh[warp] = pre, sh[NW + warp] = all;
    __syncthreads();
    AttnParts r;
    int64_t N = 0;
    pre = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        pre += sh[w];
        N += sh[NW + w];
    }
    if (N < nc) nc = (int)N;
    const int64_t tiles = attn_tiles<TL>(a, b, 1), s = pre + unit * tiles;
    r.c0 = attn_block_of(s + TL::OV, N, nc);
    r.c1 = attn_block_of(s + tiles - 1, N, nc);
    r.first = attn_first_tile(r.c0, N, nc) >= s ? 0 : 1;
    return r;
}

// A row's running maximum, sum and this lane's E = D / 32 outputs, and one more partial result.
template <int E>
struct AttnSum {
    float m = kAttnLow, l = 0.f, o[E];
    __device__ __forceinline__ AttnSum() {
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = 0.f;
    }
    // four parts at once, their loads in flight together; absent ones are null
    template <int ROWS, int D>
    __device__ __forceinline__ void add4(const float *const (&x)[4], int row, int lane) {
        float pm[4], pl[4], v[4][E];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            pm[k] = kAttnLow;
            pl[k] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) v[k][e] = 0.f;
            if (x[k]) {
                pm[k] = x[k][ROWS * D + row];
                pl[k] = x[k][ROWS * (D + 1) + row];
                if constexpr (E == 4) {
                    const float4 u = reinterpret_cast<const float4 *>(x[k] + row * D)[lane];
                    v[k][0] = u.x, v[k][1] = u.y, v[k][2] = u.z, v[k][3] = u.w;
                } else {
                    const float2 u = reinterpret_cast<const float2 *>(x[k] + row * D)[lane];
                    v[k][0] = u.x, v[k][1] = u.y;
                }
            }
        }
        // sums in two steps: references may lie further apart than fp32's exponents reach
        const float mn = fmaxf(fmaxf(m, fmaxf(pm[0], pm[1])), fmaxf(pm[2], pm[3])), f = ex2(.5f * (m - mn)), f2 = f * f;
        m = mn;
        l = l * f * f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= f2;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float g = ex2(.5f * (pm[k] - mn)), g2 = g * g;
            l += pl[k] * g * g;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] += v[k][e] * g2;
        }
    }
};

// Joins the partial results of each unit that more than one block worked on, in block
// order; the grid covers every unit, and blocks of units with nothing to join leave.
// Launched as a dependent of the main kernel: the place is computed meanwhile.
// WIDE: one block per row, its eight warps sharing the parts (four each in flight at a
// time): few rows, or few units, which then have many parts.  Otherwise 16 rows per
// block, one warp each: many units have few parts.
// Bound by latency (the place, then the parts from L2): joins cost 2 to 4 us of a call (32
// sequences of 100 keys, one token, 28 heads on 4: 10.4 us with them, 6.5 without; one of 20000:
// 19.3 us, and 22.1 with the parts added one after the other).
template <typename TL, int ROWS, int D, bool WIDE>
__global__ void __launch_bounds__(WIDE ? 256 : 512) attn_join_kernel(AttnArgs a, int rtiles, int per_unit, int nc) {
    constexpr int NW = WIDE ? 8 : 16, E = D / 32;
    __shared__ int64_t sh[2 * NW];
    __shared__ float sm[8], sl[8], so[WIDE ? 8 : 1][D];
    using Slot = AttnSlot<ROWS, D>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int R = a.T * a.G, units = a.c.Hk * rtiles;
    const int64_t u = blockIdx.x / per_unit;
    const int slice = blockIdx.x % per_unit;
    const int b = (int)(u / units), unit = (int)(u % units), hk = unit / rtiles, rt = unit % rtiles;
    const AttnParts p = attn_parts<TL, NW>(a, b, unit, units, nc, sh);
    pdl_wait();
    const int row = WIDE ? slice : slice * 16 + warp, grow = rt * ROWS + row;  // row of the unit, of its kv head
    if (p.c0 == p.c1 || (WIDE && grow >= R)) return;
    const int64_t o = ((int64_t)b * a.T + grow / a.G) * a.Hq + hk * a.G + grow % a.G;  // output row
    auto part = [&](int c) -> const float * { return c > p.c1 ? nullptr : Slot::at(a.ws, c, c == p.c0 ? p.first : 0); };
    AttnSum<E> s;
    if constexpr (WIDE) {
        for (int c = p.c0 + warp; c <= p.c1; c += 4 * NW) {
            const float *const x[4] = {part(c), part(c + NW), part(c + 2 * NW), part(c + 3 * NW)};
            s.template add4<ROWS, D>(x, row, lane);
        }
        if (lane == 0) sm[warp] = s.m, sl[warp] = s.l;
#pragma unroll
        for (int e = 0; e < E; ++e) so[warp][lane * E + e] = s.o[e];
        __syncthreads();
        float M = sm[0], L = 0.f, x = 0.f;
#pragma unroll
        for (int w = 1; w < NW; ++w) M = fmaxf(M, sm[w]);
        const int d = threadIdx.x;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float g = ex2(.5f * (sm[w] - M));
            L += sl[w] * g * g;
            if (d < D) x += so[w][d] * (g * g);
        }
        if (d < D) attn_store(a, o * D + d, L == 0.f ? 0.f : x / L);
        if (a.lse && d == 0) a.lse[o] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
    } else {
        if (grow >= R || row >= ROWS) return;
        for (int c = p.c0; c <= p.c1; c += 4) {
            const float *const x[4] = {part(c), part(c + 1), part(c + 2), part(c + 3)};
            s.template add4<ROWS, D>(x, row, lane);
        }
        const float r = s.l == 0.f ? 0.f : 1.f / s.l;
        uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + o * D + lane * E);
#pragma unroll
        for (int e = 0; e < E; e += 2) dst[e / 2] = attn_pack(a, s.o[e] * r, s.o[e + 1] * r);
        if (a.lse && lane == 0) a.lse[o] = s.l == 0.f ? -INFINITY : (s.m + log2f(s.l)) * kLn2;
    }
}

template <typename TL, int ROWS, int D, bool WIDE>
cudaError_t launch_join_w(const AttnArgs &a, int rtiles, int nc, cudaStream_t st) {
    const int R = a.T * a.G, rows = R < ROWS ? R : ROWS, per_unit = WIDE ? rows : (rows + 15) / 16;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)a.B * a.c.Hk * rtiles * per_unit), 1, 1);
    cfg.blockDim = dim3(WIDE ? 256 : 512, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<TL, ROWS, D, WIDE>, a, rtiles, per_unit, nc);
}

template <typename TL, int ROWS, int D>
cudaError_t launch_join(const AttnArgs &a, int rtiles, int nc, cudaStream_t st) {
    // one block per row while all of them run at once (eight blocks of 256 threads per SM)
    const int64_t rows = (int64_t)a.B * a.c.Hk * a.T * a.G;
    return rows <= 1216 ? launch_join_w<TL, ROWS, D, true>(a, rtiles, nc, st) : launch_join_w<TL, ROWS, D, false>(a, rtiles, nc, st);
}

}  // namespace tl
