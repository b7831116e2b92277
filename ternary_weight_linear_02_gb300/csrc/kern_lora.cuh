// kern_lora.cuh -- low-rank adapters of many requests beside a shared layer:
//     h = s_a (x A_a^T) (fp32),  out = y + h B_a^T       for the tokens of adapter a,
// y the shared layer's output, S stacked shards with ranks of their own; and the same with the
// SiLU-gated product of a fused gate/up layer behind it.
//
// One launch.  Work is dealt in tiles of up to TM tokens of one adapter, a cluster of C blocks a tile:
//   * shrink: each block takes a run of K and keeps h's partial sums (TM x S R) in shared
//     memory; they are added over the cluster in a fixed order through distributed
//     shared memory;
//   * expand: each block takes a share of the output columns, adds h B^T to y and writes.
// So x and y are read once and out is written once, A and B once per tile.  Two forms:
//   * few tokens an adapter: tiles of 16, the adapter's matrices are the traffic.  Warp MMAs fed
//     straight from global memory (an MMA sums over k: any order of k will do that both operands
//     share, so every lane loads 16 contiguous bytes);
//   * many: tiles of 128, the activations are the traffic.  Rows of x and A go through a ring of shared-memory
//     stages (16-byte copies, whatever the tokens' order) into tcgen05 MMAs, and so do the split h and B.
// Either way there are 0.7 R operations a byte: memory should bound it.  Measured: 16 tokens of 8 adapters, rank 16,
// fused QKV of 3584: 7.4 us (finding the tile 0.9, shrink 2.2, sums 1.5, expand 1.3); 333 tokens of 40 adapters,
// rank 16, gated layer of 2 x 18944: 30 us, 98 MB, 14.4 at a copy's rate: finding the tile 2.6, shrink 6 (a burst
// of 12 MB), sums 3, expand 10 (where three blocks share an SM 15); 8192 tokens of 6 adapters, rank 64,
// 18944 to 3584, f16: 103 us, 445 MB, 65.6 at a copy's rate: the plan 6, shrink 52 (6.5 TB/s), sums 8, expand 19 to 28
// (where two blocks share an SM).
//
// h enters the second product in 16 bits.  One rounding there would add as much error as that of a 16-bit
// output, so h is split into two numbers of T (three where bf16 feeds an fp32 output), each the
// rounded rest of those before: 2^-17 of h or less.  f16 into fp32 keeps to two, 2^-22, less than an fp32 sum of K
// products loses: with three, 8192 tokens of 6 adapters, rank 64, 18944 to 3584, took 190 us instead of 130 (shared memory for one
// block on an SM).  f16 takes a row scaled by a power of two, so that
// large sums do not overflow.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "launch.h"
#include "tc.cuh"

namespace tl {

// ------------------------------------------------------------ tiles
// Tokens of an adapter in tiles of TM; tokens without one are tiles of "adapter" n, which are copied.
__device__ __forceinline__ int lora_key(const LoraArgs &a, int64_t t) {
    const int w = a.which[t];
    return w >= 0 && w < a.adapters ? w : a.adapters;
}

constexpr int kLoraFind = 1024;  // tokens and adapters up to which each block finds its tile by itself

namespace lora {

constexpr int kThreads = 256, kWarps = 8;

template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// the same with nothing to add to
template <typename T>
__device__ __forceinline__ void mma16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816_first<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
template <>
__device__ __forceinline__ void mma16816_first<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f<float>(float x) { return x; }
template <typename T>
__device__ __forceinline__ T of_f(float x);
template <>
__device__ __forceinline__ __half of_f<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 of_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ float of_f<float>(float x) { return x; }

// 8 16-bit elements p[0..8) of which the first n exist (vec: p is 16-byte aligned and n is 0 or 8 at least)
template <typename T>
__device__ __forceinline__ uint4 load8(const T *p, int n, bool vec) {
    uint4 r = make_uint4(0, 0, 0, 0);
    if (vec) {
        if (n > 0) r = ldg_nc_v4(p);
    } else {
        const uint16_t *u = reinterpret_cast<const uint16_t *>(p);
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) w[i >> 1] |= (uint32_t)u[i] << (16 * (i & 1));
        r = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return r;
}

// N (4 or 8) contiguous elements of y as they are, of which the first n exist.  Not through the read-only path:
// out may be y.
template <typename O, int N>
struct Raw {
    static constexpr int WORDS = N * sizeof(O) / 4;
    uint32_t w[WORDS];
    __device__ __forceinline__ void load(const O *p, int n, bool vec) {
        if (vec && n >= N) {
            if constexpr (WORDS == 2) {
                const uint2 r = *reinterpret_cast<const uint2 *>(p);
                w[0] = r.x, w[1] = r.y;
            } else {
#pragma unroll
                for (int i = 0; i < WORDS; i += 4) {
                    const uint4 r = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint32_t *>(p) + i);
                    w[i] = r.x, w[i + 1] = r.y, w[i + 2] = r.z, w[i + 3] = r.w;
                }
            }
        } else if constexpr (sizeof(O) == 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = i < n ? __float_as_uint(p[i]) : 0u;
        } else {
            const uint16_t *u = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
            for (int i = 0; i < WORDS; ++i) w[i] = 0;
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (i < n) w[i >> 1] |= (uint32_t)u[i] << (16 * (i & 1));
        }
    }
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (sizeof(O) == 4) {
            return __uint_as_float(w[i]);
        } else {
            const uint16_t h = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
            return to_f(*reinterpret_cast<const O *>(&h));
        }
    }
};
template <typename O, int N>
__device__ __forceinline__ void store_out(O *p, int n, bool vec, const float (&v)[N]) {
    if (vec && n >= N) {
        if constexpr (sizeof(O) == 4) {
#pragma unroll
            for (int i = 0; i < N; i += 4) *reinterpret_cast<float4 *>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        } else {
            O h[N];
#pragma unroll
            for (int i = 0; i < N; ++i) h[i] = of_f<O>(v[i]);
            if constexpr (N == 8) *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(h);
            else *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(h);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) p[i] = of_f<O>(v[i]);
    }
}

__device__ __forceinline__ float cl_ld_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void cl_st_v2(uint32_t addr, uint2 v) {
    asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(v.x), "r"(v.y) : "memory");
}
__device__ __forceinline__ float4 cl_ld_v4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// For fp32 outputs as the layers' own gated products take it.  For 16-bit outputs the
// special functions' own instructions, 2^x within 2 ulp and 1/x within 1, without the scaling that the functions
// put around them for subnormal numbers (a third of the instructions): with the rounding of g log2(e), within 5 + 1.2
// |g| ulp, 2^-16 of the result, where its rounding takes 2^-9 or 2^-12; 0 instead of less than 2^-119 (g below -87).
template <typename O>
__device__ __forceinline__ float silu(float g) {
    if constexpr (sizeof(O) == 4) {
        return g / (1.f + expf(-g));
    } else {
        float e, r;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
        return g * r;
    }
}

// 16 bytes from global to shared memory, or zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint2 lds8(uint32_t at) {
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(at) : "memory");
    return r;
}
__device__ __forceinline__ void sts16(uint32_t at, uint4 r) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(at) : "memory");
    return r;
}

template <bool BIG>
struct Form {
    static constexpr int TM = BIG ? 128 : 16;  // tokens of a tile
    static constexpr int NT = 6;               // small: n-tiles of 8 ranks a pass of the shrink
    static constexpr int STAGES = 4, LAG = 2;  // BIG: stages of 64 k; copies in flight behind the newest
    static_assert(STAGES * (128 + 16) * 128 + 1024 >= tc::kSmemHolder, "holds tensor memory at the cluster's barriers");
};

// Sizes of a block's shared memory (bytes), the same on the host.
struct Smem {
    int ranks, npad;  // S R, and rounded up to 16
    int pstride;      // floats between rows of the partial sums: 16-byte stores of 8 rows hit other banks
    int hstride;      // small: elements of T between rows of the split h: 8-byte loads of 4 rows hit other banks
    int stage;        // BIG: a stage of the shrink
    int hper, htiles; // BIG: shards in a tile of the split h (64 ranks, each shard's rounded up to 16), such tiles
    int split;        // where the split h begins
    int blocks, red;  // small: where the stages of B and y, and the warps' sums begin
    int total;
    // small_stage: bytes of a stage of ExpandSmall (0: not used)
    __host__ __device__ Smem(bool big, bool gated, int S, int R, int ns, int small_stage) {
        const int tm = big ? 128 : 16;
        ranks = S * R;
        npad = (ranks + 15) & ~15;
        pstride = ranks + 4;
        const int steps = S * ((R + 15) / 16);
        hstride = steps * 16 + (steps % 2 ? 0 : 16);
        stage = (128 + npad) * 128;
        split = tm * pstride * 4;
        hper = big ? 4 / ((R + 15) / 16) : 1;
        htiles = (S + hper - 1) / hper;
        if (big) {  // four stages of B and two of y, when the sums are joined; h begins on 1024 bytes
            const int expand = 4 * 8192 + kWarps * 4096;
            split = ((split > expand ? split : expand) + 1023) & ~1023;
        }
        blocks = split + (big ? ns * htiles * 16384 : ns * tm * hstride * 2);
        const int red_bytes = 4 * 16 * Form<false>::NT * 8 * 4, stages = 2 * kWarps * small_stage;
        // (gated: a third block on each SM is worth more than copying before the sums are added)
        red = blocks + (gated ? 0 : stages);
        total = big ? blocks : gated ? blocks + (red_bytes > stages ? red_bytes : stages) : red + red_bytes;
        if (big) {
            const int ring = Form<true>::STAGES * stage;  // done with before the sums are stored
            total = (total > ring ? total : ring) + 1024; // stages lie on 1024 bytes
        }
    }
};

// What a block knows of its tile.
template <int TM>
struct Tile {
    int toks[TM];   // tokens, -1 behind the last
    int adapter, nth, count;
};

// ---- the tile: looked up in the plan, or found by each block.  False: there are fewer tiles.
template <int TM>
__device__ __forceinline__ bool find_tile(const LoraArgs &a, Tile<TM> &tile, int unit, bool report) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (a.plan != nullptr) {
        if (unit >= min(a.plan[0], a.max_tiles)) return false;
        const int *p = a.plan + 4 + 3 * unit;
        // (the bounds hold unless the workspace is written meanwhile)
        const int n = min(max(p[2], 1), TM), first = (int)min((int64_t)max(p[1], 0), a.M - n);
        if (tid < TM) {
            const int tk = tid < n ? a.plan[4 + 3 * a.max_tiles + max(first, 0) + tid] : 0;
            tile.toks[tid] = tk >= 0 && tk < a.M ? tk : 0;
        }
        if (tid == 0) tile.adapter = min(max(p[0], 0), a.adapters), tile.count = n;
        __syncthreads();
        return true;
    }
    const int M = (int)a.M, keys = a.adapters + 1;
    if (M <= 32) {  // one warp sees them all: the tokens of an adapter by their lanes
        if (warp == 0) {
            const int key = lane < M ? lora_key(a, lane) : -1;
            if (report && lane < M && a.which[lane] >= a.adapters) flag_value(a.status);
            const uint32_t same = __match_any_sync(0xffffffffu, key);
            const int tiles = key >= 0 && lane == __ffs(same) - 1 ? (__popc(same) + TM - 1) / TM : 0;
            int upto = tiles;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += u;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, unit >= upto - tiles && unit < upto);
            const int who = hit ? __ffs(hit) - 1 : 0;
            const uint32_t mine = __shfl_sync(0xffffffffu, same, who);
            const int nth = unit - __shfl_sync(0xffffffffu, upto - tiles, who), ad = __shfl_sync(0xffffffffu, key, who);
            const int r = __popc(mine & ((1u << lane) - 1u)) - nth * TM;
            if (hit && (mine >> lane & 1u) && r >= 0 && r < TM) tile.toks[r] = lane;
            if (lane == 0) {
                tile.adapter = hit ? ad : -1;
                tile.count = min(TM, __popc(mine) - nth * TM);
            }
        }
        __syncthreads();
        return tile.adapter >= 0;
    }
    __shared__ int hist[kLoraFind + 1], wsum[kWarps], tok_cnt[4][kWarps];
    int key[4];
    for (int i = tid; i < keys; i += kThreads) hist[i] = 0;
    if (tid < TM) tile.toks[tid] = -1;
    if (tid == 0) tile.adapter = -1;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int tk = i * kThreads + tid;
        key[i] = -1;
        if (tk < M) {
            key[i] = lora_key(a, tk);
            if (report && a.which[tk] >= a.adapters) flag_value(a.status);
            atomicAdd(&hist[key[i]], 1);
        }
    }
    __syncthreads();
    const int each = (keys + kThreads - 1) / kThreads;  // adapters of a thread, neighbours
    int mine = 0;
    for (int i = 0; i < each; ++i) {
        const int k = tid * each + i;
        if (k < keys) mine += (hist[k] + TM - 1) / TM;
    }
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += u;
    }
    if (lane == 31) wsum[warp] = upto;
    __syncthreads();
    int before = upto - mine;
    for (int i = 0; i < warp; ++i) before += wsum[i];
    if (mine > 0 && unit >= before && unit < before + mine) {
        int u = unit - before;
        for (int i = 0; i < each; ++i) {
            const int k = tid * each + i;
            if (k >= keys) break;
            const int n = (hist[k] + TM - 1) / TM;
            if (u < n) {
                tile.adapter = k;
                tile.nth = u;
                tile.count = min(TM, hist[k] - u * TM);
                break;
            }
            u -= n;
        }
    }
    __syncthreads();
    if (tile.adapter < 0) return false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t hit = __ballot_sync(0xffffffffu, key[i] == tile.adapter);
        if (lane == 0) tok_cnt[i][warp] = __popc(hit);
    }
    __syncthreads();
    int at = -tile.nth * TM;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t hit = __ballot_sync(0xffffffffu, key[i] == tile.adapter);
        int r = at;
        for (int w = 0; w < kWarps; ++w) {
            const int c = tok_cnt[i][w];
            if (w < warp) r += c;
            at += c;
        }
        r += __popc(hit & ((1u << lane) - 1u));
        if (key[i] == tile.adapter && r >= 0 && r < TM) tile.toks[r] = i * kThreads + tid;
    }
    __syncthreads();
    return true;
}

// ---- shrink, few tokens: 16 rows, the warps take chunks of 32 k (U in flight), operands from global memory to registers.
// VEC: rows start on 16 bytes.  NT: n-tiles of 8 ranks a pass.
template <typename T, int U, int NT, bool VEC>
__device__ __forceinline__ void shrink_small(const LoraArgs &a, const Tile<16> &tile, const Smem &sz, const T *A, int c0, int c1,
                                             float *part, float *red) {
    static_assert(NT <= Form<false>::NT, "the sums' buffer");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3, K = (int)a.K;
    const T *xr[2];
    bool live[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        live[i] = i * 8 + g < tile.count;
        xr[i] = static_cast<const T *>(a.x) + (int64_t)(live[i] ? tile.toks[i * 8 + g] : tile.toks[0]) * a.xs;
    }
    const int tiles = sz.ranks >> 3, passes = (tiles + NT - 1) / NT, np = (tiles + passes - 1) / passes;
    for (int j0 = 0; j0 < tiles; j0 += np) {
        const int nt = min(np, tiles - j0);
        float acc[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
        for (int c = c0 + warp; c < c1; c += U * kWarps) {
            uint4 xv[U][2], av[U][NT];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = (c + u * kWarps) * 32 + t * 8, n = c + u * kWarps < c1 ? K - k : 0;
#pragma unroll
                for (int i = 0; i < 2; ++i) xv[u][i] = load8(xr[i] + k, live[i] ? n : 0, VEC);
#pragma unroll
                for (int j = 0; j < NT; ++j) av[u][j] = load8(A + (int64_t)((j0 + j) * 8 + g) * K + k, j < nt ? n : 0, VEC);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t f0[4] = {xv[u][0].x, xv[u][1].x, xv[u][0].y, xv[u][1].y};
                const uint32_t f1[4] = {xv[u][0].z, xv[u][1].z, xv[u][0].w, xv[u][1].w};
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    if (j < nt) {
                        mma16816<T>(acc[j], f0, av[u][j].x, av[u][j].y);
                        mma16816<T>(acc[j], f1, av[u][j].z, av[u][j].w);
                    }
            }
        }
        // the warps' sums: of w and w + 4 by one of the two, then those four by all threads, in a fixed order
        constexpr int SUMS = 16 * NT * 8;
        float *const mine = red + (warp & 3) * SUMS + lane;
        __syncthreads();
        if (warp >= 4) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) mine[(j * 4 + e) * 32] = acc[j][e];
        }
        __syncthreads();
        if (warp < 4) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) mine[(j * 4 + e) * 32] += acc[j][e];
        }
        __syncthreads();
        for (int i = tid; i < nt * 128; i += kThreads) {
            const float *p = red + i;
            const int e = i >> 5 & 3, l = i & 31;
            part[((e >> 1) * 8 + (l >> 2)) * sz.pstride + (j0 + (i >> 7)) * 8 + 2 * (l & 3) + (e & 1)] =
                ((p[0] + p[SUMS]) + p[2 * SUMS]) + p[3 * SUMS];
        }
    }
}

// ---- shrink, many tokens: 128 rows of x and the adapter's rows of A, 64 k a stage (rows of 128 bytes, swizzled as the
// MMA reads them), copied by all warps; one of them issues a stage's MMAs once all have its copies.  (A ninth warp
// for that would leave 96 registers a thread instead of 128 with two blocks on an SM.)  Every wait gives up after a
// while: the sums are NaN then.  On return the sums are stored.
constexpr uint32_t kTmemCols = 128;  // of a block: the shrink's sums (up to 128 ranks), then two blocks of columns

// Returns the tensor memory, which the caller frees.
template <typename T>
__device__ __forceinline__ uint32_t shrink_big(const LoraArgs &a, const Tile<128> &tile, const Smem &sz, const T *A, int k0, int k1,
                                               unsigned char *ring, float *part) {
    using F = Form<true>;
    constexpr int ST = F::STAGES, LAG = F::LAG;
    __shared__ uint64_t full[ST], empty[ST], done, never;
    __shared__ uint32_t tmem_slot;
    __shared__ int dead;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&full[i], kThreads);
            mbar_init(&empty[i], 1);
        }
        mbar_init(&done, 1);
        mbar_init(&never, 1);
        dead = 0;
        fence_barrier_init();
    }
    constexpr int kIssuer = kWarps - 1;
    if (warp == kIssuer) tc::tmem_alloc(&tmem_slot, kTmemCols);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = tmem_slot;
    const int n = (k1 - k0 + 63) / 64;
    const uint32_t idesc = tc::idesc_f16(16, std::is_same<T, __nv_bfloat16>::value) - (2u << 17) + ((uint32_t)(sz.npad >> 3) << 17);
    // eight lanes copy a row's 128 bytes: a warp's request is four whole lines
    const int row = tid >> 3, c = tid & 7;  // rows row + 32 i
    const T *x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = row + 32 * i;
        x[i] = static_cast<const T *>(a.x) + (int64_t)tile.toks[r < tile.count ? r : 0] * a.xs + c * 8;
    }
    const T *const w = A + (int64_t)row * a.K + c * 8;
    const uint32_t base = smem_u32(ring) + row * 128 + ((c ^ (row & 7)) << 4);  // (32 i rows on, the swizzle is the same)
    bool ok = true;
    if (a.stall && warp == kIssuer) ok = __all_sync(0xffffffffu, mbar_wait_bounded(&never, 0, a.wait_limit));
    // a stage's copies of this thread have landed: say so; the issuer waits for all and multiplies
    const auto landed = [&](int it) {
        const int s = it % ST;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        mbar_arrive(&full[s]);
        if (warp != kIssuer) return;
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&full[s], (it / ST) & 1, a.wait_limit));
        if (!ok) return;
        tc::fence_after_sync();
        if (tc::elect_one()) {
            const uint64_t xd = tc::desc_sw128(ring + s * sz.stage), ad = tc::desc_sw128(ring + s * sz.stage + 128 * 128);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) tc::mma_ss(tm, xd + kk * 2, ad + kk * 2, idesc, (it | kk) != 0);
            tc::commit(&empty[s]);
        }
        __syncwarp();
    };
    for (int it = 0; it < n && ok; ++it) {
        const int s = it % ST;
        if (it >= ST) ok = __all_sync(0xffffffffu, mbar_wait_bounded(&empty[s], (it / ST - 1) & 1, a.wait_limit));
        if (!ok) break;
        const uint32_t dst = base + s * sz.stage;
        const int k = k0 + it * 64;
        const bool in = k + c * 8 < k1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = row + 32 * i;
            const bool xi = in && r < tile.count, wi = in && r < sz.ranks;
            copy16(dst + i * 4096, xi ? x[i] + k : static_cast<const T *>(a.x), xi);
            if (r < sz.npad) copy16(dst + 16384 + i * 4096, wi ? w + (int64_t)(32 * i) * a.K + k : A, wi);
        }
        copies_commit();
        if (it >= LAG) {
            copies_wait<LAG>();
            landed(it - LAG);
        }
    }
    copies_wait<0>();
    for (int it = max(0, n - LAG); it < n && ok; ++it) landed(it);
    if (!ok) dead = 1;
    if (warp == kIssuer) {
        if (tc::elect_one()) tc::commit(&done);
        __syncwarp();
    }
    // all MMAs that were issued have ended (or the default limit is over): nothing reads the ring
    if (!mbar_wait_bounded(&done, 0)) dead = 1;
    __syncthreads();
    tc::fence_after_sync();
    const bool bad = dead != 0;
    if (bad && tid == 0) atomicExch(a.status, kStatusTimeout);
    if (warp < 4) {  // lane = row
        float *const row = part + (warp * 32 + lane) * sz.pstride;
        for (int c = 0; c < sz.npad; c += 16) {
            uint32_t r[16];
            tc::ld_32x32b_x16(tm + ((uint32_t)(warp * 32) << 16) + c, r);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                if (c + i < sz.ranks) {
                    const float none = bad ? __uint_as_float(0x7FC00000u) : 0.f;  // (a run of K may be empty)
                    *reinterpret_cast<float4 *>(row + c + i) =
                        bad || n == 0 ? make_float4(none, none, none, none)
                                      : make_float4(__uint_as_float(r[i]), __uint_as_float(r[i + 1]), __uint_as_float(r[i + 2]), __uint_as_float(r[i + 3]));
                }
        }
        tc::fence_before_sync();
    }
    __syncthreads();
    return tm;
}

// ---- expand, few tokens: a block of 8 J columns (gated: of either half), any sizes.  B's loads of a step of 16 ranks are waited for
// one after the other: 16 tokens of 8 adapters over the fused QKV of 3584 take 10.5 us at rank 24, 12.7 at 40, 16.5 at 64 and 33 at
// 128, where ExpandSmall takes 7.1 at 16 and 9.1 at 32; over a gated layer of 2 x 18944 39 us at 24 and 62 at 64, 11 at 16.
template <typename T, typename O, bool GATED>
__device__ __forceinline__ void expand(const LoraArgs &a, const Tile<16> &tile, const Smem &sz, const T *hs, const float *up, const T *B,
                                       int sh, int64_t off, int64_t wide, int64_t blk) {
    constexpr int TM = 16, G = 1, r0 = 0;
    constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
    constexpr int NS = kBf && sizeof(O) == 4 ? 3 : 2;
    constexpr int J = GATED ? 2 : 4, W = 2 * J, H = GATED ? 2 : 1;  // n-tiles a block; contiguous columns of a thread; halves
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, R = a.R, steps = (R + 15) / 16;
    const bool has = B != nullptr;
    const O *const y = static_cast<const O *>(a.y);
    O *const out = static_cast<O *>(a.out);
    const int64_t col = off + blk * (J * 8);
    const int left = (int)min((int64_t)(J * 8), wide - blk * (J * 8)), n = left - t * W;
    Raw<O, W> yv[H][2 * G];
#pragma unroll
    for (int i = 0; i < 2 * G; ++i) {
        const int row = r0 + i * 8 + g;
        if (row < tile.count && n > 0) {
            const O *p = y + tile.toks[row] * a.ys + col + t * W;
#pragma unroll
            for (int q = 0; q < H; ++q) yv[q][i].load(p + q * wide, n, a.vec_y);
        }
    }
    float acc[H][G][J][4];
#pragma unroll
    for (int q = 0; q < H; ++q)
#pragma unroll
        for (int i = 0; i < G; ++i)
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[q][i][j][e] = 0.f;
    for (int st = 0; has && st < steps; ++st) {
        uint2 bv[H][J];
        const int r = st * 16 + 4 * t;
#pragma unroll
        for (int q = 0; q < H; ++q)
#pragma unroll
            for (int j = 0; j < J; ++j) {
                // column of the fragment's n = g: such that a thread's results are neighbours
                const int c = (g >> 1) * W + 2 * j + (g & 1);
                bv[q][j] = c < left && r < R ? ldg_nc_v2(B + (q * wide + col + c) * R + r) : make_uint2(0, 0);
            }
#pragma unroll
        for (int i = 0; i < G; ++i)
#pragma unroll
            for (int q = 0; q < H; ++q)
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    const T *h = hs + (s * TM + r0 + i * 16 + g) * sz.hstride + ((GATED ? q : sh) * steps + st) * 16 + 4 * t;
                    const uint2 x = *reinterpret_cast<const uint2 *>(h), z = *reinterpret_cast<const uint2 *>(h + 8 * sz.hstride);
                    const uint32_t f[4] = {x.x, z.x, x.y, z.y};
#pragma unroll
                    for (int j = 0; j < J; ++j) mma16816<T>(acc[q][i][j], f, bv[q][j].x, bv[q][j].y);
                }
    }
#pragma unroll
    for (int i = 0; i < 2 * G; ++i) {
        const int row = r0 + i * 8 + g;
        if (row >= tile.count || n <= 0) continue;
        const float f = !has ? 0.f : kBf ? 1.f : up[row];
        float v[W];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            v[j] = yv[0][i][j];
            if (has) v[j] = __fmaf_rn(acc[0][i >> 1][j >> 1][2 * (i & 1) + (j & 1)], f, v[j]);
            if constexpr (GATED) {
                float w = yv[1][i][j];
                if (has) w = __fmaf_rn(acc[1][i >> 1][j >> 1][2 * (i & 1) + (j & 1)], f, w);
                v[j] = silu<O>(v[j]) * w;
            }
        }
        store_out<O, W>(out + tile.toks[row] * a.os + col + t * W, n, a.vec_y, v);
    }
}

// ---- expand, few tokens, where blocks of columns are whole and start on 16 bytes and the rank is 8, 16 or 32.  B's
// rows (columns of the output) are the wide side of the MMA and 8 tokens the narrow one, so that no MMA row is idle
// with 8 tokens or more, and a thread has W neighbouring columns of two tokens.  Each warp copies its blocks' B and y
// into two stages of its own, the first ones before the shrink (gated: while the sums are joined).
template <typename O, bool GATED>
struct Blocks {
    static constexpr int W = GATED ? 4 : 8, H = GATED ? 2 : 1;  // columns of a thread; halves
    static constexpr int COLS = 8 * W;                          // columns of a block (gated: of either half)
    static constexpr int YROW = COLS * sizeof(O);               // bytes of a token's columns
    static constexpr int YBYTES = 16 * H * YROW;
    __host__ __device__ static constexpr int stage(int R) { return H * COLS * R * 2 + YBYTES; }
    __host__ __device__ static bool ranks(int R) { return R == 8 || R == 16 || R == 32; }
    // place of byte `at` of a half's rows of B that belongs to the columns of threads g: 32-byte granules of 4 threads'
    // columns exchange places, which leaves no bank conflicts
    __device__ static uint32_t b_place(int at, int g) { return (uint32_t)(at ^ ((g & 3) << 5)); }
    // place of 16-byte piece c of token row r (rows of 64 bytes: two of them span the banks)
    __device__ static uint32_t y_piece(int r, int c) { return (uint32_t)(r * YROW + ((c ^ ((r & 3) << (YROW == 64 ? 0 : 1))) << 4)); }
    // place of token row r in the split h: a thread's two tokens are t and t + 4 of a group of 8, so that groups of up to
    // 4 tokens take half the work
    __device__ static int h_row(int r) { return (r & 8) | ((r & 3) << 1) | ((r >> 2) & 1); }
};

// What a thread reads and writes lies at places that it works out once (R is a template's for that): a block of columns took
// three times the instructions with places worked out anew.
template <typename T, typename O, bool GATED, int R>
struct ExpandSmall {
    using L = Blocks<O, GATED>;
    static constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
    static constexpr int NS = kBf && sizeof(O) == 4 ? 3 : 2, STEPS = (R + 15) / 16;
    static constexpr int W = L::W, H = L::H, I = W / 2, STAGE = L::stage(R);
    static constexpr int BHALF = L::COLS * R * 2, YHALF = 16 * L::YROW;      // bytes of a half's B and y in a stage
    static constexpr int BI = BHALF / 512, C = L::YROW / 16, YI = 16 * C / 32, YSTEP = 32 / C;  // copies of a lane; pieces and rows
    static constexpr int SHIFT = W * R == 32 ? 2 : W * R == 64 ? 3 : W * R == 128 ? 4 : 5;  // log2 of the pieces of a thread's columns
    static constexpr int YX = L::YROW == 64 ? 0 : 1;
    const LoraArgs &a;
    const T *bp;       // the lane's first piece of block 0's B
    const O *yp[YI];   // and of its rows of y
    uint32_t base, bto, yto;
    int first, kk, total, count, lane;
    bool has;          // there is an adapter: else y goes through as it is (gated: through the product)

    __device__ __forceinline__ ExpandSmall(const LoraArgs &args, const Tile<16> &tile, const T *B, uint32_t base_, int first_, int kk_)
        : a(args), base(base_), first(first_), kk(kk_), count(tile.count), lane(threadIdx.x & 31), has(B != nullptr) {
        // (shards are whole blocks: block n has columns n COLS on, whatever shard they are in)
        total = (int)((GATED ? a.shard[0] : launch_columns()) / L::COLS);
        bp = B + a.col0 * R + lane * 8;
        bto = (uint32_t)(lane * 16 ^ ((lane >> SHIFT & 3) << 5));
        yto = H * BHALF + L::y_piece(lane / C, lane % C);
#pragma unroll
        for (int i = 0; i < YI; ++i) {
            const int r = i * YSTEP + lane / C;
            yp[i] = static_cast<const O *>(a.y) + (int64_t)tile.toks[r < count ? r : 0] * a.ys + a.col0 + lane % C * (16 / (int)sizeof(O));
        }
    }
    __device__ __forceinline__ int64_t launch_columns() const {
        int64_t n = 0;
        for (int i = 0; i < a.S; ++i) n += a.shard[i];
        return n;
    }
    __device__ __forceinline__ void copy(int stage, int n) const {
        if (n < total) {
            const uint32_t to = base + stage * STAGE;
            const T *b = bp + (int64_t)n * (L::COLS * R);
#pragma unroll
            for (int q = 0; q < H; ++q) {
                if (!has) break;
#pragma unroll
                for (int i = 0; i < BI; ++i)
                    copy16(to + q * BHALF + i * 512 + (bto ^ ((((i << (5 - SHIFT)) & 3) << 5))), b + i * 256, true);
                b += a.shard[0] * R;
            }
#pragma unroll
            for (int i = 0; i < YI; ++i)
                if (i * YSTEP + lane / C < count) {
                    const O *y = yp[i] + (int64_t)n * L::COLS;
#pragma unroll
                    for (int q = 0; q < H; ++q) {
                        copy16(to + q * YHALF + i * YSTEP * L::YROW + (yto ^ ((i * YSTEP & 3) << YX << 4)), y, true);
                        y += a.shard[0];
                    }
                }
        }
        copies_commit();
    }
    __device__ __forceinline__ void copy_first() const {
        copy(0, first);
        copy(1, first + kk);
    }
    // rows: where the tile's tokens are in out
    __device__ __forceinline__ void run(const Smem &sz, const T *hs, const float *up, char *const *rows) const {
        const int g = lane >> 2, t = lane & 3;
        const bool two = count > 8;  // the second group of 8 tokens has some
        const T *h0 = hs + g * sz.hstride + 4 * t;
        // the rows of B of a thread's columns: the bits that are exchanged (5 and 6) in four registers, the others are added
        uint32_t bx[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) bx[j] = base + (uint32_t)((g * W * R * 2 + 8 * t) ^ (((g & 3) ^ j) << 5));
        // (a row of 16 bytes has two loads of 8: threads t < 2)
        const uint32_t y0 = base + H * BHALF + t * L::YROW +
                            (W * sizeof(O) == 8 ? (((g >> 1) ^ (t << YX)) << 4) + (g & 1) * 8 : ((g * (W * (int)sizeof(O) / 16)) ^ (t << YX)) << 4);
        const uint32_t at = (uint32_t)(a.col0 + g * W);
        int sh = 0, end = GATED ? total : (int)(a.shard[0] / L::COLS);
        int stage = 0;
        for (int now = first; now < total; now += kk) {
            copies_wait<1>();
            __syncwarp();
            if constexpr (!GATED) {
                while (now >= end) {
                    ++sh;
                    end += (int)(a.shard[sh] / L::COLS);
                    h0 += STEPS * 16;
                }
            }
            const uint32_t off = (uint32_t)(stage * STAGE);
#pragma unroll
            for (int n8 = 0; n8 < 2; ++n8) {
                if (n8 == 1 && !two) break;
                float acc[H][I][4];
                if (!has) {
#pragma unroll
                    for (int q = 0; q < H; ++q)
#pragma unroll
                        for (int m = 0; m < I; ++m)
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[q][m][e] = 0.f;
                } else
#pragma unroll
                for (int z = 0; z < STEPS; ++z)
#pragma unroll
                    for (int q = 0; q < H; ++q) {
                        uint2 h[NS];
#pragma unroll
                        for (int n = 0; n < NS; ++n)
                            h[n] = *reinterpret_cast<const uint2 *>(h0 + (n * 16 + n8 * 8) * sz.hstride + (q * STEPS + z) * 16);
#pragma unroll
                        for (int m = 0; m < I; ++m) {
                            uint2 x = make_uint2(0, 0), v = make_uint2(0, 0);
                            const int c0 = 2 * m * R * 2 + z * 32, c1 = c0 + R * 2;  // (fields of bits apart from g's and t's)
                            if (R >= 16 || t < 2) {
                                x = lds8(bx[c0 >> 5 & 3] + off + q * BHALF + (c0 & ~96));
                                v = lds8(bx[c1 >> 5 & 3] + off + q * BHALF + (c1 & ~96));
                            }
                            const uint32_t f[4] = {x.x, v.x, x.y, v.y};
                            if (z == 0) mma16816_first<T>(acc[q][m], f, h[0].x, h[0].y);
#pragma unroll
                            for (int n = z == 0 ? 1 : 0; n < NS; ++n) mma16816<T>(acc[q][m], f, h[n].x, h[n].y);
                        }
                    }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = n8 * 8 + t + 4 * e;
                    if (row >= count) continue;
                    const float f = kBf || !has ? 1.f : up[row];
                    Raw<O, W> yv[H];
#pragma unroll
                    for (int q = 0; q < H; ++q) {
                        const uint32_t yr = y0 + off + q * YHALF + (n8 * 8 + 4 * e) * L::YROW;
                        if constexpr (Raw<O, W>::WORDS == 2) {
                            const uint2 r = lds8(yr);
                            yv[q].w[0] = r.x, yv[q].w[1] = r.y;
                        } else {
#pragma unroll
                            for (int c = 0; c < Raw<O, W>::WORDS / 4; ++c) {
                                const uint4 r = lds16(yr + c * 16);
                                yv[q].w[4 * c] = r.x, yv[q].w[4 * c + 1] = r.y, yv[q].w[4 * c + 2] = r.z, yv[q].w[4 * c + 3] = r.w;
                            }
                        }
                    }
                    float o[W];
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        o[j] = __fmaf_rn(acc[0][j >> 1][2 * (j & 1) + e], f, yv[0][j]);
                        if constexpr (GATED) o[j] = silu<O>(o[j]) * __fmaf_rn(acc[1][j >> 1][2 * (j & 1) + e], f, yv[1][j]);
                    }
                    O *const p = reinterpret_cast<O *>(rows[row]) + (at + (uint32_t)now * (uint32_t)L::COLS);
                    store_out<O, W>(p, W, true, o);
                }
            }
            __syncwarp();  // the stage is read by all
            copy(stage, now + 2 * kk);
            stage ^= 1;
        }
        copies_wait<0>();
    }
};

// f with R as a constant, where Blocks::ranks(R)
template <typename F>
__device__ __forceinline__ void with_rank(int R, F f) {
    if (R == 8) f(std::integral_constant<int, 8>{});
    else if (R == 16) f(std::integral_constant<int, 16>{});
    else f(std::integral_constant<int, 32>{});
}

// ---- expand, many tokens: blocks of 64 columns (32 of fp32) of a shard, dealt to the cluster's blocks; a shard's last may
// be cut short (to eights that start on 16 bytes: the launcher's rule).  The split h (K-major, swizzled as the MMA reads it) times a block's rows of B on tcgen05,
// into one of two accumulators while the other's columns are added to y.  B is copied three blocks of columns ahead, y
// two; a warp has 32 rows of half the columns, reads a row of its accumulator a thread, and goes through its
// stage of y, so that global memory is read and written in 64-byte pieces of rows.  8192 tokens of 6 adapters, 18944 to 3584:
// 103 us; by warp MMAs with B in registers 119 (their rate alone 20).  Stores hold it up most (12 us, the products 6, y 3).
// B null: y goes through as it is.
template <typename T, typename O>
struct ExpandBig {
    static constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
    static constexpr int NS = kBf && sizeof(O) == 4 ? 3 : 2;
    static constexpr int COLS = 128 / sizeof(O), HALF = COLS / 2, W = 16 / sizeof(O);  // columns of a block, of a warp, of 16 bytes
    static constexpr int B_STAGE = COLS * 128, B_STAGES = 4, Y_STAGE = 2048;

    const LoraArgs &a;
    const Smem &sz;
    unsigned char *const smem;
    const T *const B;
    const char *const *const yrow;
    char *const *const orow;
    const int count, rank, lane, warp, steps;

    __device__ __forceinline__ static uint32_t y_place(int row, int c) { return (uint32_t)(row * 64 + ((c ^ (row >> 1 & 3)) << 4)); }
    __device__ __forceinline__ uint32_t y_stage(int s) const { return smem_u32(smem) + B_STAGES * B_STAGE + (warp * 2 + s) * Y_STAGE; }
    // block n: its shard, first column and columns
    struct Place {
        int sh, col, left;
    };
    __device__ __forceinline__ Place locate(int n) const {
        Place p{0, (int)a.col0, (int)a.shard[0]};
        for (int blocks; n >= (blocks = (p.left + COLS - 1) / COLS) && p.sh + 1 < a.S; n -= blocks) p.col += p.left, p.left = (int)a.shard[++p.sh];
        p.col += n * COLS;
        p.left -= n * COLS;
        return p;
    }
    // the lane's 16 bytes of rows of the warp's half: where they begin; none where the block is cut short before them
    __device__ __forceinline__ uint32_t y_column(const Place &p) const {
        return (uint32_t)(p.col + (warp >> 2) * HALF + (lane & 3) * W) * (uint32_t)sizeof(O);
    }
    __device__ __forceinline__ bool y_there(const Place &p) const { return (warp >> 2) * HALF + (lane & 3) * W < p.left; }
    __device__ __forceinline__ void copy_b(const Place &at, int s) const {
        if (B) {
            const int c = threadIdx.x >> 2;
            if (c < COLS && c < at.left) {  // (what is behind stays what it was: columns do not meet)
                const T *const b = B + (int64_t)(at.col + c) * a.R;
                const uint32_t to = smem_u32(smem) + s * B_STAGE + c * 128;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int p = (threadIdx.x & 3) + 4 * i;  // (zeros up to whole steps of 16 ranks)
                    if (p < 2 * steps) copy16(to + ((p ^ (c & 7)) << 4), p * 8 < a.R ? b + p * 8 : b, p * 8 < a.R);
                }
            }
        }
    }
    __device__ __forceinline__ void copy_y(const Place &p, int s) const {
        const uint32_t at = y_column(p), to = y_stage(s);
        const int rows = y_there(p) ? count : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = i * 8 + (lane >> 2), all = (warp & 3) * 32 + row;
            if (all < rows) copy16(to + y_place(row, lane & 3), yrow[all] + at, true);
        }
    }
    // tm: tensor memory of two accumulators; done: their barriers.  False: a wait gave up (the results are NaN).
    __device__ __forceinline__ bool run(const float *up, uint32_t tm, uint64_t *done) const {
        int blocks = 0;
        for (int i = 0; i < a.S; ++i) blocks += ((int)a.shard[i] + COLS - 1) / COLS;
        const int C = a.C, n = rank < blocks ? (blocks - 1 - rank) / C + 1 : 0;
        const uint32_t idesc = tc::idesc_f16(COLS, kBf);
        bool ok = true;
        const auto copy = [&](int i, bool b, bool y) {
            if (i >= n) return;
            const Place p = locate(rank + i * C);
            if (b) copy_b(p, i % B_STAGES);
            if (y) copy_y(p, i & 1);
        };
        const auto multiply = [&](int i) {
            const int sh = locate(rank + i * C).sh;
            tc::fence_after_sync();
            if (tc::elect_one()) {
                const uint64_t bd = tc::desc_sw128(smem + i % B_STAGES * B_STAGE);
                for (int q = 0; q < NS; ++q) {
                    const uint64_t hd = tc::desc_sw128(smem + sz.split + (q * sz.htiles + sh / sz.hper) * 16384) + sh % sz.hper * steps * 2;
                    for (int z = 0; z < steps; ++z) tc::mma_ss(tm + (i & 1) * COLS, hd + z * 2, bd + z * 2, idesc, (q | z) != 0);
                }
                tc::commit(&done[i & 1]);
            }
            __syncwarp();
        };
        // groups of copies, in the order in which they are waited for
        copy(0, true, false);
        copies_commit();
        copy(1, true, false);
        copy(0, false, true);
        copies_commit();
        copy(2, true, false);
        copies_commit();
        copy(1, false, true);
        copies_commit();
        copies_wait<3>();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();
        if (B && n > 0 && warp == 0) multiply(0);
        const int row0 = (warp & 3) * 32;
        for (int i = 0; i < n; ++i) {
            const int s = i & 1;
            copy(i + 3, true, false);
            copies_commit();
            copies_wait<3>();  // the next block's B and this one's y have landed
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            tc::fence_before_sync();
            __syncthreads();
            if (B && i + 1 < n && warp == 0) multiply(i + 1);
            if (B && ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(&done[s], (i >> 1) & 1));
            if (row0 < count) {
                uint32_t acc[HALF];
                if (B && ok) {
                    tc::fence_after_sync();
                    const uint32_t from = tm + ((uint32_t)row0 << 16) + s * COLS + (warp >> 2) * HALF;
                    if constexpr (HALF == 32) tc::ld_32x32b_x32(from, acc);
                    else tc::ld_32x32b_x16(from, acc);
                    tc::wait_ld();
                } else {
#pragma unroll
                    for (int c = 0; c < HALF; ++c) acc[c] = ok ? 0u : 0x7FC00000u;
                }
                const float f = kBf || !B ? 1.f : up[row0 + lane];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t at = y_stage(s) + y_place(lane, c);
                    const uint4 q = lds16(at);
                    Raw<O, W> y;
                    y.w[0] = q.x, y.w[1] = q.y, y.w[2] = q.z, y.w[3] = q.w;
                    O v[W];
#pragma unroll
                    for (int e = 0; e < W; ++e) v[e] = of_f<O>(__fmaf_rn(__uint_as_float(acc[c * W + e]), f, y[e]));
                    sts16(at, *reinterpret_cast<const uint4 *>(v));
                }
                __syncwarp();
                const Place p = locate(rank + i * C);
                const uint32_t at = y_column(p);
                const int rows = y_there(p) ? count : 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int row = j * 8 + (lane >> 2);
                    if (row0 + row < rows) *reinterpret_cast<uint4 *>(orow[row0 + row] + at) = lds16(y_stage(s) + y_place(row, lane & 3));
                }
                __syncwarp();  // the stage is read by all
            }
            copy(i + 2, false, true);
            copies_commit();
        }
        copies_wait<0>();
        return ok;
    }
};

// O: type of y and out.
template <typename T, typename O, bool BIG, bool GATED>
__global__ void __launch_bounds__(kThreads, GATED ? 3 : 2) lora_kernel(const __grid_constant__ LoraArgs a) {
    static_assert(!(BIG && GATED), "gated layers keep to tiles of 16");
    using F = Form<BIG>;
    constexpr int TM = F::TM;
    constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
    constexpr int NS = kBf && sizeof(O) == 4 ? 3 : 2;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    unsigned char *const smem = BIG ? smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u) : smem_raw;
    __shared__ Tile<TM> tile;
    __shared__ float up[TM];       // what a row of the split h has to be multiplied by (f16)
    __shared__ float row_top[TM];  // f16: largest magnitude of a row of the partial sums
    __shared__ char *out_row[TM];
    __shared__ const char *y_row[BIG ? TM : 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = a.C, rank = (int)(blockIdx.x % (unsigned)C);
    const int unit = (int)(blockIdx.x / (unsigned)C);
    if (C > 1) cluster_arrive_relaxed();
    // (tiles of 128 hold tensor memory: a kernel that came early might take it first and wait for this one)
    if (!BIG) pdl_launch_dependents();
    pdl_wait();
    const bool any = find_tile<TM>(a, tile, unit, unit == 0 && rank == 0);
    const int ad = any ? tile.adapter : a.adapters;
    const bool has = ad < a.adapters;
    if (!any || (!has && !GATED && a.out == a.y)) {  // fewer tiles, or tokens to which nothing is added in place
        // (meeting the others at every barrier all the same: should `which` change meanwhile, a block that found a
        // tile reads this one's memory)
        if (C > 1) {
            cluster_wait();
            for (int i = 0; i < 2; ++i) {
                cl_arrive_release();
                cl_wait_acquire();
            }
        }
        return;
    }
    const int S = a.S, R = a.R, K = (int)a.K, steps = (R + 15) / 16;
    using L = Blocks<O, GATED>;
    const bool whole = !BIG && a.whole;  // blocks of columns for ExpandSmall
    const Smem sz(BIG, GATED, S, R, NS, whole ? L::stage(R) : 0);
    float *const part = reinterpret_cast<float *>(smem);
    T *const hs = reinterpret_cast<T *>(smem + sz.split);
    const T *const B = has ? static_cast<const T *>(a.b) + (int64_t)ad * a.N * R : nullptr;
    const int w0 = rank * kWarps + warp, kk = C * kWarps;
    uint32_t tmem = 0;
    if (BIG && tid < tile.count) y_row[tid] = reinterpret_cast<const char *>(static_cast<const O *>(a.y) + tile.toks[tid] * a.ys);
    if ((BIG || whole) && tid < tile.count) out_row[tid] = reinterpret_cast<char *>(static_cast<O *>(a.out) + tile.toks[tid] * a.os);
    const auto copy_first = [&] {
        if constexpr (!BIG)
            with_rank(R, [&](auto r) {
                ExpandSmall<T, O, GATED, decltype(r)::value>(a, tile, B, smem_u32(smem + sz.blocks) + warp * 2 * L::stage(R), w0, kk).copy_first();
            });
    };
    if constexpr (!BIG && !GATED) {
        if (whole) copy_first();
    }
    if (has) {
        const T *const A = static_cast<const T *>(a.a) + ((int64_t)ad * a.ranks + a.rank0) * K;
        if constexpr (BIG) {
            const int chunks = (K + 63) / 64, per = (chunks + C - 1) / C, c0 = min(chunks, rank * per), c1 = min(chunks, c0 + per);
            tmem = shrink_big<T>(a, tile, sz, A, c0 * 64, min(K, c1 * 64), smem, part);
        } else {
            const int chunks = (K + 31) / 32, per = (chunks + C - 1) / C, c0 = min(chunks, rank * per), c1 = min(chunks, c0 + per);
            float *const red = reinterpret_cast<float *>(smem + sz.red);
            constexpr int NT = GATED ? 4 : Form<false>::NT;  // (gated: what 80 registers hold with two loads of each in flight)
            if (a.vec_x) shrink_small<T, 2, NT, true>(a, tile, sz, A, c0, c1, part, red);
            else shrink_small<T, 1, NT, false>(a, tile, sz, A, c0, c1, part, red);
            __syncthreads();
        }
    }
    if (GATED && whole) copy_first();
    if (!kBf && has) {
        for (int row = warp; row < tile.count; row += kWarps) {
            float top = 0.f;
            bool odd = false;
            for (int e = lane; e < sz.ranks; e += 32) {
                const float v = fabsf(part[row * sz.pstride + e]);
                odd = odd || !isfinite(v);
                top = fmaxf(top, v);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            odd = __any_sync(0xffffffffu, odd);
            if (lane == 0) row_top[row] = odd ? __uint_as_float(0x7F800000u) : top;
        }
        __syncthreads();
    }
    if (C > 1) {
        cluster_wait();  // (every block has started)
        cl_arrive_release();
        cl_wait_acquire();
    }
    if (has) {
        // ---- h = s (the blocks' sums, in their order), split into NS numbers of T
        const float s = a.scale ? a.scale[ad] : 1.f;
        if constexpr (!kBf) {
            // f16: a row scaled such that the sum of its blocks' largest lies in [2^14, 2^15); one with an infinity or a
            // NaN as it is
            if (tid < TM) {
                float top = 0.f;
                for (int i = 0; i < C; ++i) top += C > 1 ? cl_ld_f32(cl_map(smem_u32(&row_top[tid]), i)) : row_top[tid];
                const uint32_t ex = max((__float_as_uint(top * s) & 0x7FFFFFFFu) >> 23, 15u);
                up[tid] = ex < 255u ? __uint_as_float((ex - 14u) << 23) : 1.f;
            }
            __syncthreads();
        }
        const int quads = steps * 4, row_quads = S * quads;
        constexpr int U = BIG ? 4 : 2;
        // BIG: a block joins a share of the rows and gives them to all; few tokens: every block joins all
        const int per_block = BIG ? (tile.count + C - 1) / C : tile.count, row0 = BIG ? min(rank * per_block, tile.count) : 0;
        const int rows_end = min(row0 + per_block, tile.count);
        for (int i0 = tid; i0 < (rows_end - row0) * row_quads; i0 += U * kThreads) {
            float4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * kThreads, in = i / row_quads, row = row0 + in, e = i - in * row_quads, sh = e / quads, r = (e - sh * quads) * 4;
                v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (row < rows_end && r < R) {
                    const float *p = part + row * sz.pstride + sh * R + r;
                    if (C == 1) {
                        v[u] = *reinterpret_cast<const float4 *>(p);
                    } else {
                        const uint32_t at = smem_u32(p);
                        for (int c = 0; c < C; ++c) {
                            const float4 x = cl_ld_v4(cl_map(at, c));
                            v[u].x += x.x, v[u].y += x.y, v[u].z += x.z, v[u].w += x.w;
                        }
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * kThreads, in = i / row_quads, row = row0 + in, e = i - in * row_quads;
                if (row >= rows_end) continue;
                const float f = kBf ? 1.f : 1.f / up[row];  // (a power of two)
                const int place = whole ? L::h_row(row) : row;
                float z[4] = {v[u].x * s * f, v[u].y * s * f, v[u].z * s * f, v[u].w * s * f};
#pragma unroll
                for (int n = 0; n < NS; ++n) {
                    T h[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        h[j] = of_f<T>(z[j]);
                        z[j] = isfinite(to_f(h[j])) ? z[j] - to_f(h[j]) : 0.f;
                    }
                    const uint2 w = *reinterpret_cast<const uint2 *>(h);
                    if constexpr (BIG) {
                        const int sh = e / quads, k = sh % sz.hper * steps * 16 + (e - sh * quads) * 4;
                        unsigned char *const at = smem + sz.split + (n * sz.htiles + sh / sz.hper) * 16384 + row * 128 +
                                                  (((k >> 3) ^ (row & 7)) << 4) + (k & 4) * 2;
                        if (C == 1) *reinterpret_cast<uint2 *>(at) = w;
                        else
                            for (int c = 0; c < C; ++c) cl_st_v2(cl_map(smem_u32(at), c), w);
                    } else {
                        *reinterpret_cast<uint2 *>(hs + (n * TM + place) * sz.hstride + e * 4) = w;
                    }
                }
            }
        }
    }
    if (BIG) asm volatile("fence.proxy.async;" ::: "memory");  // (h, of any block of the cluster, is read by MMAs)
    __syncthreads();
    if (C > 1) cl_arrive_release();  // the others' sums are read
    if constexpr (BIG) {
        __shared__ uint64_t expanded[2];
        if (C > 1) cl_wait_acquire();  // (the stages of B and y lie where the sums were)
        if (tid == 0) {
            mbar_init(&expanded[0], 1);
            mbar_init(&expanded[1], 1);
            fence_barrier_init();
        }
        __syncthreads();
        const ExpandBig<T, O> ex{a, sz, smem, B, y_row, out_row, tile.count, rank, lane, warp, steps};
        const bool ok = ex.run(up, tmem, expanded);
        if (!ok && lane == 0) atomicExch(a.status, kStatusTimeout);
        tc::fence_before_sync();
        __syncthreads();
        if (has && warp == kWarps - 1) tc::tmem_dealloc(tmem, kTmemCols);
    } else {
        // columns in blocks, dealt to the cluster's warps
        constexpr int J = GATED ? 2 : 4;
        if (whole)
            with_rank(R, [&](auto r) {
                ExpandSmall<T, O, GATED, decltype(r)::value>(a, tile, B, smem_u32(smem + sz.blocks) + warp * 2 * L::stage(R), w0, kk)
                    .run(sz, hs, up, out_row);
            });
        int64_t skip = w0, off = a.col0;  // blocks before this warp's next one
        for (int sh = 0; sh < (GATED ? 1 : S) && !whole; ++sh) {
            const int64_t wide = a.shard[sh], blocks = (wide + J * 8 - 1) / (J * 8);
            for (int64_t blk = skip; blk < blocks; blk += kk) expand<T, O, GATED>(a, tile, sz, hs, up, B, sh, off, wide, blk);
            skip = skip >= blocks ? skip - blocks : kk - 1 - (blocks - 1 - skip) % kk;
            off += wide;
        }
    }
    if (!BIG && C > 1) cl_wait_acquire();
}

constexpr int kMaxSmem = 200 * 1024;

template <typename T, typename O, bool BIG, bool GATED>
cudaError_t launch_one(const LoraArgs &a, int units, cudaStream_t st) {
    constexpr int NS = std::is_same<T, __nv_bfloat16>::value && sizeof(O) == 4 ? 3 : 2;
    using L = Blocks<O, GATED>;
    LoraArgs b = a;
    b.whole = !BIG && a.vec_y && L::ranks(a.R);
    for (int i = 0; i < a.S; ++i) b.whole = b.whole && a.shard[i] % L::COLS == 0;
    Smem sz(BIG, GATED, a.S, a.R, NS, b.whole ? L::stage(a.R) : 0);
    if (sz.total > kMaxSmem && b.whole) {
        b.whole = 0;
        sz = Smem(BIG, GATED, a.S, a.R, NS, 0);
    }
    static std::atomic<uint64_t> done{0};
    if (const cudaError_t e = allow_smem(done, lora_kernel<T, O, BIG, GATED>, kMaxSmem)) return e;
    return launch_chained(lora_kernel<T, O, BIG, GATED>, (unsigned)units * (unsigned)a.C, kThreads, sz.total, (unsigned)a.C, st, b);
}

template <typename T>
cudaError_t launch_type(const LoraArgs &a, bool f32, bool big, int units, cudaStream_t st) {
    if (a.gated) return f32 ? launch_one<T, float, false, true>(a, units, st) : launch_one<T, T, false, true>(a, units, st);
    if (f32) return big ? launch_one<T, float, true, false>(a, units, st) : launch_one<T, float, false, false>(a, units, st);
    return big ? launch_one<T, T, true, false>(a, units, st) : launch_one<T, T, false, false>(a, units, st);
}

}  // namespace lora
}  // namespace tl
