// kern_lora.cuh -- low-rank adapters of many requests beside a shared layer:
//     h = s_a (x A_a^T) (fp32),  out = y + h B_a^T       for the tokens of adapter a,
// y the shared layer's output, S stacked shards with ranks of their own; and the same with the
// SiLU-gated product of a fused gate/up layer behind it.
//
// One launch.  Work is dealt in tiles of up to TM tokens of one adapter, a cluster of C blocks a tile:
//   * shrink: each block takes a run of K, its warps chunks of it, and keeps h's partial sums (TM x S R)
//     in shared memory; they are added over the cluster in a fixed order through distributed
//     shared memory, by every block for itself;
//   * expand: each block takes a run of output columns, adds h B^T to y and writes.
// So x and y are read once and out is written once, A and B once per tile.  With few tokens a tile is
// 16 rows and the adapter's matrices are the traffic; with many it is 64 and the
// activations are: 0.7 R operations a byte either way, far below what the tensor cores would need to bound
// it, so warp MMAs fed straight from global memory serve (operands are loaded in the order
// the fragments want: an MMA sums over k, any order of k will do if both sides share it).
//
// h enters the second product in 16 bits.  One rounding there would double the error of a 16-bit
// output, so h is split into two numbers of T (three where bf16 feeds an fp32 output), each the
// rounded rest of those before: 2^-17 of h or less.  f16 takes a row scaled by a power of two, so that
// large sums do not overflow.
#pragma once

#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

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

// 8 (or 4) contiguous outputs as floats, of which the first n exist.  Not through the read-only path:
// out may be y.
template <typename O, int N>
__device__ __forceinline__ void load_out(const O *p, int n, bool vec, float (&v)[N]) {
    if (vec && n >= N) {
        if constexpr (sizeof(O) == 4) {
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(p + i);
                v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
            }
        } else {
            O h[N];
            if constexpr (N == 8) *reinterpret_cast<uint4 *>(h) = *reinterpret_cast<const uint4 *>(p);
            else *reinterpret_cast<uint2 *>(h) = *reinterpret_cast<const uint2 *>(p);
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = to_f(h[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = i < n ? to_f(p[i]) : 0.f;
    }
}
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

__device__ __forceinline__ float silu(float g) { return g / (1.f + expf(-g)); }

// Sizes of a block's shared memory (bytes), the same on the host.
struct Smem {
    int ranks;   // S R
    int hstride; // elements of T between rows of the split h: LDS.64 of 4 rows hit other banks
    int part, split, total;  // ends of: partial sums; split h or warps' sums; a row of each warp
    __host__ __device__ Smem(int tm, int S, int R, int ns, int nt) {
        ranks = S * R;
        const int steps = S * ((R + 15) / 16);
        hstride = steps * 16 + (steps % 2 ? 0 : 16);
        part = tm * ranks * 4;
        const int hs = ns * tm * hstride * 2, red = 4 * tm * nt * 8 * 4;
        split = part + (hs > red ? hs : red);
        total = split + kWarps * ranks * 4;
    }
};

// TM = 16 G tokens a tile.  O: type of y and out.
template <typename T, typename O, int G, bool GATED>
__global__ void __launch_bounds__(kThreads) lora_kernel(const __grid_constant__ LoraArgs a) {
    constexpr int TM = 16 * G, NT = G == 1 ? 8 : 4;  // n-tiles of 8 ranks a pass of the shrink
    constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
    constexpr int NS = kBf && sizeof(O) == 4 ? 3 : 2;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ int toks[TM];
    __shared__ float up[TM];  // what a row of the split h has to be multiplied by
    __shared__ int tile_a, tile_k, tile_n;
    __shared__ int hist[kLoraFind + 1], wsum[kWarps], tok_cnt[4][kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int C = a.C, rank = (int)(blockIdx.x % (unsigned)C);
    const int unit = (int)(blockIdx.x / (unsigned)C);
    if (C > 1) cluster_arrive_relaxed();
    // ---- the tile
    if (a.plan != nullptr) {
        pdl_wait();
        if (unit >= a.plan[0]) {
            if (C > 1) cluster_wait();
            return;
        }
        const int *tile = a.plan + 4 + 3 * unit;
        const int ad = tile[0], first = tile[1], n = tile[2];
        if (tid < TM) toks[tid] = tid < n ? a.plan[4 + 3 * a.max_tiles + first + tid] : -1;
        if (tid == 0) tile_a = ad, tile_n = n;
    } else {
        const int M = (int)a.M, keys = a.adapters + 1;
        int key[4];
        for (int i = tid; i < keys; i += kThreads) hist[i] = 0;
        if (tid < TM) toks[tid] = -1;
        if (tid == 0) tile_a = -1;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int tk = i * kThreads + tid;
            key[i] = -1;
            if (tk < M) {
                key[i] = lora_key(a, tk);
                if (unit == 0 && rank == 0 && a.which[tk] >= a.adapters) flag_value(a.status);
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
                    tile_a = k;
                    tile_k = u;
                    tile_n = min(TM, hist[k] - u * TM);
                    break;
                }
                u -= n;
            }
        }
        __syncthreads();
        if (tile_a < 0) {  // fewer tiles than there might have been
            if (C > 1) cluster_wait();
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t hit = __ballot_sync(0xffffffffu, key[i] == tile_a);
            if (lane == 0) tok_cnt[i][warp] = __popc(hit);
        }
        __syncthreads();
        int at = -tile_k * TM;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t hit = __ballot_sync(0xffffffffu, key[i] == tile_a);
            int r = at;
            for (int w = 0; w < kWarps; ++w) {
                const int c = tok_cnt[i][w];
                if (w < warp) r += c;
                at += c;
            }
            r += __popc(hit & ((1u << lane) - 1u));
            if (key[i] == tile_a && r >= 0 && r < TM) toks[r] = i * kThreads + tid;
        }
    }
    __syncthreads();
    const int ad = tile_a, count = tile_n;
    const bool has = ad < a.adapters;
    if (!has && !GATED && a.out == a.y) {  // nothing is added to these
        if (C > 1) cluster_wait();
        return;
    }
    const int S = a.S, R = a.R, K = (int)a.K;
    const Smem sz(TM, S, R, NS, NT);
    float *const part = reinterpret_cast<float *>(smem);
    T *const hs = reinterpret_cast<T *>(smem + sz.part);
    float *const red = reinterpret_cast<float *>(smem + sz.part);
    const O *const y = static_cast<const O *>(a.y);
    O *const out = static_cast<O *>(a.out);
    if (has) {
        // ---- shrink
        const T *const A = static_cast<const T *>(a.a) + (int64_t)ad * sz.ranks * K;
        const T *xr[2 * G];
        bool live[2 * G];
#pragma unroll
        for (int i = 0; i < 2 * G; ++i) {
            const int row = (i >> 1) * 16 + (i & 1) * 8 + g;
            live[i] = row < count;
            xr[i] = static_cast<const T *>(a.x) + (int64_t)(live[i] ? toks[row] : toks[0]) * a.xs;
        }
        const int chunks = (K + 31) / 32, per = (chunks + C - 1) / C;
        const int c0 = min(chunks, rank * per), c1 = min(chunks, c0 + per);
        for (int r0 = 0; r0 < sz.ranks; r0 += NT * 8) {
            const int nt = min(NT, (sz.ranks - r0) >> 3);
            float acc[G][NT][4];
#pragma unroll
            for (int i = 0; i < G; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.f;
            for (int c = c0 + warp; c < c1; c += kWarps) {
                const int k = c * 32 + t * 8, n = K - k;
                uint4 xv[2 * G], av[NT];
#pragma unroll
                for (int i = 0; i < 2 * G; ++i) xv[i] = live[i] ? load8(xr[i] + k, n, a.vec_x) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    av[j] = j < nt ? load8(A + (int64_t)(r0 + j * 8 + g) * K + k, n, a.vec_a) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < G; ++i) {
                    const uint32_t f0[4] = {xv[2 * i].x, xv[2 * i + 1].x, xv[2 * i].y, xv[2 * i + 1].y};
                    const uint32_t f1[4] = {xv[2 * i].z, xv[2 * i + 1].z, xv[2 * i].w, xv[2 * i + 1].w};
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        if (j < nt) {
                            mma16816<T>(acc[i][j], f0, av[j].x, av[j].y);
                            mma16816<T>(acc[i][j], f1, av[j].z, av[j].w);
                        }
                }
            }
            // the warps' sums: halves added in a fixed order
#pragma unroll
            for (int half = kWarps / 2; half > 0; half >>= 1) {
                __syncthreads();
                if (warp >= half && warp < 2 * half) {
                    float *p = red + (warp - half) * (TM * NT * 8);
#pragma unroll
                    for (int i = 0; i < G; ++i)
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int e = 0; e < 4; ++e) p[((i * NT + j) * 4 + e) * 32 + lane] = acc[i][j][e];
                }
                __syncthreads();
                if (warp < half) {
                    const float *p = red + warp * (TM * NT * 8);
#pragma unroll
                    for (int i = 0; i < G; ++i)
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[i][j][e] += p[((i * NT + j) * 4 + e) * 32 + lane];
                }
            }
            if (warp == 0) {
#pragma unroll
                for (int i = 0; i < G; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        if (j < nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                part[(i * 16 + (e >> 1) * 8 + g) * sz.ranks + r0 + j * 8 + 2 * t + (e & 1)] = acc[i][j][e];
            }
        }
        __syncthreads();
    }
    if (C > 1) {
        cluster_wait();  // (every block has started)
        cl_arrive_release();
        cl_wait_acquire();
    }
    if (has) {
        // ---- h = s (the blocks' sums, in their order), split into NS numbers of T; a warp per row
        const float s = a.scale ? a.scale[ad] : 1.f;
        const int steps = (R + 15) / 16;
        float *const mine = reinterpret_cast<float *>(smem + sz.split) + warp * sz.ranks;
        for (int row = warp; row < TM; row += kWarps) {
            uint32_t top = 0;
            for (int e = lane; e < sz.ranks; e += 32) {
                float v = 0.f;
                if (row < count) {
                    if (C > 1) {
                        const uint32_t at = smem_u32(part + row * sz.ranks + e);
                        for (int i = 0; i < C; ++i) v += cl_ld_f32(cl_map(at, i));
                    } else {
                        v = part[row * sz.ranks + e];
                    }
                    v *= s;
                }
                top = max(top, __float_as_uint(v) & 0x7FFFFFFFu);
                mine[e] = v;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            // f16: the row's largest to [2^14, 2^15); a row with an infinity or a NaN as it is
            const uint32_t ex = max(top >> 23, 15u);
            const bool turn = !kBf && ex < 255u;
            const float down = turn ? __uint_as_float((268u - ex) << 23) : 1.f;
            if (lane == 0) up[row] = turn ? __uint_as_float((ex - 14u) << 23) : 1.f;
            __syncwarp();
            for (int e = lane; e < S * steps * 16; e += 32) {
                const int sh = e / (steps * 16), r = e - sh * steps * 16;
                float v = r < R ? mine[sh * R + r] * down : 0.f;
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    const T h = of_f<T>(v);
                    hs[(i * TM + row) * sz.hstride + e] = h;
                    v = isfinite(to_f(h)) ? v - to_f(h) : 0.f;
                }
            }
            __syncwarp();
        }
    }
    __syncthreads();
    if (C > 1) cl_arrive_release();  // the others' sums are read
    // ---- expand: columns in blocks of 32 (gated: 16 of either half), dealt to the cluster's warps
    {
        constexpr int J = GATED ? 2 : 4, W = 2 * J;  // n-tiles a block; contiguous columns of a thread
        const T *const B = static_cast<const T *>(a.b) + (has ? (int64_t)ad * a.N * R : 0);
        const int steps = (R + 15) / 16, kk = C * kWarps;
        const int shards = GATED ? 1 : S;
        int skip = rank * kWarps + warp;  // blocks of columns before this warp's next one
        int64_t off = 0;
        for (int sh = 0; sh < shards; ++sh) {
            const int64_t wide = a.shard[sh];
            const int64_t blocks = (wide + J * 8 - 1) / (J * 8);
            int64_t blk = skip;
            for (; blk < blocks; blk += kk) {
                const int64_t col0 = off + blk * (J * 8);       // first column
                const int left = (int)min((int64_t)(J * 8), wide - blk * (J * 8));
                constexpr int H = GATED ? 2 : 1;
                float acc[H][G][J][4];
#pragma unroll
                for (int p = 0; p < H; ++p)
#pragma unroll
                    for (int i = 0; i < G; ++i)
#pragma unroll
                        for (int j = 0; j < J; ++j)
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[p][i][j][e] = 0.f;
                if (has) {
                    for (int st = 0; st < steps; ++st) {
                        uint2 bv[H][J];
                        const int r = st * 16 + 4 * t;
#pragma unroll
                        for (int p = 0; p < H; ++p)
#pragma unroll
                            for (int j = 0; j < J; ++j) {
                                // column of the fragment's n = g: such that a thread's results are neighbours
                                const int c = (g >> 1) * W + 2 * j + (g & 1);
                                bv[p][j] = c < left && r < R ? ldg_nc_v2(B + (p * wide + col0 + c) * R + r) : make_uint2(0, 0);
                            }
#pragma unroll
                        for (int i = 0; i < G; ++i)
#pragma unroll
                            for (int p = 0; p < H; ++p)
#pragma unroll
                                for (int n = 0; n < NS; ++n) {
                                    const T *h = hs + (n * TM + i * 16 + g) * sz.hstride + ((GATED ? p : sh) * steps + st) * 16 + 4 * t;
                                    const uint2 lo = *reinterpret_cast<const uint2 *>(h), hi = *reinterpret_cast<const uint2 *>(h + 8 * sz.hstride);
                                    const uint32_t f[4] = {lo.x, hi.x, lo.y, hi.y};
#pragma unroll
                                    for (int j = 0; j < J; ++j) mma16816<T>(acc[p][i][j], f, bv[p][j].x, bv[p][j].y);
                                }
                    }
                }
                const int n = left - t * W;
                if (n > 0) {
#pragma unroll
                    for (int i = 0; i < G; ++i)
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const int row = i * 16 + q * 8 + g;
                            if (row >= count) continue;
                            const int64_t tok = toks[row], col = col0 + t * W;
                            const float f = has ? up[row] : 0.f;
                            float v[W];
                            load_out<O, W>(y + tok * a.ys + col, n, a.vec_y, v);
#pragma unroll
                            for (int j = 0; j < W; ++j)
                                if (has) v[j] = __fmaf_rn(acc[0][i][j >> 1][2 * q + (j & 1)], f, v[j]);
                            if constexpr (GATED) {
                                float w[W];
                                load_out<O, W>(y + tok * a.ys + wide + col, n, a.vec_y, w);
#pragma unroll
                                for (int j = 0; j < W; ++j) {
                                    if (has) w[j] = __fmaf_rn(acc[1][i][j >> 1][2 * q + (j & 1)], f, w[j]);
                                    v[j] = silu(v[j]) * w[j];
                                }
                            }
                            store_out<O, W>(out + tok * a.os + col, n, a.vec_y, v);
                        }
                }
            }
            skip = (int)(blk - blocks);
            off += wide;
        }
    }
    if (C > 1) cl_wait_acquire();
}

// Raises the kernel's shared-memory limit on the current device, once per device.
constexpr int kMaxSmem = 200 * 1024;
template <typename K>
cudaError_t allow_smem(std::atomic<uint64_t> &done, K *kernel) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

template <typename T, typename O, int G, bool GATED>
cudaError_t launch_one(const LoraArgs &a, int units, cudaStream_t st) {
    constexpr int TM = 16 * G, NT = G == 1 ? 8 : 4;
    constexpr int NS = std::is_same<T, __nv_bfloat16>::value && sizeof(O) == 4 ? 3 : 2;
    const Smem sz(TM, a.S, a.R, NS, NT);
    static std::atomic<uint64_t> done{0};
    if (const cudaError_t e = allow_smem(done, lora_kernel<T, O, G, GATED>)) return e;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)units * (unsigned)a.C);
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = sz.total;
    c.stream = st;
    cudaLaunchAttribute at[2];
    int n = 0;
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = (unsigned)a.C;
    at[n].val.clusterDim.y = at[n].val.clusterDim.z = 1;
    ++n;
    if (a.plan) {
        at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    c.attrs = at;
    c.numAttrs = n;
    return cudaLaunchKernelEx(&c, lora_kernel<T, O, G, GATED>, a);
}

template <typename T>
cudaError_t launch_type(const LoraArgs &a, bool f32, bool big, int units, cudaStream_t st) {
    if (a.gated) {
        if (f32) return big ? launch_one<T, float, 2, true>(a, units, st) : launch_one<T, float, 1, true>(a, units, st);
        return big ? launch_one<T, T, 2, true>(a, units, st) : launch_one<T, T, 1, true>(a, units, st);
    }
    if (f32) return big ? launch_one<T, float, 4, false>(a, units, st) : launch_one<T, float, 1, false>(a, units, st);
    return big ? launch_one<T, T, 4, false>(a, units, st) : launch_one<T, T, 1, false>(a, units, st);
}

}  // namespace lora
}  // namespace tl
