// attn_stream.cuh -- attention for few rows per kv head (single tokens, small trees):
// the cache streams through registers once, fed to warp MMAs.
//
//   S^T = K Q^T, P = exp2(S sk f - r) sv, O^T += V^T P^T    (f = scale log2 e)
//
// For at most 16 rows the bytes of the cache bound the call (16 rows x 4 flops per
// 8-bit element: about 32 flops a byte), so everything is laid out for the stream:
//  * keys are the 16-wide side of mma.m16n8k16 and rows the 8-wide one: blocks of up to 8
//    rows (NB = 1) need half the MMAs, exponentials and registers of the other way round.
//  * a tile is 64 keys, 16 for each of the block's 4 warps; warps share nothing until a
//    unit ends.  Pages hold multiples of 16 keys, so a warp's 16 keys lie in one page.
//  * each thread copies exactly the bytes that its own MMA fragments need, with
//    cp.async into a ring of its warp, several tiles ahead: no block barriers in the
//    loop, and no fragment is exchanged.  The order of the contracted axis and of the
//    output's elements is free, so thread t of a quad takes 16 neighbouring elements of
//    keys g and g + 8 (and of the next 64) for S, and of its four keys' values the
//    elements [g D/8, (g + 1) D/8): every global read is 64 or 128 bytes of one row
//    over a quad or eight lanes.
//  * P changes from (keys x rows) to (rows x keys) fragments by one movmatrix per 8 keys.
//  * codes become f16 (exact); the products are exact, sums fp32.  Queries in bf16
//    enter as f16 scaled by a power of two per row (QueryScale in attn_sched.cuh).
//  * P is rounded to f16 (2^-11 relative) with its value scale in it, kept so far up that
//    products down to 2^-24 of a row's largest keep all 11 bits.  A row's reference is that of
//    its own products (kAttnRoom in attn_sched.cuh), so neither a key of a negligible weight
//    nor one that another row sees takes bits from it.  It moves only when exceeded by a
//    factor of 4, and then a factor of 8 beyond: the accumulators are rescaled a few times
//    per unit, not per tile.
// Measured: 64 sequences of 4096 to 8192 keys, 28 query heads on 4, int8, one token each:
// 91 to 95 us, 4.3 to 4.5 TB/s (0.64 to 0.66 of a copy's rate; 5.5 TB/s with 28 kv heads): issue slots (50 % used, half of them by the codes'
// conversions) and the equal division of tiles among blocks whose speeds differ by some
// 18 %.  One sequence of 131072 keys: 40 us.  16 rows, 6 sequences of up to 4099 keys, 32
// heads, int4: 73 us.
#pragma once

#include "attn_sched.cuh"
#include "kv.cuh"
#include "rope.cuh"

namespace tl {

namespace {

constexpr int kStreamThreads = 128;
// GR: groups of 16 keys that a warp takes per tile
template <int GR>
using StreamTiling = AttnTiling<64 * GR, 2 / GR>;  // (a unit costs about 128 keys beside its own)

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void *src, bool valid) {
    const int n = valid ? BYTES : 0;  // 0: the bytes are filled with zeros
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n)
                     : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int FMT, int D, int NB>
struct StreamCfg {
    static constexpr int ROWS = 8 * NB;
    static constexpr int RB = D * KvCode<FMT>::bits / 8;  // bytes per row of codes
    static constexpr int KB = RB / 4;                     // bytes of a key per thread (scores)
    static constexpr int KC = KB > 16 ? 16 : KB;          // bytes per copy
    static constexpr int NKC = KB / KC;
    static constexpr int VB = RB / 8;                     // bytes of a key per thread (values)
    static constexpr int KSTEPS = D / 16;
    // one stage of one warp: keys' copies, values' copies, 16 + 16 scales
    static constexpr int KOFF = 0, VOFF = 2 * NKC * KC * 32, SOFF = VOFF + 4 * VB * 32;
    static constexpr int GROUP = SOFF + 128;              // bytes of one group
    static constexpr int GR = NB == 1 ? 2 : 1;            // groups per tile and warp
    static constexpr int STAGE = GR * GROUP;
    static constexpr int BLOCKS = 3;                      // per SM (registers)
    static constexpr int NS = (GROUP > 3000 ? 2 + 2 / NB : GROUP > 2000 ? 6 : 8) / GR;  // stages per warp
    static constexpr bool QSMEM = NB > 1;                 // the queries' fragments stay in shared memory
    static constexpr int PITCH = D + 4;                   // floats per row of the join buffer
    // [stages of 4 warps][join rows; at a unit's start, its queries in f16]
    // [row factors][per-warp maxima and sums][place]
    static constexpr int JOFF = 4 * NS * STAGE;
    static constexpr int FOFF = JOFF + ROWS * PITCH * 4;
    static constexpr int WOFF = FOFF + ROWS * 4;
    static constexpr int POFF = WOFF + 2 * 4 * ROWS * 4;
    static constexpr int GOFF = POFF + 64;                // fragments [n][step][lane]
    static constexpr int SMEM = GOFF + (QSMEM ? NB * KSTEPS * 256 : 0);
    static_assert(BLOCKS * (SMEM + 1024) <= 228 * 1024, "blocks per SM");
};

template <int FMT, int D, int NB>
__global__ void __launch_bounds__(kStreamThreads, StreamCfg<FMT, D, NB>::BLOCKS) attn_stream_kernel(AttnArgs a) {
    using C = StreamCfg<FMT, D, NB>;
    constexpr int GR = C::GR;
    using TL = StreamTiling<GR>;
    constexpr int KT = TL::KT, ROWS = C::ROWS, NT = D / 16;
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int R = a.T * a.G;
    pdl_launch_dependents();

    uint8_t *ring = smem + warp * C::NS * C::STAGE;
    AttnWalk in, out;  // the tile being copied, the tile being computed
    if (!in.template start_block<TL, kStreamThreads>(a, 1, reinterpret_cast<int64_t *>(smem + C::POFF))) return;
    out = in;

    // Queries of a unit: TPR threads per row, EPT elements each (the first unit's are fetched
    // before its keys).
    constexpr int TPR = kStreamThreads / ROWS, EPT = D / TPR;
    const int row = threadIdx.x / TPR, part = threadIdx.x % TPR;
    uint32_t raw[EPT / 2];
    auto fetch_queries = [&](const AttnWalk &w) {
        const int r = min(row, R - 1), tok = r / a.G;
        const uint16_t *q = static_cast<const uint16_t *>(a.q) + w.b * a.qb + (int64_t)tok * a.qt +
                     (int64_t)(w.hk * a.G + r - tok * a.G) * a.qh + part * EPT;
        if (a.q_vec) {
            if constexpr (EPT >= 8) {
#pragma unroll
                for (int i = 0; i < EPT / 8; ++i) {
                    const uint4 u = __ldg(reinterpret_cast<const uint4 *>(q) + i);
                    raw[4 * i] = u.x, raw[4 * i + 1] = u.y, raw[4 * i + 2] = u.z, raw[4 * i + 3] = u.w;
                }
            } else {
                const uint2 u = __ldg(reinterpret_cast<const uint2 *>(q));
                raw[0] = u.x, raw[1] = u.y;
            }
        } else {
            const uint16_t *u = q;
#pragma unroll
            for (int i = 0; i < EPT / 2; ++i) raw[i] = u[2 * i] | (uint32_t)u[2 * i + 1] << 16;
        }
    };
    fetch_queries(out);

    // Copies run NS - 1 tiles ahead; the page of the tile after that is already on its way.
    AttnPages where[GR];
    int page[GR];
    auto locate = [&](bool start) {
#pragma unroll
        for (int i = 0; i < GR; ++i) {
            if (start) where[i].start(a, in, in.tile * KT + i * 64 + warp * 16);
            else where[i].next(a, KT);
            page[i] = where[i].fetch(a, in.b);
        }
    };
    locate(true);
    const uint32_t dst0 = smem_u32(ring) + lane * C::KC;
    const int ksrc = g * C::RB + t * C::KC, vsrc = 2 * t * C::RB + g * C::VB;
    int put = 0;  // stage being filled
    auto issue = [&]() {
        if (!in.inside()) {
            cp_commit();
            return;
        }
#pragma unroll
        for (int i = 0; i < GR; ++i) {
            const int left = in.ctx + a.T - (in.tile * KT + i * 64 + warp * 16);  // keys from the group's first one on
            if (left > 0) {
                const int64_t row = (int64_t)attn_group(a, page[i], in.hk, where[i].off) << 4;
                const uint8_t *kp = a.c.kc + row * C::RB + ksrc, *vp = a.c.vc + row * C::RB + vsrc;
                const uint32_t st = dst0 + (uint32_t)(put * C::STAGE + i * C::GROUP);
                const uint32_t sv = st + C::VOFF - lane * (C::KC - C::VB);
                auto copy = [&](auto whole) {  // whole: no key of the 16 lies beyond the last
                    constexpr bool ALL = decltype(whole)::value;
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int j = 0; j < C::NKC; ++j)
                            cp_async<C::KC>(st + C::KOFF + (n * C::NKC + j) * 32 * C::KC, kp + n * 8 * C::RB + j * 4 * C::KC,
                                            ALL || n * 8 + g < left);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = (j & 1) + (j >> 1) * 8;
                        cp_async<C::VB>(sv + j * 32 * C::VB, vp + r * C::RB, ALL || 2 * t + r < left);
                    }
                };
                if (left >= 16) copy(std::true_type());
                else copy(std::false_type());
                if (lane < 8)
                    cp_async<16>(st + C::SOFF + lane * (16 - C::KC), (lane < 4 ? a.c.ks : a.c.vs) + row + (lane & 3) * 4, true);
            }
        }
        cp_commit();
        put = put + 1 == C::NS ? 0 : put + 1;
        const bool start = in.template next<TL>(a, 1);
        if (in.inside()) locate(start);
    };
#pragma unroll 1
    for (int i = 0; i < C::NS - 1; ++i) issue();

    uint32_t qf[C::QSMEM ? 1 : NB][C::QSMEM ? 1 : C::KSTEPS][2];
    uint2 *const qsm = reinterpret_cast<uint2 *>(smem + C::GOFF) + lane;
    float f[NB][2];                        // score factors of rows 8 n + 2t and + 1
    float ref[NB][2], l[NB][2];            // reference of the products, sum of the weights
    float acc[NB][NT][4];
    uint32_t nans = 0;                     // e4m3: a new token's values hold a NaN code
    bool fresh = true, whole = true;       // the next tile begins a unit (for this block); the unit from its start
    int which = 0, get = 0;                // slot of a partial result; stage being read

#pragma unroll 1
    for (bool first = true; out.inside(); first = false) {
        if (fresh) {
            // ---------------- queries of the unit: rows as f16 in shared memory, then fragments
            fresh = false;
            whole = out.tile == 0;
            if (!first) fetch_queries(out);
            float v[EPT];
#pragma unroll
            for (int i = 0; i < EPT; i += 2) {
                const float2 x = attn_unpack(a, row < R ? raw[i / 2] : 0u);
                v[i] = x.x;
                v[i + 1] = x.y;
            }
            float down = 1.f, up = 1.f;
            if (a.bf) {
                float mx = 0.f;
#pragma unroll
                for (int i = 0; i < EPT; ++i) mx = fmaxf(mx, fabsf(v[i]));
#pragma unroll
                for (int o = TPR / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const QueryScale by(__float_as_uint(mx) >> 23);
                down = by.down;
                up = by.up;
            }
            __half *qs = reinterpret_cast<__half *>(smem + C::JOFF) + row * (D + 8) + part * EPT;
#pragma unroll
            for (int i = 0; i < EPT; i += 2)
                *reinterpret_cast<__half2 *>(qs + i) = __floats2half2_rn(v[i] * down, v[i + 1] * down);
            float *fac = reinterpret_cast<float *>(smem + C::FOFF);
            if (part == 0) fac[row] = a.scale * kLog2e * up;
            __syncthreads();
            const uint16_t *qr = reinterpret_cast<const uint16_t *>(smem + C::JOFF);
            // the elements of this thread in step s, in the order its code words give
            auto fragment = [&](int n, int s) {
                const uint16_t *r = qr + (8 * n + g) * (D + 8);
                if constexpr (FMT == kKvInt4) {
                    const uint16_t *p = r + t * (D / 4) + (s >> 1) * 8 + (s & 1) * 2;
                    return make_uint2(p[0] | ((uint32_t)p[4] << 16), p[1] | ((uint32_t)p[5] << 16));
                } else {
                    return *reinterpret_cast<const uint2 *>(r + (s >> 2) * 64 + t * 16 + (s & 3) * 4);
                }
            };
            if constexpr (C::QSMEM) {
                for (int i = warp; i < NB * C::KSTEPS; i += 4) qsm[i * 32] = fragment(i / C::KSTEPS, i % C::KSTEPS);
            }
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                if constexpr (!C::QSMEM) {
#pragma unroll
                    for (int s = 0; s < C::KSTEPS; ++s) {
                        const uint2 u = fragment(n, s);
                        qf[n][s][0] = u.x;
                        qf[n][s][1] = u.y;
                    }
                }
                f[n][0] = fac[8 * n + 2 * t];
                f[n][1] = fac[8 * n + 2 * t + 1];
                ref[n][0] = ref[n][1] = kAttnLow;
                l[n][0] = l[n][1] = 0.f;
#pragma unroll
                for (int i = 0; i < NT; ++i) acc[n][i][0] = acc[n][i][1] = acc[n][i][2] = acc[n][i][3] = 0.f;
            }
            __syncthreads();  // the queries' buffer is the join buffer too
        }

        // ---------------- GR groups of 16 keys (independent chains up to the weights)
        issue();
        cp_wait<C::NS - 1>();
        __syncwarp();  // the scales were copied by other lanes
        const int key = out.tile * KT + warp * 16;
        if (key < out.ctx + a.T) {
            const uint8_t *const stage = ring + get * C::STAGE;
            // z: scores in powers of two; [0], [1]: key g of rows 2t, 2t + 1; [2], [3]: key g + 8
            float z[GR][NB][4], sv[GR][2];
#pragma unroll
            for (int gr = 0; gr < GR; ++gr) {
                const uint8_t *st = stage + gr * C::GROUP;
                float s[NB][4];
#pragma unroll
                for (int n = 0; n < NB; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
                uint32_t w[2][C::KB / 4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int j = 0; j < C::NKC; ++j) {
                        const uint8_t *p = st + C::KOFF + ((n * C::NKC + j) * 32 + lane) * C::KC;
                        if constexpr (C::KC == 16) {
                            const uint4 u = *reinterpret_cast<const uint4 *>(p);
                            w[n][4 * j] = u.x, w[n][4 * j + 1] = u.y, w[n][4 * j + 2] = u.z, w[n][4 * j + 3] = u.w;
                        } else {
                            const uint2 u = *reinterpret_cast<const uint2 *>(p);
                            w[n][0] = u.x, w[n][1] = u.y;
                        }
                    }
#pragma unroll
                for (int i = 0; i < C::KSTEPS; ++i) {
                    uint32_t x[4];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        if constexpr (FMT == kKvInt4) {
                            const uint32_t u = i & 1 ? w[n][i >> 1] >> 8 : w[n][i >> 1];
                            x[n] = int4_lo(u);
                            x[2 + n] = int4_hi(u);
                        } else if constexpr (FMT == kKvInt8) {
                            const uint32_t u = w[n][i] ^ 0x80808080u;
                            x[n] = int8_f16x2(__byte_perm(u, 0x64646464u, 0x4140));
                            x[2 + n] = int8_f16x2(__byte_perm(u, 0x64646464u, 0x4342));
                        } else {
                            x[n] = e4m3x2_f16x2(w[n][i]);
                            x[2 + n] = e4m3x2_f16x2(w[n][i] >> 16);
                        }
                    }
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        if constexpr (C::QSMEM) {
                            const uint2 u = qsm[(n * C::KSTEPS + i) * 32];
                            mma16816(s[n], x, u.x, u.y);
                        } else {
                            mma16816(s[n], x, qf[n][i][0], qf[n][i][1]);
                        }
                    }
                }
                const float *sc = reinterpret_cast<const float *>(st + C::SOFF);
                const float sk[2] = {sc[g], sc[g + 8]};
                sv[gr][0] = sc[16 + g];
                sv[gr][1] = sc[24 + g];
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) z[gr][n][j] = s[n][j] * (sk[j >> 1] * f[n][j & 1]);
            }
            uint32_t unseen = 0;
            const bool edge = key + (GR - 1) * 64 + 16 > out.ctx;  // new tokens' keys, or the end
            if (edge) {
                const uint8_t *tree = a.tree ? a.tree + out.b * a.tree_b : nullptr;
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) {
#pragma unroll
                    for (int n = 0; n < NB; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int i = key + gr * 64 + g + (j >> 1) * 8 - out.ctx;  // index of the new token
                            const int tok = min(R - 1, 8 * n + 2 * t + (j & 1)) / a.G;
                            bool u = i < 0;
                            if (i >= 0 && i < a.T) u = tree ? tree[tok * a.tree_r + i] != 0 : i <= tok;
                            if (!u) z[gr][n][j] = -INFINITY, unseen |= 1u << (4 * (gr * NB + n) + j);
                        }
                }
            }
            // the largest product of each row; the size of an unseen scale is finite too
            float top[NB][2];
#pragma unroll
            for (int n = 0; n < NB; ++n) top[n][0] = top[n][1] = -INFINITY;
#pragma unroll
            for (int gr = 0; gr < GR; ++gr) {
                const float x0 = attn_size(sv[gr][0]), x1 = attn_size(sv[gr][1]);
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int r = 0; r < 2; ++r) top[n][r] = fmaxf(top[n][r], fmaxf(z[gr][n][r] + x0, z[gr][n][2 + r] + x1));
            }
            bool move = false;
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) move = move || attn_above(top[n][r]) - ref[n][r] > kAttnFull;
            if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float x = top[n][r];
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                        const float was = x;
                        x = attn_above(x) - ref[n][r] > kAttnFull ? fmaxf(x - kAttnRoom, ref[n][r]) : ref[n][r];
                        if (__any_sync(0xffffffffu, fabsf(was) > kAttnCoarse)) {
                            float left = -INFINITY;
#pragma unroll
                            for (int gr = 0; gr < GR; ++gr)
                                left = fmaxf(left, fmaxf(z[gr][n][r] - x + attn_size(sv[gr][0]), z[gr][n][2 + r] - x + attn_size(sv[gr][1])));
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1) left = fmaxf(left, __shfl_xor_sync(0xffffffffu, left, o));
                            if (left > kAttnFull) x = __fadd_ru(x, left - kAttnRoom);
                        }
                        // in two steps: the sum may outlive a factor that fp32 cannot hold
                        const float h = ex2(.5f * (ref[n][r] - x)), c = h * h;
                        ref[n][r] = x;
                        l[n][r] = l[n][r] * h * h;
#pragma unroll
                        for (int i = 0; i < NT; ++i) {
                            acc[n][i][r] *= c;
                            acc[n][i][2 + r] *= c;
                        }
                    }
            }
#pragma unroll
            for (int gr = 0; gr < GR; ++gr) {
                const uint8_t *st = stage + gr * C::GROUP;
                const float wv[2] = {sv[gr][0] * kAttnUnbias, sv[gr][1] * kAttnUnbias};
                uint32_t pb[NB][2];
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    float p[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float e = ex2(z[gr][n][j] - ref[n][j & 1]);
                        l[n][j & 1] += e;
                        p[j] = e * wv[j >> 1];
                    }
                    if (unseen) {  // an unseen scale may be a NaN or an infinity
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (unseen >> (4 * (gr * NB + n) + j) & 1u) p[j] = 0.f;
                    }
                    pb[n][0] = transpose8x8(pack2(__half(), p[0], p[1]));
                    pb[n][1] = transpose8x8(pack2(__half(), p[2], p[3]));
                }
                // values: elements 2i and 2i + 1 of lane group g's run are its rows of MMA i
                uint32_t v[4][C::VB / 4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint8_t *p = st + C::VOFF + (j * 32 + lane) * C::VB;
                    if constexpr (C::VB == 16) {
                        const uint4 u = *reinterpret_cast<const uint4 *>(p);
                        v[j][0] = u.x, v[j][1] = u.y, v[j][2] = u.z, v[j][3] = u.w;
                    } else if constexpr (C::VB == 8) {
                        const uint2 u = *reinterpret_cast<const uint2 *>(p);
                        v[j][0] = u.x, v[j][1] = u.y;
                    } else {
                        v[j][0] = *reinterpret_cast<const uint32_t *>(p);
                    }
                }
                if constexpr (FMT == kKvFp8) {
                    if (edge) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int i0 = key + gr * 64 + 2 * t + (j & 1) + (j >> 1) * 8 - out.ctx;  // index of the new token
                            if (i0 < 0) continue;
                            uint32_t met = 0;
#pragma unroll
                            for (int i = 0; i < C::VB / 4; ++i) v[j][i] = e4m3_finite(v[j][i], met);
                            if (i0 < a.T) nans |= met;
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < C::VB / 4; ++i) {
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        if constexpr (FMT == kKvInt4) {  // elements 0-3, then 4-7, of the two keys of a pair
                            const uint32_t sel = hh ? 0x7632 : 0x5410;
                            const uint32_t x = __byte_perm(v[0][i], v[1][i], sel), y = __byte_perm(v[2][i], v[3][i], sel);
                            const uint32_t a0[4] = {int4_lo(x), int4_hi(x), int4_lo(y), int4_hi(y)};
                            const uint32_t a1[4] = {int4_lo(x >> 8), int4_hi(x >> 8), int4_lo(y >> 8), int4_hi(y >> 8)};
#pragma unroll
                            for (int n = 0; n < NB; ++n) {
                                mma16816(acc[n][4 * i + 2 * hh], a0, pb[n][0], pb[n][1]);
                                mma16816(acc[n][4 * i + 2 * hh + 1], a1, pb[n][0], pb[n][1]);
                            }
                        } else {  // bytes 0, 1, then 2, 3, interleaved over the pair's keys
                            const uint32_t sel = hh ? 0x7362 : 0x5140;
                            uint32_t x = __byte_perm(v[0][i], v[1][i], sel), y = __byte_perm(v[2][i], v[3][i], sel);
                            uint32_t a0[4];
                            if constexpr (FMT == kKvInt8) {
                                x ^= 0x80808080u;
                                y ^= 0x80808080u;
                                a0[0] = int8_f16x2(__byte_perm(x, 0x64646464u, 0x4140));
                                a0[1] = int8_f16x2(__byte_perm(x, 0x64646464u, 0x4342));
                                a0[2] = int8_f16x2(__byte_perm(y, 0x64646464u, 0x4140));
                                a0[3] = int8_f16x2(__byte_perm(y, 0x64646464u, 0x4342));
                            } else {
                                a0[0] = e4m3x2_f16x2(x);
                                a0[1] = e4m3x2_f16x2(x >> 16);
                                a0[2] = e4m3x2_f16x2(y);
                                a0[3] = e4m3x2_f16x2(y >> 16);
                            }
#pragma unroll
                            for (int n = 0; n < NB; ++n) mma16816(acc[n][2 * i + hh], a0, pb[n][0], pb[n][1]);
                        }
                    }
                }
            }
        }
        __syncwarp();  // every lane is done with the stage (its scales are shared)
        get = get + 1 == C::NS ? 0 : get + 1;

        // ---------------- the end of a unit, or of the run: join the warps, write
        const bool last = out.last_of_unit();
        if (last || !out.template more<TL>()) {
            whole = whole && last;
            float *wm = reinterpret_cast<float *>(smem + C::WOFF), *wl = wm + 4 * ROWS;
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) l[n][r] += __shfl_xor_sync(0xffffffffu, l[n][r], o);
                    if (g == 0) {
                        wm[warp * ROWS + 8 * n + 2 * t + r] = ref[n][r];
                        wl[warp * ROWS + 8 * n + 2 * t + r] = l[n][r];
                    }
                }
            bool nan_seen = false;
            if constexpr (FMT == kKvFp8) nan_seen = __syncthreads_or(nans != 0), nans = 0;
            else __syncthreads();
            float *jb = reinterpret_cast<float *>(smem + C::JOFF);
            float c[NB][2];
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float *p = wm + 8 * n + 2 * t + r;
                    const float M = fmaxf(fmaxf(p[0], p[ROWS]), fmaxf(p[2 * ROWS], p[3 * ROWS]));
                    c[n][r] = ex2(ref[n][r] - M) * kAttnRebias;  // in units of the weights' sum
                }
#pragma unroll 1
            for (int turn = 0; turn < 4; ++turn) {
                if (turn == warp) {
#pragma unroll
                    for (int n = 0; n < NB; ++n)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            // pair i of lane group g's run lies at place (i + g) % NT of it: no
                            // two lanes of a half-warp meet in a bank
                            float2 *d = reinterpret_cast<float2 *>(jb + (8 * n + 2 * t + r) * C::PITCH + g * (D / 8));
#pragma unroll
                            for (int i = 0; i < NT; ++i) {
                                float2 *p = d + ((i + g) & (NT - 1));
                                float2 u = make_float2(acc[n][i][r] * c[n][r], acc[n][i][2 + r] * c[n][r]);
                                if (turn > 0) u.x += p->x, u.y += p->y;
                                *p = u;
                            }
                        }
                }
                __syncthreads();
            }
            if (row < R) {
                float M = wm[row], Ls = 0.f;
#pragma unroll
                for (int i = 1; i < 4; ++i) M = fmaxf(M, wm[i * ROWS + row]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float h = ex2(.5f * (wm[i * ROWS + row] - M));
                    Ls += wl[i * ROWS + row] * h * h;
                }
                float v[EPT];
#pragma unroll
                for (int e = 0; e < EPT; e += 2) {
                    const int i = (part * EPT + e) / 2, h = i / NT;  // pair of the row, lane group that wrote it
                    const float2 u = *reinterpret_cast<const float2 *>(jb + row * C::PITCH + h * (D / 8) + 2 * ((i + h) & (NT - 1)));
                    v[e] = u.x, v[e + 1] = u.y;
                }
                if (whole) {
                    const float rl = Ls == 0.f ? 0.f : 1.f / Ls;
                    const int64_t out_row = ((int64_t)out.b * a.T + row / a.G) * a.Hq + out.hk * a.G + row % a.G;
                    uint32_t *o = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + out_row * D + part * EPT);
#pragma unroll
                    for (int e = 0; e < EPT; e += 2) o[e / 2] = attn_pack(a, v[e] * rl, v[e + 1] * rl);
                    if (FMT == kKvFp8 && nan_seen) attn_put_nans<D>(a, out, row / a.G, part * EPT, EPT, o - part * (EPT / 2), nullptr);
                    if (a.lse && part == 0) a.lse[out_row] = Ls == 0.f ? -INFINITY : (M + log2f(Ls)) * kLn2;
                } else {
                    float *slot = AttnSlot<ROWS, D>::at(a.ws, blockIdx.x, which);
                    float *o = slot + row * D + part * EPT;
#pragma unroll
                    for (int e = 0; e < EPT; e += 4)
                        *reinterpret_cast<float4 *>(o + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                    if (FMT == kKvFp8 && nan_seen) attn_put_nans<D>(a, out, row / a.G, part * EPT, EPT, nullptr, slot + row * D);
                    if (part == 0) {
                        slot[ROWS * D + row] = M;
                        slot[ROWS * (D + 1) + row] = Ls;
                    }
                }
            }
            which = 1;
            fresh = true;
            __syncthreads();  // the join buffers may be written again
        }
        out.template next<TL>(a, 1);
    }
    cp_wait<0>();
}

template <int FMT, int D, int NB>
cudaError_t launch_stream_d(const AttnArgs &a, int sms, cudaStream_t st) {
    using C = StreamCfg<FMT, D, NB>;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = attn_allow_smem(allowed, attn_stream_kernel<FMT, D, NB>, C::SMEM);
    if (e != cudaSuccess) return e;
    const int nc = a.direct ? a.B * a.c.Hk : sms * C::BLOCKS;
    attn_stream_kernel<FMT, D, NB><<<nc, kStreamThreads, C::SMEM, st>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess || a.direct) return e;
    return launch_join<StreamTiling<C::GR>, C::ROWS, D>(a, 1, nc, st);
}

template <int FMT, int D>
cudaError_t launch_stream_n(const AttnArgs &a, int sms, cudaStream_t st) {
    const int rows = a.T * a.G;
    return rows <= 8 ? launch_stream_d<FMT, D, 1>(a, sms, st) : launch_stream_d<FMT, D, 2>(a, sms, st);
}

template <int FMT>
cudaError_t launch_stream(const AttnArgs &a, int sms, cudaStream_t st) {
    return a.c.D == 128 ? launch_stream_n<FMT, 128>(a, sms, st) : launch_stream_n<FMT, 64>(a, sms, st);
}

}  // namespace

}  // namespace tl
