// attn_stream.cuh -- attention for few rows per kv head (single tokens, small trees):
// the cache streams through registers once, fed to warp MMAs.
//
//   S = Q K^T, P = exp2(S sk f - m) sv, O += P V    (f = scale log2 e)
//
// For at most 16 rows the bytes of the cache bound the call (16 rows x 4 flops per
// 8-bit element: about 32 flops a byte), so everything is laid out for the stream:
//  * a tile is 64 keys, 16 for each of the block's 4 warps; warps share nothing until a
//    unit ends.  Pages hold multiples of 16 keys, so a warp's 16 keys lie in one page.
//  * each thread copies exactly the bytes that its own MMA fragments need, with
//    cp.async into a ring of its warp, several tiles ahead: no block barriers in the
//    loop, and no fragment is exchanged.  mma.m16n8k16 leaves the order of the
//    contracted axis free, so thread t of a quad takes 16 neighbouring elements of a
//    key (and of the next 64) for S, and for V its four keys' elements
//    [g D/8, (g + 1) D/8) of column group g: every global read is 64 or 128 bytes of
//    one row over a quad or eight lanes.
//  * S comes out in the layout in which P enters the second product.
//  * codes become f16 (exact); the products are exact, sums fp32.  Queries in bf16
//    enter as f16 scaled by the power of two of their row's largest element: exact
//    within 2^-14 of it, below that rounded at 2^-25 of it, far under the fp32 sums.
//  * P is rounded to f16 (2^-11 relative).  Weights are kept 2^14 up, so that those down to
//    2^-28 of the largest keep all 11 bits and none above 2^-39 vanishes.
//  * The value scales multiply P, relative to twice the largest scale met (svref).  The
//    running maximum moves only when exceeded by a factor of 4, svref only when
//    exceeded: the accumulators are rescaled a few times per unit, not per tile.
#pragma once

#include "attn_sched.cuh"
#include "kv.cuh"
#include "rope.cuh"

namespace tl {

namespace {

constexpr int kStreamKeys = 64, kStreamRows = 16, kStreamThreads = 128;

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

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// e4m3 for keys: NaN codes stay NaN (such a key's scores are its own)
__device__ __forceinline__ uint32_t e4m3x2_raw(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
        : "=r"(r)
        : "r"(w));
    return r;
}

// fields of 4 bits at bits 0-3 / 4-7 of each half, as f16x2 of field - 8
__device__ __forceinline__ uint32_t int4_lo(uint32_t x) {
    return h2_bits(__hsub2(h2_of((x & 0x000F000Fu) | 0x64006400u), __float2half2_rn(1032.f)));
}
__device__ __forceinline__ uint32_t int4_hi(uint32_t x) {  // 1024 + 16 u
    return h2_bits(__hfma2(h2_of((x & 0x00F000F0u) | 0x64006400u), __float2half2_rn(0.0625f), __float2half2_rn(-72.f)));
}

template <int FMT, int D>
struct StreamCfg {
    static constexpr int RB = D * KvCode<FMT>::bits / 8;  // bytes per row of codes
    static constexpr int KB = RB / 4;                     // bytes of a key per thread (scores)
    static constexpr int KC = KB > 16 ? 16 : KB;          // bytes per copy
    static constexpr int NKC = KB / KC;
    static constexpr int VB = RB / 8;                     // bytes of a key per thread (values)
    static constexpr int KSTEPS = D / 16;
    // one stage of one warp: keys' copies, values' copies, 16 + 16 scales
    static constexpr int KOFF = 0, VOFF = 2 * NKC * KC * 32, SOFF = VOFF + 4 * VB * 32;
    static constexpr int STAGE = SOFF + 128;
    static constexpr int NS = STAGE > 3000 ? 3 : STAGE > 2000 ? 5 : 8;  // stages per warp
    static constexpr int PITCH = D == 128 ? 144 : 80;     // floats per row of the join buffer
    // [stages of 4 warps][join rows][queries f16][row factors][per-warp max, sum, svref]
    static constexpr int JOFF = 4 * NS * STAGE;
    static constexpr int QOFF = JOFF + kStreamRows * PITCH * 4;
    static constexpr int FOFF = QOFF + kStreamRows * (D + 8) * 2;
    static constexpr int WOFF = FOFF + kStreamRows * 4;
    static constexpr int POFF = WOFF + 3 * 4 * kStreamRows * 4;
    static constexpr int SMEM = POFF + 64;
    static_assert(3 * (SMEM + 1024) <= 228 * 1024, "three blocks per SM");
};

template <int FMT, bool BF, int D>
__global__ void __launch_bounds__(kStreamThreads, 3) attn_stream_kernel(AttnArgs a, int rtiles) {
    using C = StreamCfg<FMT, D>;
    using T = typename std::conditional<BF, __nv_bfloat16, __half>::type;
    constexpr int KT = kStreamKeys, ROWS = kStreamRows, NT = D / 8;
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int nc = gridDim.x, units = a.c.Hk * rtiles, R = a.T * a.G;
    pdl_launch_dependents();

    AttnPlace place = attn_place<KT, kStreamThreads>(a, units, reinterpret_cast<int64_t *>(smem + C::POFF),
                                                     [&](int64_t N) { return attn_first_tile(blockIdx.x, N, nc); });
    const int64_t x0 = attn_first_tile(blockIdx.x, place.N, nc), x1 = attn_first_tile(blockIdx.x + 1, place.N, nc);
    if (x0 == x1) return;
    const int steps = (int)(x1 - x0);

    uint8_t *ring = smem + warp * C::NS * C::STAGE;
    const uint32_t ring_u32 = smem_u32(ring);
    AttnWalk in, out;  // the tile being copied, the tile being computed
    in.template start<KT>(a, place, x0);
    out = in;

    // Copies run NS - 1 tiles ahead; the page of the tile after that is already on its way.
    auto first_key = [&](const AttnWalk &w) { return w.tile * KT + warp * 16; };
    auto page_of = [&](const AttnWalk &w) {
        const int key = first_key(w);
        return key < w.ctx + a.T ? attn_page(a, w.b, key) : -1;
    };
    int page = page_of(in);
    auto issue = [&](int step) {
        const int key = first_key(in), L = in.ctx + a.T;
        const uint32_t st = ring_u32 + (uint32_t)(step % C::NS) * C::STAGE;
        if (page >= 0) {
            const int hk = in.unit / rtiles;
            const int64_t row = ((int64_t)page * a.c.Hk + hk) * a.c.P + (unsigned)key % (unsigned)a.c.P;
            const uint8_t *kp = a.c.kc + row * C::RB, *vp = a.c.vc + row * C::RB;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int j = 0; j < C::NKC; ++j)
                    cp_async<C::KC>(st + C::KOFF + ((n * C::NKC + j) * 32 + lane) * C::KC,
                                    kp + (n * 8 + g) * C::RB + j * 4 * C::KC + t * C::KC, key + n * 8 + g < L);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = 2 * t + (j & 1) + (j >> 1) * 8;
                cp_async<C::VB>(st + C::VOFF + (j * 32 + lane) * C::VB, vp + r * C::RB + g * C::VB, key + r < L);
            }
            if (lane < 8)
                cp_async<16>(st + C::SOFF + lane * 16, (lane < 4 ? a.c.ks : a.c.vs) + row + (lane & 3) * 4, true);
        }
        cp_commit();
        if (step + 1 < steps) {
            in.template next<KT>(a, units);
            page = page_of(in);
        }
    };
    int issued = 0;
#pragma unroll 1
    for (; issued < C::NS - 1; ++issued) {
        if (issued < steps) issue(issued);
        else cp_commit();
    }

    uint32_t qf[C::KSTEPS][4];
    float f0 = 0.f, f1 = 0.f;              // score factors of rows g and g + 8
    float m0 = kAttnLow, m1 = kAttnLow, l0 = 0.f, l1 = 0.f, svref = 1e-30f;
    float acc[NT][4];
    int tok0 = 0, tok1 = 0;                // new token of rows g and g + 8
    bool fresh = true;                     // the next tile begins a unit (for this block)
    int which = 0;                         // slot of a partial result

#pragma unroll 1
    for (int step = 0; step < steps; ++step) {
        const int hk = out.unit / rtiles, rt = out.unit % rtiles;
        if (fresh) {
            // ---------------- queries of the unit: rows as f16 in shared memory, then fragments
            fresh = false;
            const int row = threadIdx.x >> 3, part = threadIdx.x & 7, grow = rt * ROWS + row;
            constexpr int EPT = D / 8;
            float v[EPT];
            if (grow < R) {
                const T *q = static_cast<const T *>(a.q) + out.b * a.qb + (int64_t)(grow / a.G) * a.qt +
                             (int64_t)(hk * a.G + grow % a.G) * a.qh + part * EPT;
                if (a.q_vec) {
#pragma unroll
                    for (int i = 0; i < EPT; i += 8) {
                        float u[8];
                        ld8(q + i, u);
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[i + k] = u[k];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < EPT; ++i) v[i] = to_f32(q[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < EPT; ++i) v[i] = 0.f;
            }
            float down = 1.f, up = 1.f;
            if constexpr (BF) {
                float mx = 0.f;
#pragma unroll
                for (int i = 0; i < EPT; ++i) mx = fmaxf(mx, fabsf(v[i]));
#pragma unroll
                for (int o = 4; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const int e = (int)(__float_as_uint(mx) >> 23);  // biased exponent of the largest
                if (e > 0 && e < 254) {
                    down = __uint_as_float((uint32_t)(254 - e) << 23);
                    up = __uint_as_float((uint32_t)e << 23);
                }
            }
            __half *qs = reinterpret_cast<__half *>(smem + C::QOFF) + row * (D + 8) + part * EPT;
#pragma unroll
            for (int i = 0; i < EPT; i += 2)
                *reinterpret_cast<__half2 *>(qs + i) = __floats2half2_rn(v[i] * down, v[i + 1] * down);
            float *fac = reinterpret_cast<float *>(smem + C::FOFF);
            if (part == 0) fac[row] = a.scale * kLog2e * up;
            __syncthreads();
            const __half *qr = reinterpret_cast<const __half *>(smem + C::QOFF);
            auto pair = [&](int r, int d0, int d1) {
                const uint32_t lo = __half_as_ushort(qr[r * (D + 8) + d0]), hi = __half_as_ushort(qr[r * (D + 8) + d1]);
                return lo | (hi << 16);
            };
#pragma unroll
            for (int s = 0; s < C::KSTEPS; ++s) {
                int d0, d1, d2, d3;  // the elements of this thread in step s, in the order its code words give
                if constexpr (FMT == kKvInt4) {
                    const int e = t * (D / 4) + (s >> 1) * 8 + (s & 1) * 2;
                    d0 = e, d1 = e + 4, d2 = e + 1, d3 = e + 5;
                } else {
                    const int e = (s >> 2) * 64 + t * 16 + (s & 3) * 4;
                    d0 = e, d1 = e + 1, d2 = e + 2, d3 = e + 3;
                }
                qf[s][0] = pair(g, d0, d1);
                qf[s][1] = pair(g + 8, d0, d1);
                qf[s][2] = pair(g, d2, d3);
                qf[s][3] = pair(g + 8, d2, d3);
            }
            f0 = fac[g];
            f1 = fac[g + 8];
            tok0 = min(R - 1, rt * ROWS + g) / a.G;
            tok1 = min(R - 1, rt * ROWS + g + 8) / a.G;
            m0 = m1 = kAttnLow;
            l0 = l1 = 0.f;
            svref = 1e-30f;
#pragma unroll
            for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
            __syncthreads();  // the queries' buffer may be written again
        }

        // ---------------- one group of 16 keys
        if (issued < steps) issue(issued);
        else cp_commit();
        ++issued;
        cp_wait<C::NS - 1>();
        __syncwarp();  // the scales were copied by other lanes
        const int key = first_key(out), L = out.ctx + a.T;
        if (key < L) {
            const uint8_t *st = ring + (step % C::NS) * C::STAGE;
            float s[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
                uint32_t w[C::KB / 4];
#pragma unroll
                for (int j = 0; j < C::NKC; ++j) {
                    const uint8_t *p = st + C::KOFF + ((n * C::NKC + j) * 32 + lane) * C::KC;
                    if constexpr (C::KC == 16) {
                        const uint4 u = *reinterpret_cast<const uint4 *>(p);
                        w[4 * j] = u.x, w[4 * j + 1] = u.y, w[4 * j + 2] = u.z, w[4 * j + 3] = u.w;
                    } else {
                        const uint2 u = *reinterpret_cast<const uint2 *>(p);
                        w[0] = u.x, w[1] = u.y;
                    }
                }
                if constexpr (FMT == kKvInt4) {
#pragma unroll
                    for (int i = 0; i < C::KSTEPS / 2; ++i) {
                        mma16816(s[n], qf[2 * i], int4_lo(w[i]), int4_hi(w[i]));
                        mma16816(s[n], qf[2 * i + 1], int4_lo(w[i] >> 8), int4_hi(w[i] >> 8));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < C::KSTEPS; ++i) {
                        uint32_t b0, b1;
                        if constexpr (FMT == kKvInt8) {
                            const uint32_t u = w[i] ^ 0x80808080u;
                            b0 = int8_f16x2(__byte_perm(u, 0x64646464u, 0x4140));
                            b1 = int8_f16x2(__byte_perm(u, 0x64646464u, 0x4342));
                        } else {
                            b0 = e4m3x2_raw(w[i]);
                            b1 = e4m3x2_raw(w[i] >> 16);
                        }
                        mma16816(s[n], qf[i], b0, b1);
                    }
                }
            }
            // keys of this thread: key + 2t, + 1, + 8 + 2t, + 1
            const float2 ka = *reinterpret_cast<const float2 *>(st + C::SOFF + t * 8);
            const float2 kb = *reinterpret_cast<const float2 *>(st + C::SOFF + 32 + t * 8);
            const float2 va = *reinterpret_cast<const float2 *>(st + C::SOFF + 64 + t * 8);
            const float2 vb = *reinterpret_cast<const float2 *>(st + C::SOFF + 96 + t * 8);
            const float sk[4] = {ka.x, ka.y, kb.x, kb.y};
            float sv[4] = {va.x, va.y, vb.x, vb.y};
            // z: scores in powers of two, rows g and g + 8
            float z0[4], z1[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                z0[j] = s[j >> 1][j & 1] * sk[j] * f0;
                z1[j] = s[j >> 1][2 + (j & 1)] * sk[j] * f1;
            }
            uint32_t see0 = 0xFu, see1 = 0xFu;
            const bool edge = key + 16 > out.ctx;  // new tokens' keys, or the end
            if (edge) {
                see0 = see1 = 0u;
                const uint8_t *tree = a.tree ? a.tree + out.b * a.tree_b : nullptr;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int i = key + 2 * t + (j & 1) + (j >> 1) * 8 - out.ctx;  // index of the new token
                    bool u0 = i < 0, u1 = i < 0;
                    if (i >= 0 && i < a.T) {
                        u0 = tree ? tree[tok0 * a.tree_r + i] != 0 : i <= tok0;
                        u1 = tree ? tree[tok1 * a.tree_r + i] != 0 : i <= tok1;
                    }
                    if (u0) see0 |= 1u << j;
                    else z0[j] = -INFINITY;
                    if (u1) see1 |= 1u << j;
                    else z1[j] = -INFINITY;
                    if (!u0 && !u1) sv[j] = 0.f;  // unseen scales may hold anything
                }
            }
            const float x0v = fmaxf(fmaxf(z0[0], z0[1]), fmaxf(z0[2], z0[3]));
            const float x1v = fmaxf(fmaxf(z1[0], z1[1]), fmaxf(z1[2], z1[3]));
            const float svm = fmaxf(fmaxf(sv[0], sv[1]), fmaxf(sv[2], sv[3]));
            if (__any_sync(0xffffffffu, x0v > m0 + kAttnSlack || x1v > m1 + kAttnSlack || svm > svref)) {
                float r0 = x0v, r1 = x1v, rv = svm;
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    r0 = fmaxf(r0, __shfl_xor_sync(0xffffffffu, r0, o));
                    r1 = fmaxf(r1, __shfl_xor_sync(0xffffffffu, r1, o));
                }
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) rv = fmaxf(rv, __shfl_xor_sync(0xffffffffu, rv, o));
                r0 = fmaxf(r0, m0);
                r1 = fmaxf(r1, m1);
                const float c0 = ex2(m0 - r0), c1 = ex2(m1 - r1);
                float cv = 1.f;
                if (rv > svref) {  // twice the largest: the next slightly larger one changes nothing
                    cv = svref / (2.f * rv);
                    svref = 2.f * rv;
                }
                m0 = r0;
                m1 = r1;
                l0 *= c0;
                l1 *= c1;
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    acc[i][0] *= c0 * cv;
                    acc[i][1] *= c0 * cv;
                    acc[i][2] *= c1 * cv;
                    acc[i][3] *= c1 * cv;
                }
            }
            const float inv = __frcp_rn(svref);
            float p0[4], p1[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float e0 = ex2(z0[j] - m0 + kAttnUp), e1 = ex2(z1[j] - m1 + kAttnUp);
                l0 += e0;
                l1 += e1;
                const float w = sv[j] * inv;
                p0[j] = e0 * w;
                p1[j] = e1 * w;
            }
            if (edge) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (!(see0 >> j & 1u)) p0[j] = 0.f;
                    if (!(see1 >> j & 1u)) p1[j] = 0.f;
                }
            }
            uint32_t pa[4];
            pa[0] = pack2(__half(), p0[0], p0[1]);
            pa[1] = pack2(__half(), p1[0], p1[1]);
            pa[2] = pack2(__half(), p0[2], p0[3]);
            pa[3] = pack2(__half(), p1[2], p1[3]);
            // values: column d = (D / 8) n + i of MMA i belongs to lane group n
            uint32_t w[4][C::VB / 4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint8_t *p = st + C::VOFF + (j * 32 + lane) * C::VB;
                if constexpr (C::VB == 16) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(p);
                    w[j][0] = u.x, w[j][1] = u.y, w[j][2] = u.z, w[j][3] = u.w;
                } else if constexpr (C::VB == 8) {
                    const uint2 u = *reinterpret_cast<const uint2 *>(p);
                    w[j][0] = u.x, w[j][1] = u.y;
                } else {
                    w[j][0] = *reinterpret_cast<const uint32_t *>(p);
                }
            }
#pragma unroll
            for (int i = 0; i < C::VB / 4; ++i) {
                if constexpr (FMT == kKvInt4) {
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {  // elements 0-3, then 4-7, of the two keys of a pair
                        const uint32_t sel = hh ? 0x7632 : 0x5410;
                        const uint32_t x = __byte_perm(w[0][i], w[1][i], sel), y = __byte_perm(w[2][i], w[3][i], sel);
                        mma16816(acc[8 * i + 4 * hh], pa, int4_lo(x), int4_lo(y));
                        mma16816(acc[8 * i + 4 * hh + 1], pa, int4_hi(x), int4_hi(y));
                        mma16816(acc[8 * i + 4 * hh + 2], pa, int4_lo(x >> 8), int4_lo(y >> 8));
                        mma16816(acc[8 * i + 4 * hh + 3], pa, int4_hi(x >> 8), int4_hi(y >> 8));
                    }
                } else {
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {  // bytes 0, 1, then 2, 3, interleaved over the pair's keys
                        const uint32_t sel = hh ? 0x7362 : 0x5140;
                        uint32_t x = __byte_perm(w[0][i], w[1][i], sel), y = __byte_perm(w[2][i], w[3][i], sel);
                        uint32_t xa, xb, ya, yb;
                        if constexpr (FMT == kKvInt8) {
                            x ^= 0x80808080u;
                            y ^= 0x80808080u;
                            xa = int8_f16x2(__byte_perm(x, 0x64646464u, 0x4140));
                            xb = int8_f16x2(__byte_perm(x, 0x64646464u, 0x4342));
                            ya = int8_f16x2(__byte_perm(y, 0x64646464u, 0x4140));
                            yb = int8_f16x2(__byte_perm(y, 0x64646464u, 0x4342));
                        } else {
                            xa = e4m3x2_f16x2(x);
                            xb = e4m3x2_f16x2(x >> 16);
                            ya = e4m3x2_f16x2(y);
                            yb = e4m3x2_f16x2(y >> 16);
                        }
                        mma16816(acc[4 * i + 2 * hh], pa, xa, ya);
                        mma16816(acc[4 * i + 2 * hh + 1], pa, xb, yb);
                    }
                }
            }
        }
        __syncwarp();  // every lane is done with the stage (its scales are shared)

        // ---------------- the end of a unit, or of the run: join the warps, write
        const bool last = out.tile + 1 == out.tiles;
        if (last || step + 1 == steps) {
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                l0 += __shfl_xor_sync(0xffffffffu, l0, o);
                l1 += __shfl_xor_sync(0xffffffffu, l1, o);
            }
            float *wm = reinterpret_cast<float *>(smem + C::WOFF), *wl = wm + 4 * ROWS;
            if (t == 0) {
                wm[warp * ROWS + g] = m0;
                wm[warp * ROWS + g + 8] = m1;
                wl[warp * ROWS + g] = l0;
                wl[warp * ROWS + g + 8] = l1;
            }
            __syncthreads();
            float M0 = wm[g], M1 = wm[g + 8];
#pragma unroll
            for (int i = 1; i < 4; ++i) {
                M0 = fmaxf(M0, wm[i * ROWS + g]);
                M1 = fmaxf(M1, wm[i * ROWS + g + 8]);
            }
            const float c0 = ex2(m0 - M0) * svref, c1 = ex2(m1 - M1) * svref;
            float *jb = reinterpret_cast<float *>(smem + C::JOFF);
            constexpr int RUN = D / 4;  // this thread's neighbouring elements of a row
#pragma unroll 1
            for (int turn = 0; turn < 4; ++turn) {
                if (turn == warp) {
                    float *r0 = jb + g * C::PITCH + t * (RUN + 4), *r1 = r0 + 8 * C::PITCH;
#pragma unroll
                    for (int e = 0; e < RUN; e += 4) {
                        float4 u, v;
                        float *pu = &u.x, *pv = &v.x;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int i = (e + k) % NT, h = (e + k) / NT;
                            pu[k] = acc[i][h] * c0;
                            pv[k] = acc[i][2 + h] * c1;
                        }
                        float4 *d0 = reinterpret_cast<float4 *>(r0 + e), *d1 = reinterpret_cast<float4 *>(r1 + e);
                        if (turn > 0) {
                            const float4 x = *d0, y = *d1;
                            u.x += x.x, u.y += x.y, u.z += x.z, u.w += x.w;
                            v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
                        }
                        *d0 = u;
                        *d1 = v;
                    }
                }
                __syncthreads();
            }
            const bool whole = last && step >= out.tile;  // the block saw the unit from its first tile on
            const int row = threadIdx.x >> 3, part = threadIdx.x & 7, grow = rt * ROWS + row;
            if (grow < R) {
                float M = wm[row], Ls = 0.f;
#pragma unroll
                for (int i = 1; i < 4; ++i) M = fmaxf(M, wm[i * ROWS + row]);
#pragma unroll
                for (int i = 0; i < 4; ++i) Ls += wl[i * ROWS + row] * ex2(wm[i * ROWS + row] - M);
                constexpr int EPT = D / 8;
                const float *src = jb + row * C::PITCH + (part * EPT) / RUN * (RUN + 4) + (part * EPT) % RUN;
                float v[EPT];
#pragma unroll
                for (int e = 0; e < EPT; e += 4) {
                    const float4 u = *reinterpret_cast<const float4 *>(src + e);
                    v[e] = u.x, v[e + 1] = u.y, v[e + 2] = u.z, v[e + 3] = u.w;
                }
                if (whole) {
                    const float rl = Ls == 0.f ? 0.f : 1.f / Ls;
                    const int64_t out_row = ((int64_t)out.b * a.T + grow / a.G) * a.Hq + hk * a.G + grow % a.G;
                    T *o = static_cast<T *>(a.out) + out_row * D + part * EPT;
#pragma unroll
                    for (int e = 0; e < EPT; e += 8) {
                        float u[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) u[k] = v[e + k] * rl;
                        st8(o + e, u);
                    }
                    if (a.lse && part == 0) a.lse[out_row] = Ls == 0.f ? -INFINITY : (M - kAttnUp + log2f(Ls)) * kLn2;
                } else {
                    float *slot = AttnSlot<ROWS, D>::at(a.ws, blockIdx.x, which);
                    float *o = slot + row * D + part * EPT;
#pragma unroll
                    for (int e = 0; e < EPT; e += 4)
                        *reinterpret_cast<float4 *>(o + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                    if (part == 0) {
                        slot[ROWS * D + row] = M - kAttnUp;
                        slot[ROWS * (D + 1) + row] = Ls;
                    }
                }
            }
            which = 1;
            fresh = true;
            __syncthreads();  // the join buffers may be written again
        }
        if (step + 1 < steps) out.template next<KT>(a, units);
    }
    cp_wait<0>();
}

template <int FMT, bool BF, int D>
cudaError_t launch_stream_d(const AttnArgs &a, int nc, int rtiles, cudaStream_t st) {
    using C = StreamCfg<FMT, D>;
    static const cudaError_t attr = cudaFuncSetAttribute(
        attn_stream_kernel<FMT, BF, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (attr != cudaSuccess) return attr;
    attn_stream_kernel<FMT, BF, D><<<nc, kStreamThreads, C::SMEM, st>>>(a, rtiles);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)a.B * a.c.Hk * rtiles * kStreamRows), 1, 1);
    cfg.blockDim = dim3(128, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<BF, kStreamKeys, kStreamRows, D>, a, rtiles, nc);
}

template <int FMT>
cudaError_t launch_stream(const AttnArgs &a, bool bf, int nc, cudaStream_t st) {
    const int rtiles = (a.T * a.G + kStreamRows - 1) / kStreamRows;
    if (a.c.D == 128)
        return bf ? launch_stream_d<FMT, true, 128>(a, nc, rtiles, st) : launch_stream_d<FMT, false, 128>(a, nc, rtiles, st);
    return bf ? launch_stream_d<FMT, true, 64>(a, nc, rtiles, st) : launch_stream_d<FMT, false, 64>(a, nc, rtiles, st);
}

}  // namespace

}  // namespace tl
