// attn_tile.cuh -- attention for many rows per kv head (drafted trees, chunks of a prompt)
// on the 5th-generation tensor cores.
//
//   S = Q K^T, P = exp2(S sk f - m) sv, O += P V    (f = scale log2 e)
//
// A block owns 128 rows of one (sequence, kv head) -- TMEM lanes, one softmax thread
// each -- and walks tiles of 128 keys; two blocks per SM, so that one's softmax runs
// under the other's products:
//  * Warps 4-7 decode: codes go from global memory to registers a tile ahead, become f16
//    (exact) and are stored to shared memory in 128-byte-swizzled rows, keys and values
//    alike: keys are read as a K-major operand, values as an MN-major one, so neither
//    is transposed.  They also place the queries at a unit's start (f16; from bf16 scaled
//    by the power of two of the row's largest element) and the tile's scales.
//  * Warp 8 issues tcgen05.mma (kind::f16, fp32 in TMEM): S = Q K^T from shared memory,
//    O += P V with P from TMEM.
//  * Warps 0-3: a row's 128 scores are read twice from TMEM, once for the maximum, once for
//    the weights; P (f16) overwrites the first half of S.  The weights hold the value scale
//    relative to a power of two svref at least twice the largest scale met, 2^14 up, so
//    that weights down to 2^-28 of the largest keep all 11 bits.  The maximum moves only
//    when exceeded by a factor of 4, and svref when exceeded: then O is rescaled in TMEM.
// Per 128 keys and 128 rows: 1024 tensor cycles, 128 x 128 exponentials and about 1000
// issue slots of decode and softmax per scheduler set: the three are near one another.
// Every mbarrier wait is bounded; one that gives up sets the device status word, and the
// block stops issuing work, frees its TMEM and returns.
#pragma once

#include "attn_sched.cuh"
#include "kv.cuh"
#include "rope.cuh"
#include "tc.cuh"

namespace tl {

namespace {

constexpr int kLowExp = -80;  // of the value scale before any key
constexpr int kTileKeys = 128, kTileRows = 128, kTileThreads = 288;

template <int FMT, int D>
struct AttnTileCfg {
    static constexpr int HALVES = D / 64;                 // 64-element (128-byte) column blocks
    static constexpr int BLOCK = 128 * 128;               // bytes of one: 128 rows of 128 B
    static constexpr int UB = 16 * KvCode<FMT>::bits / 8; // bytes of 16 codes
    static constexpr int RB = D / 16 * UB;                // bytes per row of codes
    static constexpr int LANES = D / 16;                  // threads per row
    static constexpr int RPI = 128 / LANES;               // rows per pass of the four warps: 16 or 32
    static constexpr int PASSES = 128 / RPI;
    static constexpr uint32_t SCOL = 0, OCOL = 128, COLS = 256;
    static constexpr int QOFF = 0, KOFF = HALVES * BLOCK, VOFF = 2 * HALVES * BLOCK;
    static constexpr int SKOFF = 3 * HALVES * BLOCK;      // key scales [2][128], value scales [2][128],
    static constexpr int SVOFF = SKOFF + 1024;
    static constexpr int SMOFF = SVOFF + 1024;            // largest value scale [2],
    static constexpr int FOFF = SMOFF + 16;               // row factors [2][128]
    static constexpr int BOFF = FOFF + 1024;              // barriers, TMEM slot, abort flag
    static constexpr int POFF = BOFF + 64;                // place of the run (11 words)
    static constexpr int SMEM = POFF + 96 + 1024;         // 1 KB of alignment slack
    // no more blocks per SM than its 512 TMEM columns serve
    static constexpr int REQ = SMEM > 80 * 1024 ? SMEM : 80 * 1024;
    static_assert(2 * (REQ + 1024) <= 228 * 1024 && 3 * (REQ + 1024) > 228 * 1024, "two blocks per SM");
};

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)),
          "l"(reinterpret_cast<uint64_t &>(c)));
    return d;
}

template <int FMT, bool BF, int D>
__global__ void __launch_bounds__(kTileThreads, 2) attn_tile_kernel(AttnArgs a, int rtiles) {
    using C = AttnTileCfg<FMT, D>;
    using T = typename std::conditional<BF, __nv_bfloat16, __half>::type;
    constexpr int KT = kTileKeys, ROWS = kTileRows;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::BOFF);
    uint64_t *kfull = bars, *vfull = bars + 1, *sdone = bars + 2, *pfull = bars + 3, *odone = bars + 4;
    uint64_t *fin = bars + 5;  // after a give-up: every product issued has ended
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 6);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nc = gridDim.x, R = a.T * a.G, units = a.c.Hk * rtiles;
    pdl_launch_dependents();

    if (threadIdx.x == 0) {
        mbar_init(kfull, 4);  // one arrival per decoder warp
        mbar_init(vfull, 4);
        mbar_init(sdone, 1);
        mbar_init(pfull, 4);  // one per softmax warp
        mbar_init(odone, 1);
        mbar_init(fin, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    const AttnPlace place = attn_place<KT, kTileThreads>(a, units, reinterpret_cast<int64_t *>(smem + C::POFF),
                                                         [&](int64_t N) { return attn_first_tile(blockIdx.x, N, nc); });
    const int64_t x0 = attn_first_tile(blockIdx.x, place.N, nc), x1 = attn_first_tile(blockIdx.x + 1, place.N, nc);
    if (x0 == x1) return;
    const int steps = (int)(x1 - x0);
    if (warp == 8) tc::tmem_alloc(tmem_slot, C::COLS);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;

    auto wait = [&](uint64_t *bar, int phase) -> bool {  // completion of the barrier's phase 0, 1, 2 ..
        if (!*abort_flag && mbar_wait_bounded(bar, (uint32_t)phase & 1u)) return true;
        *abort_flag = 1;
        if (a.status) atomicExch(a.status, kStatusTimeout);
        return false;
    };

    AttnWalk at;
    at.template start<KT>(a, place, x0);

    if (warp >= 4 && warp < 8) {
        // ---------------- decoders
        const int dw = warp - 4;
        // LANES threads per row of codes; the store order keeps each 8 lanes' 16-byte
        // chunks in different banks
        const int cu = C::LANES == 8 ? (lane & 3) + 4 * (lane >> 4) : lane & 3;
        const int r0 = C::LANES == 8 ? dw * 4 + ((lane >> 2) & 3) : dw * 8 + (lane >> 2);
        // first row of group i of 16 keys: lane i holds it for the tile that is loaded next
        int64_t rowbase = 0;
        auto locate = [&](const AttnWalk &w) {
            const int key = w.tile * KT + (lane & 7) * 16;
            if (key < w.ctx + a.T)
                rowbase = ((int64_t)attn_page(a, w.b, key) * a.c.Hk + w.unit / rtiles) * a.c.P + (unsigned)key % (unsigned)a.c.P;
        };
        using Unit = typename std::conditional<C::UB == 16, uint4, uint2>::type;
        Unit kreg[C::PASSES], vreg[C::PASSES];
        float4 sreg = make_float4(0.f, 0.f, 0.f, 0.f);  // warp 4: key scales, warp 5: value scales, 4 per lane
        auto load = [&](const AttnWalk &w, const uint8_t *codes, Unit(&reg)[C::PASSES]) {
            const int left = w.ctx + a.T - w.tile * KT;
#pragma unroll
            for (int i = 0; i < C::PASSES; ++i) {
                const int r = i * C::RPI + r0;
                const int64_t base = __shfl_sync(0xffffffffu, rowbase, r >> 4);
                reg[i] = Unit{};
                if (r < left) {
                    const uint8_t *p = codes + (base + (r & 15)) * C::RB + cu * C::UB;
                    if constexpr (C::UB == 16) reg[i] = ldg_nc_v4(p);
                    else reg[i] = ldg_nc_v2(p);
                }
            }
        };
        auto load_scales = [&](const AttnWalk &w) {
            if (dw > 1) return;
            const int left = w.ctx + a.T - w.tile * KT, r = lane * 4;
            const int64_t base = __shfl_sync(0xffffffffu, rowbase, r >> 4);
            sreg = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < left) {
                sreg = *reinterpret_cast<const float4 *>((dw ? a.c.vs : a.c.ks) + base + (r & 15));
                if (r + 1 >= left) sreg.y = 0.f;
                if (r + 2 >= left) sreg.z = 0.f;
                if (r + 3 >= left) sreg.w = 0.f;
            }
        };
        auto store = [&](uint8_t *dst, const Unit(&reg)[C::PASSES]) {
#pragma unroll
            for (int i = 0; i < C::PASSES; ++i) {
                const int r = i * C::RPI + r0;
                uint32_t w[4], h[8];
                if constexpr (C::UB == 16) w[0] = reg[i].x, w[1] = reg[i].y, w[2] = reg[i].z, w[3] = reg[i].w;
                else w[0] = reg[i].x, w[1] = reg[i].y;
                codes16_f16<FMT>(w, h);
                uint8_t *row = dst + (cu >> 2) * C::BLOCK + r * 128;
                const int ch = 2 * (cu & 3);
                *reinterpret_cast<uint4 *>(row + ((ch ^ (r & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4 *>(row + (((ch + 1) ^ (r & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
            }
        };
        auto queries = [&](const AttnWalk &w, int parity) {
            const int r = dw * 32 + lane, grow = (w.unit % rtiles) * ROWS + r, hk = w.unit / rtiles;
            const bool has = grow < R;
            const T *q = static_cast<const T *>(a.q) + w.b * a.qb + (int64_t)(has ? grow / a.G : 0) * a.qt +
                         (int64_t)(hk * a.G + (has ? grow % a.G : 0)) * a.qh;
            auto get8 = [&](int i, float(&v)[8]) {
                if (!has) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] = 0.f;
                } else if (a.q_vec) {
                    ld8(q + i, v);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] = to_f32(q[i + k]);
                }
            };
            float down = 1.f, up = 1.f;
            if constexpr (BF) {
                float mx = 0.f;
#pragma unroll 4
                for (int i = 0; i < D; i += 8) {
                    float v[8];
                    get8(i, v);
#pragma unroll
                    for (int k = 0; k < 8; ++k) mx = fmaxf(mx, fabsf(v[k]));
                }
                const int e = (int)(__float_as_uint(mx) >> 23);  // biased exponent of the largest
                if (e > 0 && e < 254) {
                    down = __uint_as_float((uint32_t)(254 - e) << 23);
                    up = __uint_as_float((uint32_t)e << 23);
                }
            }
#pragma unroll 4
            for (int i = 0; i < D; i += 8) {
                float v[8];
                get8(i, v);
                uint4 h;
                h.x = pack2(__half(), v[0] * down, v[1] * down);
                h.y = pack2(__half(), v[2] * down, v[3] * down);
                h.z = pack2(__half(), v[4] * down, v[5] * down);
                h.w = pack2(__half(), v[6] * down, v[7] * down);
                *reinterpret_cast<uint4 *>(smem + C::QOFF + (i >> 6) * C::BLOCK + r * 128 + ((((i >> 3) & 7) ^ (r & 7)) << 4)) = h;
            }
            reinterpret_cast<float *>(smem + C::FOFF)[parity * 128 + r] = a.scale * kLog2e * up;
        };
        auto publish = [&](uint64_t *bar) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };

        locate(at);
        load(at, a.c.kc, kreg);
        load(at, a.c.vc, vreg);
        load_scales(at);
        AttnWalk ahead = at;  // the tile that is loaded next
        int parity = 0;
        bool fresh = true;
#pragma unroll 1
        for (int j = 0; j < steps; ++j) {
            const bool more = j + 1 < steps;
            const AttnWalk now = ahead;
            if (more) {
                ahead.template next<KT>(a, units);
                locate(ahead);
            }
            if (j > 0 && !wait(sdone, j - 1)) break;  // S of the last tile is computed: Q and K are free
            if (fresh) queries(now, parity);
            store(smem + C::KOFF, kreg);
            if (dw < 2) {
                reinterpret_cast<float4 *>(smem + (dw ? C::SVOFF : C::SKOFF) + (j & 1) * 512)[lane] = sreg;
                if (dw == 1) {  // the largest value scale among keys that every row sees
                    const int k = now.tile * KT + lane * 4;
                    float mx = 0.f;
                    if (k < now.ctx) mx = sreg.x;
                    if (k + 1 < now.ctx) mx = fmaxf(mx, sreg.y);
                    if (k + 2 < now.ctx) mx = fmaxf(mx, sreg.z);
                    if (k + 3 < now.ctx) mx = fmaxf(mx, sreg.w);
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    if (lane == 0) reinterpret_cast<float *>(smem + C::SMOFF)[j & 1] = mx;
                }
            }
            publish(kfull);
            if (more) {
                load(ahead, a.c.kc, kreg);
                load_scales(ahead);
            }
            if (j > 0 && !wait(odone, j - 1)) break;
            store(smem + C::VOFF, vreg);
            publish(vfull);
            if (more) load(ahead, a.c.vc, vreg);
            fresh = now.tile + 1 == now.tiles;
            if (fresh) parity ^= 1;
        }
    } else if (warp == 8) {
        // ---------------- MMA issuer
        if (lane == 0) {
            constexpr uint32_t idesc_s = tc::idesc_f16(KT, false);
            constexpr uint32_t idesc_o = tc::idesc_f16(D, false) | tc::kIdescBTransposed;
            bool fresh = true;
#pragma unroll 1
            for (int j = 0; j < steps; ++j) {
                // P of the last tile lies in S's columns: its product has to be done
                if ((j > 0 && !wait(odone, j - 1)) || !wait(kfull, j)) break;
                tc::fence_after_sync();
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t qd = tc::desc_sw128(smem + C::QOFF + (k >> 2) * C::BLOCK) + (uint64_t)((k & 3) * 2);
                    const uint64_t kd = tc::desc_sw128(smem + C::KOFF + (k >> 2) * C::BLOCK) + (uint64_t)((k & 3) * 2);
                    tc::mma_ss(tmem + C::SCOL, qd, kd, idesc_s, k > 0);
                }
                tc::commit(sdone);
                if (!wait(pfull, j) || !wait(vfull, j)) break;
                tc::fence_after_sync();
                const uint64_t vd = tc::desc_sw128_mn(smem + C::VOFF, C::BLOCK);
#pragma unroll
                for (int k = 0; k < KT / 16; ++k)
                    tc::mma_ts(tmem + C::OCOL, tmem + C::SCOL + k * 8, vd + (uint64_t)(k * 128), idesc_o, !fresh || k > 0);
                tc::commit(odone);
                fresh = at.tile + 1 == at.tiles;
                if (j + 1 < steps) at.template next<KT>(a, units);
            }
        }
        __syncwarp();
    } else {
        // ---------------- softmax: thread = row = TMEM lane
        const int row = threadIdx.x;
        const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
        float m = kAttnLow, l = 0.f, f = 0.f;
        int ve = kLowExp;                     // svref = 2^ve
        int parity = 0, which = 0;
        bool fresh = true;
#pragma unroll 1
        for (int j = 0; j < steps; ++j) {
            const int rt = at.unit % rtiles, hk = at.unit / rtiles, grow = rt * ROWS + row;
            const bool live = rt * ROWS + warp * 32 < R;  // the warp has rows
            const bool last = at.tile + 1 == at.tiles;
            if (!wait(sdone, j)) break;
            tc::fence_after_sync();
            if (live) {
                if (fresh) {
                    f = reinterpret_cast<const float *>(smem + C::FOFF)[parity * 128 + row];
                    m = kAttnLow;
                    l = 0.f;
                    ve = kLowExp;
                }
                const float4 *sk = reinterpret_cast<const float4 *>(smem + C::SKOFF + (j & 1) * 512);
                const float4 *sv = reinterpret_cast<const float4 *>(smem + C::SVOFF + (j & 1) * 512);
                float svmax = reinterpret_cast<const float *>(smem + C::SMOFF)[j & 1];
                const int key = at.tile * KT;
                const bool edge = key + KT > at.ctx;  // new tokens' keys, or the end
                uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};
                if (edge) {
                    const int tok = min(grow, R - 1) / a.G;
                    const uint8_t *tree = a.tree ? a.tree + at.b * a.tree_b + (int64_t)tok * a.tree_r : nullptr;
                    const float *svs = reinterpret_cast<const float *>(sv);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int i0 = key + 32 * c - at.ctx;  // index of the new token at the chunk's start
                        if (i0 + 32 <= 0) continue;
                        uint32_t bits = 0;
                        for (int k = 0; k < 32; ++k) {
                            const int i = i0 + k;
                            bool u = i < 0;
                            if (i >= 0 && i < a.T) u = tree ? tree[i] != 0 : i <= tok;
                            if (u) {
                                bits |= 1u << k;
                                svmax = fmaxf(svmax, svs[32 * c + k]);
                            }
                        }
                        see[c] = bits;
                    }
                }
                // ---- the row's largest score
                float top = -INFINITY;
                auto largest = [&](auto masked) {
                    constexpr bool EDGE = decltype(masked)::value;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t s[32];
                    tc::ld_32x32b_x32(lane_base + C::SCOL + c * 32, s);
                    tc::wait_ld();
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        const float4 w = sk[c * 8 + k / 4];
                        float2 x = mul2(make_float2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), make_float2(w.x, w.y));
                        float2 y = mul2(make_float2(__uint_as_float(s[k + 2]), __uint_as_float(s[k + 3])), make_float2(w.z, w.w));
                        if constexpr (EDGE) {
                            if (!(see[c] >> k & 1u)) x.x = -INFINITY;
                            if (!(see[c] >> (k + 1) & 1u)) x.y = -INFINITY;
                            if (!(see[c] >> (k + 2) & 1u)) y.x = -INFINITY;
                            if (!(see[c] >> (k + 3) & 1u)) y.y = -INFINITY;
                        }
                        top = fmaxf(fmaxf(top, x.x), x.y);
                        top = fmaxf(fmaxf(top, y.x), y.y);
                    }
                }
                };
                if (edge) largest(std::true_type());
                else largest(std::false_type());
                top *= f;
                const bool bigger = svmax > __uint_as_float((uint32_t)(ve + 127) << 23);
                const bool move = top > m + kAttnSlack || bigger;
                if (__any_sync(0xffffffffu, move)) {
                    const float mn = fmaxf(m, top);
                    // a power of two in (2 svmax, 4 svmax]
                    const int vn = bigger ? min(120, (int)(__float_as_uint(svmax) >> 23) - 127 + 2) : ve;
                    const float c = ex2(m - mn + (float)(ve - vn));
                    m = mn;
                    ve = vn;
                    l *= c;
                    if (!fresh) {
#pragma unroll
                        for (int h = 0; h < D / 32; ++h) {
                            uint32_t o[32];
                            tc::ld_32x32b_x32(lane_base + C::OCOL + h * 32, o);
                            tc::wait_ld();
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * c);
                            tc::st_32x32b_x32(lane_base + C::OCOL + h * 32, o);
                        }
                        tc::wait_st();
                    }
                }
                // ---- the weights
                const float off = kAttnUp - m - (float)ve;
                const float2 f2 = make_float2(f, f), off2 = make_float2(off, off);
                float2 l2 = make_float2(0.f, 0.f);
                auto weigh = [&](auto masked) {
                    constexpr bool EDGE = decltype(masked)::value;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t s[32], p[16];
                    tc::ld_32x32b_x32(lane_base + C::SCOL + c * 32, s);
                    tc::wait_ld();
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        const float4 w = sk[c * 8 + k / 4], v = sv[c * 8 + k / 4];
                        float2 x = mul2(make_float2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), make_float2(w.x, w.y));
                        float2 y = mul2(make_float2(__uint_as_float(s[k + 2]), __uint_as_float(s[k + 3])), make_float2(w.z, w.w));
                        x = fma2(x, f2, off2);
                        y = fma2(y, f2, off2);
                        x = make_float2(ex2(x.x), ex2(x.y));
                        y = make_float2(ex2(y.x), ex2(y.y));
                        if constexpr (EDGE) {
                            if (!(see[c] >> k & 1u)) x.x = 0.f;
                            if (!(see[c] >> (k + 1) & 1u)) x.y = 0.f;
                            if (!(see[c] >> (k + 2) & 1u)) y.x = 0.f;
                            if (!(see[c] >> (k + 3) & 1u)) y.y = 0.f;
                        }
                        l2 = add2(l2, add2(x, y));
                        x = mul2(x, make_float2(v.x, v.y));
                        y = mul2(y, make_float2(v.z, v.w));
                        if constexpr (EDGE) {  // an unseen scale may be a NaN
                            if (!(see[c] >> k & 1u)) x.x = 0.f;
                            if (!(see[c] >> (k + 1) & 1u)) x.y = 0.f;
                            if (!(see[c] >> (k + 2) & 1u)) y.x = 0.f;
                            if (!(see[c] >> (k + 3) & 1u)) y.y = 0.f;
                        }
                        p[k / 2] = pack2(__half(), x.x, x.y);
                        p[k / 2 + 1] = pack2(__half(), y.x, y.y);
                    }
                    tc::st_32x32b_x16(lane_base + C::SCOL + c * 16, p);
                }
                };
                if (edge) weigh(std::true_type());
                else weigh(std::false_type());
                l += l2.x + l2.y;
                tc::wait_st();
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(pfull);
            fresh = false;
            if (last || j + 1 == steps) {
                // ---------------- the unit's output, or this block's part of it
                if (!wait(odone, j)) break;
                tc::fence_after_sync();
                if (live) {
                    const bool whole = last && j >= at.tile;  // the block saw the unit from its first tile on
                    const float rl = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
                    const int64_t out_row = ((int64_t)at.b * a.T + min(grow, R - 1) / a.G) * a.Hq + hk * a.G + min(grow, R - 1) % a.G;
                    float *slot = AttnSlot<ROWS, D>::at(a.ws, blockIdx.x, which);
#pragma unroll
                    for (int h = 0; h < D / 32; ++h) {
                        uint32_t o[32];
                        tc::ld_32x32b_x32(lane_base + C::OCOL + h * 32, o);
                        tc::wait_ld();
                        if (grow < R) {
                            if (whole) {
                                uint4 *dst = reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + out_row * D + h * 32);
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    uint32_t w[4];
#pragma unroll
                                    for (int i = 0; i < 4; ++i)
                                        w[i] = pack2(T(), __uint_as_float(o[8 * k + 2 * i]) * rl, __uint_as_float(o[8 * k + 2 * i + 1]) * rl);
                                    dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
                                }
                            } else {
                                uint4 *dst = reinterpret_cast<uint4 *>(slot + row * D + h * 32);
#pragma unroll
                                for (int k = 0; k < 8; ++k) dst[k] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                            }
                        }
                    }
                    if (grow < R) {
                        // l counts in units of 2^(kAttnUp - ve), and so does O
                        if (whole) {
                            if (a.lse) a.lse[out_row] = l == 0.f ? -INFINITY : (m - kAttnUp + (float)ve + log2f(l)) * kLn2;
                        } else {
                            slot[ROWS * D + row] = m - kAttnUp + (float)ve;
                            slot[ROWS * (D + 1) + row] = l;
                        }
                    }
                }
                tc::fence_before_sync();
                which = 1;
                fresh = true;
                parity ^= 1;
            }
            if (j + 1 < steps) at.template next<KT>(a, units);
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 8) {
        tc::fence_after_sync();
        if (*abort_flag && lane == 0) {  // products may still be running: wait for them before TMEM goes
            tc::commit(fin);
            mbar_wait_bounded(fin, 0);
        }
        __syncwarp();
        tc::tmem_dealloc(tmem, C::COLS);
    }
}

template <int FMT, bool BF, int D>
cudaError_t launch_tile_d(const AttnArgs &a, int sms, cudaStream_t st) {
    using C = AttnTileCfg<FMT, D>;
    static const cudaError_t attr =
        cudaFuncSetAttribute(attn_tile_kernel<FMT, BF, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::REQ);
    if (attr != cudaSuccess) return attr;
    const int nc = sms * 2, rtiles = (a.T * a.G + kTileRows - 1) / kTileRows;
    attn_tile_kernel<FMT, BF, D><<<nc, kTileThreads, C::REQ, st>>>(a, rtiles);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_join<BF, kTileKeys, kTileRows, D, false>(a, rtiles, nc, st);
}

template <int FMT>
cudaError_t launch_tile(const AttnArgs &a, bool bf, int sms, cudaStream_t st) {
    if (a.c.D == 128) return bf ? launch_tile_d<FMT, true, 128>(a, sms, st) : launch_tile_d<FMT, false, 128>(a, sms, st);
    return bf ? launch_tile_d<FMT, true, 64>(a, sms, st) : launch_tile_d<FMT, false, 64>(a, sms, st);
}

}  // namespace

}  // namespace tl
