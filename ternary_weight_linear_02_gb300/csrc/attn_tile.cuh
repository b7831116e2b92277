// attn_tile.cuh -- attention for many rows per kv head (drafted trees, chunks of a prompt)
// on the 5th-generation tensor cores.
//
//   S = Q K^T, P = exp2(S sk f - r) sv, O += P V    (f = scale log2 e)
//
// A block owns 128 rows of one (sequence, kv head) -- TMEM lanes, one softmax thread
// each -- and walks tiles of 64 keys; two blocks per SM.
//  * Warp 4 copies: a tile's codes and scales land in shared memory as they lie in the cache
//    (bulk copies of 16 keys of one page), keys three tiles ahead and values two.  It
//    also issues tcgen05.mma (kind::f16, fp32 in TMEM): S = Q K^T from shared memory into
//    one of two buffers, so that the scores of the next tile are computed during the
//    softmax of this one, and O += P V with P from TMEM.
//  * Warps 5-7 decode codes to f16 (exact) in 128-byte-swizzled rows, keys and values alike:
//    keys are read as a K-major operand, values as an MN-major one, so neither is
//    transposed.  They also place the queries at a unit's start (f16; bf16 scaled by a power
//    of two per row, QueryScale in attn_sched.cuh).  Codes that came through registers
//    instead, a tile ahead, were waited for with every other load of their warp
//    (page table, scales): 5000 cycles a tile against 3500.
//  * Warps 0-3: a row's 64 scores are read in halves, for the maximum and then for the
//    weights; P (f16) overwrites the first half of them in TMEM.  The weights hold the
//    value scale, so far up that products down to 2^-24 of the row's largest keep all 11 bits
//    (kAttnRoom in attn_sched.cuh).  A row's reference moves only when exceeded by a factor of
//    4, and then a factor of 8 beyond: then O is rescaled in TMEM.  The largest score and the
//    largest value scale together bound a tile's products; only where that bound exceeds the
//    reference and the scales that the row sees lie far apart is the largest product looked for.
// Measured: 8 trees of 64 over 16384 keys, 28 query heads on 4, fp8: 204 us, 428
// TFLOP/s of both products; 6 trees of 23, 32 heads, up to 4099 keys, int4: 75 us.
// Bound by the instruction streams of the three kinds of warps: 44 % of the issue slots are
// used, the tensor pipe 22 %, and the stalls are waits for loads and for results.  Short code
// without spills matters (39 %, and waits for instructions, before it): loops over the halves of a tile and one decoder for keys and values took
// these two cases from 255 and 85 us, a rolled loop for the rescaling the first in int4 from
// 217 to 197.  Two more warps (ten, one for the copies and four decoders) decoded in half
// the time but slowed the softmax by more.
// Softmax warps without a row that decode too (23 rows: three more) were slower: 99 us
// against 90 (fp8).
// Every mbarrier wait is bounded and answered alike in all lanes of a warp; one that gives up
// sets the device status word, and the block stops issuing work, lets its copies and products
// in flight end, makes the partial results it owes NaN, frees its TMEM and returns.
#pragma once

#include <cfloat>
#include <climits>

#include "attn_sched.cuh"
#include "kv.cuh"
#include "rope.cuh"
#include "tc.cuh"

namespace tl {

namespace {

using TileTiling = AttnTiling<64, 4>;  // (a unit costs about four tiles beside its own)
constexpr int kTileKeys = TileTiling::KT, kTileRows = 128, kTileThreads = 256;

template <int FMT, int D>
struct AttnTileCfg {
    static constexpr int HALVES = D / 64;                 // 64-element (128-byte) column blocks
    static constexpr int QBLOCK = 128 * 128, KBLOCK = kTileKeys * 128;  // bytes of one: rows of 128 B
    static constexpr int UB = 16 * KvCode<FMT>::bits / 8; // bytes of 16 codes
    static constexpr int RB = D / 16 * UB;                // bytes per row of codes
    static constexpr int LANES = D / 16;                  // threads per row
    // A pass is one load and store of a warp: RPP rows; the three decoder warps take turns.
    static constexpr int RPP = 32 / LANES, PASSES = kTileKeys / RPP, MANY = (PASSES + 2) / 3;
    static constexpr uint32_t SCOL = 0, OCOL = 128, COLS = 256;  // S: two buffers of 64 columns
    static constexpr int TILE = HALVES * KBLOCK;          // keys or values of a tile as f16
    static constexpr int QOFF = 0, KOFF = HALVES * QBLOCK, VOFF = KOFF + TILE;
    // codes as they lie in the cache: two stages of keys, two of values; scales of four tiles
    static constexpr int CODES = kTileKeys * RB, CKOFF = VOFF + TILE, CVOFF = CKOFF + 2 * CODES;
    static constexpr int SKOFF = CVOFF + 2 * CODES, SVOFF = SKOFF + 4 * kTileKeys * 4;
    static constexpr int SXOFF = SVOFF + 4 * kTileKeys * 4;  // sizes of the value scales, as them
    static constexpr int SMOFF = SXOFF + 4 * kTileKeys * 4;  // largest, smallest of committed keys [4]
    static constexpr int NOFF = SMOFF + 32;               // units with NaN codes among new values [4]
    static constexpr int FOFF = NOFF + 16;                // row factors [4][128]
    static constexpr int BOFF = FOFF + 4 * 512;           // barriers, TMEM slot, abort flag
    static constexpr int POFF = BOFF + 128;               // place of the run (10 words)
    static constexpr int SMEM = POFF + 80 + 1024;         // 1 KB of alignment slack
    // no more blocks per SM than its 512 TMEM columns serve
    static constexpr int REQ = SMEM > 80 * 1024 ? SMEM : 80 * 1024;
    static_assert(2 * (REQ + 1024) <= 228 * 1024 && 3 * (REQ + 1024) > 228 * 1024, "two blocks per SM");
};

__device__ __forceinline__ void sts_v4(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void lds(uint32_t at, uint32_t (&w)[4]) {
    if constexpr (BYTES == 16)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
    else
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at) : "memory");
}
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

// The largest product of a row (a lane's scores of one tile at scol) over 2^base, in powers of two.
__device__ __forceinline__ float largest_product(uint32_t scol, const float *sk, const float *sx, float f, uint32_t see0, uint32_t see1, float base) {
    float top = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < kTileKeys; c += 16) {
        uint32_t s[16];
        tc::ld_32x32b_x16(scol + c, s);
        tc::wait_ld();
        const uint32_t see = (c & 32 ? see1 : see0) >> (c & 16);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float y = fmaf(__uint_as_float(s[k]) * sk[c + k], f, -base) + sx[c + k];
            top = fmaxf(top, see >> k & 1u ? y : -INFINITY);
        }
    }
    return top;
}
// The reference of a row after a tile from its largest product.  By a whole warp.  Rarely called, and
// not inlined: in place its code made every tile dearer.
__device__ __noinline__ float exact_reference(uint32_t scol, const float *sk, const float *sx, float f, uint32_t see0, uint32_t see1, float ref) {
    const float y = largest_product(scol, sk, sx, f, see0, see1, 0.f);
    float rn = attn_above(y) - ref > kAttnFull ? fmaxf(y - kAttnRoom, ref) : ref;
    if (__any_sync(0xffffffffu, fabsf(y) > kAttnCoarse)) {
        const float left = largest_product(scol, sk, sx, f, see0, see1, rn);
        if (left > kAttnFull) rn = __fadd_ru(rn, left - kAttnRoom);
    }
    return rn;
}

// The rest of a wait that has not succeeded at once, by a whole warp: all lanes see the phase
// complete, or all give up (a warp may not part before its tcgen05 instructions).
__device__ __noinline__ bool wait_or_give_up(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int *status, long long limit) {
    const long long t0 = clock64();
    for (;;) {
        if (__all_sync(0xffffffffu, mbar_try_wait_sleep(bar, parity, 200u))) return true;
        if (__any_sync(0xffffffffu, *abort_flag || clock64() - t0 > limit)) break;
    }
    *abort_flag = 1;
    if (status && (threadIdx.x & 31) == 0) atomicExch(status, kStatusTimeout);
    return false;
}

// Makes the e4m3 codes finite that a thread decodes of a tile's staged values (16 bytes at `codes`
// of row r0 and every STEP-th after it), from row `held` on: the new tokens' and what lies beyond.
// Whether a new token's held a NaN.  Not inlined: it is for the last tiles of a unit alone.
template <int STEP, int RB>
__device__ __noinline__ bool finite_rows(uint8_t *codes, int r0, int held, int T) {
    uint32_t nans = 0;
    for (int r = r0; r < kTileKeys; r += STEP, codes += STEP * RB) {
        if (r < held) continue;
        uint4 *const p = reinterpret_cast<uint4 *>(codes);
        uint4 w = *p;
        uint32_t met = 0;
        w.x = e4m3_finite(w.x, met), w.y = e4m3_finite(w.y, met), w.z = e4m3_finite(w.z, met), w.w = e4m3_finite(w.w, met);
        if (met) *p = w;
        if (r - held < T) nans |= met;
    }
    return nans != 0;
}

template <int FMT, int D>
__global__ void __launch_bounds__(kTileThreads, 2) attn_tile_kernel(AttnArgs a, int rtiles) {
    using C = AttnTileCfg<FMT, D>;
    using TL = TileTiling;
    constexpr int KT = TL::KT, ROWS = kTileRows;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    // tile j: number j & 1 in phase j >> 1 of the pairs, phase j of the single ones
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::BOFF);
    uint64_t *ckfull = bars, *cvfull = bars + 2, *sdone = bars + 4, *pfull = bars + 6, *odone = bars + 8;
    uint64_t *kfull = bars + 10, *vfull = bars + 11;
    uint64_t *fin = bars + 12;  // after a give-up: every product issued has ended
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 13);
    uint64_t *never = bars + 14;  // nothing arrives on it (testing aid)
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int R = a.T * a.G;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(ckfull + i, 1);  // the copies' bytes
            mbar_init(cvfull + i, 1);
            mbar_init(sdone + i, 1);
            mbar_init(pfull + i, 4);  // one arrival per softmax warp
            mbar_init(odone + i, 1);
        }
        mbar_init(kfull, 3);  // one per decoder warp
        mbar_init(vfull, 3);
        mbar_init(fin, 1);
        mbar_init(never, 1);
        *abort_flag = 0;
        *reinterpret_cast<int4 *>(smem + C::NOFF) = make_int4(0, 0, 0, 0);
        fence_barrier_init();
    }
    AttnWalk at;
    if (!at.template start_block<TL, kTileThreads>(a, rtiles, reinterpret_cast<int64_t *>(smem + C::POFF))) return;
    if (warp == 4) tc::tmem_alloc(tmem_slot, C::COLS);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    // Dependents may start once every block of this grid holds its TMEM (or has left for want
    // of a run): a linear layer that follows the direct form allocates columns of its own before
    // it waits for this grid, and a block that found none left would wait for it in turn.
    pdl_launch_dependents();

    auto wait_phase = [&](uint64_t *bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || wait_or_give_up(bar, parity, abort_flag, a.status, a.wait_limit);
    };
    auto wait = [&](uint64_t *pair, int j) -> bool { return wait_phase(pair + (j & 1), (uint32_t)(j >> 1) & 1u); };
    auto wait1 = [&](uint64_t *bar, int j) -> bool { return wait_phase(bar, (uint32_t)j & 1u); };

    if (warp == 4) {
        // ---------------- copies and products: the whole warp walks; lane i of the first four
        // copies group i of 16 keys, and one lane issues the products, so that descriptors
        // stay in uniform registers
        constexpr uint32_t idesc_s = tc::idesc_f16(KT, false);
        constexpr uint32_t idesc_o = tc::idesc_f16(D, false) | tc::kIdescBTransposed;
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        AttnWalk ahead = at;  // the tile that is copied next; its page is fetched a tile before
        AttnPages where;
        where.start(a, ahead, ahead.tile * KT + (lane & 3) * 16);
        int page = where.fetch(a, ahead.b);
        uint32_t group = 0, group1 = 0;  // of the tile whose keys were copied last, and of the one before
        int groups = 0, groups1 = 0;     // (none: 0)
        bool one = false, one1 = false;  // whole, within one page: one copy (each takes the warp about 70 cycles)
        constexpr uint32_t codes = 16 * C::RB;
        auto copy_keys = [&](int j) {  // and both sides' scales
            group1 = group;
            groups1 = groups;
            one1 = one;
            groups = 0;
            one = false;
            if (!ahead.inside()) return;
            groups = min(KT / 16, (ahead.ctx + a.T - ahead.tile * KT + 15) >> 4);
            group = attn_group(a, page, ahead.hk, where.off);
            one = groups == KT / 16 && __shfl_sync(0xffffffffu, where.off, 0) + KT <= a.c.P;
            uint64_t *bar = ckfull + (j & 1);
            if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)groups * (codes + 128));
            __syncwarp();
            if (lane < (one ? 1 : groups)) {
                const int64_t row = (int64_t)group << 4;
                const uint32_t n = one ? KT / 16 : 1;
                bulk_g2s(smem + C::CKOFF + (j & 1) * C::CODES + lane * codes, a.c.kc + row * C::RB, n * codes, bar);
                bulk_g2s(smem + C::SKOFF + (j & 3) * KT * 4 + lane * 64, a.c.ks + row, n * 64, bar);
                bulk_g2s(smem + C::SVOFF + (j & 3) * KT * 4 + lane * 64, a.c.vs + row, n * 64, bar);
            }
            __syncwarp();
            const bool start = ahead.template next<TL>(a, rtiles);
            if (!ahead.inside()) return;
            if (start) where.start(a, ahead, (lane & 3) * 16);
            else where.next(a, KT);
            page = where.fetch(a, ahead.b);
        };
        auto copy_values = [&](int j, uint32_t grp, int n, bool single) {
            if (n == 0) return;
            uint64_t *bar = cvfull + (j & 1);
            if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)n * codes);
            __syncwarp();
            if (lane < (single ? 1 : n))
                bulk_g2s(smem + C::CVOFF + (j & 1) * C::CODES + lane * codes, a.c.vc + ((int64_t)grp << 4) * C::RB,
                         single ? (uint32_t)C::CODES : codes, bar);
            __syncwarp();
        };
        auto scores = [&](int j) -> bool {
            // S buffer j & 1 holds P of tile j - 2: its product has to be done
            if ((j > 1 && !wait(odone, j - 2)) || !wait1(kfull, j)) return false;
            tc::fence_after_sync();
            const uint64_t qd = tc::desc_sw128(smem + C::QOFF), kd = tc::desc_sw128(smem + C::KOFF);
            const uint32_t d = tm + C::SCOL + (uint32_t)(j & 1) * KT;
            if (tc::elect_one()) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    tc::mma_ss(d, qd + (uint64_t)((k >> 2) * (C::QBLOCK >> 4) + (k & 3) * 2),
                               kd + (uint64_t)((k >> 2) * (C::KBLOCK >> 4) + (k & 3) * 2), idesc_s, k > 0);
                tc::commit(sdone + (j & 1));
            }
            __syncwarp();
            return true;
        };
        auto values = [&](int j, bool first) -> bool {
            if (!wait(pfull, j) || !wait1(vfull, j)) return false;
            tc::fence_after_sync();
            const uint64_t vd = tc::desc_sw128_mn(smem + C::VOFF, C::KBLOCK);
            const uint32_t p = tm + C::SCOL + (uint32_t)(j & 1) * KT;
            if (tc::elect_one()) {
#pragma unroll
                for (int k = 0; k < KT / 16; ++k)
                    tc::mma_ts(tm + C::OCOL, p + k * 8, vd + (uint64_t)(k * 128), idesc_o, !first || k > 0);
                tc::commit(odone + (j & 1));
            }
            __syncwarp();
            return true;
        };
        copy_keys(0);
        copy_values(0, group, groups, one);
        copy_keys(1);
        copy_values(1, group, groups, one);
        bool fresh = true;  // the tile begins a unit (for this block)
        bool ok = scores(0);
        if (ok) copy_keys(2);
        int j = 0;
#pragma unroll 1
        for (; ok && at.inside(); ++j) {
            // The next tile's scores, computed during this one's softmax.  Free since then: the
            // stage of the last tile's values (vfull, in values), of the next tile's keys
            // (kfull, in scores), and the scales of the last tile (odone, in scores).
            if (at.template more<TL>()) ok = scores(j + 1);
            if (ok && j > 0) copy_values(j + 1, group1, groups1, one1);
            if (ok) copy_keys(j + 3);
            ok = ok && values(j, fresh);
            fresh = at.last_of_unit();
            at.template next<TL>(a, rtiles);
        }
        if (!ok) {  // given up: the copies in flight still land before the block ends
            for (int i = j; i < j + 4; ++i) {
                mbar_wait_bounded(ckfull + (i & 1), (uint32_t)(i >> 1) & 1u, 1ll << 22);
                mbar_wait_bounded(cvfull + (i & 1), (uint32_t)(i >> 1) & 1u, 1ll << 22);
            }
        }
    } else if (warp >= 5) {
        // ---------------- decoders
        const int dw = warp - 5;
        // LANES threads per row of codes; the store order keeps each 8 lanes' 16-byte
        // chunks in different banks
        const int cu = C::LANES == 8 ? (lane & 3) + 4 * (lane >> 4) : lane & 3;
        const int rin = C::LANES == 8 ? (lane >> 2) & 3 : lane >> 2;  // row within a pass
        // Passes turn, turn + 3 .. of a tile.  A row's 16-byte chunk c lies at c ^ (row & 7): with
        // four rows to a pass every second pass flips bit 2 of the row (and of the chunk),
        // with eight all passes agree.
        const uint32_t smem0 = smem_u32(smem);
        auto decode = [&](int turn, uint32_t from, uint32_t to) {
            const int r0 = turn * C::RPP + rin;
            const uint32_t src = smem0 + from + (uint32_t)(r0 * C::RB + cu * C::UB);
            const uint32_t dst = smem0 + to + (uint32_t)((cu >> 2) * C::KBLOCK + r0 * 128);
            const uint32_t ch0 = (uint32_t)((2 * (cu & 3)) ^ (r0 & 7)) << 4;
            uint32_t w[C::MANY][4];
#pragma unroll
            for (int i = 0; i < C::MANY; ++i)
                if (turn + 3 * i < C::PASSES) lds<C::UB>(src + i * 3 * C::RPP * C::RB, w[i]);
#pragma unroll
            for (int i = 0; i < C::MANY; ++i) {
                if (turn + 3 * i >= C::PASSES) break;
                uint32_t h[8];
                codes16_mma<FMT>(w[i], h);
                const uint32_t ch = C::RPP == 4 && (i & 1) ? ch0 ^ 64u : ch0;
                sts_v4(dst + i * 3 * C::RPP * 128 + ch, h[0], h[1], h[2], h[3]);
                sts_v4(dst + i * 3 * C::RPP * 128 + (ch ^ 16u), h[4], h[5], h[6], h[7]);
            }
        };
        // The unit's rows as f16, D / 8 lanes per row; rows beyond the last repeat it or are left
        // as they are (a row only ever meets its own scores and outputs).
        auto queries = [&](const AttnWalk &w, int buf) {
            constexpr int QL = D / 8, QR = 32 / QL;  // lanes per row, rows per pass
            const int c = lane % QL, r1 = min(ROWS, R - w.rt * ROWS);
            float *fac = reinterpret_cast<float *>(smem + C::FOFF) + buf * 128;
#pragma unroll 1
            for (int n0 = dw * 8 * QR; n0 < r1; n0 += 24 * QR) {  // eight passes at a time
                uint4 raw[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int g = min(w.rt * ROWS + n0 + i * QR + lane / QL, R - 1), tok = g / a.G;
                    const uint16_t *q = static_cast<const uint16_t *>(a.q) + w.b * a.qb + (int64_t)tok * a.qt +
                                 (int64_t)(w.hk * a.G + g - tok * a.G) * a.qh + c * 8;
                    if (a.q_vec) {
                        raw[i] = __ldg(reinterpret_cast<const uint4 *>(q));
                    } else {
                        const uint16_t *u = q;
                        raw[i] = make_uint4(u[0] | (uint32_t)u[1] << 16, u[2] | (uint32_t)u[3] << 16,
                                            u[4] | (uint32_t)u[5] << 16, u[6] | (uint32_t)u[7] << 16);
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = n0 + i * QR + lane / QL;
                    uint4 h = raw[i];
                    float up = 1.f;
                    if (a.bf) {
                        const uint32_t x[4] = {h.x, h.y, h.z, h.w};
                        // bf16 magnitudes compare as their bits
                        uint32_t mx = 0;
#pragma unroll
                        for (int k = 0; k < 4; ++k) mx = max(mx, max(x[k] & 0x7FFFu, (x[k] >> 16) & 0x7FFFu));
                        mx = __reduce_max_sync(((1u << QL) - 1u) << (lane & ~(QL - 1)), mx);  // the row's lanes
                        const QueryScale by(mx >> 7);
                        const float down = by.down;
                        up = by.up;
                        uint32_t y[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 f = unpack2(__nv_bfloat16(), x[k]);
                            y[k] = pack2(__half(), f.x * down, f.y * down);
                        }
                        h = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                    h = mma_order<FMT>(h);
                    *reinterpret_cast<uint4 *>(smem + C::QOFF + (c >> 3) * C::QBLOCK + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = h;
                    if (c == 0) fac[r] = fmaxf(a.scale * kLog2e * up, FLT_MIN);  // (0 would meet infinities)
                }
            }
        };
        auto publish = [&](uint64_t *bar) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };

        int unit = 0;         // row factors' buffer
        // Turns of a tile's keys and the values of the tile before, so that the scores are computed
        // first; one copy of the code serves both.
        bool fresh = true;  // `at` begins a unit
        int held = 0, held1 = 0, unit1 = 0;  // committed keys of the keys' tile, and of the values'; the latter's unit
#pragma unroll 1
        for (int i = 0, last = INT_MAX;; ++i) {
            const int j = (i >> 1) - (i & 1);  // keys of tiles 0 1 2 .., values of tiles -1 0 1 ..
            const bool vals = i & 1;
            if (vals) {
                if (j < 0) continue;
            } else {
                held1 = held;
                unit1 = unit;
                if (j > last) continue;
                held = at.ctx - at.tile * KT;
            }
            uint64_t *const from = vals ? cvfull : ckfull, *const gone = vals ? odone : sdone;
            // the codes have landed, and what was made of the tile before has been read
            if (!wait(from, j) || (j > 0 && !wait(gone, j - 1))) break;
            if (!vals && fresh) queries(at, unit++ & 3);  // (and the last unit's queries)
            if (!vals && dw == 2) {  // (the warp with the fewest passes) value scales: sizes, and unbiased
                const int k = at.tile * KT + lane * 2;
                float2 *const v = reinterpret_cast<float2 *>(smem + C::SVOFF + (j & 3) * KT * 4 + lane * 8);
                const float2 w = *v, x = make_float2(attn_size(w.x), attn_size(w.y));
                *v = make_float2(w.x * kAttnUnbias, w.y * kAttnUnbias);
                *reinterpret_cast<float2 *>(smem + C::SXOFF + (j & 3) * KT * 4 + lane * 8) = x;
                // from kAttnSmall on, where they compare as their bits
                const uint32_t b0 = __float_as_uint(x.x - kAttnSmall), b1 = __float_as_uint(x.y - kAttnSmall), most = __float_as_uint(128.f - kAttnSmall);
                const int n = at.ctx - k;
                const uint32_t mx = __reduce_max_sync(0xffffffffu, max(n > 0 ? b0 : 0u, n > 1 ? b1 : 0u));
                const uint32_t mn = __reduce_min_sync(0xffffffffu, min(n > 0 ? b0 : most, n > 1 ? b1 : most));
                if (lane == 0)
                    reinterpret_cast<float2 *>(smem + C::SMOFF)[j & 3] = make_float2(__uint_as_float(mx) + kAttnSmall, __uint_as_float(mn) + kAttnSmall);
            }
            const int turn = vals ? 2 - dw : dw;
            if (FMT == kKvFp8 && vals && held1 < KT) {  // new tokens' values
                const int r0 = turn * C::RPP + rin;
                if (finite_rows<3 * C::RPP, C::RB>(smem + C::CVOFF + (j & 1) * C::CODES + r0 * C::RB + cu * C::UB, r0, held1, a.T))
                    reinterpret_cast<volatile int *>(smem + C::NOFF)[unit1 & 3] = unit1;  // (counted from 1 here)
            }
            decode(turn, (vals ? C::CVOFF : C::CKOFF) + (j & 1) * C::CODES, vals ? C::VOFF : C::KOFF);
            publish(vals ? vfull : kfull);
            if (vals) {
                if (j == last) break;
            } else if (at.template more<TL>()) {
                fresh = at.template next<TL>(a, rtiles);
            } else {
                last = j;
            }
        }
    } else {
        // ---------------- softmax: thread = row = TMEM lane
        const int row = threadIdx.x;
        const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
        float ref = kAttnLow, l = 0.f, f = 0.f;
        int unit = 0, which = 0;
        bool fresh = true, whole = true;      // whole: the block sees the unit from its first tile on
        if (a.stall && !wait_or_give_up(never, 0, abort_flag, a.status, a.wait_limit)) at.end = at.at;
#pragma unroll 1
        for (int j = 0; at.inside(); ++j) {
            const int grow = at.rt * ROWS + row;
            const bool live = at.rt * ROWS + warp * 32 < R;  // the warp has rows
            const bool last = at.last_of_unit();
            const uint32_t scol = lane_base + C::SCOL + (uint32_t)(j & 1) * KT;
            if (!wait(sdone, j)) break;
            tc::fence_after_sync();
            if (live) {
                if (fresh) {
                    whole = at.tile == 0;
                    f = grow < R ? reinterpret_cast<const float *>(smem + C::FOFF)[(unit & 3) * 128 + row] : 0.f;
                    ref = kAttnLow;
                    l = 0.f;
                }
                const float4 *sk = reinterpret_cast<const float4 *>(smem + C::SKOFF + (j & 3) * KT * 4);
                const float4 *sv = reinterpret_cast<const float4 *>(smem + C::SVOFF + (j & 3) * KT * 4);
                const float4 *sx = reinterpret_cast<const float4 *>(smem + C::SXOFF + (j & 3) * KT * 4);
                float2 size = reinterpret_cast<const float2 *>(smem + C::SMOFF)[j & 3];  // the largest and the smallest that the row sees
                uint32_t see0 = ~0u, see1 = ~0u;
                const bool edge = at.tile * KT + KT > at.ctx;  // new tokens' keys, or the end
                if (edge) {
                    const int tok = min(grow, R - 1) / a.G;
                    const uint8_t *tree = a.tree ? a.tree + at.b * a.tree_b + (int64_t)tok * a.tree_r : nullptr;
                    const float *sizes = reinterpret_cast<const float *>(sx);
#pragma unroll 1
                    for (int c = 0; c < 2; ++c) {
                        const int i0 = at.tile * KT + 32 * c - at.ctx;  // index of the new token at the chunk's start
                        if (i0 + 32 <= 0) continue;
                        uint32_t bits = 0;
#pragma unroll 4
                        for (int k = 0; k < 32; ++k) {
                            const int i = i0 + k;
                            bool u = i < 0;
                            if (i >= 0 && i < a.T) u = tree ? tree[i] != 0 : i <= tok;
                            if (u) {
                                bits |= 1u << k;
                                size = make_float2(fmaxf(size.x, sizes[32 * c + k]), fminf(size.y, sizes[32 * c + k]));
                            }
                        }
                        if (c) see1 = bits;
                        else see0 = bits;
                    }
                }
                // ---- scores of half a tile, times the key scales.  The second half is read twice and the
                // halves share their code: all 64 held at once spilled, and the longer code cost more.
                uint32_t s[32];
                auto half = [&](int c) {
                    tc::ld_32x32b_x32(scol + 32 * c, s);
                    tc::wait_ld();
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        const float4 w = sk[c * 8 + k / 4];
                        const float2 x = mul2(make_float2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), make_float2(w.x, w.y));
                        const float2 y = mul2(make_float2(__uint_as_float(s[k + 2]), __uint_as_float(s[k + 3])), make_float2(w.z, w.w));
                        s[k] = __float_as_uint(x.x), s[k + 1] = __float_as_uint(x.y);
                        s[k + 2] = __float_as_uint(y.x), s[k + 3] = __float_as_uint(y.y);
                    }
                    if (edge) {
                        const uint32_t see = c ? see1 : see0;
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (!(see >> k & 1u)) s[k] = 0xFF800000u;  // -infinity
                    }
                };
                float top = -INFINITY;
#pragma unroll 1
                for (int c = 1; c >= 0; --c) {
                    half(c);
                    float tops[4] = {top, -INFINITY, -INFINITY, -INFINITY};  // four short chains
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        float &x = tops[(k >> 1) & 3];
                        x = fmaxf(fmaxf(x, __uint_as_float(s[k])), __uint_as_float(s[k + 1]));
                    }
                    top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                }
                // No product is larger than top and size say; z - r by the same operation as for the weights.
                if (__any_sync(0xffffffffu, grow < R && fmaf(top, f, -ref) + size.x > kAttnFull)) {
                    float rn = top * f + size.x - kAttnRoom;
                    const float left = fmaf(top, f, -rn) + size.x;
                    if (left > kAttnFull) rn = __fadd_ru(rn, left - kAttnRoom);
                    if (!(fmaf(top, f, -ref) + size.x > kAttnFull)) rn = ref;
                    const bool far = rn != ref && size.x - size.y > kAttnSpread;  // no product may be near the bound
                    if (__any_sync(0xffffffffu, grow < R && far)) {
                        const float y = exact_reference(scol, reinterpret_cast<const float *>(sk), reinterpret_cast<const float *>(sx), f, see0, see1, ref);
                        if (far) rn = y;
                    }
                    // in two steps: the sum may outlive a factor that fp32 cannot hold
                    const float h = ex2(.5f * (ref - rn)), c2 = h * h;
                    ref = rn;
                    l = l * h * h;
                    if (!fresh) {
                        if (!wait(odone, j - 1)) break;  // O holds every product so far
                        tc::fence_after_sync();
#pragma unroll 1
                        for (int h = 0; h < D / 16; ++h) {
                            uint32_t o[16];
                            tc::ld_32x32b_x16(lane_base + C::OCOL + h * 16, o);
                            tc::wait_ld();
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * c2);
                            tc::st_32x32b_x16(lane_base + C::OCOL + h * 16, o);
                        }
                    }
                }
                // ---- weights, over S's first columns
                const float off = -ref;
                const float2 f2 = make_float2(f, f), off2 = make_float2(off, off);
                float2 l2 = make_float2(0.f, 0.f), l3 = l2;
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    if (c) half(1);
                    uint32_t p[16];
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        const float4 v = sv[c * 8 + k / 4];
                        float2 x = fma2(make_float2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), f2, off2);
                        float2 y = fma2(make_float2(__uint_as_float(s[k + 2]), __uint_as_float(s[k + 3])), f2, off2);
                        x = make_float2(ex2(x.x), ex2(x.y));
                        y = make_float2(ex2(y.x), ex2(y.y));
                        l2 = add2(l2, x);
                        l3 = add2(l3, y);
                        x = mul2(x, make_float2(v.x, v.y));
                        y = mul2(y, make_float2(v.z, v.w));
                        p[k / 2] = pack2(__half(), x.x, x.y);
                        p[k / 2 + 1] = pack2(__half(), y.x, y.y);
                    }
                    if (edge) {  // an unseen scale may be a NaN
                        const uint32_t see = c ? see1 : see0;
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            if (!(see >> (2 * k) & 1u)) p[k] &= 0xFFFF0000u;
                            if (!(see >> (2 * k + 1) & 1u)) p[k] &= 0x0000FFFFu;
                        }
                    }
                    tc::st_32x32b_x16(scol + c * 16, p);
                }
                l += (l2.x + l2.y) + (l3.x + l3.y);
                tc::wait_st();
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(pfull + (j & 1));
            fresh = false;
            if (last || !at.template more<TL>()) {
                // ---------------- the unit's output, or this block's part of it
                if (!wait(odone, j)) break;
                tc::fence_after_sync();
                if (live) {
                    whole = whole && last;
                    // O lacks the bias that l counts
                    const float rl = whole ? (l == 0.f ? 0.f : kAttnRebias / l) : kAttnRebias;
                    const int g = min(grow, R - 1);
                    const int64_t out_row = ((int64_t)at.b * a.T + g / a.G) * a.Hq + at.hk * a.G + g % a.G;
                    float *slot = AttnSlot<ROWS, D>::at(a.ws, blockIdx.x, which);
#pragma unroll
                    for (int h = 0; h < D / 32; ++h) {
                        uint32_t x[32], o[32];
                        tc::ld_32x32b_x32(lane_base + C::OCOL + h * 32, x);
                        tc::wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[mma_element<FMT>(k)] = x[k];  // (registers renamed)
                        if (grow < R) {
                            if (whole) {
                                uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + out_row * D + h * 32);
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    uint32_t w[4];
#pragma unroll
                                    for (int i = 0; i < 4; ++i)
                                        w[i] = attn_pack(a, __uint_as_float(o[8 * k + 2 * i]) * rl, __uint_as_float(o[8 * k + 2 * i + 1]) * rl);
                                    dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
                                }
                            } else {
                                uint4 *dst = reinterpret_cast<uint4 *>(slot + row * D + h * 32);
#pragma unroll
                                for (int k = 0; k < 8; ++k) {
                                    uint32_t w[4];
#pragma unroll
                                    for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(__uint_as_float(o[4 * k + i]) * rl);
                                    dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
                                }
                            }
                        }
                    }
                    if (grow < R) {
                        if (FMT == kKvFp8 && reinterpret_cast<volatile int *>(smem + C::NOFF)[(unit + 1) & 3] == unit + 1)
                            attn_put_nans<D>(a, at, g / a.G, 0, D, whole ? static_cast<uint16_t *>(a.out) + out_row * D : nullptr, slot + row * D);
                        if (whole) {
                            if (a.lse) a.lse[out_row] = l == 0.f ? -INFINITY : (ref + log2f(l)) * kLn2;
                        } else {
                            slot[ROWS * D + row] = ref;
                            slot[ROWS * (D + 1) + row] = l;
                        }
                    }
                }
                tc::fence_before_sync();
                which = 1;
                fresh = true;
                ++unit;
            }
            at.template next<TL>(a, rtiles);
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 4) {
        tc::fence_after_sync();
        if (*abort_flag) {  // products may still be running: wait for them before TMEM goes
            if (tc::elect_one()) tc::commit(fin);
            __syncwarp();
            mbar_wait_bounded(fin, 0);
            if (!a.direct)
                for (int i = lane; i < 2 * ROWS; i += 32)
                    AttnSlot<ROWS, D>::at(a.ws, blockIdx.x, i / ROWS)[ROWS * (D + 1) + i % ROWS] = __uint_as_float(0x7FC00000u);
        }
        __syncwarp();
        tc::tmem_dealloc(tmem, C::COLS);
    }
}

template <int FMT, int D>
cudaError_t launch_tile_d(const AttnArgs &a, int sms, cudaStream_t st) {
    using C = AttnTileCfg<FMT, D>;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = attn_allow_smem(allowed, attn_tile_kernel<FMT, D>, C::REQ);
    if (e != cudaSuccess) return e;
    const int rtiles = (a.T * a.G + kTileRows - 1) / kTileRows, nc = a.direct ? a.B * a.c.Hk * rtiles : sms * 2;
    attn_tile_kernel<FMT, D><<<nc, kTileThreads, C::REQ, st>>>(a, rtiles);
    e = cudaGetLastError();
    if (e != cudaSuccess || a.direct) return e;
    return launch_join<TileTiling, kTileRows, D>(a, rtiles, nc, st);
}

template <int FMT>
cudaError_t launch_tile(const AttnArgs &a, int sms, cudaStream_t st) {
    return a.c.D == 128 ? launch_tile_d<FMT, 128>(a, sms, st) : launch_tile_d<FMT, 64>(a, sms, st);
}

}  // namespace

}  // namespace tl
