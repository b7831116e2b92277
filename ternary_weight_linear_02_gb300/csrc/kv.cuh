// kv.cuh -- the codes of the quantised cache as fp32 or f16 values.
//
//   TL_KV_INT8: two's complement bytes; TL_KV_FP8: e4m3; TL_KV_INT4: two per byte,
//   field value + 8, the even element in the low bits.
// Every code is exact in f16 (8 bits of an int8, 4 of an e4m3 with its exponent
// range), so products of f16 values of codes are exact in fp32.
#pragma once

#include "common.cuh"

namespace tl {

enum { kKvInt8 = 0, kKvFp8 = 1, kKvInt4 = 2 };

template <int FMT>
struct KvCode {
    static constexpr int bits = FMT == kKvInt4 ? 4 : 8;
    static constexpr float qmax = FMT == kKvInt8 ? 127.f : FMT == kKvFp8 ? 448.f : 7.f;
};

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<const uint32_t *>(&h); }
__device__ __forceinline__ __half2 h2_of(uint32_t w) { return *reinterpret_cast<const __half2 *>(&w); }

// two e4m3 bytes (the low 16 bits of w) as f16x2; the two NaN patterns, which no append writes
// but a caller or an unwritten page may hold, stay NaN
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
        : "=r"(r)
        : "r"(w));
    return r;
}

// Four e4m3 bytes with the NaN patterns turned into the largest value, for values that some rows
// of a block do not see: with a weight of 0 they contribute 0.  found: not 0 after any.
__device__ __forceinline__ uint32_t e4m3_finite(uint32_t w, uint32_t &found) {
    const uint32_t n = ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
    found |= n;
    return w ^ (n >> 7);
}

// Two int8 bytes already moved to the low byte of each half and offset by 128
// (b ^ 0x80), under the byte 0x64: the f16 value 1024 + 128 + q, less 1152.
__device__ __forceinline__ uint32_t int8_f16x2(uint32_t halves) {
    return h2_bits(__hsub2(h2_of(halves), __float2half2_rn(1152.f)));
}

// 16 codes, in order, as 8 f16x2 registers.  w: 16 bytes of 8-bit codes, or (INT4) 8
// bytes in w[0], w[1].
template <int FMT>
__device__ __forceinline__ void codes16_f16(const uint32_t *w, uint32_t (&r)[8]) {
    if constexpr (FMT == kKvInt8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t u = w[i] ^ 0x80808080u;
            r[2 * i] = int8_f16x2(__byte_perm(u, 0x64646464u, 0x4140));
            r[2 * i + 1] = int8_f16x2(__byte_perm(u, 0x64646464u, 0x4342));
        }
    } else if constexpr (FMT == kKvFp8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r[2 * i] = e4m3x2_f16x2(w[i]);
            r[2 * i + 1] = e4m3x2_f16x2(w[i] >> 16);
        }
    } else {
        // byte b holds elements (2b, 2b + 1): spread byte b to both halves, keep the low
        // field of the one and the high field (16 times its value) of the other
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t b = (w[i >> 2] >> (8 * (i & 3))) & 0xFFu;
            const uint32_t x = (b & 0xFu) | ((b >> 4) << 16) | 0x64006400u;
            r[i] = h2_bits(__hsub2(h2_of(x), __float2half2_rn(1032.f)));
        }
    }
}

// Fields of 4 bits at bits 0-3 / 4-7 of each half, as f16x2 of field - 8.
__device__ __forceinline__ uint32_t int4_lo(uint32_t x) {
    return h2_bits(__hsub2(h2_of((x & 0x000F000Fu) | 0x64006400u), __float2half2_rn(1032.f)));
}
__device__ __forceinline__ uint32_t int4_hi(uint32_t x) {  // 1024 + 16 u
    return h2_bits(__hfma2(h2_of((x & 0x00F000F0u) | 0x64006400u), __float2half2_rn(0.0625f), __float2half2_rn(-72.f)));
}

// The order in which codes16_mma gives the elements of each 8: the registers' pairs are
// (0,1) (2,3) (4,5) (6,7), or for INT4 (0,4) (1,5) (2,6) (3,7), which takes 9 instructions per
// word instead of 20.  element(i): the element at place i.
template <int FMT>
__host__ __device__ constexpr int mma_element(int i) {
    return FMT == kKvInt4 ? (i & ~7) + ((i & 7) >> 1) + (i & 1) * 4 : i;
}
template <int FMT>
__device__ __forceinline__ void codes16_mma(const uint32_t *w, uint32_t (&r)[8]) {
    if constexpr (FMT == kKvInt4) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            r[4 * i] = int4_lo(w[i]);
            r[4 * i + 1] = int4_hi(w[i]);
            r[4 * i + 2] = int4_lo(w[i] >> 8);
            r[4 * i + 3] = int4_hi(w[i] >> 8);
        }
    } else {
        codes16_f16<FMT>(w, r);
    }
}
// 8 16-bit values (4 words) in that order
template <int FMT>
__device__ __forceinline__ uint4 mma_order(uint4 h) {
    if constexpr (FMT == kKvInt4)
        return make_uint4(__byte_perm(h.x, h.z, 0x5410), __byte_perm(h.x, h.z, 0x7632), __byte_perm(h.y, h.w, 0x5410),
                          __byte_perm(h.y, h.w, 0x7632));
    return h;
}

// The same 16 codes as fp32.
template <int FMT>
__device__ __forceinline__ void codes16_f32(const uint32_t *w, float (&v)[16]) {
    uint32_t r[8];
    codes16_f16<FMT>(w, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = __half22float2(h2_of(r[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

}  // namespace tl
