// rope.cuh -- the rotation shared by kern_rope.cu and kern_kv.cu, and 8-element
// loads and stores of the 16- and 32-bit types as fp32.
#pragma once

#include "common.cuh"

namespace tl {

__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }

__device__ __forceinline__ uint32_t pack2(__half, float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack2(__nv_bfloat16, float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack2(__half, uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
__device__ __forceinline__ float2 unpack2(__nv_bfloat16, uint32_t w) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w));
}

// 8 elements at a 16-byte aligned address
template <typename T>
__device__ __forceinline__ void ld8(const T *p, float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        const float4 x = *reinterpret_cast<const float4 *>(p), y = *reinterpret_cast<const float4 *>(p + 4);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
    } else {
        const uint4 w = *reinterpret_cast<const uint4 *>(p);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2(T(), u[i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}
template <typename T>
__device__ __forceinline__ void st8(T *p, const float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint4 w;
        w.x = pack2(T(), v[0], v[1]);
        w.y = pack2(T(), v[2], v[3]);
        w.z = pack2(T(), v[4], v[5]);
        w.w = pack2(T(), v[6], v[7]);
        *reinterpret_cast<uint4 *>(p) = w;
    }
}

// The turned pair.  Each product and each sum is rounded on its own (no fused
// multiply-add): a cache written from these values then holds the same codes as
// the formula evaluated operation by operation in fp32.
__device__ __forceinline__ float rope_a(float a, float b, float c, float s) {
    return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
}
__device__ __forceinline__ float rope_b(float a, float b, float c, float s) {
    return __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

// Column group c of a head, two runs of 8 elements at a and b.  Rotated groups
// (c < R/16) hold 8 whole pairs: half layout, the runs 8c of either half;
// interleaved, 16 neighbours.  The groups after them hold 16 neighbours beyond R.
template <bool INTER>
struct RopeCols {
    int a, b;
    bool rotated;
    __device__ __forceinline__ RopeCols(uint32_t c, int R) {
        rotated = (int)c < R / 16;
        a = rotated && !INTER ? 8 * (int)c : 16 * (int)c;
        b = rotated && !INTER ? a + R / 2 : a + 8;
    }
};

// cosines and sines of a rotated group's pairs
template <bool INTER>
__device__ __forceinline__ void rope_row(const float *row, const RopeCols<INTER> &rc, int R, int inverse,
                                         float (&cs)[8], float (&sn)[8]) {
    const int i = INTER ? rc.a / 2 : rc.a;  // first pair
    ld8(row + i, cs);
    ld8(row + R / 2 + i, sn);
    if (inverse) {
#pragma unroll
        for (int k = 0; k < 8; ++k) sn[k] = -sn[k];
    }
}

template <bool INTER>
__device__ __forceinline__ void rope_turn(float (&lo)[8], float (&hi)[8], const float (&cs)[8],
                                          const float (&sn)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        float *pa, *pb;
        if constexpr (INTER) {
            float *v = k < 4 ? lo : hi;
            pa = v + 2 * (k & 3);
            pb = pa + 1;
        } else {
            pa = lo + k;
            pb = hi + k;
        }
        const float a = *pa, b = *pb;
        *pa = rope_a(a, b, cs[k], sn[k]);
        *pb = rope_b(a, b, cs[k], sn[k]);
    }
}

}  // namespace tl
