// kern_kv.cu -- the quantised cache: writing it (with the rotation of queries and
// keys in the same pass) and reading it back.
//
// A row y (one token, one kv head, keys after their rotation) is stored as codes
// and one fp32 scale: scale = max|y| (1/Q), code = y / scale rounded to nearest even on
// the format's grid (Q = 127, 448, 7; 1/Q rounded to fp32).  The division is rounded to
// nearest: a reciprocal would move values next to a tie to the other code.
#include "kernels.h"
#include "kv.cuh"
#include "rope.cuh"

namespace tl {

namespace {

template <typename T, bool VEC>
__device__ __forceinline__ void ld8_any(const T *p, float (&v)[8]) {
    if constexpr (VEC) {
        ld8(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f32(p[i]);
    }
}
template <typename T, bool VEC>
__device__ __forceinline__ void st8_any(T *p, const float (&v)[8]) {
    if constexpr (VEC) {
        st8(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = from_f32<T>(v[i]);
    }
}

// 8 values as codes (8 bytes, or 4 for INT4, low element first).  Adding 1.5 * 2^23
// rounds |z| < 2^22 to nearest even in the low bits; the clamp only acts where a
// scale near the smallest fp32 number lost its bits.
template <int FMT>
__device__ __forceinline__ uint2 quant8(const float (&y)[8], float s) {
    uint2 w = make_uint2(0u, 0u);
    if (!(s > 0.f)) {  // zero rows, and rows with a NaN or an infinity
        if constexpr (FMT == kKvInt4) w.x = 0x88888888u;
        return w;
    }
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float q = KvCode<FMT>::qmax;
        const float z = fminf(q, fmaxf(-q, __fdiv_rn(y[i], s)));
        b[i] = FMT == kKvFp8 ? __float_as_uint(z) : __float_as_uint(__fadd_rn(z, 12582912.f));
    }
    if constexpr (FMT == kKvFp8) {
        uint16_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
                : "=h"(h[i])
                : "f"(__uint_as_float(b[2 * i + 1])), "f"(__uint_as_float(b[2 * i])));
        w.x = h[0] | ((uint32_t)h[1] << 16);
        w.y = h[2] | ((uint32_t)h[3] << 16);
    } else if constexpr (FMT == kKvInt8) {
        w.x = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
        w.y = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) w.x |= ((b[i] + 8u) & 0xFu) << (4 * i);
    }
    return w;
}

// One thread per column group of 16 elements (RopeCols) of one row; the D/16 threads
// of a row are neighbours in a warp and share its largest magnitude by shuffles.
// Rows of a token: Hq query heads, Hk keys, Hk values.
template <typename T, int FMT, int D, bool INTER, bool VEC>
__global__ void __launch_bounds__(256) kv_append_kernel(KvAppendArgs a, uint32_t rows, uint32_t total) {
    constexpr uint32_t C = D / 16;
    const uint32_t id0 = blockIdx.x * 256u + threadIdx.x;
    const bool inside = id0 < total;
    const uint32_t id = inside ? id0 : total - 1;
    const uint32_t c = id % C, r = id / C;
    const int64_t t = r / rows;
    const int hh = (int)(r % rows);
    const int side = hh < a.Hq ? 0 : hh < a.Hq + a.c.Hk ? 1 : 2;  // q, k, v
    const int h = side == 0 ? hh : side == 1 ? hh - a.Hq : hh - a.Hq - a.c.Hk;

    bool ok = inside;
    int64_t pos = 0;
    if (a.R > 0) {
        pos = a.positions[t];
        if (pos < 0 || pos >= a.table_rows) {
            ok = false;
            flag_value(a.status);
        }
    }
    const RopeCols<INTER> rc(c, side == 2 ? 0 : a.R);
    float lo[8], hi[8];
    if (ok) {
        const T *x = static_cast<const T *>(side == 0 ? a.q : side == 1 ? a.k : a.v) +
                     t * (side == 0 ? a.qt : side == 1 ? a.kt : a.vt) +
                     h * (side == 0 ? a.qh : side == 1 ? a.kh : a.vh);
        ld8_any<T, VEC>(x + rc.a, lo);
        ld8_any<T, VEC>(x + rc.b, hi);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) lo[i] = hi[i] = 0.f;
    }
    if (ok && rc.rotated) {
        float cs[8], sn[8];
        rope_row<INTER>(a.table + pos * a.R, rc, a.R, 0, cs, sn);
        rope_turn<INTER>(lo, hi, cs, sn);
    }
    if (side == 0 && ok) {
        T *o = static_cast<T *>(a.qo) + t * a.qot + h * a.qoh;
        st8_any<T, VEC>(o + rc.a, lo);
        st8_any<T, VEC>(o + rc.b, hi);
    }
    // magnitudes compare as their bits, an infinity or a NaN above every number
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = max(m, max(__float_as_uint(lo[i]) & 0x7FFFFFFFu, __float_as_uint(hi[i]) & 0x7FFFFFFFu));
#pragma unroll
    for (int o = C / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (side == 0 || !ok) return;
    const int64_t slot = a.slots[t];
    if (slot < 0) return;
    if (slot >= a.c.pages * a.c.P) {
        flag_value(a.status);
        return;
    }
    const float s = m >= 0x7F800000u ? __uint_as_float(0x7FC00000u)
                                     : __fmul_rn(__uint_as_float(m), 1.f / KvCode<FMT>::qmax);
    const int64_t page = slot / a.c.P;
    const int64_t row = (page * a.c.Hk + h) * a.c.P + (slot - page * a.c.P);
    uint8_t *w = (side == 1 ? a.c.kc : a.c.vc) + row * (D * KvCode<FMT>::bits / 8);
    const uint2 x = quant8<FMT>(lo, s), y = quant8<FMT>(hi, s);
    if constexpr (FMT == kKvInt4) {
        *reinterpret_cast<uint32_t *>(w + rc.a / 2) = x.x;
        *reinterpret_cast<uint32_t *>(w + rc.b / 2) = y.x;
    } else {
        *reinterpret_cast<uint2 *>(w + rc.a) = x;
        *reinterpret_cast<uint2 *>(w + rc.b) = y;
    }
    if (c == 0) (side == 1 ? a.c.ks : a.c.vs)[row] = s;
}

template <typename T, int FMT, int D>
cudaError_t append_d(const KvAppendArgs &a, bool inter, bool vec, cudaStream_t st) {
    const uint32_t rows = (uint32_t)(a.Hq + 2 * a.c.Hk);
    // tokens per launch such that every thread index fits 31 bits
    const int64_t chunk = ((int64_t)1 << 30) / ((int64_t)rows * (D / 16));
    for (int64_t t0 = 0; t0 < a.tokens; t0 += chunk) {
        KvAppendArgs b = a;
        b.tokens = a.tokens - t0 < chunk ? a.tokens - t0 : chunk;
        b.k = static_cast<const T *>(a.k) + t0 * a.kt;
        b.v = static_cast<const T *>(a.v) + t0 * a.vt;
        b.slots = a.slots + t0;
        if (a.Hq) {
            b.q = static_cast<const T *>(a.q) + t0 * a.qt;
            b.qo = static_cast<T *>(a.qo) + t0 * a.qot;
        }
        if (a.R) b.positions = a.positions + t0;
        const uint32_t total = (uint32_t)(b.tokens * rows * (D / 16));
        const unsigned grid = (total + 255) / 256;
        if (inter) {
            if (vec) kv_append_kernel<T, FMT, D, true, true><<<grid, 256, 0, st>>>(b, rows, total);
            else kv_append_kernel<T, FMT, D, true, false><<<grid, 256, 0, st>>>(b, rows, total);
        } else {
            if (vec) kv_append_kernel<T, FMT, D, false, true><<<grid, 256, 0, st>>>(b, rows, total);
            else kv_append_kernel<T, FMT, D, false, false><<<grid, 256, 0, st>>>(b, rows, total);
        }
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <typename T, int FMT>
cudaError_t append_f(const KvAppendArgs &a, bool inter, bool vec, cudaStream_t st) {
    return a.c.D == 128 ? append_d<T, FMT, 128>(a, inter, vec, st) : append_d<T, FMT, 64>(a, inter, vec, st);
}

template <typename T>
cudaError_t append_t(const KvAppendArgs &a, bool inter, bool vec, cudaStream_t st) {
    return a.c.fmt == kKvInt8  ? append_f<T, kKvInt8>(a, inter, vec, st)
           : a.c.fmt == kKvFp8 ? append_f<T, kKvFp8>(a, inter, vec, st)
                               : append_f<T, kKvInt4>(a, inter, vec, st);
}

// Reading back: one thread per 16 elements of one row, keys then values of a token.
template <typename T, int FMT, int D>
__global__ void __launch_bounds__(256) kv_read_kernel(KvReadArgs a, uint32_t rows, uint32_t total) {
    constexpr uint32_t C = D / 16;
    constexpr int UB = 16 * KvCode<FMT>::bits / 8;  // bytes of 16 codes
    const uint32_t id = blockIdx.x * 256u + threadIdx.x;
    if (id >= total) return;
    const uint32_t c = id % C, r = id / C;
    const int64_t t = r / rows;
    const int hh = (int)(r % rows);
    const bool value = a.k == nullptr || hh >= a.c.Hk;
    const int h = hh >= a.c.Hk ? hh - a.c.Hk : hh;
    const int64_t slot = a.slots[t];
    float lo[8], hi[8];
    if (slot < 0 || slot >= a.c.pages * a.c.P) {
        if (slot >= 0) flag_value(a.status);
#pragma unroll
        for (int i = 0; i < 8; ++i) lo[i] = hi[i] = 0.f;
    } else {
        const int64_t page = slot / a.c.P;
        const int64_t row = (page * a.c.Hk + h) * a.c.P + (slot - page * a.c.P);
        const uint8_t *p = (value ? a.c.vc : a.c.kc) + row * (C * UB) + c * UB;
        const float s = (value ? a.c.vs : a.c.ks)[row];
        uint32_t w[4];
        if constexpr (UB == 16) {
            const uint4 x = ldg_nc_v4(p);
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
        } else {
            const uint2 x = ldg_nc_v2(p);
            w[0] = x.x, w[1] = x.y;
        }
        float v[16];
        codes16_f32<FMT>(w, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo[i] = __fmul_rn(v[i], s);
            hi[i] = __fmul_rn(v[8 + i], s);
        }
    }
    T *o = static_cast<T *>(value ? a.v : a.k) + (t * a.c.Hk + h) * D + c * 16;
    st8(o, lo);
    st8(o + 8, hi);
}

template <typename T, int FMT, int D>
cudaError_t read_d(const KvReadArgs &a, cudaStream_t st) {
    const uint32_t rows = (uint32_t)(a.c.Hk * (a.k && a.v ? 2 : 1));
    const int64_t chunk = ((int64_t)1 << 30) / ((int64_t)rows * (D / 16));
    for (int64_t t0 = 0; t0 < a.tokens; t0 += chunk) {
        KvReadArgs b = a;
        b.tokens = a.tokens - t0 < chunk ? a.tokens - t0 : chunk;
        b.slots = a.slots + t0;
        if (a.k) b.k = static_cast<T *>(a.k) + t0 * a.c.Hk * D;
        if (a.v) b.v = static_cast<T *>(a.v) + t0 * a.c.Hk * D;
        const uint32_t total = (uint32_t)(b.tokens * rows * (D / 16));
        kv_read_kernel<T, FMT, D><<<(total + 255) / 256, 256, 0, st>>>(b, rows, total);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <typename T>
cudaError_t read_t(const KvReadArgs &a, cudaStream_t st) {
    const bool w = a.c.D == 128;
    switch (a.c.fmt) {
    case kKvInt8: return w ? read_d<T, kKvInt8, 128>(a, st) : read_d<T, kKvInt8, 64>(a, st);
    case kKvFp8: return w ? read_d<T, kKvFp8, 128>(a, st) : read_d<T, kKvFp8, 64>(a, st);
    default: return w ? read_d<T, kKvInt4, 128>(a, st) : read_d<T, kKvInt4, 64>(a, st);
    }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs &a, bool bf, bool interleaved, bool vec, cudaStream_t st) {
    return bf ? append_t<__nv_bfloat16>(a, interleaved, vec, st) : append_t<__half>(a, interleaved, vec, st);
}

cudaError_t launch_kv_read(const KvReadArgs &a, int out_dtype, cudaStream_t st) {
    return out_dtype == 0 ? read_t<__half>(a, st) : out_dtype == 1 ? read_t<__nv_bfloat16>(a, st) : read_t<float>(a, st);
}

}  // namespace tl
