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

// 8 values as codes (8 bytes, or 4 for INT4, low element first): y / s rounded to nearest,
// then to nearest even on the grid.  s > 0, r = 1 / s rounded to nearest.
//  * The quotient takes one step of Markstein's correction (P. W. Markstein, IBM J. Res.
//    Dev. 34, 1990): the residual of the first quotient y r is exact in a fused
//    multiply-add.  Three instructions an element for about twelve; it holds where
//    neither step overflows or underflows, and PLAIN rows divide instead.
//  * Adding 1.5 * 2^23 rounds to nearest even in the low bits (INT4: the 8 of the field comes
//    with it).
//  * The clamp only acts where a scale near the smallest fp32 number lost its bits.
template <int FMT, bool PLAIN>
__device__ __forceinline__ uint2 quant8(const float (&y)[8], float s, float r) {
    constexpr float q = KvCode<FMT>::qmax, magic = 12582912.f + (FMT == kKvInt4 ? 8.f : 0.f);
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float z;
        if constexpr (PLAIN) {
            z = fminf(q, fmaxf(-q, __fdiv_rn(y[i], s)));
        } else {
            z = __fmul_rn(y[i], r);
            z = __fmaf_rn(__fmaf_rn(-z, s, y[i]), r, z);
        }
        b[i] = FMT == kKvFp8 ? __float_as_uint(z) : __float_as_uint(__fadd_rn(z, magic));
    }
    if constexpr (FMT == kKvFp8) {
        uint16_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
                : "=h"(h[i])
                : "f"(__uint_as_float(b[2 * i + 1])), "f"(__uint_as_float(b[2 * i])));
        return make_uint2(h[0] | ((uint32_t)h[1] << 16), h[2] | ((uint32_t)h[3] << 16));
    } else {
        const uint32_t x = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
        const uint32_t w = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
        if constexpr (FMT == kKvInt8) return make_uint2(x, w);
        return make_uint2(__byte_perm(x | (x >> 4), w | (w >> 4), 0x6420), 0u);  // bytes of two fields
    }
}

// Stores one row's column group as codes; the D/16 threads of a row are neighbours in a warp
// and share its largest magnitude by shuffles (all lanes take part).
template <int FMT, int D, bool INTER>
__device__ __forceinline__ void put_row(const RopeCols<INTER> &rc, const float (&lo)[8], const float (&hi)[8],
                                        uint8_t *codes, float *scales, int64_t row, bool store, bool first) {
    constexpr int C = D / 16;
    // magnitudes compare as their bits, an infinity or a NaN above every number
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = max(m, max(__float_as_uint(lo[i]) & 0x7FFFFFFFu, __float_as_uint(hi[i]) & 0x7FFFFFFFu));
#pragma unroll
    for (int o = C / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (!store) return;
    const float s = m >= 0x7F800000u ? __uint_as_float(0x7FC00000u)
                                     : __fmul_rn(__uint_as_float(m), 1.f / KvCode<FMT>::qmax);
    uint2 x, y;
    if (s > 1e-30f && s < 1e30f) {  // far from where the correction's steps leave fp32
        const float r = __frcp_rn(s);
        x = quant8<FMT, false>(lo, s, r);
        y = quant8<FMT, false>(hi, s, r);
    } else if (s > 0.f) {
        x = quant8<FMT, true>(lo, s, 0.f);
        y = quant8<FMT, true>(hi, s, 0.f);
    } else {  // zero rows, and rows with a NaN or an infinity
        x = y = make_uint2(FMT == kKvInt4 ? 0x88888888u : 0u, 0u);
    }
    uint8_t *w = codes + row * (D * KvCode<FMT>::bits / 8);
    if constexpr (FMT == kKvInt4) {
        *reinterpret_cast<uint32_t *>(w + rc.a / 2) = x.x;
        *reinterpret_cast<uint32_t *>(w + rc.b / 2) = y.x;
    } else {
        *reinterpret_cast<uint2 *>(w + rc.a) = x;
        *reinterpret_cast<uint2 *>(w + rc.b) = y;
    }
    if (first) scales[row] = s;
}

// One thread per column group of 16 elements (RopeCols) of a query head, or of a kv head's key and
// value together (their loads in flight at once).  Rows are requested before their position
// is looked at.  9973 tokens of 32 heads, f16 to INT4, half rotated: 82 us, 4.6 TB/s (rows,
// codes and scales; a copy's rate is 6.7); with divisions in the place of the corrected
// reciprocal it was bound by them.  Two rows of one tensor per thread were slower.
template <typename T, int FMT, int D, bool INTER, bool VEC>
__global__ void __launch_bounds__(256, 4) kv_append_kernel(KvAppendArgs a, uint32_t items, uint32_t total) {
    constexpr uint32_t C = D / 16;
    const uint32_t id0 = blockIdx.x * 256u + threadIdx.x;
    const uint32_t id = min(id0, total - 1);
    const uint32_t c = id % C, r = id / C;
    const int64_t t = r / items;
    const int item = (int)(r - (uint32_t)t * items);
    const bool kv = item >= a.Hq;
    const int h = kv ? item - a.Hq : item;
    const int64_t pos = a.R > 0 ? a.positions[t] : 0;
    const int64_t slot = kv ? a.slots[t] : -1;
    const RopeCols<INTER> rc(c, a.R), rv(c, 0);
    const T *x = kv ? static_cast<const T *>(a.k) + t * a.kt + h * a.kh : static_cast<const T *>(a.q) + t * a.qt + h * a.qh;
    float lo[8], hi[8], lo2[8], hi2[8];
    ld8_any<T, VEC>(x + rc.a, lo);
    ld8_any<T, VEC>(x + rc.b, hi);
    if (kv) {
        const T *y = static_cast<const T *>(a.v) + t * a.vt + h * a.vh;
        ld8_any<T, VEC>(y + rv.a, lo2);
        ld8_any<T, VEC>(y + rv.b, hi2);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) lo2[i] = hi2[i] = 0.f;
    }
    bool ok = id0 < total;
    if (a.R > 0 && (pos < 0 || pos >= a.table_rows)) {
        ok = false;
        flag_value(a.status);
    }
    if (ok && rc.rotated) {
        float cs[8], sn[8];
        rope_row<INTER>(a.table + pos * a.R, rc, a.R, 0, cs, sn);
        rope_turn<INTER>(lo, hi, cs, sn);
    }
    if (!kv && ok) {
        T *o = static_cast<T *>(a.qo) + t * a.qot + h * a.qoh;
        st8_any<T, VEC>(o + rc.a, lo);
        st8_any<T, VEC>(o + rc.b, hi);
    }
    if (!__any_sync(0xffffffffu, kv)) return;
    bool store = ok && slot >= 0;
    if (store && slot >= a.c.pages * a.c.P) {
        flag_value(a.status);
        store = false;
    }
    int64_t row = 0;
    if (store) {
        const int64_t page = (slot >> 31) == 0 ? (int64_t)((uint32_t)slot / (uint32_t)a.c.P) : slot / a.c.P;
        row = (page * a.c.Hk + h) * a.c.P + (slot - page * a.c.P);
    }
    put_row<FMT, D>(rc, lo, hi, a.c.kc, a.c.ks, row, store, c == 0);
    put_row<FMT, D>(rv, lo2, hi2, a.c.vc, a.c.vs, row, store, c == 0);
}

template <typename T, int FMT, int D>
cudaError_t append_d(const KvAppendArgs &a, bool inter, bool vec, cudaStream_t st) {
    const uint32_t items = (uint32_t)(a.Hq + a.c.Hk);
    // tokens per launch such that every thread index fits 31 bits
    const int64_t chunk = ((int64_t)1 << 30) / ((int64_t)items * (D / 16));
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
        const uint32_t total = (uint32_t)(b.tokens * items * (D / 16));
        const unsigned grid = (total + 255) / 256;
        if (inter) {
            if (vec) kv_append_kernel<T, FMT, D, true, true><<<grid, 256, 0, st>>>(b, items, total);
            else kv_append_kernel<T, FMT, D, true, false><<<grid, 256, 0, st>>>(b, items, total);
        } else {
            if (vec) kv_append_kernel<T, FMT, D, false, true><<<grid, 256, 0, st>>>(b, items, total);
            else kv_append_kernel<T, FMT, D, false, false><<<grid, 256, 0, st>>>(b, items, total);
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

// Reading back: one thread per 16 elements of one kv head's key and value row, both loads in
// flight together.  131072 tokens of 4 heads, e4m3 to bf16: 65 us, 6.3 TB/s, 0.94 of a
// copy's rate.
template <typename T, int FMT, int D>
__global__ void __launch_bounds__(256) kv_read_kernel(KvReadArgs a, uint32_t total) {
    constexpr uint32_t C = D / 16;
    constexpr int UB = 16 * KvCode<FMT>::bits / 8;  // bytes of 16 codes
    const uint32_t id = blockIdx.x * 256u + threadIdx.x;
    if (id >= total) return;
    const uint32_t c = id % C, r = id / C, heads = (uint32_t)a.c.Hk;
    const int64_t t = r / heads;
    const int h = (int)(r - (uint32_t)t * heads);
    const int64_t slot = a.slots[t];
    uint32_t w[2][4];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) w[0][i] = w[1][i] = FMT == kKvInt4 ? 0x88888888u : 0u;  // zeros
    if (slot >= 0 && slot < a.c.pages * a.c.P) {
        const int64_t page = (slot >> 31) == 0 ? (int64_t)((uint32_t)slot / (uint32_t)a.c.P) : slot / a.c.P;
        const int64_t row = (page * a.c.Hk + h) * a.c.P + (slot - page * a.c.P);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const uint8_t *p = (v ? a.c.vc : a.c.kc) + row * (C * UB) + c * UB;
            s[v] = (v ? a.c.vs : a.c.ks)[row];
            if constexpr (UB == 16) {
                const uint4 x = ldg_nc_v4(p);
                w[v][0] = x.x, w[v][1] = x.y, w[v][2] = x.z, w[v][3] = x.w;
            } else {
                const uint2 x = ldg_nc_v2(p);
                w[v][0] = x.x, w[v][1] = x.y;
            }
        }
    } else if (slot >= 0) {
        flag_value(a.status);
    }
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        T *o = static_cast<T *>(v ? a.v : a.k);
        if (o == nullptr) continue;
        o += (t * a.c.Hk + h) * D + c * 16;
        float x[16], lo[8], hi[8];
        codes16_f32<FMT>(w[v], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo[i] = __fmul_rn(x[i], s[v]);
            hi[i] = __fmul_rn(x[8 + i], s[v]);
        }
        st8(o, lo);
        st8(o + 8, hi);
    }
}

template <typename T, int FMT, int D>
cudaError_t read_d(const KvReadArgs &a, cudaStream_t st) {
    const int64_t per = (int64_t)a.c.Hk * (D / 16);
    const int64_t chunk = ((int64_t)1 << 30) / per;  // tokens per launch: thread indexes fit 31 bits
    for (int64_t t0 = 0; t0 < a.tokens; t0 += chunk) {
        KvReadArgs b = a;
        b.tokens = a.tokens - t0 < chunk ? a.tokens - t0 : chunk;
        b.slots = a.slots + t0;
        if (a.k) b.k = static_cast<T *>(a.k) + t0 * a.c.Hk * D;
        if (a.v) b.v = static_cast<T *>(a.v) + t0 * a.c.Hk * D;
        const uint32_t total = (uint32_t)(b.tokens * per);
        kv_read_kernel<T, FMT, D><<<(total + 255) / 256, 256, 0, st>>>(b, total);
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
