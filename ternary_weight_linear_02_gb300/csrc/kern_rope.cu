// kern_rope.cu -- rotary positions: the table of cosines and sines, and the
// rotation of query / key heads by it.
//
// A head's elements below R form R/2 pairs (a, b); pair i of a token at position
// p turns by the angle p f_i:  (a, b) -> (a c - b s, b c + a s).  Half layout:
// (x[i], x[i + R/2]); interleaved: (x[2i], x[2i + 1]).  The inverse (and the
// gradient) turns by the negative angle.
#include "rope.cuh"
#include "kernels.h"

namespace tl {

namespace {

// One entry per thread and pair.  The angle p f_i reaches 10^5 radians and more,
// where fp32 would keep two digits of it after reduction, so it is computed (and
// reduced, by sincos) in fp64; this runs once per model.
__global__ void __launch_bounds__(256) rope_table_kernel(RopeTableArgs a) {
    const int half = a.R / 2;
    const int64_t n = a.positions * half;
    for (int64_t e = blockIdx.x * 256ll + threadIdx.x; e < n; e += gridDim.x * 256ll) {
        const int64_t p = e / half;
        const int i = (int)(e - p * half);
        double f = pow(a.base, -2.0 * i / a.R);
        double keep = 0.0;
        if (a.original_len > 0 && a.ramp_hi > a.ramp_lo) {
            const double turns = a.original_len * f / 6.283185307179586476925;
            keep = fmin(1.0, fmax(0.0, (turns - a.ramp_lo) / (a.ramp_hi - a.ramp_lo)));
        }
        f *= keep + (1.0 - keep) / a.factor;
        double s, c;
        sincos((double)p * f, &s, &c);
        a.table[p * a.R + i] = (float)(a.magnitude * c);
        a.table[p * a.R + half + i] = (float)(a.magnitude * s);
    }
}

// Vector form: rows whose starts are 16-byte aligned, R and D multiples of 16.  A thread owns one
// column group of 16 elements (RopeCols) of one head: measured against two and four
// heads per thread, which read a table row less often but keep fewer warps in flight
// (16384 tokens x 32 heads of 128, half rotated: 48.5 us, 5.6 TB/s, against 72 and 128; a plain copy of
// the same bytes takes 43).  The head's elements are requested before the position is
// looked at, so that only the table row waits for it.
template <typename T, bool INTER>
__global__ void __launch_bounds__(256) rope_kernel(RopeArgs a, uint32_t cols, uint32_t total) {
    const uint32_t id = blockIdx.x * 256u + threadIdx.x;
    if (id >= total) return;
    const uint32_t c = id % cols, r = id / cols;
    const int64_t t = r / (uint32_t)a.heads;
    const int h = (int)(r - (uint32_t)t * (uint32_t)a.heads);
    const int64_t pos = a.positions[t];
    const RopeCols<INTER> rc(c, a.R);
    const T *x = static_cast<const T *>(a.x) + t * a.xt + h * a.xh;
    float lo[8], hi[8];
    ld8(x + rc.a, lo);
    ld8(x + rc.b, hi);
    if (pos < 0 || pos >= a.table_rows) {
        flag_value(a.status);
        return;
    }
    if (rc.rotated) {
        float cs[8], sn[8];
        rope_row<INTER>(a.table + pos * a.R, rc, a.R, a.inverse, cs, sn);
        rope_turn<INTER>(lo, hi, cs, sn);
    }
    T *o = static_cast<T *>(a.out) + t * a.ot + h * a.oh;
    st8(o + rc.a, lo);
    st8(o + rc.b, hi);
}

// Any alignment, any even R: one pair (or one copied element) per thread.
template <typename T, bool INTER>
__global__ void __launch_bounds__(256) rope_plain_kernel(RopeArgs a) {
    const int half = a.R / 2, per = half + (a.D - a.R);
    const int64_t n = a.tokens * a.heads * per;
    for (int64_t e = blockIdx.x * 256ll + threadIdx.x; e < n; e += gridDim.x * 256ll) {
        const int i = (int)(e % per);
        const int64_t r = e / per, t = r / a.heads;
        const int h = (int)(r - t * a.heads);
        const int64_t pos = a.positions[t];
        if (pos < 0 || pos >= a.table_rows) {
            flag_value(a.status);
            continue;
        }
        const T *x = static_cast<const T *>(a.x) + t * a.xt + h * a.xh;
        T *o = static_cast<T *>(a.out) + t * a.ot + h * a.oh;
        if (i >= half) {
            o[half + i] = x[half + i];  // element R + (i - half)
            continue;
        }
        const int ia = INTER ? 2 * i : i, ib = INTER ? 2 * i + 1 : i + half;
        const float *row = a.table + pos * a.R;
        const float c = row[i], s = a.inverse ? -row[half + i] : row[half + i];
        const float va = to_f32(x[ia]), vb = to_f32(x[ib]);
        o[ia] = from_f32<T>(rope_a(va, vb, c, s));
        o[ib] = from_f32<T>(rope_b(va, vb, c, s));
    }
}

template <typename T, bool INTER>
cudaError_t launch_rope_t(const RopeArgs &a, bool vec, int sm_count, cudaStream_t st) {
    if (!vec) {
        const int64_t n = a.tokens * a.heads * (a.R / 2 + a.D - a.R);
        const int64_t blocks = (n + 255) / 256, most = (int64_t)sm_count * 32;
        rope_plain_kernel<T, INTER><<<(unsigned)(blocks < most ? blocks : most), 256, 0, st>>>(a);
        return cudaGetLastError();
    }
    const int64_t cols = a.D / 16;
    // tokens per launch such that every thread index fits 31 bits
    const int64_t chunk = ((int64_t)1 << 30) / (cols * a.heads);
    for (int64_t t0 = 0; t0 < a.tokens; t0 += chunk) {
        RopeArgs b = a;
        b.tokens = a.tokens - t0 < chunk ? a.tokens - t0 : chunk;
        b.x = static_cast<const T *>(a.x) + t0 * a.xt;
        b.out = static_cast<T *>(a.out) + t0 * a.ot;
        b.positions = a.positions + t0;
        const uint32_t total = (uint32_t)(b.tokens * cols * a.heads);
        rope_kernel<T, INTER><<<(total + 255) / 256, 256, 0, st>>>(b, (uint32_t)cols, total);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_rope_table(const RopeTableArgs &a, cudaStream_t st) {
    const int64_t blocks = (a.positions * (a.R / 2) + 255) / 256;
    rope_table_kernel<<<(unsigned)(blocks < 65536 ? blocks : 65536), 256, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_rope(const RopeArgs &a, int dtype, bool interleaved, bool vec, int sm_count,
                        cudaStream_t st) {
    if (dtype == 0)
        return interleaved ? launch_rope_t<__half, true>(a, vec, sm_count, st)
                           : launch_rope_t<__half, false>(a, vec, sm_count, st);
    if (dtype == 1)
        return interleaved ? launch_rope_t<__nv_bfloat16, true>(a, vec, sm_count, st)
                           : launch_rope_t<__nv_bfloat16, false>(a, vec, sm_count, st);
    return interleaved ? launch_rope_t<float, true>(a, vec, sm_count, st)
                       : launch_rope_t<float, false>(a, vec, sm_count, st);
}

}  // namespace tl
