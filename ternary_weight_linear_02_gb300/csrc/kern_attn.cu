// kern_attn.cu -- attention of new tokens (one, a chain or a tree of drafts) over the
// quantised paged cache.
//
//   o = sum_j p_j sv_j vc_j / sum_j p_j,  p_j = exp(scale sk_j (q . kc_j) - max)
// over the keys j that the row sees: every committed key, and of the new tokens'
// keys those its tree row names.
//
// One warp per query row; lanes take 32 keys at a time for the scores and D/32 elements
// each for the output.
#include "kernels.h"
#include "kv.cuh"
#include "rope.cuh"

namespace tl {

namespace {

template <typename T, int FMT, int D>
__global__ void __launch_bounds__(128) attn_rows_kernel(AttnArgs a) {
    constexpr int RB = D * KvCode<FMT>::bits / 8;  // bytes per row of codes
    constexpr int UB = RB / (D / 16);
    constexpr int E = D / 32;
    __shared__ float sq[4][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = blockIdx.x * 4ll + warp;
    if (row >= (int64_t)a.B * a.T * a.Hq) return;
    const int h = (int)(row % a.Hq);
    const int t = (int)(row / a.Hq % a.T);
    const int64_t b = row / a.Hq / a.T;
    const int hk = h / a.G;
    const T *q = static_cast<const T *>(a.q) + b * a.qb + t * a.qt + h * a.qh;
    for (int d = lane; d < D; d += 32) sq[warp][d] = to_f32(q[d]) * a.scale;
    __syncwarp();
    int64_t ctx = a.ctx[b];
    if (ctx < 0 || ctx > a.max_keys - a.T) {
        flag_value(a.status);
        ctx = ctx < 0 ? 0 : a.max_keys - a.T;
    }
    const uint8_t *tree = a.tree ? a.tree + b * a.tree_b + t * a.tree_r : nullptr;
    auto row_of = [&](int64_t j) -> int64_t {
        int64_t page = a.pages[b * a.pages_stride + j / a.c.P];
        if (page < 0 || page >= a.c.pages) {
            flag_value(a.status);
            page = 0;
        }
        return (page * a.c.Hk + hk) * a.c.P + j % a.c.P;
    };
    float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int64_t j0 = 0; j0 < ctx + a.T; j0 += 32) {
        const int64_t j = j0 + lane;
        bool see = j < ctx + a.T;
        if (see && j >= ctx) see = tree ? tree[j - ctx] != 0 : j - ctx <= t;
        float s = -INFINITY, sv = 0.f;
        int64_t kr = 0;
        if (see) {
            kr = row_of(j);
            float dot = 0.f;
            for (int c = 0; c < D / 16; ++c) {
                uint32_t w[4];
                for (int i = 0; i < UB / 4; ++i)
                    w[i] = *reinterpret_cast<const uint32_t *>(a.c.kc + kr * RB + c * UB + 4 * i);
                float v[16];
                codes16_f32<FMT>(w, v);
                for (int i = 0; i < 16; ++i) dot = fmaf(sq[warp][c * 16 + i], v[i], dot);
            }
            s = dot * a.c.ks[kr];
            sv = a.c.vs[kr];
        }
        float mx = s;
        for (int i = 16; i > 0; i >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, i));
        const float mn = fmaxf(m, mx), base = mn == -INFINITY ? 0.f : mn;
        const float corr = expf(m - base), p = see ? expf(s - base) : 0.f;
        m = mn;
        float ps = p;
        for (int i = 16; i > 0; i >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, i);
        l = l * corr + ps;
        for (int e = 0; e < E; ++e) o[e] *= corr;
        const float pv = see ? p * sv : 0.f;
        uint32_t seen = __ballot_sync(0xffffffffu, see);
        while (seen) {
            const int k = __ffs(seen) - 1;
            seen &= seen - 1;
            const float w = __shfl_sync(0xffffffffu, pv, k);
            const int64_t r = __shfl_sync(0xffffffffu, kr, k);
            const int d0 = lane * E;
            uint32_t u[4] = {0u, 0u, 0u, 0u};
            const int c = d0 / 16;
            for (int i = 0; i < UB / 4; ++i)
                u[i] = *reinterpret_cast<const uint32_t *>(a.c.vc + r * RB + c * UB + 4 * i);
            float v[16];
            codes16_f32<FMT>(u, v);
            for (int i = 0; i < 16; ++i)
                for (int e = 0; e < E; ++e)
                    if (i == d0 % 16 + e) o[e] = fmaf(w, v[i], o[e]);
        }
    }
    T *out = static_cast<T *>(a.out) + row * D + lane * E;
    for (int e = 0; e < E; ++e) out[e] = from_f32<T>(l == 0.f ? 0.f : o[e] / l);
    if (a.lse && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : m + logf(l);
}

template <typename T, int FMT>
cudaError_t launch_rows(const AttnArgs &a, cudaStream_t st) {
    const int64_t rows = (int64_t)a.B * a.T * a.Hq;
    const unsigned grid = (unsigned)((rows + 3) / 4);
    if (a.c.D == 128) attn_rows_kernel<T, FMT, 128><<<grid, 128, 0, st>>>(a);
    else attn_rows_kernel<T, FMT, 64><<<grid, 128, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const AttnArgs &a, cudaStream_t st) {
    return a.c.fmt == kKvInt8  ? launch_rows<T, kKvInt8>(a, st)
           : a.c.fmt == kKvFp8 ? launch_rows<T, kKvFp8>(a, st)
                               : launch_rows<T, kKvInt4>(a, st);
}

}  // namespace

int64_t tree_attention_workspace(int64_t, int64_t, int, int, int) { return 0; }

cudaError_t launch_tree_attention(const AttnArgs &a, bool bf, int sm_count, cudaStream_t st) {
    (void)sm_count;
    return bf ? launch_t<__nv_bfloat16>(a, st) : launch_t<__half>(a, st);
}

}  // namespace tl
