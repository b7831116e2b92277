// kern_move.cu -- entries of the cache moved as they are, in all layers of a model by one
// launch: whole pages and parts of them (copies, forks), and entries closed up in place.
//
// A head's codes of a page are contiguous (page_size rows of rb bytes), so are its scales.
#include "common.cuh"
#include "kernels.h"

namespace tl {

namespace {

// The first n places of one head of a page to another page: keys, values, and their scales.
__device__ __forceinline__ void copy_head(const KvMove &m, int layer, int h, int src, int dst, int n) {
    const int64_t s = ((int64_t)src * m.Hk + h) * m.P, d = ((int64_t)dst * m.Hk + h) * m.P;
    const int pieces = n * (m.rb >> 4);
    const uint4 *k = reinterpret_cast<const uint4 *>(m.kc[layer] + s * m.rb), *v = reinterpret_cast<const uint4 *>(m.vc[layer] + s * m.rb);
    uint4 *ko = reinterpret_cast<uint4 *>(m.kc[layer] + d * m.rb), *vo = reinterpret_cast<uint4 *>(m.vc[layer] + d * m.rb);
    for (int i0 = 0; i0 < pieces; i0 += 512) {
        const int i = i0 + threadIdx.x, j = i + 256;
        uint4 a, b, c, e;
        if (i < pieces) a = k[i], b = v[i];
        if (j < pieces) c = k[j], e = v[j];
        if (i < pieces) ko[i] = a, vo[i] = b;
        if (j < pieces) ko[j] = c, vo[j] = e;
    }
    for (int i = threadIdx.x; i < n; i += 256) {
        const float a = m.ks[layer][s + i], b = m.vs[layer][s + i];
        m.ks[layer][d + i] = a;
        m.vs[layer][d + i] = b;
    }
}

__global__ void __launch_bounds__(256) kv_copy_kernel(const __grid_constant__ KvMove m, const int *src, const int *dst, const int *tokens,
                                                      int64_t n) {
    const uint32_t per = (uint32_t)(m.L * m.Hk);
    const int64_t units = n * per;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t i = u / per;
        const uint32_t lh = (uint32_t)(u - i * per), layer = lh / (uint32_t)m.Hk;
        const int s = src[i], d = dst[i], t = tokens ? tokens[i] : m.P;
        if (s < 0 || d < 0) continue;
        if (s >= m.pages || d >= m.pages || t < 0 || t > m.P) {
            if (threadIdx.x == 0) flag_value(m.status);
            continue;
        }
        copy_head(m, (int)layer, (int)(lh - layer * (uint32_t)m.Hk), s, d, t);
    }
}

// The rows that pages_take listed (list[0] of them): a unit that shares the full pages, and one for
// each head and layer of the last page's entries.
__global__ void __launch_bounds__(256) fork_apply_kernel(const __grid_constant__ KvMove m, KvPages g, const int *parent, const int *list, int share) {
    const uint32_t per = (uint32_t)(m.L * m.Hk) + (uint32_t)share;
    const int64_t units = (int64_t)list[0] * per;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t i = u / per;
        const uint32_t j = (uint32_t)(u - i * per);
        const int r = list[1 + i], p = parent[r];
        const uint32_t n = (uint32_t)g.lens[p], full = n / (uint32_t)g.P;
        const int *from = g.table + p * g.stride;
        int *to = g.table + r * g.stride;
        if (share && j == 0) {
            for (uint32_t e = threadIdx.x; e < full; e += 256) {
                const int page = from[e];
                to[e] = page;
                if ((uint32_t)page < (uint32_t)g.pages) atomicAdd(g.refs + page, 1);
                else flag_value(m.status);
            }
            continue;
        }
        const int part = (int)(n - full * (uint32_t)g.P);
        if (part == 0) continue;
        const uint32_t lh = j - (uint32_t)share, layer = lh / (uint32_t)m.Hk;
        const int s = from[full], d = to[full];
        if ((uint32_t)s >= (uint32_t)g.pages || (uint32_t)d >= (uint32_t)g.pages) {
            if (threadIdx.x == 0) flag_value(m.status);
            continue;
        }
        copy_head(m, (int)layer, (int)(lh - layer * (uint32_t)m.Hk), s, d, part);
    }
}

// ---------------------------------------------------------------- closing up
// Entry i of a sequence moves from place start + keep[i] to start + i, keep ascending, so dst_i <=
// src_i < src_j for i < j: what an entry overwrites is no later entry's source.  Moves done in
// order, a group's reads before its writes, therefore give what reading everything first
// would, and the next group may be read before this one is written.

// Row (place of one head of the pool) of a sequence's place; -1 for a page that the pool does not have.
__device__ __forceinline__ int64_t row_of(const KvMove &m, const KvCompactArgs &a, const int *pages, uint32_t place) {
    const uint32_t p = place / (uint32_t)m.P;
    const int page = pages[p];
    if ((uint32_t)page >= (uint32_t)m.pages) {
        flag_value(m.status);
        return -1;
    }
    return (int64_t)page * m.Hk * m.P + (place - p * (uint32_t)m.P);
}

struct Moves {
    int start, n;  // first place; moves of the sequence
    const int *keep, *pages;
    __device__ __forceinline__ Moves(const KvMove &m, const KvCompactArgs &a, int64_t b) {
        start = a.start[b];
        n = a.count[b];
        keep = a.keep + b * a.keep_stride;
        pages = a.table + b * a.table_stride;
        if (n < 0 || n > a.n || start < 0) {
            flag_value(m.status);
            n = start < 0 || n < 0 ? 0 : (int)a.n;
        }
    }
    // rows of move i, or false where the sequence's moves end
    __device__ __forceinline__ bool at(const KvMove &m, const KvCompactArgs &a, int i, int64_t &src, int64_t &dst) const {
        const int k = keep[i], before = i > 0 ? keep[i - 1] : -1;
        const int64_t place = (int64_t)start + k;
        if (k <= before || k < i || place >= a.max_places) {  // (k < i: an earlier one did not ascend)
            flag_value(m.status);
            return false;
        }
        src = row_of(m, a, pages, (uint32_t)place);
        dst = k == i ? src : row_of(m, a, pages, (uint32_t)(start + i));
        return true;
    }
};

// Few moves a sequence: a warp per (sequence, layer, head), 16 moves at a time, keys and values
// together.  PIECES: 16-byte pieces of a row of codes.
template <int PIECES>
__global__ void __launch_bounds__(256) compact_warp_kernel(const __grid_constant__ KvMove m, KvCompactArgs a, int64_t units) {
    constexpr int ROWS = 32 / PIECES, PASSES = 16 / ROWS;  // rows a pass of the warp
    const int lane = threadIdx.x & 31;
    const int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (u >= units) return;
    const uint32_t per = (uint32_t)(m.L * m.Hk);
    const int64_t b = u / per;
    const uint32_t lh = (uint32_t)(u - b * per), layer = lh / (uint32_t)m.Hk;
    const int64_t head = (int64_t)(lh - layer * (uint32_t)m.Hk) * m.P;
    const Moves mv(m, a, b);
    uint8_t *const kc = m.kc[layer], *const vc = m.vc[layer];
    float *const ks = m.ks[layer], *const vs = m.vs[layer];
    bool more = true;
    for (int i0 = 0; i0 < mv.n && more; i0 += 16) {
        int64_t src = -1, dst = -1;
        bool ok = true;
        if (lane < 16 && i0 + lane < mv.n) ok = mv.at(m, a, i0 + lane, src, dst);
        const uint32_t bad = __ballot_sync(0xffffffffu, !ok);
        if (bad) {  // nothing from the first bad move on
            more = false;
            if (lane >= __ffs(bad) - 1) src = dst = -1;
        }
        if (src < 0 || dst < 0 || src == dst) src = dst = -1;
        uint4 k[PASSES], v[PASSES];
        int64_t to[PASSES];
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int row = p * ROWS + lane / PIECES;
            const int64_t s = __shfl_sync(0xffffffffu, src, row), d = __shfl_sync(0xffffffffu, dst, row);
            to[p] = d < 0 ? -1 : ((head + d) * PIECES + lane % PIECES) * 16;
            if (d >= 0) {
                const int64_t from = ((head + s) * PIECES + lane % PIECES) * 16;
                k[p] = *reinterpret_cast<const uint4 *>(kc + from);
                v[p] = *reinterpret_cast<const uint4 *>(vc + from);
            }
        }
        float x = 0.f, y = 0.f;
        if (dst >= 0) x = ks[head + src], y = vs[head + src];
        __syncwarp();
#pragma unroll
        for (int p = 0; p < PASSES; ++p)
            if (to[p] >= 0) {
                *reinterpret_cast<uint4 *>(kc + to[p]) = k[p];
                *reinterpret_cast<uint4 *>(vc + to[p]) = v[p];
            }
        if (dst >= 0) ks[head + dst] = x, vs[head + dst] = y;
        __syncwarp();
    }
}

// Many moves: a block per (sequence, layer, head, keys or values), eight 16-byte pieces a thread in
// flight, the next group's rows looked up and requested before this one is written.
template <int PIECES>
__global__ void __launch_bounds__(256) compact_block_kernel(const __grid_constant__ KvMove m, KvCompactArgs a) {
    constexpr int ROWS = 256 * 8 / PIECES, EACH = ROWS / 256;  // moves a group; looked up by each thread
    __shared__ int64_t rows[2][2][ROWS];                       // [buffer][from, to]; -1: nothing to move
    __shared__ int end;
    const uint32_t per = (uint32_t)(m.L * m.Hk) * 2u, tid = threadIdx.x;
    const int64_t u = blockIdx.x, b = u / per;
    const uint32_t rest = (uint32_t)(u - b * per), lh = rest >> 1, layer = lh / (uint32_t)m.Hk;
    const int64_t head = (int64_t)(lh - layer * (uint32_t)m.Hk) * m.P;
    const Moves mv(m, a, b);
    uint8_t *const codes = rest & 1u ? m.vc[layer] : m.kc[layer];
    float *const scales = rest & 1u ? m.vs[layer] : m.ks[layer];
    if (tid == 0) end = mv.n;
    __syncthreads();
    const auto look = [&](int i0, int buf) {
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            const int k = e * 256 + tid, i = i0 + k;
            int64_t src = -1, dst = -1;
            if (i < mv.n && !mv.at(m, a, i, src, dst)) atomicMin(&end, i);
            if (src < 0 || dst < 0 || src == dst) src = dst = -1;
            rows[buf][0][k] = src;
            rows[buf][1][k] = dst;
        }
    };
    uint4 piece[8];
    float scale[EACH];
    const auto load = [&](int i0, int buf) {
        const int lim = end - i0;
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const int k = p * (ROWS / 8) + (int)tid / PIECES;
            const int64_t s = rows[buf][0][k];
            if (s >= 0 && k < lim) piece[p] = *reinterpret_cast<const uint4 *>(codes + ((head + s) * PIECES + tid % PIECES) * 16);
        }
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            const int64_t s = rows[buf][0][e * 256 + tid];
            if (s >= 0 && e * 256 + (int)tid < lim) scale[e] = scales[head + s];
        }
    };
    look(0, 0);
    __syncthreads();
    load(0, 0);
    int buf = 0;
    for (int i0 = 0; i0 < end; i0 += ROWS, buf ^= 1) {
        look(i0 + ROWS, buf ^ 1);
        const uint4 was[8] = {piece[0], piece[1], piece[2], piece[3], piece[4], piece[5], piece[6], piece[7]};
        float had[EACH];
#pragma unroll
        for (int e = 0; e < EACH; ++e) had[e] = scale[e];
        __syncthreads();  // the group is read by all, the next one's rows are known to all
        const int lim = end - i0;
        load(i0 + ROWS, buf ^ 1);
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const int k = p * (ROWS / 8) + (int)tid / PIECES;
            const int64_t d = rows[buf][1][k];
            if (d >= 0 && k < lim) *reinterpret_cast<uint4 *>(codes + ((head + d) * PIECES + tid % PIECES) * 16) = was[p];
        }
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            const int64_t d = rows[buf][1][e * 256 + tid];
            if (d >= 0 && e * 256 + (int)tid < lim) scales[head + d] = had[e];
        }
        __syncthreads();  // rows of this group are done with
    }
}

template <int PIECES>
cudaError_t compact(const KvMove &m, const KvCompactArgs &a, cudaStream_t st) {
    const int64_t per = (int64_t)m.L * m.Hk;
    // sequences of a launch, such that blocks are counted in 31 bits
    const int64_t chunk = ((int64_t)1 << 29) / per;
    for (int64_t b0 = 0; b0 < a.batch; b0 += chunk) {
        KvCompactArgs c = a;
        c.batch = a.batch - b0 < chunk ? a.batch - b0 : chunk;
        c.table += b0 * a.table_stride;
        c.keep += b0 * a.keep_stride;
        c.start += b0;
        c.count += b0;
        const int64_t units = c.batch * per;
        if (a.n <= 64) compact_warp_kernel<PIECES><<<(unsigned)((units + 7) / 8), 256, 0, st>>>(m, c, units);
        else compact_block_kernel<PIECES><<<(unsigned)(units * 2), 256, 0, st>>>(m, c);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_kv_copy(const KvMove &m, const int *src, const int *dst, const int *tokens, int64_t n, int sm_count, cudaStream_t st) {
    const int64_t units = n * m.L * m.Hk, most = (int64_t)sm_count * 8;
    kv_copy_kernel<<<(unsigned)(units < most ? units : most), 256, 0, st>>>(m, src, dst, tokens, n);
    return cudaGetLastError();
}

cudaError_t launch_fork_apply(const KvMove &m, const KvPages &g, const int *parent, const int *list, bool share, int sm_count, cudaStream_t st) {
    const int64_t units = (int64_t)g.rows * (m.L * m.Hk + (share ? 1 : 0)), most = (int64_t)sm_count * 8;
    fork_apply_kernel<<<(unsigned)(units < most ? units : most), 256, 0, st>>>(m, g, parent, list, share);
    return cudaGetLastError();
}

cudaError_t launch_kv_compact(const KvMove &m, const KvCompactArgs &a, cudaStream_t st) {
    return m.rb == 128 ? compact<8>(m, a, st) : m.rb == 64 ? compact<4>(m, a, st) : compact<2>(m, a, st);
}

}  // namespace tl
