// kern_move.cu -- entries of the cache moved as they are, in all layers of a model by one
// launch: whole pages and parts of them (copies, forks), and entries closed up in place.
//
// A head's codes of a page are contiguous (page_size rows of rb bytes), so are its scales.  HBM-bound: nothing is
// computed.
#include "common.cuh"
#include "kernels.h"
#include "launch.h"

namespace tl {

namespace {

constexpr int kMovers = 512, kPieces = 4;  // threads of a block that closes up a long context; pieces in flight a group of each

// Copies are dealt to warps: a warp moves the first n places of one head of a page, keys or values, codes
// and scales, eight 16-byte pieces a lane in flight.  `task` counts (layer, head, keys or values).
// 224 rows forked in 28 layers: 45 us for 358 MB read and written (part of it stays in the L2), 52.8 at a copy's rate;
// a block per page and head, dividing the unit's number by each thread, took 65.
// kv_copy of 224 whole pages in 28 layers (fp8): 128 us, 125 at a copy's rate; of 4 pages 4.2 us; of 30 places of 224 pages (int4) 40, 30
// at a copy's rate.
__device__ __forceinline__ void copy_head(const KvMove &m, uint32_t task, int src, int dst, int n) {
    const int lane = threadIdx.x & 31;
    const uint32_t lh = task >> 1, layer = lh / (uint32_t)m.Hk, h = lh - layer * (uint32_t)m.Hk;
    uint8_t *const codes = task & 1u ? m.vc[layer] : m.kc[layer];
    float *const scales = task & 1u ? m.vs[layer] : m.ks[layer];
    const int64_t s = ((int64_t)src * m.Hk + h) * m.P, d = ((int64_t)dst * m.Hk + h) * m.P;
    const uint4 *const from = reinterpret_cast<const uint4 *>(codes + s * m.rb);
    uint4 *const to = reinterpret_cast<uint4 *>(codes + d * m.rb);
    const int pieces = n * (m.rb >> 4);
    float sc[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
        if (e * 32 + lane < n) sc[e] = scales[s + e * 32 + lane];
    int i = lane;
    for (; i + 7 * 32 < pieces; i += 8 * 32) {
        uint4 v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = from[i + e * 32];
#pragma unroll
        for (int e = 0; e < 8; ++e) to[i + e * 32] = v[e];
    }
    {
        uint4 v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (i + e * 32 < pieces) v[e] = from[i + e * 32];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (i + e * 32 < pieces) to[i + e * 32] = v[e];
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
        if (e * 32 + lane < n) scales[d + e * 32 + lane] = sc[e];
    for (int e = 64 + lane; e < n; e += 32) scales[d + e] = scales[s + e];
}

__global__ void __launch_bounds__(256) kv_copy_kernel(const __grid_constant__ KvMove m, const int *src, const int *dst, const int *tokens,
                                                      uint32_t n) {
    pdl_launch_dependents();
    pdl_wait();
    const uint32_t per = (uint32_t)(m.L * m.Hk) * 2u, total = n * per;
    for (uint32_t u = blockIdx.x * 8u + (threadIdx.x >> 5); u < total; u += gridDim.x * 8u) {
        const uint32_t i = u / per;
        const int s = src[i], d = dst[i], t = tokens ? tokens[i] : m.P;
        if (s < 0 || d < 0) continue;
        if (s >= m.pages || d >= m.pages || t < 0 || t > m.P) {
            if ((threadIdx.x & 31) == 0) flag_value(m.status);
            continue;
        }
        copy_head(m, u - i * per, s, d, t);
    }
}

// The rows that pages_take listed: their full pages, `runs` of 256 a row (0: not in this launch), and copies of the
// places in use of their last pages.  A warp a task.
__global__ void __launch_bounds__(256) fork_apply_kernel(const __grid_constant__ KvMove m, KvPages g, const int *listed,
                                                         const ForkItem *items, uint32_t runs) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const uint32_t per = (uint32_t)(m.L * m.Hk) * 2u + runs;
    const uint64_t total = (uint64_t)*listed * per;
    for (uint64_t w = blockIdx.x * 8u + (threadIdx.x >> 5); w < total; w += gridDim.x * 8u) {
        const uint32_t i = total >> 32 ? (uint32_t)(w / per) : (uint32_t)w / per, u = (uint32_t)(w - (uint64_t)i * per);
        const ForkItem it = items[i];
        if (u < runs) {
            const int *const from = g.table + it.parent * g.stride;
            int *const to = g.table + it.row * g.stride;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int64_t at = (int64_t)u * 256 + e * 32 + lane;
                if (at < it.full) {
                    const int page = from[at];
                    to[at] = page;
                    if ((uint32_t)page < (uint32_t)g.pages) atomicAdd(g.refs + page, 1);
                    else flag_value(m.status);
                }
            }
            continue;
        }
        if (it.places == 0) continue;
        if ((uint32_t)it.src >= (uint32_t)m.pages || (uint32_t)it.dst >= (uint32_t)m.pages) {
            if (lane == 0) flag_value(m.status);
            continue;
        }
        copy_head(m, u - runs, it.src, it.dst, it.places);
    }
}

// ---------------------------------------------------------------- closing up
// Entry i of a sequence moves from place start + keep[i] to start + i, keep ascending, so dst_i <=
// src_i < src_j for i < j: what an entry overwrites is no later entry's source.  Moves done in
// order, a group's reads before its writes, therefore give what reading everything first
// would, and the next group may be read before this one is written.

// Rows of a cache are counted in 32 bits (the call checks it: more would not fit this GPU's memory).
constexpr uint32_t kNone = 0xFFFFFFFFu;

// A place of a sequence on its way to its row of the pool (of one head): first the entry of the page table is requested,
// then, when it is there, looked at.
struct Place {
    int page;
    uint32_t off;
    __device__ __forceinline__ void request(const KvMove &m, const int *pages, uint32_t place) {
        const uint32_t p = m.shift >= 0 ? place >> m.shift : place / (uint32_t)m.P;
        page = pages[p];
        off = place - p * (uint32_t)m.P;
    }
    // kNone for a page that the pool does not have
    __device__ __forceinline__ uint32_t row(const KvMove &m) const {
        if ((uint32_t)page >= (uint32_t)m.pages) {
            flag_value(m.status);
            return kNone;
        }
        return (uint32_t)page * (uint32_t)(m.Hk * m.P) + off;
    }
};

struct Moves {
    int start, n;  // first place; moves of the sequence
    int64_t places;  // that the sequence has
    const int *keep, *pages;
    __device__ __forceinline__ Moves(const KvMove &m, const KvCompactArgs &a, int64_t b) {
        start = a.start[b];
        n = a.count[b];
        keep = a.keep + b * a.keep_stride;
        pages = a.table + b * a.table_stride;
        places = a.max_places;
        if (a.held) {  // entries of the table behind the held ones are nobody's, or 0
            const int64_t has = (int64_t)a.held[b] * m.P;
            if (has < 0 || has > places) flag_value(m.status);
            places = has <= places ? has : 0;
        }
        if (n < 0 || n > a.n || start < 0) {
            flag_value(m.status);
            n = start < 0 || n < 0 ? 0 : (int)a.n;
        }
    }
    // move i (k = keep[i], before = keep[i - 1]): where its entry lies and goes; false where the sequence's moves end
    __device__ __forceinline__ bool request(const KvMove &m, int i, int k, int before, Place &src, Place &dst) const {
        const int64_t place = (int64_t)start + k;
        if (k <= before || k < i || place >= places) {  // (k < i: an earlier one did not ascend)
            flag_value(m.status);
            return false;
        }
        src.request(m, pages, (uint32_t)place);
        dst.request(m, pages, (uint32_t)(start + i));
        return true;
    }
    // their rows; both kNone where nothing moves
    __device__ __forceinline__ void rows(const KvMove &m, const Place &from, const Place &to, uint32_t &src, uint32_t &dst) const {
        src = from.row(m);
        dst = to.row(m);
        if (src == kNone || dst == kNone || src == dst) src = dst = kNone;
    }
};

// Few moves a sequence: a warp per (sequence, layer, head), 16 moves at a time, keys and values
// together.  PIECES: 16-byte pieces of a row of codes.  The accepted paths of 64 trees in 28 layers: 5.5 us (2.5 at a
// copy's rate): one wave of four dependent trips to memory.
template <int PIECES>
__global__ void __launch_bounds__(256) compact_warp_kernel(const __grid_constant__ KvMove m, KvCompactArgs a, int64_t units) {
    constexpr int ROWS = 32 / PIECES, PASSES = 16 / ROWS;  // rows a pass of the warp
    const int lane = threadIdx.x & 31;
    const int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    pdl_launch_dependents();
    pdl_wait();
    if (u >= units) return;
    const uint32_t per = (uint32_t)(m.L * m.Hk);
    const int64_t b = u / per;
    const uint32_t lh = (uint32_t)(u - b * per), layer = lh / (uint32_t)m.Hk;
    const uint32_t head = (lh - layer * (uint32_t)m.Hk) * (uint32_t)m.P;
    const Moves mv(m, a, b);
    uint8_t *const kc = m.kc[layer], *const vc = m.vc[layer];
    float *const ks = m.ks[layer], *const vs = m.vs[layer];
    bool more = true;
    for (int i0 = 0; i0 < mv.n && more; i0 += 16) {
        uint32_t src = kNone, dst = kNone;
        bool ok = true;
        if (lane < 16 && i0 + lane < mv.n) {
            Place from, to;
            ok = mv.request(m, i0 + lane, mv.keep[i0 + lane], i0 + lane > 0 ? mv.keep[i0 + lane - 1] : -1, from, to);
            if (ok) mv.rows(m, from, to, src, dst);
        }
        const uint32_t bad = __ballot_sync(0xffffffffu, !ok);
        if (bad) {  // nothing from the first bad move on
            more = false;
            if (lane >= __ffs(bad) - 1) src = dst = kNone;
        }
        uint4 k[PASSES], v[PASSES];
        int64_t to[PASSES];
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int row = p * ROWS + lane / PIECES;
            const uint32_t s = __shfl_sync(0xffffffffu, src, row), d = __shfl_sync(0xffffffffu, dst, row);
            to[p] = d == kNone ? -1 : ((int64_t)(head + d) * PIECES + lane % PIECES) * 16;
            if (d != kNone) {
                const int64_t from = ((int64_t)(head + s) * PIECES + lane % PIECES) * 16;
                k[p] = *reinterpret_cast<const uint4 *>(kc + from);
                v[p] = *reinterpret_cast<const uint4 *>(vc + from);
            }
        }
        float x = 0.f, y = 0.f;
        if (dst != kNone) x = ks[head + src], y = vs[head + src];
        __syncwarp();
#pragma unroll
        for (int p = 0; p < PASSES; ++p)
            if (to[p] >= 0) {
                *reinterpret_cast<uint4 *>(kc + to[p]) = k[p];
                *reinterpret_cast<uint4 *>(vc + to[p]) = v[p];
            }
        if (dst != kNone) ks[head + dst] = x, vs[head + dst] = y;
        __syncwarp();
    }
}

__device__ __forceinline__ void copy_async(void *dst, const void *src, int bytes) {  // 4 or 16
    const uint32_t d = smem_u32(dst);
    if (bytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(d), "l"(src) : "memory");
}

// Many moves: a block per (sequence, layer, head, keys or values), in groups of 512 x 4 pieces of 16 bytes.  Two groups
// travel to shared memory while a third is written: a thread writes what it copied itself, so the one barrier a
// group says only that all of its reads are done.  Each lane looks up EACH moves of its warp: keep is
// requested two groups before an entry is, the page a group before.
// 8 contexts of 16384 closed up to half in 4 layers (int4): 46 us, 3.5 TB/s of the memory's traffic: the longest
// context's blocks have 16 groups of 2.6 us, bound by what a row costs in instructions and in requests of the
// load-store unit (11 cycles a row and SM), not by the trips, which are hidden.  1024 threads: 43.5, but one block
// to an SM; 256 threads of eight pieces: 50; pieces through registers: 51.
template <int PIECES>
struct CompactSmem {
    static constexpr int WARP = 32 * kPieces / PIECES, EACH = (WARP + 31) / 32;  // moves of a warp; looked up by a lane
    uint4 piece[3][kPieces][kMovers];  // (two blocks of these share an SM)
    float scale[3][EACH][kMovers];
};
template <int PIECES>
__global__ void __launch_bounds__(kMovers) compact_block_kernel(const __grid_constant__ KvMove m, KvCompactArgs a) {
    using Smem = CompactSmem<PIECES>;
    constexpr int EACH = Smem::EACH, WARP = Smem::WARP, ROWS = kMovers / 32 * WARP, STEP = 32 / PIECES;  // ROWS: moves of a group
    extern __shared__ __align__(16) unsigned char raw[];
    Smem &sm = *reinterpret_cast<Smem *>(raw);
    __shared__ int end;
    const uint32_t per = (uint32_t)(m.L * m.Hk) * 2u, tid = threadIdx.x;
    const int lane = tid & 31, w0 = (int)(tid >> 5) * WARP;
    const int64_t u = blockIdx.x, b = u / per;
    pdl_launch_dependents();
    pdl_wait();
    const uint32_t rest = (uint32_t)(u - b * per), lh = rest >> 1, layer = lh / (uint32_t)m.Hk;
    const uint32_t head = (lh - layer * (uint32_t)m.Hk) * (uint32_t)m.P;
    const Moves mv(m, a, b);
    uint8_t *const codes = rest & 1u ? m.vc[layer] : m.kc[layer];
    float *const scales = rest & 1u ? m.vs[layer] : m.ks[layer];
    uint8_t *const mine = codes + lane % PIECES * 16;
    if (tid == 0) end = mv.n;
    __syncthreads();
    int k[EACH], before[EACH];
    uint32_t src[EACH], dst[EACH], to[2][EACH];  // rows, or kNone: of the group looked up, and where those in flight go
    const auto fetch = [&](int i0) {
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            const int i = i0 + w0 + e * 32 + lane;
            if (e * 32 + lane < WARP && i < mv.n) {
                k[e] = mv.keep[i];
                before[e] = i > 0 ? mv.keep[i - 1] : -1;
            }
        }
    };
    Place from[EACH], into[EACH];
    bool good[EACH];
    const auto look = [&](int i0) {  // entries of the page table are requested ..
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            const int i = i0 + w0 + e * 32 + lane;
            good[e] = e * 32 + lane < WARP && i < mv.n;
            if (good[e] && !mv.request(m, i, k[e], before[e], from[e], into[e])) {
                good[e] = false;
                atomicMin(&end, i);
            }
        }
    };
    const auto found = [&] {  // .. and looked at, a group later
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            src[e] = dst[e] = kNone;
            if (good[e]) mv.rows(m, from[e], into[e], src[e], dst[e]);
        }
    };
    const auto request = [&](int stage) {
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const uint32_t s = __shfl_sync(0xffffffffu, src[p * STEP / 32], (p * STEP + lane / PIECES) & 31);
            if (s != kNone) copy_async(&sm.piece[stage][p][tid], mine + (int64_t)(head + s) * (PIECES * 16), 16);
        }
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            if (src[e] != kNone) copy_async(&sm.scale[stage][e][tid], scales + (head + src[e]), 4);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch(0);
    look(0);
    fetch(ROWS);
    found();
    request(0);
#pragma unroll
    for (int e = 0; e < EACH; ++e) to[0][e] = dst[e];
    look(ROWS);
    fetch(2 * ROWS);
    found();
    request(1);
#pragma unroll
    for (int e = 0; e < EACH; ++e) to[1][e] = dst[e];
    look(2 * ROWS);
    fetch(3 * ROWS);
    int stage = 0;
    for (int i0 = 0;; i0 += ROWS) {
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();  // the group is read by all, and its last good move is known:
        if (i0 >= end) break;  // only later groups lower `end` from here on, so all leave the loop together
        found();
        request(stage == 0 ? 2 : stage - 1);
        look(i0 + 3 * ROWS);
        fetch(i0 + 4 * ROWS);
        const int lim = end - i0 - w0;
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const int r = p * STEP + lane / PIECES;
            const uint32_t d = __shfl_sync(0xffffffffu, to[0][p * STEP / 32], r & 31);
            if (d != kNone && r < lim) *reinterpret_cast<uint4 *>(mine + (int64_t)(head + d) * (PIECES * 16)) = sm.piece[stage][p][tid];
        }
#pragma unroll
        for (int e = 0; e < EACH; ++e)
            if (to[0][e] != kNone && e * 32 + lane < lim) scales[head + to[0][e]] = sm.scale[stage][e][tid];
#pragma unroll
        for (int e = 0; e < EACH; ++e) to[0][e] = to[1][e], to[1][e] = dst[e];
        stage = stage == 2 ? 0 : stage + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <int PIECES>
cudaError_t compact(const KvMove &m, const KvCompactArgs &a, int sm_count, cudaStream_t st) {
    // Which form: a warp takes about 1.2 us for 16 moves, more where many warps share the SMs; a block 2.3 us and 6.5 ns a
    // move, two of them for each unit, two on an SM.  Measured (us, warps / blocks; sequences x layers of 4 heads, moves
    // of 128 bytes): 1 x 28, 64: 6.8 / 3.7; 4 x 28, 64: 6.8 / 8.4, 128: 11.1 / 8.7; 16 x 28, 64: 8.6 / 29, 256: 34 / 44, 512:
    // 63 / 62; 64 x 28, 128: 46 / 132; 8 x 4, 128: 11.1 / 3.9.
    const double units_all = (double)a.batch * m.L * m.Hk, share = units_all / sm_count;
    const bool blocks = (share > 1 ? share : 1) * (2.3 + 0.0065 * (double)a.n) < (double)((a.n + 15) / 16) * (1.2 + 0.00075 * units_all);
    static std::atomic<uint64_t> done{0};
    constexpr int bytes = sizeof(CompactSmem<PIECES>);
    if (blocks)
        if (const cudaError_t e = allow_smem(done, compact_block_kernel<PIECES>, bytes)) return e;
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
        if (c.held) c.held += b0;
        const int64_t units = c.batch * per;
        const cudaError_t e = blocks ? launch_chained(compact_block_kernel<PIECES>, (unsigned)(units * 2), kMovers, bytes, 0, st, m, c)
                                     : launch_chained(compact_warp_kernel<PIECES>, (unsigned)((units + 7) / 8), 256, 0, 0, st, m, c, units);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_kv_copy(const KvMove &m, const int *src, const int *dst, const int *tokens, int64_t n, int sm_count, cudaStream_t st) {
    const int64_t per = (int64_t)m.L * m.Hk * 2, chunk = ((int64_t)1 << 31) / per;  // copies of a launch: tasks fit 32 bits
    for (int64_t i0 = 0; i0 < n; i0 += chunk) {
        const int64_t c = n - i0 < chunk ? n - i0 : chunk, blocks = (c * per + 7) / 8, most = (int64_t)sm_count * 8;
        const cudaError_t e = launch_chained(kv_copy_kernel, (unsigned)(blocks < most ? blocks : most), 256, 0, 0, st, m, src + i0, dst + i0,
                                             tokens ? tokens + i0 : nullptr, (uint32_t)c);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_fork_apply(const KvMove &m, const KvPages &g, const int *listed, const ForkItem *items, bool share, int sm_count,
                              cudaStream_t st) {
    const int64_t runs = share ? (g.max_pages + 255) / 256 : 0, blocks = (g.rows * ((int64_t)m.L * m.Hk * 2 + runs) + 7) / 8,
                  most = (int64_t)sm_count * 8;
    return launch_chained(fork_apply_kernel, (unsigned)(blocks < most ? blocks > 0 ? blocks : 1 : most), 256, 0, 0, st, m, g, listed, items,
                          (uint32_t)runs);
}

cudaError_t launch_kv_compact(const KvMove &m, const KvCompactArgs &a, int sm_count, cudaStream_t st) {
    return m.rb == 128  ? compact<8>(m, a, sm_count, st)
           : m.rb == 64 ? compact<4>(m, a, sm_count, st)
                        : compact<2>(m, a, sm_count, st);
}

}  // namespace tl
