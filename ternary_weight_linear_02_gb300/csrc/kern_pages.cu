// kern_pages.cu -- the pages of a pool: giving them back, taking them for the next tokens,
// and for sequences that continue another one.
//
// A page is free where its reference count is 0, so there is no list of free pages to keep: taking
// looks through the counts and gives the lowest-numbered free pages to the rows in order, by prefix
// sums.  Which page a row gets depends on the counts alone, never on timing.
#include "common.cuh"
#include "kernels.h"
#include "launch.h"

namespace tl {

namespace {

constexpr uint32_t kSat = (1u << 30) - 1;  // where page counts saturate
constexpr uint32_t kNeeds = 1u << 31, kBad = 1u << 30;
constexpr int kListed = 4096;  // free pages that a block lists at a time

// One warp per row: the pages behind the kept ones.  Three dependent trips to memory: 3 us for 1021 rows.
__global__ void __launch_bounds__(256) pages_free_kernel(KvPages g, const int *keep, int *status) {
    const int r = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    pdl_launch_dependents();
    pdl_wait();
    if (r >= g.rows) return;
    const int n = keep[r], held = g.held[r];
    if (n < 0) return;
    if (held < 0 || held > g.max_pages || n > (int64_t)held * g.P) {
        if (lane == 0) flag_value(status);
        return;
    }
    const int stay = (int)(((uint32_t)n + (uint32_t)g.P - 1u) / (uint32_t)g.P);
    int *row = g.table + r * g.stride;
    for (int i = stay + lane; i < held; i += 32) {
        const int page = row[i];
        if ((uint32_t)page >= (uint32_t)g.pages) {
            flag_value(status);
        } else if (atomicSub(g.refs + page, 1) <= 0) {
            atomicAdd(g.refs + page, 1);
            flag_value(status);
        }
        row[i] = 0;
    }
    __syncwarp();
    if (lane == 0) {
        g.held[r] = stay;
        g.lens[r] = n;
    }
}

// What a row wants: pages (at most kSat; kBad for a row that cannot be served), the place in its table where
// they go, and the tokens that it has.
struct Want {
    uint32_t need;
    int place, tokens;
};
template <bool FORK>
__device__ __forceinline__ Want want_of(const PagesTakeArgs &a, int r) {
    const KvPages &g = a.g;
    const int w = a.want[r], lens = FORK ? 0 : g.lens[r], held = g.held[r];
    if (w < 0) return {0u, 0, lens};
    if constexpr (FORK) {
        if (w >= g.rows || held != 0) return {kBad, 0, 0};
        const int grand = a.want[w], n = g.lens[w], has = g.held[w];
        if (grand >= 0 || n < 0 || has < 0 || has > g.max_pages || n > (int64_t)has * g.P) return {kBad, 0, 0};
        const uint32_t full = (uint32_t)n / (uint32_t)g.P;
        return {(uint32_t)n > full * (uint32_t)g.P ? 1u : 0u, (int)full, n};
    } else {
        const int64_t most = g.max_pages * g.P;
        if (lens < 0 || held < 0 || held > g.max_pages || lens + (int64_t)w > most) return {kBad, 0, lens};
        const uint32_t P = (uint32_t)g.P, last = (uint32_t)lens / P;
        if (w > 0 && (uint32_t)lens > last * P && last < (uint32_t)held) {  // the next token goes into a page in use
            const int page = g.table[r * g.stride + last];
            if ((uint32_t)page >= (uint32_t)g.pages || g.refs[page] > 1) return {kBad, 0, lens};
        }
        const uint32_t upto = ((uint32_t)lens + (uint32_t)w + P - 1u) / P;
        return {upto > (uint32_t)held ? min(upto - (uint32_t)held, kSat) : 0u, held, lens};
    }
}

__device__ __forceinline__ uint32_t sat(uint32_t x) { return min(x, kSat); }

// Inclusive prefix sum over the block's threads (saturating where SAT), and the total.
template <bool SAT>
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *part, uint32_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v = SAT ? sat(v + u) : v + u;
    }
    __syncthreads();  // part may still be read by the call before
    if (lane == 31) part[warp] = v;
    __syncthreads();
    uint32_t s = lane < (int)(blockDim.x >> 5) ? part[lane] : 0u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s = SAT ? sat(s + u) : s + u;
    }
    total = __shfl_sync(0xffffffffu, s, 31);
    const uint32_t before = __shfl_sync(0xffffffffu, s, (warp + 31) & 31);
    if (warp > 0) v = SAT ? sat(v + before) : v + before;
    return v;
}

// Which of 1024 pages from p0 on are free: lane j holds the word of pages p0 + 32 j ...
__device__ __forceinline__ uint32_t free_words(const int *refs, int64_t p0, int64_t end) {
    const int lane = threadIdx.x & 31;
    const int *const p = refs + p0 + lane;
    const int left = (int)max(min(end - p0, (int64_t)1024), (int64_t)0) - lane;  // pages from the lane's first on
    uint32_t mine = 0;
    int v[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = 32 * j < left ? p[32 * j] : 1;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        const uint32_t w = __ballot_sync(0xffffffffu, v[j] == 0);
        if (lane == j) mine = w;
    }
    return mine;
}

// One cluster of up to 8 blocks (one block up to 32768 pages) serves all rows:
//   free pages counted, each block a run of pages, which needs nothing of the rows;
//   needs of the rows and their running sums (every block for itself, kept in shared memory);
//   the free page of rank k goes to the row whose sum passes k, as far as whole rows are covered;
//   lengths, slots and answers.
// Bound by latency: three dependent loads, the cluster's two barriers, the table's new entries read back for the
// slots.  1021 rows over 200 thousand pages: 13 us, of which
// counting 4, needs 2, the exchange 1.4, giving out 3.3, slots 1.7.  Each lane giving out the pages that it found
// took 38 us: free pages lie together, so one warp had most of them.
template <bool FORK>
__global__ void __launch_bounds__(1024) pages_take_kernel(PagesTakeArgs a) {
    extern __shared__ uint32_t cum[];  // [rows] sums, then places and tokens
    __shared__ uint32_t part[32], counts[8];
    __shared__ uint16_t list[kListed];
    const KvPages &g = a.g;
    const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31, warp = tid >> 5;
    const int C = gridDim.x, rank = blockIdx.x;
    int *const place = reinterpret_cast<int *>(cum) + g.rows, *const tokens = place + g.rows;
    if (C > 1) cluster_arrive_relaxed();
    pdl_launch_dependents();
    pdl_wait();
    const int64_t batch = threads * 32, per = (g.pages + C * 1024 - 1) / (C * 1024) * 1024;
    const int64_t lo = rank * per, hi = min(lo + per, g.pages);
    uint32_t words = 0, free_here = 0;
    for (int64_t p0 = lo; p0 < hi; p0 += batch) {
        words = free_words(g.refs, p0 + warp * 1024, hi);
        free_here += __popc(words);
    }
    uint32_t total = 0;
    for (int r0 = 0; r0 < g.rows; r0 += threads) {
        const int r = r0 + tid;
        const Want w = r < g.rows ? want_of<FORK>(a, r) : Want{0u, 0, 0};
        const bool bad = w.need == kBad;
        if (bad && rank == 0) flag_value(a.status);
        uint32_t sum;
        const uint32_t upto = block_scan<true>(bad ? 0u : w.need, part, sum);
        if (r < g.rows) {
            cum[r] = sat(total + upto) | (bad ? kBad : w.need ? kNeeds : 0u);
            place[r] = w.place;
            tokens[r] = w.tokens;
        }
        total = sat(total + sum);
    }
    uint32_t below = 0, have = 0;
    block_scan<false>(free_here, part, have);
    if (C > 1) {
        cluster_wait();  // every block has started
        if (tid < C) cl_st_u32(cl_map(smem_u32(&counts[rank]), tid), have);
        cl_arrive_release();
        cl_wait_acquire();
        have = 0;
        for (int i = 0; i < C; ++i) {
            if (i == rank) below = have;
            have += counts[i];
        }
    } else {
        __syncthreads();
    }
    if (total > 0) {
        // pages given out: the largest sum of needs that the free pages cover
        uint32_t given = 0;
        {
            int x = 0, y = g.rows;  // rows before x are covered, from y on not
            while (x < y) {
                const int m = (x + y) >> 1;
                if ((cum[m] & kSat) <= have) x = m + 1;
                else y = m;
            }
            if (x > 0) given = cum[x - 1] & kSat;
        }
        for (int64_t p0 = lo; p0 < hi && below < given; p0 += batch) {
            if (per > batch) words = free_words(g.refs, p0 + warp * 1024, hi);
            uint32_t sum;
            const uint32_t n = __popc(words);
            const uint32_t k0 = block_scan<false>(n, part, sum) - n;  // the lane's free pages before its own
            const uint32_t take = min(sum, given - below);
            // the batch's free pages in order, a part of them at a time, then a thread for each
            for (uint32_t a0 = 0; a0 < take; a0 += kListed) {
                uint32_t w = words, k = k0;
                while (w && k < a0 + kListed) {
                    const int bit = __ffs(w) - 1;
                    if (k >= a0) list[k - a0] = (uint16_t)(warp * 1024 + 32 * lane + bit);
                    w &= w - 1u;
                    ++k;
                }
                __syncthreads();
                for (uint32_t i = tid; i < min(take - a0, (uint32_t)kListed); i += threads) {
                    const uint32_t nth = below + a0 + i;
                    int x = 0, y = g.rows - 1;  // the first row whose sum is above nth
                    while (x < y) {
                        const int m = (x + y) >> 1;
                        if ((cum[m] & kSat) > nth) y = m;
                        else x = m + 1;
                    }
                    const uint32_t before = x > 0 ? cum[x - 1] & kSat : 0u;
                    const int page = (int)(p0 + list[i]);
                    g.table[x * g.stride + place[x] + (nth - before)] = page;
                    g.refs[page] = 1;
                }
                __syncthreads();
            }
            below += sum;
        }
    }
    // (whatever the block found: should `want` or the tables change meanwhile, blocks find other totals, and one that
    // skipped the barrier would leave the others waiting)
    if (C > 1) {
        cl_arrive_release();
        cl_wait_acquire();
    }
    const auto served = [&](int r) {
        const uint32_t c = cum[r];
        return !(c & kBad) && (!(c & kNeeds) || (c & kSat) <= have);
    };
    const uint32_t P = (uint32_t)g.P;
    if constexpr (FORK) {
        if (rank != 0) return;
        uint32_t listed = 0;
        for (int r0 = 0; r0 < g.rows; r0 += threads) {
            const int r = r0 + tid;
            const bool in = r < g.rows, ok = in && served(r);
            const int p = in ? a.want[r] : -1;
            const bool forked = ok && p >= 0;
            if (in && a.ok) a.ok[r] = ok;
            uint32_t sum;
            const uint32_t k = listed + block_scan<false>(forked, part, sum) - forked;
            if (forked) {
                const int n = tokens[r], full = place[r], places = n - full * g.P;
                g.lens[r] = n;
                g.held[r] = full + (places > 0);
                ForkItem it{r, p, full, places, -1, -1, 0, 0};
                if (places > 0) {
                    it.src = g.table[p * g.stride + full];
                    it.dst = __ldcg(g.table + r * g.stride + full);  // (written above, by any block of the cluster)
                }
                a.items[k] = it;
            }
            listed += sum;
        }
        if (tid == 0) *a.listed = (int)listed;
    } else {
        for (int r = rank * threads + tid; r < g.rows; r += C * threads) {
            const bool ok = served(r);
            if (a.ok) a.ok[r] = ok;
            if (ok && (cum[r] & kNeeds)) g.held[r] = (int)(((uint32_t)tokens[r] + (uint32_t)a.want[r] + P - 1u) / P);
        }
        if (a.slots == nullptr) return;
        const int64_t all = (int64_t)g.rows * a.width;
        for (int64_t e = rank * threads + tid; e < all; e += C * threads) {
            const int r = all >> 31 ? (int)(e / a.width) : (int)((uint32_t)e / (uint32_t)a.width), i = (int)(e - (int64_t)r * a.width);
            long long s = -1;
            if (served(r) && i < a.want[r]) {
                const uint32_t j = (uint32_t)tokens[r] + (uint32_t)i, p = j / P;
                if (p < (uint64_t)g.max_pages) {  // (holds unless extra changes during the call)
                    const int page = __ldcg(g.table + r * g.stride + p);  // (another block of the cluster may have written it)
                    if ((uint32_t)page < (uint32_t)g.pages) s = (long long)page * g.P + (j - p * P);
                    else flag_value(a.status);
                }
            }
            a.slots[e] = s;
        }
    }
}

}  // namespace

cudaError_t launch_pages_free(const KvPages &g, const int *keep, int *status, cudaStream_t st) {
    return launch_chained(pages_free_kernel, (unsigned)(g.rows + 7) / 8, 256, 0, 0, st, g, keep, status);
}

cudaError_t launch_pages_take(const PagesTakeArgs &a, bool fork, cudaStream_t st) {
    // a block's run of pages is looked through once and kept as bits: up to 32768 of them
    int C = 1;
    while (C < 8 && (int64_t)C * 32768 < a.g.pages) C *= 2;
    // 256 threads for a small server: 16 rows of 1100 pages 9.2 us against 12.5 with 1024, 250 rows 14.1 and 14.4, 1000 rows
    // 30 and 18.6 (freeing before included)
    const int threads = a.g.pages <= 8192 && a.g.rows <= 256 ? 256 : 1024, bytes = a.g.rows * 12;
    static std::atomic<uint64_t> done[2];
    const auto kernel = fork ? pages_take_kernel<true> : pages_take_kernel<false>;
    if (bytes > 32 * 1024)
        if (const cudaError_t e = allow_smem(done[fork], kernel, kMaxPageRows * 12)) return e;
    return launch_chained(kernel, (unsigned)C, (unsigned)threads, (size_t)bytes, (unsigned)C, st, a);
}

}  // namespace tl
