// kern_verify.cu -- drafted tokens checked against the target's probabilities, and the token
// that follows the accepted ones drawn, from given random numbers.
//
// At a node with target row p and drafter's row q the children are looked at in order.  After
// k of them were rejected the target's rest is
//     w_k = max(w_{k-1} - W_{k-1} q, 0),  W_k = sum w_k,  w_0 = p, W_0 = 1
// (each w normalised by its sum, less q).  Where an inner maximum is 0 the outer one is too, so
//     w_k = max(p - A_k q, 0),  A_k = W_0 + .. + W_{k-1}:
// a rejection costs one pass over p and q with one number to remember, and the last pass's sums
// serve the drawing too.  Without q (a drafter that gives tokens only) w is p without the rejected
// tokens.
//
// Which token a random number falls on hangs on sums of a whole vocabulary, next to whose borders fp32
// says nothing (an error of 1e-7 moves one draw in a hundred at 130000 tokens).  Sums are
// therefore kept as pairs of fp32 (an error-free sum and what it lost: about 47 bits; GB300 adds fp64
// at 1/64 of the rate), decisions are made in fp64.
#include "common.cuh"
#include "kernels.h"

namespace tl {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kMaxBlocks = 8;

struct Pair {
    float hi, lo;
    __device__ __forceinline__ double d() const { return (double)hi + (double)lo; }
};
// a + b and what its rounding lost (D. E. Knuth, The Art of Computer Programming 2, 4.2.2)
__device__ __forceinline__ Pair two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
    const Pair s = two_sum(a.hi, b.hi);
    const float e = __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)), h = __fadd_rn(s.hi, e);
    return {h, __fsub_rn(e, __fsub_rn(h, s.hi))};
}
__device__ __forceinline__ Pair shfl_up(Pair a, int o) {
    return {__shfl_up_sync(0xffffffffu, a.hi, o), __shfl_up_sync(0xffffffffu, a.lo, o)};
}
__device__ __forceinline__ Pair warp_total(Pair a) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        a = add(a, Pair{__shfl_xor_sync(0xffffffffu, a.hi, o), __shfl_xor_sync(0xffffffffu, a.lo, o)});
    return a;
}

template <typename T>
__device__ __forceinline__ float value(T x);
template <>
__device__ __forceinline__ float value<float>(float x) { return x; }
template <>
__device__ __forceinline__ float value<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float value<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
// what is below 0 or not a number counts as 0
template <typename T>
__device__ __forceinline__ float prob(T x) { return fmaxf(value(x), 0.f); }

// The weights that the next token is drawn from: w = max(p - A q, 0) (q: nullptr where nothing
// was rejected), without the first `gone` tokens of the list.
template <typename T>
struct Weights {
    const T *p, *q;
    float ah, al;  // A
    int gone;
    const int *list;
    __device__ __forceinline__ Pair of(float p, float q) const {
        const float t = __fmul_rn(ah, q), te = __fmaf_rn(al, q, __fmaf_rn(ah, q, -t));
        Pair d = two_sum(p, -t);
        d.lo = __fsub_rn(d.lo, te);
        return __fadd_rn(d.hi, d.lo) > 0.f ? d : Pair{0.f, 0.f};
    }
    __device__ __forceinline__ bool removed(int v) const {
        for (int i = 0; i < gone; ++i)
            if (list[i] == v) return true;
        return false;
    }
    __device__ __forceinline__ Pair at(int v) const {
        if (removed(v)) return {0.f, 0.f};
        return q ? of(prob(p[v]), prob(q[v])) : Pair{prob(p[v]), 0.f};
    }
};

template <typename T>
__device__ __forceinline__ void load16(const T *p, float (&v)[16 / sizeof(T)]) {
    const uint4 r = ldg_nc_v4(p);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = fmaxf(__uint_as_float(w[i]), 0.f);
    } else {
        const T *h = reinterpret_cast<const T *>(w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = prob(h[i]);
    }
}

// Sum of the weights of tokens [lo, hi), taken by one warp.  VEC: lo is a multiple of 8 and rows
// start on 16-byte boundaries.
template <typename T, bool VEC>
__device__ __forceinline__ Pair sum_run(const Weights<T> &w, int lo, int hi) {
    const int lane = threadIdx.x & 31;
    Pair acc{0.f, 0.f};
    const auto take = [&](Pair x) {
        const Pair s = two_sum(acc.hi, x.hi);
        acc = {s.hi, __fadd_rn(acc.lo, __fadd_rn(s.lo, x.lo))};
    };
    if constexpr (VEC) {
        constexpr int W = 16 / sizeof(T), U = sizeof(T) == 4 ? 4 : 2;  // elements a load, loads in flight
        int v = lo + lane * W;
        for (; v + (U - 1) * 32 * W + W <= hi; v += U * 32 * W) {
            float p[U][W], q[U][W];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                load16(w.p + v + u * 32 * W, p[u]);
                if (w.q) load16(w.q + v + u * 32 * W, q[u]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                for (int i = 0; i < w.gone; ++i) {
                    const unsigned at = (unsigned)(w.list[i] - (v + u * 32 * W));
#pragma unroll
                    for (int e = 0; e < W; ++e)
                        if (at == (unsigned)e) p[u][e] = 0.f;
                }
#pragma unroll
                for (int e = 0; e < W; ++e) take(w.q ? w.of(p[u][e], q[u][e]) : Pair{p[u][e], 0.f});
            }
        }
        for (; v < hi; v += 32 * W)
            for (int e = 0; e < W && v + e < hi; ++e) take(w.at(v + e));
    } else {
        constexpr int U = 8;
        int v = lo + lane;
        for (; v + (U - 1) * 32 < hi; v += U * 32) {
            float p[U], q[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                p[u] = prob(w.p[v + u * 32]);
                q[u] = w.q ? prob(w.q[v + u * 32]) : 0.f;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (w.gone && w.removed(v + u * 32)) p[u] = 0.f;
                take(w.q ? w.of(p[u], q[u]) : Pair{p[u], 0.f});
            }
        }
        for (; v < hi; v += 32) take(w.at(v));
    }
    // acc.lo may be as large as acc.hi's last bits; the pairs' sum puts that right
    return warp_total(add(Pair{0.f, 0.f}, acc));
}

// One cluster of C blocks per sequence; block r holds tokens [r per, (r + 1) per), warp w of it a run
// of them.  Every block follows the accepted path by itself (the entries that it turns on
// are gathered first); sums are exchanged through distributed shared memory.
// Bound by latency: the gather (two dependent loads), a pass, the cluster's barrier, the drawing.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) verify_kernel(VerifyArgs a) {
    __shared__ float px[kMaxDraft], qx[kMaxDraft], un[kMaxDraft + 1];
    __shared__ int tok[kMaxDraft], par[kMaxDraft], path[kMaxDraft], gone[kMaxDraft];
    __shared__ Pair warp_sum[kWarps], part[kWarps], block_sum[2][kMaxBlocks];
    __shared__ struct {
        int todo;  // 0: a pass over p, 1: over p and q, 2: done
        int node, count, gone, next;
        double A, W;
    } st;
    __shared__ int found;
    const int C = (int)a.blocks, rank = (int)(blockIdx.x % (unsigned)C), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t b = blockIdx.x / (unsigned)C;
    const int n = a.T, V = a.V;
    const T *target = static_cast<const T *>(a.target) + b * a.target_b;
    const T *draft = a.draft ? static_cast<const T *>(a.draft) + b * a.draft_b : nullptr;
    if (C > 1) cluster_arrive_relaxed();
    for (int i = tid; i <= n; i += kThreads) {
        un[i] = a.uniform[b * a.uniform_b + i];
        if (i == n) break;
        const int64_t x = a.tokens[b * a.tokens_b + i];
        const int at = a.parent ? a.parent[b * a.parent_b + i] : i - 1;
        const bool ok = x >= 0 && x < V && at >= -1 && at < i;
        if (!ok && rank == 0) flag_value(a.status);
        tok[i] = (int)x;
        par[i] = ok ? at : -2;
        px[i] = ok ? prob(target[(at + 1) * a.target_n + x]) : 0.f;
        qx[i] = ok && draft ? prob(draft[(at + 1) * a.draft_n + x]) : 1.f;
    }
    if (tid == 0) {
        st.node = st.count = st.gone = st.next = 0;
        st.A = 0.;
        st.W = 1.;
    }
    // tokens of this block, and of each of its warps
    const int per = (((V + C - 1) / C) + 255) & ~255, lo = min(V, rank * per), hi = min(V, lo + per);
    const int run = (((hi - lo + kWarps - 1) / kWarps) + 7) & ~7;
    __syncthreads();
    if (C > 1) cluster_wait();  // every block has started
    Weights<T> w;
    w.list = gone;
    int buf = 0;
    double before = 0., all = 0.;  // sums of the blocks before this one, and of all
    const auto pass = [&] {
        const int l = min(hi, lo + warp * run), h = min(hi, l + run);
        const Pair s = sum_run<T, VEC>(w, l, h);
        if (lane == 0) warp_sum[warp] = s;
        __syncthreads();
        Pair mine{0.f, 0.f};
        for (int i = 0; i < kWarps; ++i) mine = add(mine, warp_sum[i]);
        if (C > 1) {
            if (tid < C) {
                const uint32_t at = cl_map(smem_u32(&block_sum[buf][rank]), tid);
                cl_st_f32(at, mine.hi);
                cl_st_f32(at + 4, mine.lo);
            }
            cl_arrive_release();
            cl_wait_acquire();
        } else {
            if (tid == 0) block_sum[buf][0] = mine;
            __syncthreads();
        }
        all = 0.;
        for (int i = 0; i < C; ++i) {
            if (i == rank) before = all;
            all += block_sum[buf][i].d();
        }
        buf ^= 1;  // (a block writes a buffer again only after all have passed the next barrier)
    };
    for (bool summed = false;; summed = true) {
        if (warp == 0) {  // on along the tokens, until sums are needed
            int node = st.node, count = st.count, ngone = st.gone, i = st.next, todo = -1;
            double A = st.A, W = summed ? all : st.W;
            while (todo < 0) {
                // the next child of this node
                if (a.parent) {
                    int at = n;
                    for (int j = i; j < n; j += 32) {
                        const uint32_t hit = __ballot_sync(0xffffffffu, j + lane < n && par[min(j + lane, n - 1)] == node - 1);
                        if (hit) {
                            at = j + __ffs(hit) - 1;
                            break;
                        }
                    }
                    i = at;
                } else {
                    while (i < n && par[i] != node - 1) ++i;
                }
                if (i >= n) {
                    todo = 2;
                    break;
                }
                const int x = tok[i];
                double p = (double)px[i];
                const double q = (double)qx[i];
                if (draft) {
                    p = fmax(p - A * q, 0.);
                } else {
                    for (int j = 0; j < ngone; ++j)
                        if (gone[j] == x) p = 0.;
                }
                if ((double)un[i] * (W * q) < p) {
                    if (lane == 0) path[count] = i;
                    ++count;
                    node = i + 1;
                    A = 0.;
                    W = 1.;
                    ngone = 0;
                } else if (draft) {
                    A += W;
                    todo = 1;
                } else {
                    W -= p;
                    if (lane == 0) gone[ngone] = x;
                    ++ngone;
                    __syncwarp();
                }
                ++i;
            }
            // at the end: sums of the last pass serve if they are this node's
            if (lane == 0) {
                st.node = node;
                st.count = count;
                st.gone = ngone;
                st.next = i;
                st.A = A;
                st.W = W;
                st.todo = todo == 2 && A == 0. ? 0 : todo;
            }
        }
        __syncthreads();
        const int todo = st.todo;
        if (todo == 2) break;  // (w and its sums are those of the pass before)
        w.p = target + (int64_t)st.node * a.target_n;
        w.q = todo == 1 ? draft + (int64_t)st.node * a.draft_n : nullptr;
        w.ah = (float)st.A;
        w.al = (float)(st.A - (double)w.ah);
        w.gone = st.gone;
        pass();
        if (todo == 0) break;
        __syncthreads();  // st is read by all before it changes
    }
    if (!(all > 0.) && (w.q || w.gone)) {  // nothing is left: the target's own row
        w.q = nullptr;
        w.gone = 0;
        pass();
    }
    if (rank == 0) {
        const int count = st.count;
        for (int i = tid; i < n; i += kThreads) a.path[b * n + i] = i < count ? path[i] : -1;
        for (int i = tid; i <= n; i += kThreads)
            if (i != count) a.out[b * (n + 1) + i] = i < count ? tok[path[i]] : -1;
        if (tid == 0) {
            a.count[b] = count;
            if (!(all > 0.)) {
                a.out[b * (n + 1) + count] = -1;
                flag_value(a.status);
            }
        }
    }
    if (!(all > 0.)) return;
    // the block whose tokens the number falls on: the first whose sum with those before passes it, else
    // (the number is not below 1) the last that has any
    const double t = (double)un[n] * all;
    int owner = -1;
    {
        double c = 0.;
        int last = 0;
        for (int i = 0; i < C; ++i) {
            const double s = block_sum[buf ^ 1][i].d();
            c += s;
            if (s > 0.) last = i;
            if (owner < 0 && s > 0. && c > t) owner = i;
        }
        if (owner < 0) owner = last;
    }
    if (owner != rank) return;
    // and the warp's run within it
    int which = -1, last = 0;
    Pair c{0.f, 0.f}, start{0.f, 0.f};
    for (int i = 0; i < kWarps; ++i) {
        const Pair s = warp_sum[i];
        const Pair next = add(c, s);
        if (s.hi > 0.f && which < 0 && (before + next.d() > t)) {
            which = i;
            start = c;
        }
        if (s.hi > 0.f) last = i;
        c = next;
    }
    if (which < 0) {
        which = last;
        start = Pair{0.f, 0.f};
        for (int i = 0; i < last; ++i) start = add(start, warp_sum[i]);
    }
    const double from = before + start.d();
    const int l = min(hi, lo + which * run), h = min(hi, l + run), each = (h - l + kThreads - 1) / kThreads;
    const int v0 = min(h, l + tid * each), v1 = min(h, v0 + each);
    Pair s{0.f, 0.f};
    for (int v = v0; v < v1; ++v) s = add(s, w.at(v));
    Pair upto = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Pair u = shfl_up(upto, o);
        if (lane >= o) upto = add(upto, u);
    }
    if (lane == 31) part[warp] = upto;
    if (tid == 0) found = -1;
    __syncthreads();
    Pair ahead{0.f, 0.f};
    for (int i = 0; i < warp; ++i) ahead = add(ahead, part[i]);
    const Pair prev = shfl_up(upto, 1);
    const Pair mine = lane > 0 ? add(ahead, prev) : ahead;  // of the threads before this one
    // the first thread whose tokens pass the number, else the last that has any: candidates compete
    // with the former ahead of the latter
    const bool any = s.hi > 0.f, passes = any && from + add(mine, s).d() > t;
    if (any) atomicMax(&found, passes ? 2 * kThreads - tid : tid);
    __syncthreads();
    if (!any || found != (passes ? 2 * kThreads - tid : tid)) return;
    double sum = from + mine.d();
    int v = -1;
    for (int i = v0; i < v1; ++i) {
        const double x = w.at(i).d();
        if (!(x > 0.)) continue;
        v = i;
        sum += x;
        if (sum > t) break;
    }
    a.out[b * (n + 1) + st.count] = v;
}

template <typename T>
cudaError_t launch_t(const VerifyArgs &a, bool vec, cudaStream_t st) {
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)(a.B * a.blocks));
    c.blockDim = dim3(kThreads);
    c.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)a.blocks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    c.attrs = at;
    c.numAttrs = 1;
    return vec ? cudaLaunchKernelEx(&c, verify_kernel<T, true>, a) : cudaLaunchKernelEx(&c, verify_kernel<T, false>, a);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs &args, int dtype, bool vec, cudaStream_t st) {
    VerifyArgs a = args;
    a.blocks = 1;
    while (a.blocks < kMaxBlocks && a.V > 4096 * a.blocks) a.blocks *= 2;
    return dtype == 0 ? launch_t<__half>(a, vec, st) : dtype == 1 ? launch_t<__nv_bfloat16>(a, vec, st) : launch_t<float>(a, vec, st);
}

}  // namespace tl
