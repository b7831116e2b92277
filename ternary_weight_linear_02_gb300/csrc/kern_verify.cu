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
// therefore kept as pairs of fp32 (an error-free sum and what it lost: within (V + 2^15) 2^-55 of the
// sum if all roundings fell to one side, 2^-44 as they come; GB300 adds fp64 at 1/64 of the rate),
// decisions are made in fp64.
#include "common.cuh"
#include "kernels.h"
#include "launch.h"

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
__device__ __forceinline__ bool above(Pair a, Pair b) { return add(a, Pair{-b.hi, -b.lo}).hi > 0.f; }
__device__ __forceinline__ Pair pair_of(double x) {
    const float h = (float)x;
    return {h, (float)(x - (double)h)};
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
    // a thread's own entries of the rows, kept in shared memory while a node's children are rejected one by one:
    // 0 not kept, 1 to be kept, 2 there
    uint4 *kept;
    int keep, threads;
    __device__ __forceinline__ uint4 &slot(int i) const { return kept[i * threads + (int)threadIdx.x]; }
    __device__ __forceinline__ Pair of(float p, float q) const {
        const float t = __fmul_rn(ah, q), te = __fmaf_rn(al, q, __fmaf_rn(ah, q, -t));
        // p - t and what its rounding lost: exact where p >= t, and where they are near each other; else w is 0
        const float d = __fsub_rn(p, t), e = __fsub_rn(__fsub_rn(__fsub_rn(p, d), t), te);
        return __fadd_rn(d, e) > 0.f ? Pair{d, e} : Pair{0.f, 0.f};
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
__device__ __forceinline__ void values16(uint4 r, float (&v)[16 / sizeof(T)]) {
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
// start on 16-byte boundaries.  The last, partly filled step is read under a mask like the others: a loop of
// single loads would wait for each.
// A lane's V / 2048 entries (up to 16 below 32768 tokens) go into one pair, in whose lo the lost parts are added in plain
// fp32.  Every W of them (8 without VEC) lo is brought back below half a unit of hi, so that an addition loses (W + 2) 2^-48 of
// the sum at most; left to grow, lo lost a 2^-49 n^2 of it after n (2^-29 at 2^22 tokens, one large among many small).
template <typename T, bool VEC>
__device__ __forceinline__ Pair sum_run(const Weights<T> &w, int lo, int hi) {
    const int lane = threadIdx.x & 31;
    Pair acc{0.f, 0.f};
    const auto take = [&](Pair x) {
        const Pair s = two_sum(acc.hi, x.hi);
        acc = {s.hi, __fadd_rn(acc.lo, __fadd_rn(s.lo, x.lo))};
    };
    const auto settle = [&] {
        const float h = __fadd_rn(acc.hi, acc.lo);
        acc = {h, __fsub_rn(acc.lo, __fsub_rn(h, acc.hi))};
    };
    if constexpr (VEC) {
        // two steps of U loads in flight: one travels while the other is added
        constexpr int W = 16 / sizeof(T), U = sizeof(T) == 4 ? 2 : 1, STEP = U * 32 * W;
        const int whole = lo + (hi - lo) / W * W;
        uint4 p[2][U], q[2][U];
        const auto request = [&](int v, uint4 (&x)[U], uint4 (&y)[U]) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool in = v + u * 32 * W < whole;
                const int at = 2 * ((v + u * 32 * W - lo) / (32 * W));
                x[u] = y[u] = make_uint4(0, 0, 0, 0);
                if (in && w.keep == 2) {
                    x[u] = w.slot(at);
                    y[u] = w.slot(at + 1);
                } else {
                    if (in) x[u] = ldg_nc_v4(w.p + v + u * 32 * W);
                    if (in && w.q) y[u] = ldg_nc_v4(w.q + v + u * 32 * W);
                }
            }
        };
        const auto add_up = [&](int v, const uint4 (&x)[U], const uint4 (&y)[U]) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (w.keep == 1 && v + u * 32 * W < whole) {
                    const int at = 2 * ((v + u * 32 * W - lo) / (32 * W));
                    w.slot(at) = x[u];
                    w.slot(at + 1) = y[u];
                }
                float pv[W], qv[W];
                values16<T>(x[u], pv);
                values16<T>(y[u], qv);
                for (int i = 0; i < w.gone; ++i) {
                    const unsigned at = (unsigned)(w.list[i] - (v + u * 32 * W));
#pragma unroll
                    for (int e = 0; e < W; ++e)
                        if (at == (unsigned)e) pv[e] = 0.f;
                }
#pragma unroll
                for (int e = 0; e < W; ++e) take(w.q ? w.of(pv[e], qv[e]) : Pair{pv[e], 0.f});
                settle();
            }
        };
        int v = lo + lane * W;
        request(v, p[0], q[0]);
        request(v + STEP, p[1], q[1]);
        for (; v < whole; v += 2 * STEP) {
            add_up(v, p[0], q[0]);
            request(v + 2 * STEP, p[0], q[0]);
            add_up(v + STEP, p[1], q[1]);
            request(v + 3 * STEP, p[1], q[1]);
        }
        if (whole + lane < hi) take(w.at(whole + lane));
    } else {
        constexpr int U = 8;  // (a slot holds two tokens)
        for (int v = lo + lane; v < hi; v += U * 32) {
            float p[U], q[U];
            const int at = (v - lo) / (32 * 2);
            if (w.keep == 2) {
#pragma unroll
                for (int u = 0; u < U; u += 2) {
                    const uint4 s = w.slot(at + u / 2);
                    p[u] = __uint_as_float(s.x), q[u] = __uint_as_float(s.y), p[u + 1] = __uint_as_float(s.z), q[u + 1] = __uint_as_float(s.w);
                }
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const bool in = v + u * 32 < hi;
                    p[u] = in ? prob(w.p[v + u * 32]) : 0.f;
                    q[u] = in && w.q ? prob(w.q[v + u * 32]) : 0.f;
                }
                if (w.keep == 1) {
#pragma unroll
                    for (int u = 0; u < U; u += 2)
                        w.slot(at + u / 2) =
                            make_uint4(__float_as_uint(p[u]), __float_as_uint(q[u]), __float_as_uint(p[u + 1]), __float_as_uint(q[u + 1]));
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (w.gone && w.removed(v + u * 32)) p[u] = 0.f;
                take(w.q ? w.of(p[u], q[u]) : Pair{p[u], 0.f});
            }
            settle();
        }
    }
    // acc.lo may be as large as acc.hi's last bits; the pairs' sum puts that right
    return warp_total(add(Pair{0.f, 0.f}, acc));
}

// Weights of tokens [v0, v1), at most N of them (0 beyond), by one thread.
template <typename T, bool VEC, int N>
__device__ __forceinline__ void weights_at(const Weights<T> &w, int v0, int v1, Pair (&x)[N]) {
    float p[N], q[N];
    constexpr int W = 16 / sizeof(T);
    if (VEC && v0 % W == 0 && v1 - v0 == N) {
#pragma unroll
        for (int i = 0; i < N; i += W) {
            float r[W];
            values16<T>(ldg_nc_v4(w.p + v0 + i), r);
#pragma unroll
            for (int e = 0; e < W; ++e) p[i + e] = r[e];
            if (w.q) {
                values16<T>(ldg_nc_v4(w.q + v0 + i), r);
#pragma unroll
                for (int e = 0; e < W; ++e) q[i + e] = r[e];
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            p[i] = v0 + i < v1 ? prob(w.p[v0 + i]) : 0.f;
            q[i] = v0 + i < v1 && w.q ? prob(w.q[v0 + i]) : 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (w.gone && w.removed(v0 + i)) p[i] = 0.f;
        x[i] = w.q ? w.of(p[i], q[i]) : Pair{p[i], 0.f};
    }
}

// One cluster of C blocks per sequence; block r holds tokens [r per, (r + 1) per), warp w of it a run
// of them.  Every block follows the accepted path by itself: the entries that it turns on are gathered and given to
// all first, sums are exchanged through distributed shared memory.
// Bound by latency: the gather (two dependent loads), a pass, the cluster's barrier, the drawing.  One chain of 4 over
// 32000 tokens 9.0 us (launch and gather 2, pass 3, exchange 1.6, drawing 2), 64 chains over 131072 tokens 22 us
// (67 MB: 9.9 at a copy's rate; the pass takes 10), 24 trees of 31 over 50021 tokens 41 us (the longest has
// ten rejections, one pass each).
// fp64 is left to one warp, and to one step per drafted token: at its rate here each operation of a
// warp takes the SM's unit 16 cycles.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, 4) verify_kernel(VerifyArgs a) {
    __shared__ float px[kMaxDraft], qx[kMaxDraft], un[kMaxDraft + 1];
    __shared__ int tok[kMaxDraft], par[kMaxDraft], path[kMaxDraft], gone[kMaxDraft];
    __shared__ Pair warp_sum[kWarps], part[kWarps], block_sum[2][kMaxBlocks];
    __shared__ struct {
        int todo;  // 0: a pass over p, 1: over p and q, 2: done
        int node, count, gone, next;
        double A, W;
        Pair a;  // A (made once: fp64 in every warp would hold the pass up)
    } st;
    __shared__ struct {
        int empty, owner, run;  // nothing to draw from; block and warp's run that the number falls in
        Pair rest;              // what is left of it there
    } fin;
    __shared__ int found;
    const int C = (int)a.blocks, rank = (int)(blockIdx.x % (unsigned)C), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t b = blockIdx.x / (unsigned)C;
    const int n = a.T, V = a.V;
    const T *target = static_cast<const T *>(a.target) + b * a.target_b;
    const T *draft = a.draft ? static_cast<const T *>(a.draft) + b * a.draft_b : nullptr;
    if (C > 1) cluster_arrive_relaxed();
    pdl_launch_dependents();
    pdl_wait();
    // entry i is looked up by one block and given to all (a thread for each of them): whatever happens to the inputs
    // meanwhile, all blocks take the same decisions and meet at the same barriers
    for (int e0 = 0; e0 * C + rank <= n; e0 += kThreads / C) {
        const int i = (e0 + tid / C) * C + rank, to = tid % C;
        float u = 0.f, p = 0.f, q = 1.f;
        int64_t x = 0;
        int up = -4;  // (parent, accepted as its node's first child)
        if (i <= n) u = a.uniform[b * a.uniform_b + i];
        if (i < n) {
            x = a.tokens[b * a.tokens_b + i];
            const int at = a.parent ? a.parent[b * a.parent_b + i] : i - 1;
            if (x >= 0 && x < V && at >= -1 && at < i) {
                p = prob(target[(at + 1) * a.target_n + x]);
                if (draft) q = prob(draft[(at + 1) * a.draft_n + x]);
                up = at * 2 + ((double)u * (double)q < (double)p ? 1 : 0);  // (the product of two fp32 is exact)
            } else if (to == 0) {
                flag_value(a.status);
            }
        }
        if (C > 1 && e0 == 0) cluster_wait();  // every block has started
        if (i > n) continue;
        if (C > 1) {
            cl_st_f32(cl_map(smem_u32(&un[i]), to), u);
            if (i == n) continue;
            cl_st_f32(cl_map(smem_u32(&px[i]), to), p);
            cl_st_f32(cl_map(smem_u32(&qx[i]), to), q);
            cl_st_u32(cl_map(smem_u32(&tok[i]), to), (uint32_t)x);
            cl_st_u32(cl_map(smem_u32(&par[i]), to), (uint32_t)up);
        } else {
            un[i] = u;
            if (i == n) continue;
            px[i] = p;
            qx[i] = q;
            tok[i] = (int)x;
            par[i] = up;
        }
    }
    if (C > 1 && rank > n) cluster_wait();  // (no entry was this block's)
    if (tid == 0) {
        st.node = st.count = st.gone = st.next = 0;
        st.A = 0.;
        st.W = 1.;
    }
    // tokens of this block, and of each of its warps
    const int per = (((V + C - 1) / C) + 255) & ~255, lo = min(V, rank * per), hi = min(V, lo + per);
    const int run = (((hi - lo + kWarps - 1) / kWarps) + 7) & ~7;
    if (C > 1) {
        cl_arrive_release();
        cl_wait_acquire();
    } else {
        __syncthreads();
    }
    extern __shared__ uint4 kept[];
    Weights<T> w;
    w.list = gone;
    w.kept = kept;
    w.threads = kThreads;
    w.keep = 0;
    int kept_node = -1;
    int buf = 0;
    double all = 0., upto = 0.;  // warp 0: the sum, and (lane i) the sum of blocks 0 .. i
    const auto pass = [&] {
        const int l = min(hi, lo + warp * run), h = min(hi, l + run);
        const Pair s = sum_run<T, VEC>(w, l, h);
        if (lane == 0) warp_sum[warp] = s;
        __syncthreads();
        if (warp == 0) {
            Pair mine = lane < kWarps ? warp_sum[lane] : Pair{0.f, 0.f};
#pragma unroll
            for (int o = kWarps / 2; o > 0; o >>= 1)
                mine = add(mine, Pair{__shfl_xor_sync(0xffffffffu, mine.hi, o), __shfl_xor_sync(0xffffffffu, mine.lo, o)});
            if (C > 1) {
                if (lane < C) {
                    const uint32_t at = cl_map(smem_u32(&block_sum[buf][rank]), lane);
                    cl_st_f32(at, mine.hi);
                    cl_st_f32(at + 4, mine.lo);
                }
                __syncwarp();
            } else if (lane == 0) {
                block_sum[buf][0] = mine;
            }
        }
        if (C > 1) {
            cl_arrive_release();
            cl_wait_acquire();
        } else {
            __syncthreads();
        }
        if (warp == 0) {
            upto = lane < C ? block_sum[buf][lane].d() : 0.;
#pragma unroll
            for (int o = 1; o < kMaxBlocks; o <<= 1) {
                const double u = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o && lane < C) upto += u;
            }
            all = __shfl_sync(0xffffffffu, upto, C - 1);
        }
        buf ^= 1;  // (a block writes a buffer again only after all have passed the next barrier)
    };
    for (bool summed = false;; summed = true) {
        if (warp == 0) {  // on along the tokens, until sums are needed
            int node = st.node, count = st.count, ngone = st.gone, i = st.next, todo = -1;
            double A = st.A, W = summed ? all : st.W;
            bool first = !summed;  // no child of this node was rejected
            while (todo < 0) {
                // the next child of this node
                if (a.parent) {
                    int at = n;
                    for (int j = i; j < n; j += 32) {
                        const uint32_t hit = __ballot_sync(0xffffffffu, j + lane < n && par[min(j + lane, n - 1)] >> 1 == node - 1);
                        if (hit) {
                            at = j + __ffs(hit) - 1;
                            break;
                        }
                    }
                    i = at;
                } else if (i < n && par[i] >> 1 != node - 1) {  // (a chain's node has one child)
                    i = n;
                }
                if (i >= n) {
                    todo = 2;
                    break;
                }
                const int x = tok[i];
                bool yes;
                double p = 0.;
                if (first) {
                    yes = par[i] & 1;
                    if (!yes && !draft) p = (double)px[i];
                } else {
                    p = (double)px[i];
                    if (draft) {
                        p = fmax(p - A * (double)qx[i], 0.);
                    } else {
                        for (int j = 0; j < ngone; ++j)
                            if (gone[j] == x) p = 0.;
                    }
                    yes = W * ((double)un[i] * (double)qx[i]) < p;  // (the product of two fp32 is exact)
                }
                if (yes) {
                    if (lane == 0) path[count] = i;
                    ++count;
                    node = i + 1;
                    A = 0.;
                    W = 1.;
                    ngone = 0;
                    first = true;
                } else if (draft) {
                    A += W;
                    todo = 1;
                } else {
                    W -= p;
                    if (lane == 0) gone[ngone] = x;
                    ++ngone;
                    first = false;
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
                if (todo == 1) st.a = pair_of(A);
                st.todo = todo == 2 && A == 0. ? 0 : todo;
            }
        }
        __syncthreads();
        const int todo = st.todo;
        if (todo == 2) break;  // (w and its sums are those of the pass before)
        w.p = target + (int64_t)st.node * a.target_n;
        w.q = todo == 1 ? draft + (int64_t)st.node * a.draft_n : nullptr;
        w.ah = st.a.hi;
        w.al = st.a.lo;
        w.gone = st.gone;
        w.keep = todo == 0 || !a.keep ? 0 : kept_node == st.node ? 2 : 1;
        if (w.keep) kept_node = st.node;
        pass();
        if (todo == 0) break;
        __syncthreads();  // st is read by all before it changes
    }
    for (bool again = false;; again = true) {
        if (warp == 0) {
            // the block whose tokens the number falls on: the first whose sum with those before passes it, else
            // (the number is not below 1) the last that has any; and the warp's run within it
            const Pair mine = lane < C ? block_sum[buf ^ 1][lane] : Pair{0.f, 0.f};
            const uint32_t some = __ballot_sync(0xffffffffu, mine.hi > 0.f);
            const double t = (double)un[n] * all;
            const uint32_t hit = __ballot_sync(0xffffffffu, mine.hi > 0.f && upto > t);
            const int owner = hit ? __ffs(hit) - 1 : 31 - __clz(some | 1u);
            double ahead = __shfl_sync(0xffffffffu, upto, max(owner - 1, 0));
            if (owner == 0) ahead = 0.;
            const Pair ws = lane < kWarps ? warp_sum[lane] : Pair{0.f, 0.f};
            Pair c = ws;
#pragma unroll
            for (int o = 1; o < kWarps; o <<= 1) {
                const Pair u = shfl_up(c, o);
                if (lane >= o) c = add(c, u);
            }
            const Pair rest = pair_of(t - ahead);
            const uint32_t any = __ballot_sync(0xffffffffu, ws.hi > 0.f);
            const uint32_t pass_it = __ballot_sync(0xffffffffu, ws.hi > 0.f && above(c, rest));
            const int r = pass_it ? __ffs(pass_it) - 1 : 31 - __clz(any | 1u);
            Pair start{__shfl_sync(0xffffffffu, c.hi, max(r - 1, 0)), __shfl_sync(0xffffffffu, c.lo, max(r - 1, 0))};
            if (r == 0) start = Pair{0.f, 0.f};
            if (lane == 0) {
                fin.empty = !(all > 0.);
                fin.owner = owner;
                fin.run = r;
                fin.rest = add(rest, Pair{-start.hi, -start.lo});
            }
        }
        if (tid == 0) found = -1;
        __syncthreads();
        if (again || !fin.empty || !(w.q || w.gone)) break;
        w.q = nullptr;  // nothing is left: the target's own row
        w.gone = w.keep = 0;
        pass();
        __syncthreads();
    }
    const int count = st.count;
    if (rank == 0) {
        for (int i = tid; i < n; i += kThreads) a.path[b * n + i] = i < count ? path[i] : -1;
        for (int i = tid; i <= n; i += kThreads)
            if (i != count) a.out[b * (n + 1) + i] = i < count ? tok[path[i]] : -1;
        if (tid == 0) {
            a.count[b] = count;
            if (fin.empty) {
                a.out[b * (n + 1) + count] = -1;
                flag_value(a.status);
            }
        }
    }
    if (fin.empty || fin.owner != rank) return;
    // the run's tokens dealt to the threads, neighbours to each
    const Pair rest = fin.rest;
    const int l = min(hi, lo + fin.run * run), h = min(hi, l + run), each = (((h - l + kThreads - 1) / kThreads) + 7) & ~7;
    const int v0 = min(h, l + tid * each), v1 = min(h, v0 + each);
    Pair s{0.f, 0.f}, x[8];
    for (int v = v0; v < v1; v += 8) {
        weights_at<T, VEC, 8>(w, v, min(v1, v + 8), x);
#pragma unroll
        for (int i = 0; i < 8; ++i) s = add(s, x[i]);
    }
    Pair c = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Pair u = shfl_up(c, o);
        if (lane >= o) c = add(c, u);
    }
    if (lane == 31) part[warp] = c;
    __syncthreads();
    Pair ahead{0.f, 0.f};
    for (int i = 0; i < warp; ++i) ahead = add(ahead, part[i]);
    const Pair prev = shfl_up(c, 1);
    if (lane > 0) ahead = add(ahead, prev);
    // the first thread whose tokens pass the number, else the last that has any: candidates compete
    // with the former ahead of the latter
    const bool any = s.hi > 0.f, passes = any && above(add(ahead, s), rest);
    const int key = passes ? 2 * kThreads - tid : tid;
    if (any) atomicMax(&found, key);
    __syncthreads();
    if (!any || found != key) return;
    int token = -1;
    for (int v = v0; v < v1; v += 8) {
        if (each > 8) weights_at<T, VEC, 8>(w, v, min(v1, v + 8), x);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            // (a weight's hi may be 0 or below, all of it in lo: p less A q where that rounds to p)
            if (__fadd_rn(x[i].hi, x[i].lo) > 0.f && !(token >= 0 && above(ahead, rest))) {
                token = v + i;
                ahead = add(ahead, x[i]);
            }
    }
    a.out[b * (n + 1) + count] = token;
}

template <typename T, bool VEC>
cudaError_t launch_one(const VerifyArgs &a, int sm_count, cudaStream_t st) {
    // Rows kept by the threads: only a tree looks at a node's rows more than once (24 trees of 31 over 50021 tokens 40.6 us,
    // 58.6 without), and only where the batch fits the SMs beside them.
    constexpr int kMost = 96 * 1024, kFixed = 31 * 1024, kSm = 227 * 1024;
    const int64_t per = (((a.V + (int64_t)a.blocks - 1) / a.blocks) + 255) & ~(int64_t)255, run = (((per + kWarps - 1) / kWarps) + 7) & ~(int64_t)7;
    constexpr int STEP = VEC ? 32 * (16 / (int)sizeof(T)) : 8 * 32;
    const int64_t bytes = (run + STEP - 1) / STEP * (VEC ? 2 : 4) * kThreads * 16;
    VerifyArgs b = a;
    b.keep = a.parent && a.draft && bytes <= kMost && a.B * a.blocks <= kSm / (kFixed + bytes) * sm_count;
    const auto kernel = verify_kernel<T, VEC>;
    static std::atomic<uint64_t> done{0};
    if (b.keep)
        if (const cudaError_t e = allow_smem(done, kernel, kMost)) return e;
    return launch_chained(kernel, (unsigned)(a.B * a.blocks), kThreads, b.keep ? (size_t)bytes : 0, (unsigned)a.blocks, st, b);
}

template <typename T>
cudaError_t launch_t(const VerifyArgs &a, bool vec, int sm_count, cudaStream_t st) {
    return vec ? launch_one<T, true>(a, sm_count, st) : launch_one<T, false>(a, sm_count, st);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs &args, int dtype, bool vec, int sm_count, cudaStream_t st) {
    VerifyArgs a = args;
    a.blocks = 1;  // (256 threads each: 512 took 10.4 us for a chain where 256 take 9.6, and 24 for 38 long ones where 256 take 18)
    while (a.blocks < kMaxBlocks && a.V > 4096 * a.blocks) a.blocks *= 2;
    return dtype == 0   ? launch_t<__half>(a, vec, sm_count, st)
           : dtype == 1 ? launch_t<__nv_bfloat16>(a, vec, sm_count, st)
                        : launch_t<float>(a, vec, sm_count, st);
}

}  // namespace tl
