// pi_verify.cu -- a drafted tree against the target's probabilities: the accepted path and the next token of every sequence.
//
// At a node with target probabilities p and draft probabilities q, what is left of p after some children were not accepted is
// max(p - q, 0) normalised, once per child.  Normalising and subtracting q again only moves the factor of q: after each child the weights are
// w = max(p - a q, 0) with a sum s, and the next ones have a + s instead of a.  So a rejection costs one pass over the rows p and q, an accepted
// child none, and the next token one pass (that of the last rejection, if the last node had one).
//
// A cluster of CTAs takes a sequence, each of them a contiguous share of the vocabulary, a warp of it a contiguous part of the share.  All
// CTAs make the same walk from the same numbers.  A pass leaves the warps' sums in shared memory, every CTA collects the cluster's, and
// their running sum says which warp's part holds the next token; that part is summed again, finer.
//
// A running sum is compared with a random number: an error in it would pick a neighbour's token as often as it is large.  fp32 sums over
// 10^5 tokens would do that once in a hundred calls.  Products and sums are carried in pairs of fp32 (48 bits): a GB300 has few fp64 units, and
// fewer than ten fp64 operations per child remain, in one warp.
#include "pi_mma.cuh"
#include "pi_paged.cuh"
#include "pi_step.h"

namespace pi {
namespace verify {

constexpr int THREADS = 512, WARPS = THREADS / 32;
constexpr int MAX_P = 8;  // CTAs per cluster (portable limit)
constexpr unsigned kFull = 0xffffffffu;

// A number as an unevaluated sum of two fp32.
struct Pair {
    float hi, lo;
};
// x + y exactly, hi being their rounded sum.
__device__ __forceinline__ Pair two_sum(float x, float y) {
    const float s = __fadd_rn(x, y), t = __fsub_rn(s, x);
    return Pair{s, __fadd_rn(__fsub_rn(x, __fsub_rn(s, t)), __fsub_rn(y, t))};
}
__device__ __forceinline__ Pair add(const Pair &x, const Pair &y) {
    const Pair s = two_sum(x.hi, y.hi);
    const float lo = __fadd_rn(s.lo, __fadd_rn(x.lo, y.lo)), hi = __fadd_rn(s.hi, lo);
    return Pair{hi, __fadd_rn(lo, -__fsub_rn(hi, s.hi))};
}
__device__ __forceinline__ double value(const Pair &x) { return (double)x.hi + (double)x.lo; }
__device__ __forceinline__ Pair pair_of(double x) {
    const float hi = (float)x;
    return Pair{hi, (float)(x - (double)hi)};
}
__device__ __forceinline__ Pair warp_sum(Pair x) {
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) x = add(x, Pair{__shfl_xor_sync(kFull, x.hi, w), __shfl_xor_sync(kFull, x.lo, w)});
    return x;
}

// A probability as it counts: negative or not finite, 0.
__device__ __forceinline__ float sane(float p) { return p > 0.f && p < INFINITY ? p : 0.f; }
__device__ __forceinline__ float unit(float u) { return fminf(fmaxf(u, 0.f), 0x1.fffffep-1f); }

// The node whose rows a pass reads, and its weights.
struct Weights {
    const float *p, *q;  // rows; q null: none, or a = 0
    Pair a;
    int removed;         // children's tokens without a weight (no draft probabilities)
};

struct Shared {
    int parent[kTreeMax], token[kTreeMax];
    float u[kTreeMax], p[kTreeMax], q[kTreeMax];  // of each node: its random number, its probabilities at its parent
    int path[kTreeMax], removed[kTreeMax];
    Pair mine[2][WARPS];        // the warps' sums of this pass and the one before
    Pair all[MAX_P * WARPS];    // the cluster's
    Weights w;
    int pass, len;              // whether there is another pass; the path's length
    int at;                     // the part that holds the next token, the running sum that it passes, and the one in front of it
    double goal, before;
};

__device__ __forceinline__ Pair weight(const Weights &w, const Shared &sh, int v) {
    const float p = sane(ld_now(w.p + v));
    Pair d{p, 0.f};
    if (w.q) {
        const float q = sane(ld_now(w.q + v)), h = __fmul_rn(w.a.hi, q);
        d = two_sum(p, -h);
        d.lo = __fsub_rn(d.lo, fmaf(w.a.lo, q, fmaf(w.a.hi, q, -h)));
        if (!(__fadd_rn(d.hi, d.lo) > 0.f)) d = Pair{0.f, 0.f};
    }
    for (int r = 0; r < w.removed; ++r)
        if (sh.removed[r] == v) d = Pair{0.f, 0.f};
    return d;
}
// The sum of the weights of tokens lo + lane, lo + lane + 32, ... below hi, over the warp.
__device__ __forceinline__ Pair sum_of(const Weights &w, const Shared &sh, int lo, int hi) {
    Pair s{0.f, 0.f};
#pragma unroll 4
    for (int v = lo + (int)(threadIdx.x & 31); v < hi; v += 32) s = add(s, weight(w, sh, v));
    return warp_sum(s);
}

// Sum over the lanes up to and including this one.
__device__ __forceinline__ double upto_lane(double x) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const double y = __shfl_up_sync(kFull, x, d);
        if ((int)(threadIdx.x & 31) >= d) x += y;
    }
    return x;
}
// Which of n sums (all >= 0) the running sum passes `goal` in: the last one above 0 that begins at or before it, or -1; `before`:
// the running sum in front of it, given that in front of them all.  With `scale` goal is u times the whole sum.  For a whole warp.
__device__ __forceinline__ int find_part(const Pair *sums, int n, double u, bool scale, double &goal, double &before) {
    const int lane = threadIdx.x & 31;
    constexpr int PER = MAX_P * WARPS / 32;
    double m[PER], run[PER], all = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int k = lane * PER + i;
        m[i] = k < n ? value(sums[k]) : 0.0;
        run[i] = all;
        all += m[i];
    }
    const double upto = upto_lane(all), start = before + (upto - all);
    if (scale) goal = u * __shfl_sync(kFull, upto, 31);
    int at = -1;
    double mine = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (m[i] > 0.0 && start + run[i] <= goal) {
            at = lane * PER + i;
            mine = start + run[i];
        }
    const unsigned who = __ballot_sync(kFull, at >= 0);
    if (!who) {  // (rounding: the first one above 0)
#pragma unroll
        for (int i = PER - 1; i >= 0; --i)
            if (m[i] > 0.0) {
                at = lane * PER + i;
                mine = start + run[i];
            }
        const unsigned any = __ballot_sync(kFull, at >= 0);
        if (!any) return -1;
        before = __shfl_sync(kFull, mine, __ffs(any) - 1);
        return __shfl_sync(kFull, at, __ffs(any) - 1);
    }
    before = __shfl_sync(kFull, mine, 31 - __clz(who));
    return __shfl_sync(kFull, at, 31 - __clz(who));
}

__global__ void __launch_bounds__(THREADS) verify_kernel(const __grid_constant__ VerifyArgs a, int P) {
    __shared__ Shared sh;
    const int rank = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int t0 = ld_now(a.cu + b), t1 = ld_now(a.cu + b + 1), n = t1 - t0;
    bool ok = t0 >= 0 && t0 <= t1 && t1 <= a.T && n <= kTreeMax;
    if (ok && tid < n) {
        const int parent = ld_now(a.parent + t0 + tid), token = ld_now(a.tokens + t0 + tid);
        ok = parent >= -1 && parent < tid && (tid == 0 || ((unsigned)token < (unsigned)a.V));
        sh.parent[tid] = parent;
        sh.token[tid] = token;
        if (ok && parent >= 0) {
            sh.u[tid] = unit(ld_now(a.u + t0 + tid));
            sh.p[tid] = sane(ld_now(a.target + (long long)(t0 + parent) * a.target_stride + token));
            sh.q[tid] = a.draft ? sane(ld_now(a.draft + (long long)(t0 + parent) * a.draft_stride + token)) : 1.f;
        }
    }
    if (!__syncthreads_and(ok) || n == 0) {  // (all CTAs of the cluster)
        if (tid == 0 && rank == 0) {
            if (!ok || n != 0) record_index(a.index_word);
            a.count[b] = 0;
            a.next[b] = -1;
        }
        return;
    }
    const int share = ((a.V + P - 1) / P + WARPS * 32 - 1) & ~(WARPS * 32 - 1), part = share / WARPS;
    auto part_lo = [&](int i) -> int { return (int)min((long long)a.V, (long long)(i / WARPS) * share + (i % WARPS) * part); };
    auto part_hi = [&](int i) -> int { return (int)min((long long)a.V, (long long)part_lo(i) + part); };

    // ---- the walk, by warp 0: at node x, whose children up to `last` were not accepted
    int x = 0, last = 0, len = 1, removed = 0;
    double w_a = 0.0, s = 1.0;
    bool summed = false, spent = false;  // the weights' sum is known; it is 0, and p's own is asked for
    int passes = 0;
    if (tid == 0) sh.path[0] = 0;
    for (;;) {
        if (warp == 0) {
            bool more = true;
            if (passes > 0) {  // the sum of a pass
                Pair t{0.f, 0.f};
                for (int i = lane; i < P * WARPS; i += 32) t = add(t, sh.all[i]);
                s = value(warp_sum(t));
                summed = true;
            }
            while (!spent) {
                int c = kTreeMax;  // the next child
                for (int j0 = (last + 1) & ~31; c == kTreeMax && j0 < n; j0 += 32) {
                    const unsigned who = __ballot_sync(kFull, j0 + lane > last && j0 + lane < n && sh.parent[min(j0 + lane, kTreeMax - 1)] == x);
                    if (who) c = j0 + __ffs(who) - 1;
                }
                if (c == kTreeMax) break;
                last = c;
                double w = (double)sh.p[c];
                if (a.draft) {
                    w -= w_a * (double)sh.q[c];
                } else {
                    bool gone = false;
                    for (int r = lane; r < removed; r += 32) gone = gone || sh.removed[r] == sh.token[c];
                    if (__any_sync(kFull, gone)) w = 0.0;
                }
                w = w > 0.0 ? w : 0.0;
                if ((double)sh.u[c] * (double)sh.q[c] * s < w) {
                    x = c;
                    if (lane == 0) sh.path[len] = c;
                    ++len;
                    removed = 0;
                    w_a = 0.0;
                    s = 1.0;
                    summed = false;
                } else if (a.draft) {
                    w_a += s;
                    summed = false;
                    break;  // a pass
                } else {
                    if (w > 0.0) {
                        if (lane == 0) sh.removed[removed] = sh.token[c];
                        ++removed;
                        __syncwarp();
                        s -= w;
                    }
                    summed = false;
                }
            }
            if (summed) {
                if (s > 0.0 || spent) {
                    more = false;
                } else {  // nothing is left of p: the next token is drawn from p itself
                    spent = true;
                    w_a = 0.0;
                    removed = 0;
                }
            }
            if (lane == 0) {
                const long long row = t0 + x;
                sh.w.p = a.target + row * a.target_stride;
                sh.w.q = a.draft && w_a != 0.0 ? a.draft + row * a.draft_stride : nullptr;
                sh.w.a = pair_of(w_a);
                sh.w.removed = removed;
                sh.pass = more;
                sh.len = len;
            }
        }
        __syncthreads();
        if (!sh.pass) break;
        const Weights w = sh.w;
        Pair *mine = sh.mine[passes & 1];  // (a peer may still read the other one)
        const int i = rank * WARPS + warp;
        const Pair t = sum_of(w, sh, part_lo(i), part_hi(i));
        if (lane == 0) mine[warp] = t;
        cluster_sync();
        if (tid < P * WARPS) {
            const float2 f = ld_peer2(peer_addr(smem_addr(mine + tid % WARPS), tid / WARPS));
            sh.all[tid] = Pair{f.x, f.y};
        }
        __syncthreads();
        ++passes;
    }

    // ---- the next token: the part in which the running sum passes u times the whole sum
    if (rank == 0) {
        for (int j = tid; j < n; j += THREADS) a.path[t0 + j] = j < sh.len ? sh.path[j] : -1;
        if (tid == 0) a.count[b] = sh.len;
    }
    if (warp == 0) {
        double goal = 0.0, before = 0.0;
        const int at = find_part(sh.all, P * WARPS, (double)unit(ld_now(a.u_next + b)), true, goal, before);
        if (lane == 0) {
            sh.at = at;
            sh.goal = goal;
            sh.before = before;
            if (at < 0 && rank == 0) a.next[b] = -1;
        }
    }
    __syncthreads();
    if (sh.at >= 0 && sh.at / WARPS == rank) {  // this CTA has it: the part once more, a piece of it per warp
        const Weights w = sh.w;
        const int lo = part_lo(sh.at), hi = part_hi(sh.at), piece = part / WARPS;
        const Pair t = sum_of(w, sh, min(hi, lo + warp * piece), min(hi, lo + (warp + 1) * piece));
        if (lane == 0) sh.all[warp] = t;
        __syncthreads();
        if (warp == 0) {
            double goal = sh.goal, run = sh.before;
            const int in = find_part(sh.all, WARPS, 0.0, false, goal, run);
            // token by token, 32 at a time; where rounding leaves the goal past the last one, that one
            int token = -1;
            const int end = min(hi, lo + (in + 1) * piece);
            for (int v0 = lo + in * piece; in >= 0 && v0 < end; v0 += 32) {
                const int v = v0 + lane;
                const double m = v < end ? value(weight(w, sh, v)) : 0.0, upto = run + upto_lane(m);
                const unsigned past = __ballot_sync(kFull, m > 0.0 && upto > goal), some = __ballot_sync(kFull, m > 0.0);
                if (past) {
                    token = v0 + __ffs(past) - 1;
                    break;
                }
                if (some) token = v0 + 31 - __clz(some);
                run = __shfl_sync(kFull, upto, 31);
            }
            if (lane == 0) a.next[b] = token;
        }
    }
    cluster_leave();  // a CTA's shared memory stays until the others have read it
}

}  // namespace verify

cudaError_t launch_verify(const VerifyArgs &a, cudaStream_t st) {
    using namespace verify;
    // as many CTAs per sequence as leave each at least 4096 tokens of the vocabulary and fit the SMs at once
    int P = 1;
    while (P < MAX_P && a.V / (2 * P) >= 4096 && (long long)a.B * 2 * P <= 2LL * sm_count()) P *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)P, (unsigned)a.B, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)P;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, verify_kernel, a, P);
}

}  // namespace pi
