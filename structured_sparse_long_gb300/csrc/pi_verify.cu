// pi_verify.cu -- a drafted tree against the target's probabilities: the accepted path and the next token of every sequence.
//
// At a node with target probabilities p and draft probabilities q, what is left of p after some children were not accepted is
// max(p - q, 0) normalised, once per child.  Normalising and subtracting q again only moves the factor of q: after each child the weights are
// w = max(p - a q, 0) with a sum s, and the next ones have a + s instead of a.  So a rejection costs one pass over the rows p and q, an accepted
// child none, and the next token one pass (that of the last rejection, if the last node had one).
//
// A cluster of CTAs takes a sequence, each of them a contiguous share of the vocabulary, a warp of it a contiguous part of the share.  All
// CTAs make the same walk from the same numbers.  In a pass the warps send their sums to every CTA of the cluster, and
// their running sum says which warp's part holds the next token; that part is gone through token by token.
//
// A running sum is compared with a random number: an error in it would pick a neighbour's token as often as it is large.  fp32 sums over
// 10^5 tokens would do that once in a hundred calls.  Products and sums are carried in pairs of fp32 (48 bits), two tokens to an
// instruction: a dependent fp64 operation takes 75 cycles on a GB300, the sum of two pairs 37.
//
// What bounds it: few sequences, the chain gather (0.8 us) -> tests (0.2 each; 0.4 where siblings were refused) -> pass (1.7) -> search (1.7); 32 trees
// over 128001 tokens (29.6 us), their passes one after the other: 6 us the first, whose rows come from HBM, 4.5 the others, in which warps wait
// for loads and at the cluster's barrier (issue slots are 22 % busy, HBM 17 %).  The rows kept in shared memory from pass to pass changed
// nothing (30.7 for 30.2), nor did two sets of registers in turn (30.2 for 28.9).
#include "pi_mma.cuh"
#include "pi_paged.cuh"
#include "pi_step.h"

namespace pi {
namespace verify {

// Eight warps, each with 32 loads per lane in flight: the walk and the searches are made by every warp alike and share the SM's issue slots (16
// warps with 16 loads: 6 drafted tokens of 32000 7.3 instead of 6.7 us, 16 trees of chosen tokens over 50257 12.0 instead of 10.3, 32 trees
// over 128001 the same; 4 warps: 8.3, 23, 36).
constexpr int THREADS = 256, WARPS = THREADS / 32;
static_assert(THREADS >= kTreeMax, "a node to a thread");
constexpr int MAX_P = 8;  // CTAs per cluster (portable limit)
constexpr int HELD = 8;   // tokens that a lane holds in the search, at most
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
__device__ __forceinline__ Pair sub(const Pair &x, const Pair &y) { return add(x, Pair{-y.hi, -y.lo}); }
__device__ __forceinline__ Pair mul(const Pair &x, const Pair &y) {
    const float h = __fmul_rn(x.hi, y.hi), l = fmaf(x.hi, y.lo, fmaf(x.lo, y.hi, fmaf(x.hi, y.hi, -h))), hi = __fadd_rn(h, l);
    return Pair{hi, __fadd_rn(l, -__fsub_rn(hi, h))};
}
// (both as add() and mul() leave them)
__device__ __forceinline__ bool less(const Pair &x, const Pair &y) { return x.hi < y.hi || (x.hi == y.hi && x.lo < y.lo); }
__device__ __forceinline__ bool positive(const Pair &x) { return x.hi > 0.f; }
__device__ __forceinline__ Pair warp_sum(Pair x) {
#pragma unroll 1
    for (int w = 16; w > 0; w >>= 1) x = add(x, Pair{__shfl_xor_sync(kFull, x.hi, w), __shfl_xor_sync(kFull, x.lo, w)});
    return x;
}

// A probability as it counts: the nearest number in [0, 1], NaN 0.
__device__ __forceinline__ float sane(float p) { return __saturatef(p); }
__device__ __forceinline__ float unit(float u) { return fminf(fmaxf(u, 0.f), 0x1.fffffep-1f); }

// Two numbers at a time, in packed fp32.
struct Two {
    uint64_t v;
    __device__ __forceinline__ Two(uint64_t x) : v(x) {}
    __device__ __forceinline__ Two(float x, float y) : v(tc::pack2(x, y)) {}
};
__device__ __forceinline__ Two operator+(const Two &x, const Two &y) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x.v), "l"(y.v));
    return Two(r);
}
__device__ __forceinline__ Two fma(const Two &x, const Two &y, const Two &z) { return Two(tc::fma2(x.v, y.v, z.v)); }
__device__ __forceinline__ Two operator*(const Two &x, const Two &y) { return Two(tc::mul2(x.v, y.v)); }
__device__ __forceinline__ Two operator-(const Two &x, const Two &y) { return fma(y, Two(-1.f, -1.f), x); }  // (the product is exact)

// The node whose rows a pass reads, and its weights.
struct Weights {
    const float *p, *q;  // rows; q null: none, or a = 0
    Pair a;
    int removed;         // children's tokens without a weight (no draft probabilities)
};

struct Shared {
    int parent[kTreeMax], token[kTreeMax];
    float u[kTreeMax], p[kTreeMax], q[kTreeMax];  // of each node: its random number, its probabilities at its parent
    bool first[kTreeMax];  // whether it is accepted as its parent's first child (a = 0, s = 1)
    int path[kTreeMax], removed[kTreeMax];
    Pair all[2][MAX_P * WARPS];  // the sums of the cluster's warps, of this pass and the one before
};

__device__ __forceinline__ bool is_removed(const Weights &w, const Shared &sh, int v) {
    bool gone = false;
    for (int r = 0; r < w.removed; ++r) gone = gone || sh.removed[r] == v;
    return gone;
}
// The number of tokens to look at for those without a weight, or 0 where none of lo .. hi - 1 is one.  For the whole warp.
__device__ __forceinline__ int removed_in(const Weights &w, const Shared &sh, int lo, int hi) {
    bool some = false;
    for (int r = threadIdx.x & 31; r < w.removed; r += 32) some = some || (sh.removed[r] >= lo && sh.removed[r] < hi);
    return __any_sync(kFull, some) ? w.removed : 0;
}
// The weight of token v with probabilities p and q.
__device__ __forceinline__ Pair weight(const Weights &w, const Shared &sh, int v, float p, float q) {
    p = sane(p);
    if (is_removed(w, sh, v)) return Pair{0.f, 0.f};
    if (!w.q) return Pair{p, 0.f};
    // (as in sum_of, so that a part whose sum is above 0 has a token with a weight)
    q = sane(q);
    const float d = fmaf(-w.a.hi, q, p), t = __fsub_rn(p, d), r = __fsub_rn(__fsub_rn(p, t), d);
    const Pair x = add(Pair{d, fmaf(-w.a.lo, q, __fadd_rn(fmaf(-w.a.hi, q, t), r))}, Pair{0.f, 0.f});
    return positive(x) ? x : Pair{0.f, 0.f};
}

// The sum of the weights of tokens lo .. hi - 1, over the warp; AHEAD tokens per lane in flight.
template <bool DRAFT>
__device__ __forceinline__ Pair sum_of(const Weights &w, const Shared &sh, int lo, int hi) {
    constexpr int AHEAD = DRAFT ? 16 : 32;
    const int lane = threadIdx.x & 31;
    const int removed = removed_in(w, sh, lo, hi);
    const float *pp = w.p, *qq = w.q;
    Two hi2(0.f, 0.f), lo2(0.f, 0.f);
    const Two na_hi(-w.a.hi, -w.a.hi), na_lo(-w.a.lo, -w.a.lo);
    float p[AHEAD], q[AHEAD];
    auto take = [&](int v0) {
#pragma unroll 1
        for (int r = 0; r < removed; ++r) {
            const int v = sh.removed[r] - v0;
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                if (v == 32 * i) p[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < AHEAD; i += 2) {
            Two x(sane(p[i]), sane(p[i + 1])), rest(0.f, 0.f);
            if (DRAFT) {
                // d = p - a q rounded, and what that left: p - d = t + r exactly where |d| <= p, and t is a q up to d's rounding.  The weight
                // is above 0 where d + rest is (d alone says so only down to 2^-24 of p, where p is a q up to a's low part)
                const Two y(sane(q[i]), sane(q[i + 1])), d = fma(na_hi, y, x), t = x - d, r = (x - t) - d;
                rest = fma(na_lo, y, fma(na_hi, y, t) + r);
                float s0, s1;
                tc::unpack2((d + rest).v, s0, s1);
                const Two keep(s0 > 0.f ? 1.f : 0.f, s1 > 0.f ? 1.f : 0.f);
                x = d * keep;
                rest = rest * keep;
            }
            const Two s = hi2 + x, t = s - hi2;
            const Two err = (hi2 - (s - t)) + (x - t);
            hi2 = s;
            lo2 = lo2 + (DRAFT ? err + rest : err);
        }
        // the low words back below half a step of the high ones: left to grow over a row they would be rounded ever coarser (2^26 equal
        // tokens: 10^-6 off)
        const Two s = hi2 + lo2;
        lo2 = lo2 - (s - hi2);
        hi2 = s;
    };
    int v0 = lo + lane;
#pragma unroll 1
    for (; v0 - lane + 32 * AHEAD <= hi; v0 += 32 * AHEAD) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            p[i] = ld_now(pp + v0 + 32 * i);
            if (DRAFT) q[i] = ld_now(qq + v0 + 32 * i);
        }
        take(v0);
    }
    if (v0 - lane < hi) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const bool in = v0 + 32 * i < hi;
            p[i] = in ? ld_now(pp + v0 + 32 * i) : 0.f;
            if (DRAFT) q[i] = in ? ld_now(qq + v0 + 32 * i) : 0.f;
        }
        take(v0);
    }
    Pair x, y;
    tc::unpack2(hi2.v, x.hi, y.hi);
    tc::unpack2(lo2.v, x.lo, y.lo);
    return warp_sum(add(x, y));
}

__device__ __forceinline__ Pair from_lane(const Pair &x, int lane) { return Pair{__shfl_sync(kFull, x.hi, lane), __shfl_sync(kFull, x.lo, lane)}; }
// The sum over the lanes up to and including this one, of the first N.  (A lane without a lane so far below it adds 0: with a branch
// around the addition the five steps take 670 cycles instead of 320.)
template <int N>
__device__ __forceinline__ Pair upto_lane(Pair x) {
#pragma unroll
    for (int d = 1; d < N; d <<= 1) {
        const float hi = __shfl_up_sync(kFull, x.hi, d), lo = __shfl_up_sync(kFull, x.lo, d);
        const bool in = (int)(threadIdx.x & 31) >= d;
        x = add(x, Pair{in ? hi : 0.f, in ? lo : 0.f});
    }
    return x;
}
// Of the lanes' numbers m (>= 0), the one in which the running sum `here` passes `goal`: the first lane past it, or (where
// rounding left the goal past them all) the last one above 0; -1: none is.  run: the sum in front of it (before: of lane 0).
__device__ __forceinline__ int find_lane(const Pair &m, const Pair &here, const Pair &goal, Pair &run) {
    const unsigned past = __ballot_sync(kFull, positive(m) && less(goal, here)), some = __ballot_sync(kFull, positive(m));
    if (!some) return -1;
    const int x = past ? __ffs(past) - 1 : 31 - __clz(some);
    const Pair before = from_lane(here, max(x - 1, 0));
    if (x > 0) run = before;
    return x;
}
// The same of 32 * per numbers m, per <= MOST consecutive ones to a lane, whose sum `all` is.
template <int MOST>
__device__ __forceinline__ int find_held(const Pair (&m)[MOST], int per, const Pair &all, const Pair &here, const Pair &goal, Pair &run) {
    const int x = find_lane(all, here, goal, run);
    if (x < 0) return x;
    int at = -1;
    Pair upto = run;
#pragma unroll
    for (int i = 0; i < MOST; ++i) {  // that lane's numbers, by all lanes alike
        if (i >= per) break;
        const Pair y = from_lane(m[i], x);
        const bool next = positive(y) && (at < 0 || !less(goal, upto));
        const Pair more = add(upto, y);
        at = next ? x * per + i : at;
        run = next ? upto : run;
        upto = next ? more : upto;
    }
    return at;
}

__global__ void __launch_bounds__(THREADS, 2) verify_kernel(const __grid_constant__ VerifyArgs a, int P, int part) {
    __shared__ Shared sh;
    const int rank = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.launch_dependents;");
    cluster_arrive();  // (before a CTA writes into another's shared memory, that one has to run)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int t0 = ld_now(a.cu + b), t1 = ld_now(a.cu + b + 1), n = t1 - t0;
    const float u_next = ld_now(a.u_next + b);
    bool ok = t0 >= 0 && t0 <= t1 && t1 <= a.T && n <= kTreeMax;
    if (ok && tid < n) {
        const int parent = ld_now(a.parent + t0 + tid), token = ld_now(a.tokens + t0 + tid);
        ok = parent >= -1 && parent < tid && (tid == 0 || ((unsigned)token < (unsigned)a.V));
        sh.parent[tid] = parent;
        sh.token[tid] = token;
        if (ok && parent >= 0) {
            const float u = unit(ld_now(a.u + t0 + tid)), p = sane(ld_now(a.target + (long long)(t0 + parent) * a.target_stride + token));
            const float q = a.draft ? sane(ld_now(a.draft + (long long)(t0 + parent) * a.draft_stride + token)) : 1.f;
            sh.u[tid] = u;
            sh.p[tid] = p;
            sh.q[tid] = q;
            sh.first[tid] = less(mul(Pair{u, 0.f}, Pair{q, 0.f}), Pair{p, 0.f});
        }
    }
    ok = __syncthreads_and(ok);
    cluster_wait();
    if (!ok || n == 0) {  // (all CTAs of the cluster)
        if (tid == 0 && rank == 0) {
            if (!ok) record_index(a.index_word);
            a.count[b] = 0;
            a.next[b] = -1;
        }
        return;
    }
    const int share = part * WARPS;
    auto part_lo = [&](int i) -> int { return (int)min((long long)a.V, (long long)(i / WARPS) * share + (i % WARPS) * part); };
    auto part_hi = [&](int i) -> int { return (int)min((long long)a.V, (long long)part_lo(i) + part); };

    // node 0's rows, which the first pass most often reads
    for (int v = part_lo(rank * WARPS) + 32 * tid; v < part_hi(rank * WARPS + WARPS - 1); v += 32 * THREADS) {
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.target + t0 * a.target_stride + v));
        if (a.draft) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.draft + t0 * a.draft_stride + v));
    }
    // ---- the walk, by every warp alike (shuffles in a part of the code that one warp alone runs took seven times as long, and what
    // it found would have to be handed on): at node x, whose children up to `last` were not accepted
    int x = 0, last = 0, len = 1, passes = 0;
    Weights w{};
    Pair s{1.f, 0.f};
    constexpr int PER = MAX_P * WARPS / 32;
    Pair parts[PER], mine, here;  // of the last pass: PER warps' sums, their sum, and that of all up to them
    bool summed = false, spent = false;  // the weights' sum is known; it is 0, and p's own is asked for
    if (lane == 0) sh.path[0] = 0;
    for (;;) {
        while (!spent) {
            int c = kTreeMax;  // the next child
#pragma unroll 1
            for (int j0 = (last + 1) & ~31; c == kTreeMax && j0 < n; j0 += 32) {
                const unsigned who = __ballot_sync(kFull, j0 + lane > last && j0 + lane < n && sh.parent[min(j0 + lane, kTreeMax - 1)] == x);
                if (who) c = j0 + __ffs(who) - 1;
            }
            if (c == kTreeMax) break;
            last = c;
            Pair left{sh.p[c], 0.f};
            bool yes;
            if (a.draft ? !positive(w.a) : w.removed == 0) {
                yes = sh.first[c];
            } else {
                if (a.draft) {
                    left = sub(left, mul(w.a, Pair{sh.q[c], 0.f}));
                } else {  // the same token, chosen twice
                    bool gone = false;
                    for (int r = x + 1 + lane; r < c; r += 32) gone = gone || (sh.parent[r] == x && sh.token[r] == sh.token[c]);
                    if (__any_sync(kFull, gone)) left = Pair{0.f, 0.f};
                }
                yes = positive(left) && less(mul(mul(Pair{sh.u[c], 0.f}, Pair{sh.q[c], 0.f}), s), left);
            }
            summed = false;
            if (yes) {
                x = c;
                if (lane == 0) sh.path[len] = c;
                ++len;
                w.a = Pair{0.f, 0.f};
                w.removed = 0;
                s = Pair{1.f, 0.f};
            } else if (a.draft) {
                w.a = add(w.a, s);
                break;  // a pass
            } else if (positive(left)) {
                ++w.removed;
                s = sub(s, left);
            }
        }
        if (summed) {
            if (positive(s) || spent) break;
            spent = true;  // nothing is left of p: the next token is drawn from p itself
            w.a = Pair{0.f, 0.f};
            w.removed = 0;
        }
        const long long row = t0 + x;
        w.p = a.target + row * a.target_stride;
        w.q = a.draft && positive(w.a) ? a.draft + row * a.draft_stride : nullptr;
        if (w.removed > 0) {  // the tokens without a weight: x's children (all of them, without draft probabilities)
            w.removed = 0;
#pragma unroll 1
            for (int j0 = x & ~31; j0 < n; j0 += 32) {
                const bool in = j0 + lane > x && j0 + lane < n && sh.parent[min(j0 + lane, kTreeMax - 1)] == x;
                const unsigned who = __ballot_sync(kFull, in);
                if (in) sh.removed[w.removed + __popc(who & ((1u << lane) - 1u))] = sh.token[j0 + lane];
                w.removed += __popc(who);
            }
            __syncwarp();
        }
        const int i = rank * WARPS + warp;
        const Pair t = w.q ? sum_of<true>(w, sh, part_lo(i), part_hi(i)) : sum_of<false>(w, sh, part_lo(i), part_hi(i));
        // to every CTA of the cluster (into the half that none of them still reads)
        Pair *all = sh.all[passes & 1];
        if (lane < P) st_peer2(peer_addr(smem_addr(&all[i]), lane), make_float2(t.hi, t.lo));
        cluster_sync();
        ++passes;
#pragma unroll
        for (int k = 0; k < PER; ++k) parts[k] = lane * PER + k < P * WARPS ? all[lane * PER + k] : Pair{0.f, 0.f};
        mine = parts[0];
#pragma unroll
        for (int k = 1; k < PER; ++k) mine = add(mine, parts[k]);
        here = upto_lane<32>(mine);
        s = from_lane(here, 31);
        summed = true;
    }

    // ---- the next token: the part in which the running sum passes u times the whole sum
    if (rank == 0) {
        for (int j = tid; j < n; j += THREADS) a.path[t0 + j] = j < len ? sh.path[j] : -1;  // (a warp's own writes)
        if (tid == 0) a.count[b] = len;
    }
    const Pair goal = mul(Pair{unit(u_next), 0.f}, s);
    Pair run{0.f, 0.f};
    const int at = find_held<PER>(parts, PER, mine, here, goal, run);  // by every warp alike
    if (at < 0) {
        if (tid == 0 && rank == 0) a.next[b] = -1;
    } else if (at / WARPS == rank) {  // this CTA has it: a piece of that part per warp, a few tokens of it to a lane
        const int hi = part_hi(at), piece = part / WARPS, from = part_lo(at) + warp * piece, n_mine = min(from + piece, hi) - from;
        const int per = min(HELD, (piece + 31) / 32);
        const bool held = piece <= 32 * HELD;
        w.removed = removed_in(w, sh, from, from + n_mine);
        // tokens lo + lane * per ... of the warp's, as far as its end: their weights, all of them under way at once
        Pair m[HELD], sum;
        auto hold = [&](int lo) {
            float p[HELD], q[HELD];
#pragma unroll
            for (int i = 0; i < HELD; ++i) {
                const int v = lo + lane * per + i;
                const bool in = i < per && v < n_mine;
                p[i] = in ? ld_now(w.p + from + v) : 0.f;
                q[i] = in && w.q ? ld_now(w.q + from + v) : 0.f;
            }
            sum = Pair{0.f, 0.f};
#pragma unroll
            for (int i = 0; i < HELD; ++i) {
                if (i >= per) break;
                m[i] = weight(w, sh, from + lo + lane * per + i, p[i], q[i]);
                sum = add(sum, m[i]);
            }
            here = upto_lane<32>(sum);
        };
        if (held) {
            hold(0);
            mine = from_lane(here, 31);
        } else {
            mine = w.q ? sum_of<true>(w, sh, from, from + n_mine) : sum_of<false>(w, sh, from, from + n_mine);
        }
        Pair *sums = sh.all[passes & 1];  // (its last readers are past the last pass)
        if (lane == 0) sums[warp] = mine;
        __syncthreads();
        const Pair its = lane < WARPS ? sums[lane] : Pair{0.f, 0.f};
        const int in = find_lane(its, add(run, upto_lane<WARPS>(its)), goal, run);
        if (max(in, 0) == warp) {
            int lo = 0, x = 0;
            if (!held) {  // the 32 * HELD tokens that hold it, or the last ones above 0 (rounding left the goal past them all)
                Pair upto = run;
#pragma unroll 1
                for (int t = 0; t < n_mine; t += 32 * HELD) {
                    hold(t);
                    const Pair y = from_lane(here, 31);
                    if (!positive(y)) continue;
                    lo = t;
                    run = upto;
                    upto = add(upto, y);
                    if (less(goal, upto)) break;
                }
                hold(lo);
            }
            x = find_held<HELD>(m, per, sum, add(run, here), goal, run);
            if (lane == 0) a.next[b] = from + lo + max(x, 0);  // (there is one; else the first)
        }
    }
    cluster_leave();  // a CTA's shared memory stays until the others have read it
}

}  // namespace verify

cudaError_t launch_verify(const VerifyArgs &a, cudaStream_t st) {
    using namespace verify;
    // as many CTAs per sequence as leave each at least 1024 tokens of the vocabulary and, at two CTAs per SM, run at once (clusters do
    // not fill every SM; at one per SM 32 trees over 128001 tokens took 43.0 us for 29.1)
    int P = 1;
    while (P < MAX_P && a.V / (2 * P) >= 1024 && (long long)a.B * 2 * P <= 2LL * sm_count() - 16) P *= 2;
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
    const int part = ((a.V + P - 1) / P + WARPS * 32 - 1) / (WARPS * 32) * 32;  // tokens of a warp
    return cudaLaunchKernelEx(&cfg, verify_kernel, a, P, part);
}

}  // namespace pi
