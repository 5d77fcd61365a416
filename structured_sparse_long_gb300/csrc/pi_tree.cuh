// pi_tree.cuh -- drafted trees: a sequence's nodes, each with its parent's number (below its own) or -1.
#pragma once

#include "pi_paged.cuh"
#include "pi_step.h"

namespace pi {

// Depth of node x of the n that start with packed token t0; -1: more than kTreeMax, or a parent out of range.  For the whole
// warp: its lanes hold the parents, so that a step up is a shuffle.
__device__ __forceinline__ int tree_depth(const int *parent, int t0, int n, int x) {
    if (n > kTreeMax) return -1;
    const int lane = threadIdx.x & 31;
    int held[kTreeMax / 32];
    bool ok = true;
#pragma unroll
    for (int i = 0; i < kTreeMax / 32; ++i) {
        const int j = 32 * i + lane;
        held[i] = j < n ? ld_now(parent + t0 + j) : -1;
        ok = ok && held[i] >= -1 && held[i] < j;
    }
    if (!__all_sync(0xffffffffu, ok)) return -1;
    int depth = 0;
#pragma unroll 1
    for (int at = x;; ++depth) {  // (ends: every parent's number is lower)
        int up = -1;
#pragma unroll
        for (int i = 0; i < kTreeMax / 32; ++i)
            if (at >> 5 == i) up = __shfl_sync(0xffffffffu, held[i], at & 31);
        if (up < 0) return depth;
        at = up;
    }
}

constexpr int kTreeGroup = 8;             // most nodes whose queries a CTA of the short kernel takes
constexpr int kNodeTag = -0x40000000;     // a key that is a node: this, plus the bits of the queries that attend it

// What a CTA of the short kernel knows of its nodes.
struct TreeGroup {
    int pos[kTreeGroup];        // their positions
    int ctx, node0, n_rows;     // position of the tree's roots; the first one's number; attended nodes
    uint8_t row[kTreeMax];      // their numbers
    unsigned mask[kTreeMax];    // a node's bits: u where query u has it in its band, kTreeGroup + u where it is one of its skips
    int parent[kTreeMax];
};
__device__ __forceinline__ TreeGroup *tree_group() {
    __shared__ TreeGroup group;
    return &group;
}

// A tree's parents on their way, some to a thread of the CTA (of 64 or more).
struct TreeParents {
    int held[kTreeMax / 64];
    int n, node0, ctx;
};
__device__ __forceinline__ void load_parents(TreeParents &p, const int *parent, int n, int node0, int ctx) {
    p.n = n;
    p.node0 = node0;
    p.ctx = ctx;
#pragma unroll
    for (int i = 0; i < kTreeMax / 64; ++i) {
        const int j = i * (int)blockDim.x + (int)threadIdx.x;
        p.held[i] = j < min(n, kTreeMax) ? ld_now(parent + j) : -1;
    }
}

// Nodes node0 .. node0 + n_q - 1 of a tree: their positions (lowest and highest in first, last) and the nodes that they attend.  False: more
// than kTreeMax nodes, or a parent out of range.  For the whole CTA; every thread returns the same.
__device__ __forceinline__ bool tree_walk(TreeGroup &g, const TreeParents &p, const Shape &s, int n_q, int &first, int &last) {
    const int n = p.n, node0 = p.node0, ctx = p.ctx;
    if (n > kTreeMax) return false;
    bool ok = true;
#pragma unroll
    for (int i = 0; i < kTreeMax / 64; ++i) {
        const int j = i * (int)blockDim.x + (int)threadIdx.x;
        if (j >= n) break;
        g.parent[j] = p.held[i];
        g.mask[j] = 0u;
        ok = ok && p.held[i] >= -1 && p.held[i] < j;
    }
    if (!__syncthreads_and(ok)) return false;
    if ((int)threadIdx.x < n_q) {
        int deep = 0;
        for (int at = g.parent[node0 + threadIdx.x]; at >= 0; at = g.parent[at]) ++deep;
        const int i = ctx + deep, lo = band_lo(i, s.mode, s.k_local);
        g.pos[threadIdx.x] = i;
        int at = node0 + threadIdx.x;
        for (int gap = 0; at >= 0; ++gap, at = g.parent[at]) {
            const bool band = i - gap >= lo;
            const bool skip = !band && s.mode != kModeEcp && s.S > 0 && gap % s.period == 0 && gap / s.period <= s.S;
            if (band || skip) atomicOr(&g.mask[at], 1u << (threadIdx.x + (band ? 0 : kTreeGroup)));
        }
    }
    if (threadIdx.x == 0) {
        g.ctx = ctx;
        g.node0 = node0;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        int rows = 0;
        for (int j0 = 0; j0 < node0 + n_q; j0 += 32) {
            const int j = j0 + threadIdx.x;
            const bool in = j < node0 + n_q && g.mask[j];
            const unsigned who = __ballot_sync(0xffffffffu, in);
            if (in) g.row[rows + __popc(who & ((1u << threadIdx.x) - 1u))] = (uint8_t)j;
            rows += __popc(who);
        }
        if (threadIdx.x == 0) g.n_rows = rows;
    }
    __syncthreads();
    first = last = g.pos[0];
    for (int u = 1; u < n_q; ++u) {
        first = min(first, g.pos[u]);
        last = max(last, g.pos[u]);
    }
    return true;
}

}  // namespace pi
