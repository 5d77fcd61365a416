// pi_decode_paged.cu -- one decode step of pi-Attention / ECP attention against a paged key/value cache:
// for sequence b with n = lens[b] cached rows and query head h, row n - 1 of the forward.
//
// The neighbour rows of a (sequence, KV head) -- the band, then the skips -- form a key list that is cut
// into tiles of 16 keys.  Every warp of a CTA (and of its cluster, where few sequences leave SMs idle)
// takes tiles of its own and needs nothing from the others until the end:
//   * The tile's rows are looked up by one lane each (a page-table load per key), then all of the
//     tile's K and V bytes are requested at once, straight into registers and straight into the layout
//     of the warp's matrix products, so that no shared memory and no barrier lies between HBM and
//     the arithmetic, and a warp has 8 KB (bf16, d = 128) in flight.
//   * S^T = K Q^T by mma.m16n8k16 (16 keys x 8 heads): the head group's queries are the 8 columns, so
//     grouped heads cost nothing.  A contraction may take its elements in any order as long as both
//     operands agree: lane 4 g + t holds 16 contiguous bytes of key rows g and g + 8, whose elements
//     are its share of the k steps, and the queries are loaded the same way.
//   * The softmax keeps a running maximum and sum per head in 32 bits: a lane holds heads 2t, 2t+1 of keys g,
//     g + 8, so a tile's maximum takes three shuffles per head; the sums stay per lane until the end.
//   * O^T += V^T P^T (16 elements of d x 8 heads): P^T is S^T's accumulator rounded to bf16 (half a step
//     of 2^-7 relative, as in the forward; drafted trees: two bf16 terms, whose sum is within 2^-15; one tree of 26 nodes 9.9 us either way) and
//     transposed by movmatrix; lane 4 g + t holds 16 (8-bit
//     cache: 16 or 8) contiguous bytes of V rows 2t, 2t+1, 2t+8, 2t+9, which two byte permutes per word
//     turn into the pairs of keys that the product wants.
//   * 8-bit codes become bf16 in registers (exact, see pi_paged.cuh).
// The partial states (m, l, o) meet in shared memory, and across a cluster through distributed shared
// memory.  With a few hundred keys per sequence the step is bound by the latency of its dependent
// loads (length, page table, rows) for small batches and by HBM for large ones.
#include <type_traits>

#include "pi_mma.cuh"
#include "pi_paged.cuh"
#include "pi_row.cuh"
#include "pi_tree.cuh"

#include "pi_launch.h"

namespace pi {
namespace decp {

constexpr int MAX_P = 8;   // CTAs per cluster (portable limit)
constexpr int MEET = 12;   // states of a row that meet in one turn
constexpr int KEYS = 16;   // keys per tile: the rows of S^T
constexpr unsigned kFull = 0xffffffffu;

// One step of decode (sequence b's one query at position lens[b] - 1), or a few new tokens per sequence, at most `group` of
// them per CTA: packed queries as in pi_attn_extend, or the nodes of a drafted tree.
enum Kind { kSingle, kTokens, kTree };
struct Args {
    const __nv_bfloat16 *q;
    long long q_stride;
    const float *alpha;
    const int *lens;
    PagedBatch batch;  // B, table; all but for kSingle cu, ctx and T
    __nv_bfloat16 *out;
    float *lse;
    Shape s;
    PagedCache cache;
    int *index_word;
    int m_first, group;
    const int *parent;  // kTree: [T]
    int group0;         // kTree: the launch's first group of tokens
};

// ---- what a lane holds of a tile -------------------------------------------------------------

// K: 16 bytes each of rows g and g + 8, C chunks per row; V: C chunks of VB bytes each of rows 2t, 2t+1,
// 2t+8, 2t+9.  Registers are 32-bit words.
template <int D, int KV>
struct Frag;

template <int D>
struct Frag<D, kKvBf16> {
    static constexpr int C = D / 32;       // 16-byte chunks of a K row per lane: elements 32 c + 8 t ...
    static constexpr int CV = D / 64;      // 16-byte chunks of a V row per lane: elements 64 c + 8 g ...
    uint4 k[2][C], v[4][CV];
};
template <int D>
struct Frag8 {
    static constexpr int C = D / 64;       // 16-byte chunks of a K row: elements 64 c + 16 t ...
    static constexpr int VW = D / 32;      // words of a V row: elements (D / 8) g ... : 4 (d = 128) or 2
    uint4 k[2][C];
    uint32_t v[4][VW];
    uint32_t ks[2], vs[4];                 // scale bytes of the lane's K rows (all), of its V elements
};
template <int D> struct Frag<D, kKvE4m3> : Frag8<D> {};
template <int D> struct Frag<D, kKvInt8> : Frag8<D> {};

template <int D, int KV>
__device__ __forceinline__ void load_k(Frag<D, KV> &f, const PagedCache &c, int half, int row, int t) {
    // a row of -1 (no key, or a page out of range) reads as zeros; its score is masked
    if constexpr (KV == kKvBf16) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(c.k) + (long long)row * D) + t;
#pragma unroll
        for (int x = 0; x < f.C; ++x) f.k[half][x] = row >= 0 ? ld_stream(p + 4 * x) : make_uint4(0u, 0u, 0u, 0u);
    } else {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(c.k) + (long long)row * D) + t;
#pragma unroll
        for (int x = 0; x < f.C; ++x) f.k[half][x] = row >= 0 ? ld_stream(p + 4 * x) : make_uint4(0u, 0u, 0u, 0u);
        if (D == 128) f.ks[half] = row >= 0 ? ld_now(reinterpret_cast<const uint32_t *>(c.k_scale) + row) : 0u;
        else f.ks[half] = row >= 0 ? ld_now(reinterpret_cast<const uint16_t *>(c.k_scale) + row) : 0u;
    }
}

template <int D, int KV>
__device__ __forceinline__ void load_v(Frag<D, KV> &f, const PagedCache &c, int which, int row, int g) {
    if constexpr (KV == kKvBf16) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(c.v) + (long long)row * D) + g;
#pragma unroll
        for (int x = 0; x < f.CV; ++x) f.v[which][x] = row >= 0 ? ld_stream(p + 8 * x) : make_uint4(0u, 0u, 0u, 0u);
    } else {
        const uint8_t *p = static_cast<const uint8_t *>(c.v) + (long long)row * D + g * (D / 8);
        if constexpr (D == 128) {
            const uint4 x = row >= 0 ? ld_stream(reinterpret_cast<const uint4 *>(p)) : make_uint4(0u, 0u, 0u, 0u);
            f.v[which][0] = x.x; f.v[which][1] = x.y; f.v[which][2] = x.z; f.v[which][3] = x.w;
        } else {
            const uint2 x = row >= 0 ? ld_now(reinterpret_cast<const uint2 *>(p)) : make_uint2(0u, 0u);
            f.v[which][0] = x.x; f.v[which][1] = x.y;
        }
        // elements (D / 8) g ... lie in one block of 32
        f.vs[which] = row >= 0 ? ld_now(c.v_scale + (long long)row * (D / kScaleBlock) + g * (D / 8) / kScaleBlock) : 0u;
    }
}

// ---- the two products ----------------------------------------------------------------------

// s[nh] += K (16 keys) . Q (heads 8 nh ...): q[nh][k step] from load_q
template <int D, int KV, int NH>
__device__ __forceinline__ void scores(const Frag<D, KV> &f, const uint2 (&q)[NH][D / 16], float (&s)[NH][4], int t) {
    if constexpr (KV == kKvBf16) {
#pragma unroll
        for (int x = 0; x < f.C; ++x) {
#pragma unroll
            for (int nh = 0; nh < NH; ++nh) {
                mma_bf16(s[nh], f.k[0][x].x, f.k[1][x].x, f.k[0][x].y, f.k[1][x].y, q[nh][2 * x].x, q[nh][2 * x].y);
                mma_bf16(s[nh], f.k[0][x].z, f.k[1][x].z, f.k[0][x].w, f.k[1][x].w, q[nh][2 * x + 1].x, q[nh][2 * x + 1].y);
            }
        }
    } else {
#pragma unroll
        for (int x = 0; x < f.C; ++x) {
            // elements 64 x + 16 t ... of a row lie in block 2 x + t / 2
            const Scale2<KV> s0 = scale_same<KV>(f.ks[0] >> (8 * (2 * x + (t >> 1))) & 0xffu);
            const Scale2<KV> s1 = scale_same<KV>(f.ks[1] >> (8 * (2 * x + (t >> 1))) & 0xffu);
            const uint32_t w0[4] = {f.k[0][x].x, f.k[0][x].y, f.k[0][x].z, f.k[0][x].w};
            const uint32_t w1[4] = {f.k[1][x].x, f.k[1][x].y, f.k[1][x].z, f.k[1][x].w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {  // one k step per word: four elements of each row
                uint32_t a0, a2, a1, a3;
                codes_to_bf16<KV>(w0[w], s0, s0.big, a0, a2);
                codes_to_bf16<KV>(w1[w], s1, s1.big, a1, a3);
#pragma unroll
                for (int nh = 0; nh < NH; ++nh) mma_bf16(s[nh], a0, a1, a2, a3, q[nh][4 * x + w].x, q[nh][4 * x + w].y);
            }
        }
    }
}

// The queries of head 8 nh + g in the k order of scores().
template <int D, int KV>
__device__ __forceinline__ void load_q(uint2 (&q)[D / 16], const __nv_bfloat16 *row, bool ok, int t) {
    const uint4 *p = reinterpret_cast<const uint4 *>(row);
#pragma unroll
    for (int x = 0; x < D / 32; ++x) {
        // bf16 cache: elements 32 x + 8 t ...; 8 bits: halves of 64 (x / 2) + 16 t ...
        const int at = KV == kKvBf16 ? 4 * x + t : 8 * (x >> 1) + 2 * t + (x & 1);
        const uint4 u = ok ? ld_now(p + at) : make_uint4(0u, 0u, 0u, 0u);
        q[2 * x] = make_uint2(u.x, u.y);
        q[2 * x + 1] = make_uint2(u.z, u.w);
    }
}

// o[nh][j] += V^T P^T, P being the sum of TERMS matrices; accumulator j holds elements elem(j, g), elem(j, g) + 1 of heads 2t, 2t + 1
template <int D, int KV>
__device__ __forceinline__ int elem(int j, int g) {
    return KV == kKvBf16 ? 64 * (j >> 2) + 8 * g + 2 * (j & 3) : (D / 8) * g + 2 * j;
}
template <int D, int KV, int NH, int TERMS>
__device__ __forceinline__ void accumulate(const Frag<D, KV> &f, const uint32_t (&p)[TERMS][NH][2], float (&o)[NH][D / 16][4]) {
    if constexpr (KV == kKvBf16) {
#pragma unroll
        for (int x = 0; x < f.CV; ++x) {
            const uint32_t r[4][4] = {{f.v[0][x].x, f.v[0][x].y, f.v[0][x].z, f.v[0][x].w},
                                      {f.v[1][x].x, f.v[1][x].y, f.v[1][x].z, f.v[1][x].w},
                                      {f.v[2][x].x, f.v[2][x].y, f.v[2][x].z, f.v[2][x].w},
                                      {f.v[3][x].x, f.v[3][x].y, f.v[3][x].z, f.v[3][x].w}};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t a0 = __byte_perm(r[0][w], r[1][w], 0x5410), a1 = __byte_perm(r[0][w], r[1][w], 0x7632);
                const uint32_t a2 = __byte_perm(r[2][w], r[3][w], 0x5410), a3 = __byte_perm(r[2][w], r[3][w], 0x7632);
#pragma unroll
                for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                    for (int y = 0; y < TERMS; ++y) mma_bf16(o[nh][4 * x + w], a0, a1, a2, a3, p[y][nh][0], p[y][nh][1]);
            }
        }
    } else {
        const Scale2<KV> s01 = scale_pair<KV>(f.vs[0], f.vs[1]), s23 = scale_pair<KV>(f.vs[2], f.vs[3]);
#pragma unroll
        for (int w = 0; w < f.VW; ++w) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // codes 2h, 2h + 1 of the word, each with its pair of keys
                const uint32_t sel = h ? 0x7362 : 0x5140;
                uint32_t a0, a1, a2, a3;
                codes_to_bf16<KV>(__byte_perm(f.v[0][w], f.v[1][w], sel), s01, s01.big, a0, a1);
                codes_to_bf16<KV>(__byte_perm(f.v[2][w], f.v[3][w], sel), s23, s23.big, a2, a3);
#pragma unroll
                for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                    for (int y = 0; y < TERMS; ++y) mma_bf16(o[nh][2 * w + h], a0, a1, a2, a3, p[y][nh][0], p[y][nh][1]);
            }
        }
    }
}

// Warps of a kernel that an SM holds, and the most of one CTA: by the registers that its fragments take (16 columns need twice
// the queries and accumulators).  At d = 128, bf16 spills in 128 registers, and 8 bits wait for each other's: 16 warps per SM
// instead of 12 took 11.2 instead of 10.7 us for 64 sequences x 4 KV heads, e4m3, 7.1 instead of 6.1 for 8, 12.0 instead of 10.4 for
// 16 drafts of 5; at d = 64, 12 warps instead of 16 took 7.9 instead of 6.1 us for 32 sequences x 12 KV heads, int8.
constexpr int sm_warps(int D, int KV, int NH) { return NH == 2 ? 8 : D == 128 ? 12 : 16; }
constexpr int max_warps(int D, int KV, int NH) { return sm_warps(D, KV, NH) / (NH == 2 ? 1 : 2); }

// The row of token at / H and head at % H, position i of sequence b, by itself (pi_row.cuh).
template <int D, int KV, bool TREE>
__device__ __noinline__ void again(const Args &a, int b, int i, int kvh, int at, int ctx, int t0) {
    const int tok = at / a.s.H;
    RowKeys k = row_keys(a.s, i, kvh, a.m_first, a.q + tok * a.q_stride + (at - tok * a.s.H) * D,
                         a.batch.table + (long long)b * a.cache.width, a.alpha ? a.alpha + at : nullptr);
    if (TREE) {
        k.parent = a.parent + t0;
        k.ctx = ctx;
        k.node = tok - t0;
    }
    attend_row<D, KV, TREE>(a.cache, k, a.out + (long long)at * D);
}

// NH: groups of 8 columns (1 or 2), a column being one query head of one token
template <int D, int KV, int NH, Kind KIND>
__global__ void __launch_bounds__(max_warps(D, KV, NH) * 32, sm_warps(D, KV, NH) / max_warps(D, KV, NH))
paged_rows_kernel(const __grid_constant__ Args a) {
    constexpr bool TOKENS = KIND != kSingle, TREE = KIND == kTree;
    const Shape &s = a.s;
    const PagedCache &c = a.cache;
    constexpr int PART = D + 4;  // floats of a column's partial state: o[D], m, l, padding to 16 bytes
    extern __shared__ __align__(16) float part[];  // [warps][columns][PART]
    const int P = gridDim.x, rank = blockIdx.x, kvh = blockIdx.y, warps = blockDim.x >> 5;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int G = s.H / s.Hkv, h0 = kvh * G;

    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // ---- the CTA's sequence b, its queries' positions first .. last and their first packed token tok0
    int b, first, last, tok0, n_tok = 1;
    TreeGroup *tree = nullptr;
    TreeParents parents;
    if constexpr (TREE) tree = tree_group();
    if constexpr (!TOKENS) {
        b = tok0 = blockIdx.z;
        // the table's first entries are on their way while the length is (5.76 -> 5.70 us; copied to shared memory, 5.58 instead
        // of 5.30 in a later state)
        if (32 * threadIdx.x < c.width) asm volatile("prefetch.global.L1 [%0];" ::"l"(a.batch.table + (long long)b * c.width + 32 * threadIdx.x));
        last = ld_now(a.lens + b) - 1;
        if (last < -1 || last >= (long long)c.width << c.page_log2) {
            if (threadIdx.x == 0) record_index(a.index_word);
            last = -1;
        }
        first = last;
    } else {
        if (blockIdx.z == 0 && kvh == 0 && rank == 0 && (!TREE || a.group0 == 0))  // offsets that decrease may hide their sequence from the search below
            for (int j = threadIdx.x; j < a.batch.B; j += blockDim.x)
                if (ld_now(a.batch.cu + j) > ld_now(a.batch.cu + j + 1)) record_index(a.index_word);
        const int id = (TREE ? a.group0 : 0) + blockIdx.z, B = a.batch.B;
        auto start = [&](int j, int at) -> long long { return plan::group_start(j, at, a.group); };
        int t0, t1, ctx;
        if (B <= 32) {  // a sequence per lane, so that one round of loads has everything
            const bool in = lane < B;
            const int c0 = in ? ld_now(a.batch.cu + lane) : 0, c1 = in ? ld_now(a.batch.cu + lane + 1) : 0, x = in ? ld_now(a.batch.ctx + lane) : 0;
            b = __popc(__ballot_sync(kFull, in && start(lane + 1, c1) <= id));
            t0 = __shfl_sync(kFull, c0, b & 31);
            t1 = __shfl_sync(kFull, c1, b & 31);
            ctx = __shfl_sync(kFull, x, b & 31);
            if (b >= B) return;
        } else {
            b = find_sequence(B, [&](int j) { return start(j, ld_now(a.batch.cu + j)) <= id; });
            if (b >= B) return;
            t0 = ld_now(a.batch.cu + b);
            t1 = ld_now(a.batch.cu + b + 1);
            ctx = ld_now(a.batch.ctx + b);
        }
        if (!sequence_ok(c, a.batch, t0, t1, ctx)) {
            if (threadIdx.x == 0) record_index(a.index_word);
            return;
        }
        const long long x = (id - start(b, t0)) * a.group;
        if (x < 0 || x >= t1 - t0) return;
        const int x0 = (int)x;
        tok0 = t0 + x0;
        first = ctx + x0;
        last = min(first + a.group, ctx + t1 - t0) - 1;
        n_tok = last - first + 1;
        if constexpr (TREE) load_parents(parents, a.parent + t0, t1 - t0, x0, ctx);  // (and the page table's entries)
        if constexpr (TREE) {
            const int at = (band_lo(ctx, s.mode, s.k_local) >> c.page_log2) + 32 * threadIdx.x;
            if (at <= (ctx + t1 - t0 - 1) >> c.page_log2) asm volatile("prefetch.global.L1 [%0];" ::"l"(a.batch.table + (long long)b * c.width + at));
        }
    }
    const int cols = n_tok * G;
    // column x: token x / G, head x % G
    auto row_of = [&](int x) -> long long { return TOKENS ? (long long)(tok0 + x / G) * s.H + h0 + x % G : (long long)b * s.H + h0 + x; };

    uint2 q[NH][D / 16];
    float offb[NH][2], offs[NH][2];
    int tok[NH][2];  // the token of the lane's columns
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
        const int x = 8 * nh + g;
        load_q<D, KV>(q[nh], a.q + (TOKENS ? (tok0 + x / G) * a.q_stride + (h0 + x % G) * D : b * a.q_stride + (h0 + x) * D), x < cols, t);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int y = 8 * nh + 2 * t + e;
            tok[nh][e] = TOKENS ? y / G : 0;
            const float al = a.alpha && y < cols ? ld_now(a.alpha + row_of(y)) : 1.f;
            offb[nh][e] = a.alpha ? log2f(al) : 0.f;
            offs[nh][e] = log2f(1.f - al);
        }
    }
    if constexpr (TREE) {  // first and last: the lowest and the highest position of the nodes
        if (!tree_walk(*tree, parents, s, n_tok, first, last)) {
            if (threadIdx.x == 0) record_index(a.index_word);
            return;
        }
    }
    // ---- the key list: the band lo .. last, then for each skip distance m * period, m = m_first ..., the n_tok keys that
    // many before the queries (some may lie before the sequence)
    const int lo = last >= 0 ? band_lo(first, s.mode, s.k_local) : 0;
    int n_band = last - lo + 1, n_cached = n_band;
    if constexpr (TREE) {  // the band's cached keys, then the nodes that some of the queries attend
        n_cached = max(tree->ctx - lo, 0);
        n_band = n_cached + tree->n_rows;
    }
    int n_keys = n_band;
    if (last >= 0 && s.mode != kModeEcp && s.S > 0) n_keys += n_tok * max(0, min(s.S, last / s.period) - a.m_first + 1);
    const int n_tiles = (n_keys + KEYS - 1) / KEYS;
    // Key kk: its cache row (-1: none) and, for the masks, its position (band) or -1 - u (the key of query first + u alone).
    auto key = [&](int kk, int &row, int &tag) {
        row = -1;
        tag = -0x7fffffff;  // attended by nobody
        if (kk >= n_keys) return;
        int pos;
        if (kk < n_cached) {
            pos = tag = lo + kk;
        } else if (TREE && kk < n_band) {
            const int node = tree->row[kk - n_cached];
            pos = tree->ctx + node;
            tag = kNodeTag + tree->mask[node];
        } else {
            const int x = kk - n_band, w = TOKENS ? x / n_tok : x, u = TOKENS ? x - w * n_tok : 0;
            pos = (TREE ? tree->pos[u] : first + u) - (a.m_first + w) * s.period;
            if (pos < 0 || (TREE && pos >= tree->ctx)) return;
            tag = -1 - u;
        }
        const int pg = page_of(c, a.batch.table, b, pos);
        if (pg >= 0) {
            row = row_in_page(c, pg, kvh, pos);
        } else {
            tag = -0x7fffffff;
            record_index(a.index_word);
        }
    };

    float m[NH][2], l[NH][2], o[NH][D / 16][4];
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
#pragma unroll
        for (int e = 0; e < 2; ++e) { m[nh][e] = -INFINITY; l[nh][e] = 0.f; }
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nh][j][e] = 0.f;
    }

    // ---- the warp's tiles.  Lanes 0-15 hold the rows of one tile, 16-31 those of the warp's next one.  (Requesting the next
    // tile's K after this one's scores, and its V after P V, took 64 sequences 15.8 us instead of 12.7 in an earlier state that takes
    // 10.0 now: the waits for the older loads also wait for the newer ones.)
    const int step = P * warps;
    int tile = rank * warps + warp;
    Frag<D, KV> f;
    int row, tag;
    auto load_keys = [&](int u) {
#pragma unroll
        for (int x = 0; x < 2; ++x) load_k<D, KV>(f, c, x, __shfl_sync(kFull, row, u * KEYS + g + 8 * x), t);
    };
    auto load_values = [&](int u) {
#pragma unroll
        for (int x = 0; x < 4; ++x) load_v<D, KV>(f, c, x, __shfl_sync(kFull, row, u * KEYS + 2 * t + (x & 1) + 8 * (x >> 1)), g);
    };
    if (tile < n_tiles) key((tile + (lane < KEYS ? 0 : step)) * KEYS + (lane & (KEYS - 1)), row, tag);
#pragma unroll 1
    for (int u = 0; tile < n_tiles; tile += step, u ^= 1) {
        load_keys(u);
        load_values(u);
        const int tag0 = __shfl_sync(kFull, tag, u * KEYS + g), tag1 = __shfl_sync(kFull, tag, u * KEYS + g + 8);
        float sc[NH][4] = {};
        scores<D, KV, NH>(f, q, sc, t);
        if (u == 1 && tile + step < n_tiles) key((tile + (lane < KEYS ? step : 2 * step)) * KEYS + (lane & (KEYS - 1)), row, tag);
        constexpr int TERMS = TREE ? 2 : 1;  // of a weight, bf16 each
        uint32_t p[TERMS][NH][2];
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
            float pr[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = TREE ? tree->pos[tok[nh][e]] : first + tok[nh][e];
                const int lo_i = TOKENS ? band_lo(i, s.mode, s.k_local) : lo;
                auto logit = [&](int tg, float x) -> float {
                    if (tg >= 0) return tg >= lo_i && tg <= i ? fmaf(x, s.scale_log2, offb[nh][e]) : -INFINITY;
                    if (TREE && tg < -kTreeGroup && tg >= kNodeTag) {
                        const int by = (tg - kNodeTag) >> tok[nh][e];
                        return by & 1 ? fmaf(x, s.scale_log2, offb[nh][e]) : by >> kTreeGroup & 1 ? fmaf(x, s.scale_log2, offs[nh][e]) : -INFINITY;
                    }
                    return tg == -1 - tok[nh][e] ? fmaf(x, s.scale_log2, offs[nh][e]) : -INFINITY;
                };
                const float z0 = logit(tag0, sc[nh][e]), z1 = logit(tag1, sc[nh][2 + e]);
                float mx = fmaxf(z0, z1);
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
                const float mn = fmaxf(m[nh][e], mx), ref = mn == -INFINITY ? 0.f : mn;
                const float corr = exp2f(m[nh][e] - ref);
                pr[e] = exp2f(z0 - ref);
                pr[2 + e] = exp2f(z1 - ref);
                l[nh][e] = fmaf(l[nh][e], corr, pr[e] + pr[2 + e]);
                m[nh][e] = mn;
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    o[nh][j][e] *= corr;
                    o[nh][j][2 + e] *= corr;
                }
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if constexpr (TREE) {  // the weights' high halves, and what those leave, rounded
                    const uint32_t u0 = __float_as_uint(pr[2 * x]), u1 = __float_as_uint(pr[2 * x + 1]);
                    p[0][nh][x] = transpose8(__byte_perm(u0, u1, 0x7632));
                    p[1][nh][x] = transpose8(pack_bf16x2(pr[2 * x] - __uint_as_float(u0 & 0xffff0000u), pr[2 * x + 1] - __uint_as_float(u1 & 0xffff0000u)));
                } else {
                    p[0][nh][x] = transpose8(pack_bf16x2(pr[2 * x], pr[2 * x + 1]));
                }
            }
        }
        accumulate<D, KV, NH, TERMS>(f, p, o);
    }

    // ---- the warps' partial states to shared memory
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float sum = l[nh][e];
            sum += __shfl_xor_sync(kFull, sum, 4);
            sum += __shfl_xor_sync(kFull, sum, 8);
            sum += __shfl_xor_sync(kFull, sum, 16);
            const int x = 8 * nh + 2 * t + e;
            if (x < cols) {
                float *ps = part + (warp * cols + x) * PART;
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
                    *reinterpret_cast<float2 *>(ps + elem<D, KV>(j, g)) = make_float2(o[nh][j][e], o[nh][j][2 + e]);
                if (g == 0) *reinterpret_cast<float2 *>(ps + D) = make_float2(m[nh][e], sum);
            }
        }
    // ---- and meet: four columns of a row per thread, all the cluster's states at once (a merge in each CTA first and then one
    // of the CTAs' took 10.6 us where this takes 9.1, 16 drafts of up to 5 tokens in clusters of three)
    constexpr int PER_ROW = D / 4, BATCH = MEET;  // threads of a row; states in flight
    const int states = P * warps, items = cols * PER_ROW;
    const uint32_t base = smem_addr(part);
    auto meet = [&](auto across) {
        for (int w0 = (rank * warps + warp) * 32; w0 < items; w0 += states * 32) {
            const bool in = w0 + lane < items;
            const int x = in ? (w0 + lane) / PER_ROW : cols - 1, col = 4 * (lane % PER_ROW);
            float mt = -INFINITY, lt = 0.f;
            float4 ot = make_float4(0.f, 0.f, 0.f, 0.f);
            int wp = 0, cta = 0;
#pragma unroll 1
            for (int y0 = 0; y0 < states; y0 += BATCH) {
                float2 ml[BATCH];
                float4 ov[BATCH];
#pragma unroll
                for (int y = 0; y < BATCH; ++y) {
                    ml[y] = make_float2(-INFINITY, 0.f);
                    ov[y] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (y0 + y >= states) continue;
                    const uint32_t at = (uint32_t)((wp * cols + x) * PART) * 4u;
                    if constexpr (across.value) {
                        const uint32_t there = peer_addr(base + at, cta);
                        ml[y] = ld_peer2(there + D * 4);
                        ov[y] = ld_peer4(there + col * 4);
                    } else {
                        const float *ps = part + at / 4;
                        ml[y] = *reinterpret_cast<const float2 *>(ps + D);
                        ov[y] = *reinterpret_cast<const float4 *>(ps + col);
                    }
                    if (++wp == warps) {
                        wp = 0;
                        ++cta;
                    }
                }
                float mn = mt;
#pragma unroll
                for (int y = 0; y < BATCH; ++y) mn = fmaxf(mn, ml[y].x);
                const float ref = mn == -INFINITY ? 0.f : mn, corr = exp2f(mt - ref);
                mt = mn;
                lt *= corr;
                ot = make_float4(ot.x * corr, ot.y * corr, ot.z * corr, ot.w * corr);
#pragma unroll
                for (int y = 0; y < BATCH; ++y) {
                    const float e = exp2f(ml[y].x - ref);
                    lt = fmaf(e, ml[y].y, lt);
                    ot = make_float4(fmaf(e, ov[y].x, ot.x), fmaf(e, ov[y].y, ot.y), fmaf(e, ov[y].z, ot.z), fmaf(e, ov[y].w, ot.w));
                }
            }
            const float inv = lt == 0.f ? 0.f : 1.f / lt;
            if (lt == 0.f) ot = make_float4(0.f, 0.f, 0.f, 0.f);  // no finite logit: 0, whatever the values are
            const uint2 four = make_uint2(pack_bf16x2(ot.x * inv, ot.y * inv), pack_bf16x2(ot.z * inv, ot.w * inv));
            const long long at = row_of(x);
            bool mine = in;
            if constexpr (TOKENS) {  // a value of another token's key may have made a row non-finite (pi_row.cuh)
                uint32_t seen = 0u;
                watch(seen, four.x);
                watch(seen, four.y);
                unsigned bad = __ballot_sync(kFull, in && went_bad(seen) && lt == lt);
                while (bad) {
                    const int y = __shfl_sync(kFull, x, __ffs(bad) - 1);
                    if constexpr (TREE) again<D, KV, true>(a, b, tree->pos[y / G], kvh, (int)row_of(y), tree->ctx, tok0 - tree->node0);
                    else again<D, KV, false>(a, b, first + y / G, kvh, (int)row_of(y), 0, 0);
                    bad &= ~__ballot_sync(kFull, x == y);
                    mine = mine && x != y;
                }
            }
            if (mine) *reinterpret_cast<uint2 *>(a.out + at * D + col) = four;
            if (in && col == 0) a.lse[at] = lt == 0.f ? -INFINITY : (mt + log2f(lt)) * kLn2;
        }
    };
    if (P == 1) {
        __syncthreads();
        meet(std::false_type{});
        return;
    }
    cluster_sync();
    meet(std::true_type{});
    cluster_leave();  // a CTA's shared memory stays until the others have read it
}

// Warps per CTA and CTAs per cluster for `pairs` (token group, KV head) pairs of up to `tiles` key tiles each.  A warp takes
// its tiles one after the other, each a round trip to memory; the CTAs that the SMs do not hold at once start another.
// Measured: 64 sequences x 4 KV heads, 17 tiles, bf16, d = 128: 6 warps 10.3 us, 4 warps 12.6, 3 warps in clusters of two 11.8;
// 32 x 12 pairs of 9 int8 tiles, d = 64: 5 warps 5.5, 4 warps 6.4, 6 warps (two waves) 8.2; one sequence x 4 heads, 17 e4m3
// tiles: clusters of 6 x 3 warps 5.0, 5 x 4 5.2, 3 x 6 5.3, one CTA of 6 warps 7.2.
// `most`: warps of a cluster.  Trees have up to MEET of them, whose states of up to 8 columns meet in one turn: a tree of 26 nodes, 16 heads on
// 4, d = 128, bf16: 2 warps in clusters of 5 9.5 us, 4 in clusters of 5 10.5.
struct Split {
    int warps, ctas;
};
static Split split(int sm_w, int max_w, long long tiles, long long pairs, int most = MAX_P * 32) {
    Split best{max_w, 1};
    long long least = -1;
    const long long sms = sm_count();
    for (int ctas = 1; ctas <= MAX_P; ++ctas)
        for (int w = 2; w <= max_w && w * ctas <= most; ++w) {
            const long long waves = (pairs * ctas - 1) / (sm_w / w * sms) + 1, rounds = (tiles - 1) / (w * ctas) + 1;
            // half a round for meeting across a cluster; then as few warps in all as do, then small CTAs
            const long long cost = (2 * waves * (rounds + 2) + (ctas > 1 ? 1 : 0)) * 128 + w * ctas;
            if (least < 0 || cost <= least) {
                least = cost;
                best = Split{w, ctas};
            }
        }
    return best;
}

template <int D, int KV, int NH, Kind KIND>
static cudaError_t launch(const Args &a, int groups, long long keys, cudaStream_t st) {
    const int cols = a.group * (a.s.H / a.s.Hkv);
    const Split sp = split(sm_warps(D, KV, NH), max_warps(D, KV, NH), (keys + KEYS - 1) / KEYS, (long long)groups * a.s.Hkv, KIND == kTree ? MEET : MAX_P * 32);
    auto *kernel = paged_rows_kernel<D, KV, NH, KIND>;
    static PerDeviceOnce configured;  // shared memory above the 48 KB default
    int dev = 0;
    cudaGetDevice(&dev);
    if (configured.needed(dev)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   max_warps(D, KV, NH) * 8 * NH * (D + 4) * 4);
        if (e != cudaSuccess) return e;
        configured.mark(dev);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)sp.ctas, (unsigned)a.s.Hkv, (unsigned)groups);
    cfg.blockDim = dim3((unsigned)sp.warps * 32, 1, 1);
    cfg.dynamicSmemBytes = (size_t)(sp.warps * cols * (D + 4) * 4);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)sp.ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = sp.ctas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int D, int KV, Kind KIND>
static cudaError_t launch_shape(const Args &a, int groups, long long keys, cudaStream_t st) {
    return a.group * (a.s.H / a.s.Hkv) <= 8 ? launch<D, KV, 1, KIND>(a, groups, keys, st) : launch<D, KV, 2, KIND>(a, groups, keys, st);
}

template <Kind KIND>
static cudaError_t launch_types(const Args &a, int groups, long long keys, cudaStream_t st) {
    const bool d64 = a.s.d == 64;
    switch (a.cache.kv_type) {
        case kKvBf16: return d64 ? launch_shape<64, kKvBf16, KIND>(a, groups, keys, st) : launch_shape<128, kKvBf16, KIND>(a, groups, keys, st);
        case kKvE4m3: return d64 ? launch_shape<64, kKvE4m3, KIND>(a, groups, keys, st) : launch_shape<128, kKvE4m3, KIND>(a, groups, keys, st);
        default: return d64 ? launch_shape<64, kKvInt8, KIND>(a, groups, keys, st) : launch_shape<128, kKvInt8, KIND>(a, groups, keys, st);
    }
}

// The longest band and the most skips of a query, at the last position that a page table reaches.
struct MostKeys {
    long long cap, band, windows;
    MostKeys(const Shape &s, const PagedCache &c) : cap((long long)c.width << c.page_log2), windows(0) {
        band = std::min(cap, s.mode == kModeEcp ? 2LL * s.k_local : s.k_local + 1LL);
        if (s.mode != kModeEcp && s.S > 0)
            windows = std::max(0LL, std::min<long long>(s.S, cap / s.period) - first_skip_multiple(s) + 1);
    }
    // keys of the longest list of `tokens` consecutive queries
    long long list(int tokens) const { return std::min(cap, band + tokens - 1) + windows * tokens; }
};

}  // namespace decp

cudaError_t launch_decode_paged(const DecodePagedArgs &d, cudaStream_t st) {
    using namespace decp;
    const Shape &s = d.s;
    Args a{d.q, d.q_stride, d.alpha, d.lens, PagedBatch{d.table, nullptr, nullptr, s.B, s.B}, d.out, d.lse, s, d.cache, d.index_word,
           s.mode != kModeEcp && s.S > 0 ? first_skip_multiple(s) : 1, 1, nullptr, 0};
    return launch_types<kSingle>(a, s.B, MostKeys(s, d.cache).list(1), st);
}

// Tokens per CTA: as many as 8 columns hold (16 took a batch of five drafted tokens, 4 heads per KV head, 15.0 us, 8 10.4).
static int token_group(int G) { return std::max(1, 8 / G); }

// Whether a call's chunks are so short that this kernel beats the tensor-core pipeline (pi_extend_tc.cu), whose blocks of 128
// rows take about the same time however few of them hold queries.  Judged by the sizes that the host knows, as if all
// sequences had the same length, by two estimates in us: this kernel's launch and its rounds of tiles over the SMs' warps
// (a CTA's start and merge count as six tiles), and the pipeline's launches and its turns of blocks, tile by tile, with the
// conversion of an 8-bit cache.  Fitted to 84 shapes (16 heads on 4, d = 128, and 12 on 12, d = 64; 1 to 128 sequences of 2 to
// 256 tokens; three types), of which it gets all but one right and that one 10 % wrong; of 108 others (other heads, bands and
// skips, up to 8000 tokens) nine are 8 to 30 % slower than they could be.  For instance (this kernel / pipeline):
//   16 heads on 4, d = 128, band 256, bf16:  1 sequence x 128 tokens 10.0 / 12.7, x 256 15.0 / 12.9; 32 x 4 15.6 / 14.2, x 8 16.9 / 14.1
//                                     e4m3:  32 x 8 19.2 / 21.5, x 16 34.8 / 21.2; 128 x 4 41.3 / 55.6, x 8 68.1 / 54.8
//   12 on 12, d = 64, band 128, bf16:  1 x 256 8.4 / 16.3; 32 x 16 13.6 / 17.2, x 32 23.5 / 24.0; 128 x 16 37.7 / 40.7
bool extend_few_rows(const ExtendArgs &e) {
    const Shape &s = e.s;
    const PagedCache &c = e.cache;
    const int G = s.H / s.Hkv, group = token_group(G);
    const long long T = e.batch.T, B = std::min<long long>(e.batch.B, T);
    if (G > 16 || s.Hkv > 65535 || (T + e.batch.B * (long long)(group - 1)) / group > 65535) return false;
    const decp::MostKeys most(s, c);
    if (most.list(group) >= (1LL << 30)) return false;
    const bool quant = c.kv_type != kKvBf16;
    const long long n = (T + B - 1) / B, band = most.band, windows = most.windows;
    const long long tiles = (most.list(group) + decp::KEYS - 1) / decp::KEYS;
    const long long ctas = B * ((n + group - 1) / group) * s.Hkv, sms = sm_count();
    const double rounds = (double)ctas * (double)(tiles + 6) / (double)(sms * decp::sm_warps(s.d, c.kv_type, group * G > 8 ? 2 : 1));
    const double few = 6.0 + (quant ? 1.8 : 1.4) * rounds;
    const int heads = packed_heads(G), rows = 128 / heads;
    const long long turns = (B * ((n + rows - 1) / rows) * (s.H / heads) - 1) / (2 * sms) + 1, m = std::min<long long>(n, rows);
    const double block = (double)(band + m) / 32 + 1 + (double)windows * ((double)((m - 1) / 32) + 1.5);
    const double converted = (double)(B * s.Hkv) * s.d / 64 * ((double)(band + n) / 32 + 1 + (double)windows * ((double)n / 32 + 1.5));
    return few <= 7.5 + 0.45 * (double)turns * block + (quant ? 1.0 + 0.001 * converted : 0.0);
}

cudaError_t launch_extend_few(const ExtendArgs &e, cudaStream_t st) {
    using namespace decp;
    const Shape &s = e.s;
    const int group = token_group(s.H / s.Hkv);
    Args a{e.q, e.q_stride, e.alpha, nullptr, e.batch, e.out, e.lse, s, e.cache, e.index_word,
           s.mode != kModeEcp && s.S > 0 ? first_skip_multiple(s) : 1, group, nullptr, 0};
    return launch_types<kTokens>(a, (int)((e.batch.T + e.batch.B * (long long)(group - 1)) / group), MostKeys(s, e.cache).list(group), st);
}

// Whether this kernel beats the tensor-core one for a batch of trees (pi_tree_tc.cu), and whether either can number its work.  As in
// extend_few_rows, by two estimates in us from the sizes that the host knows, all trees taken as equally large: this kernel's waves of
// rounds of tiles (split()), and the other's turns of blocks, each a start and tiles of 32 keys.  Fitted to 204 shapes (16 heads on 4, 8 on 1 and 16 on
// 16, d = 128; 12 on 12, 8 on 8 and 7 on 1, d = 64; bf16 and e4m3; 1 to 64 trees of 2 to 160 nodes), of which it gets 196 right to 5 %
// and the others wrong by 5 to 21 %.  For instance (this kernel / the other):
//   16 heads on 4, d = 128, band 256, bf16:  1 tree of 26 nodes 9.3 / 12.9, of 160 15.4 / 15.7; 8 of 32 17.8 / 13.2, 32 of 32 65.0 / 14.0
//                                     e4m3:  1 of 26 9.9 / 16.5; 8 of 8 12.3 / 15.2, 8 of 32 21.3 / 16.9
//   12 on 12, d = 64, band 128, bf16:  1 of 26 7.5 / 9.6; 16 of 16 11.5 / 12.7, 32 of 32 28.7 / 20.3
bool tree_few(const ExtendTreeArgs &t, bool &fits) {
    const ExtendArgs &e = t.e;
    const Shape &s = e.s;
    const PagedCache &c = e.cache;
    const int G = s.H / s.Hkv, group = token_group(G);
    const long long T = e.batch.T, B = std::min<long long>(e.batch.B, T), n = std::min<long long>((T + B - 1) / B, kTreeMax);
    const decp::MostKeys most(s, c);
    const int heads = tree_heads(G), rows = 128 / heads;
    const long long blocks = (T + e.batch.B * (long long)(rows - 1)) / rows * (s.H / heads);
    const bool tc_fits = blocks <= 0x7fffffffLL && most.band + kTreeMax + most.windows * kTreeMax < (1LL << 30);
    const bool few_fits = G <= 16 && s.Hkv <= 65535 && most.band + kTreeMax + most.windows * group < (1LL << 30) &&
                          (T + e.batch.B * (long long)(group - 1)) / group <= 0x7fffffffLL;
    fits = tc_fits || few_fits;
    if (!tc_fits || !few_fits) return few_fits;
    const bool quant = c.kv_type != kKvBf16, d64 = s.d == 64;
    const int nh = group * G > 8 ? 2 : 1, sm_w = decp::sm_warps(s.d, c.kv_type, nh);
    const long long tiles = (most.list(group) + std::min<long long>(n, 8 * group) + decp::KEYS - 1) / decp::KEYS;
    const long long pairs = B * ((n + group - 1) / group) * s.Hkv, sms = sm_count();
    const decp::Split sp = decp::split(sm_w, decp::max_warps(s.d, c.kv_type, nh), tiles, pairs, decp::MEET);
    const long long waves = (pairs * sp.ctas - 1) / (sm_w / sp.warps * sms) + 1, rounds = (tiles - 1) / (sp.warps * sp.ctas) + 1;
    const double few = 2.4 + (double)waves * ((double)rounds + 2.6) * (d64 ? 1.42 : 1.8);
    const long long turns = (B * ((n + rows - 1) / rows) * (s.H / heads) - 1) / (2 * sms) + 1;
    const double block_tiles = (double)(most.band + n + 6 * most.windows) / 32 + 0.5;
    return few <= 1.5 + (double)turns * (6.9 + 0.4 * block_tiles * (d64 ? 0.66 : 1.0) * (quant ? 1.93 : 1.0));
}

cudaError_t launch_extend_tree(const ExtendTreeArgs &t, cudaStream_t st) {
    using namespace decp;
    if (!t.few) return launch_tree_tc(t, st);
    const ExtendArgs &e = t.e;
    const Shape &s = e.s;
    const int group = token_group(s.H / s.Hkv);
    const MostKeys most(s, e.cache);
    const long long keys = most.band + std::min<long long>(e.batch.T, kTreeMax) + most.windows * group;
    Args a{e.q, e.q_stride, e.alpha, nullptr, e.batch, e.out, e.lse, s, e.cache, e.index_word,
           s.mode != kModeEcp && s.S > 0 ? first_skip_multiple(s) : 1, group, t.parent, 0};
    const long long groups = (e.batch.T + e.batch.B * (long long)(group - 1)) / group;
    constexpr int MOST = 65535;  // of a grid's third dimension
    for (long long g0 = 0; g0 < groups; g0 += MOST) {
        a.group0 = (int)g0;
        const cudaError_t err = launch_types<kTree>(a, (int)std::min<long long>(MOST, groups - g0), keys, st);
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

}  // namespace pi
