// pi_tree_tc.cu -- attention of drafted trees over the paged cache on the tensor cores (tcgen05), for batches whose trees have
// many nodes (pi_decode_paged.cu has the kernel for few).
//
// A block is 128 rows, the M of every product: GP query heads of one KV group x R nodes of one tree.  Its keys are a list that is cut into
// tiles of 32 without regard to positions or pages: the cached keys of the band, then the tree's nodes, then for each skip distance the
// cached keys that far before the depths that occur.  A tree's nodes share nearly all of their cached keys, so the list is hardly longer
// than one node's, and since its rows are gathered one by one the few keys of a skip window cost no tile of their own.
//   warps 0-3   softmax and epilogue, a thread per row: scores from TMEM, masks as 32 bits per tile, a running reference and sum,
//               P back to TMEM as two bf16 terms, whose sum is within 2^-15 of it (the sum takes the unrounded values; one
//               term, as in the forward: 48 trees of up to 64 nodes, bf16, 17.4 instead of 18.6 us, and 2.3e-3 instead of 1.7e-3 from
//               64 bits, of which the output's own rounding is 1.7e-3)
//   warps 4-7   producers: the tile's page-table entries a tile ahead, rows of K and V into the swizzled layout of the
//               products, by cp.async (bf16), or by way of the tile as it is, whose 8-bit codes become bf16 (exact, pi_paged.cuh)
//   warp 8      issues S = Q K^T (Q in TMEM) and O += P V (P in TMEM), S a tile ahead of P V (d = 64: three)
// The ancestors of a node are found by walking the parents in shared memory once per block; for each of its nodes and each node of
// the tree two bits say whether it lies in the band or is a skip.  Meanwhile the first tiles of cached keys, which do not depend on the tree, are
// on their way.
#include "pi_launch.h"
#include "pi_mma.cuh"
#include "pi_paged.cuh"
#include "pi_row.cuh"
#include "pi_step.h"
#include "pi_tc_ptx.cuh"
#include "pi_tile.cuh"
#include "pi_tree.cuh"

namespace pi {
namespace ttc {

using namespace tc;

constexpr int BM = 128;          // rows per block (MMA M)
constexpr int THREADS = 288;
constexpr int MMA_WARP = 8;
constexpr int TMEM_COLS = 256;   // per CTA, two CTAs per SM
constexpr int ROW_BYTES = 128;   // one 64-element bf16 swizzle row
constexpr int PRODUCERS = 128;
constexpr int SCANNED = 4 * THREADS;  // sequences whose blocks are counted by every CTA
constexpr unsigned kFull = 0xffffffffu;

struct Args {
    ExtendTreeArgs t;
    int GP, R, R_log2, ngrp;  // heads and nodes of a block, groups of heads
    int m_first;
    FastDiv div_ngrp, div_G;
};

template <int D, int KV>
struct Cfg {
    static constexpr bool QUANT = KV != kKvBf16;
    static constexpr int NB = D == 64 ? 4 : 2;  // S buffers
    static constexpr int O_COL = 128, Q_COL = D == 128 ? 64 : 192;
    static constexpr int KD = D / 64;
    static constexpr int ST = D == 64 ? 8 : QUANT ? 4 : 6;  // stages of a K and a V tile; the last two are where the queries were
    static constexpr int Q_BYTES = BM * D * 2, Q_DBLK = BM * ROW_BYTES;
    static constexpr int TILE_BYTES = CHUNK * D * 2, DBLK = CHUNK * ROW_BYTES, STAGE_BYTES = 2 * TILE_BYTES;
    static constexpr int DATA_BYTES = ST * STAGE_BYTES;
    // 8-bit caches: tiles as they are, K, V and a word for each row's scales, ahead of their conversion
    static constexpr int RAW = 4, RAW_OFF = DATA_BYTES, RAW_SCALES = 2 * CHUNK * D, RAW_BYTES = RAW_SCALES + 2 * CHUNK * 4;
    static constexpr int META_OFF = DATA_BYTES + (QUANT ? RAW * RAW_BYTES : 0);
    static_assert(Q_BYTES == 2 * STAGE_BYTES && DATA_BYTES >= BM * D * 2, "two stages; the output is staged there too");
    static constexpr int k_at(int st) { return (st + 2) % ST * STAGE_BYTES; }
    static constexpr int v_at(int st) { return k_at(st) + TILE_BYTES; }
    // barriers
    static constexpr int B_Q = 0;              // queries in shared memory (128)
    static constexpr int B_QT = 1;             // queries in TMEM
    static constexpr int B_FULL = 2;           // [ST] a tile's K and V (128)
    static constexpr int B_EMPTY = B_FULL + ST;  // [ST] its P V done
    static constexpr int B_SF = B_EMPTY + ST;  // [NB] S in TMEM
    static constexpr int B_PR = B_SF + NB;     // [NB] P written over it (128)
    static constexpr int B_OF = B_PR + NB;     // O complete
    static constexpr int B_DR = B_OF + 1;      // all products done
    static constexpr int NBARS = B_DR + 1;
    static constexpr int arrivals(int i) { return i == B_Q || (i >= B_FULL && i < B_EMPTY) || (i >= B_PR && i < B_OF) ? 128 : 1; }
};

// What the block's threads share, behind the tiles.
struct Meta {
    uint64_t bars[32];
    uint32_t tmem, abort, bad[4];  // bad: rows that came out non-finite, a bit each
    int b, t0, n, ctx, x0, taken;  // sequence, its first token, nodes and context; the block's first node; whether these are set
    int broken;                    // a parent out of range
    int sums[THREADS / 32];
    unsigned odd[4][4];            // 8-bit caches, d = 64: of each raw tile, the rows of each producer warp whose scales are a word's high half
    unsigned depths[kTreeMax / 32];  // which depths occur among them
    int parent[kTreeMax];
    int pos[BM];
    unsigned band[kTreeMax / 32][BM], skip[kTreeMax / 32][BM];  // node's bits: the nodes that it attends
};

template <int D, int KV>
constexpr int smem_bytes() { return Cfg<D, KV>::META_OFF + 1024 + (int)sizeof(Meta); }
static_assert(smem_bytes<128, kKvBf16>() <= 115712 && smem_bytes<128, kKvInt8>() <= 115712 && smem_bytes<64, kKvBf16>() <= 115712 &&
              smem_bytes<64, kKvInt8>() <= 115712, "two CTAs per SM");

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
// One of the barrier's arrivals, once this thread's copies so far have landed.  (They are writes of the generic proxy: who waits
// for them in order to issue a product fences.)
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Place of 16-byte piece c of row r in a tile (or the queries) of 64-element blocks `dblk` bytes apart.
__device__ __forceinline__ uint32_t piece_at(int r, int c, int dblk) {
    return (uint32_t)((c >> 3) * dblk + r * ROW_BYTES + (((c & 7) ^ (r & 7)) << 4));
}

// tile_exp (pi_tile.cuh) in two bf16 terms: the values' high halves in r, what those leave, rounded, in `rest`.
__device__ __forceinline__ float tile_exp_terms(uint32_t *r, uint32_t *rest, float sc, float bo) {
    const uint64_t sc2 = pack2(sc, sc), bo2 = pack2(bo, bo), minus = pack2(-1.f, -1.f);
    uint64_t acc0 = pack2(0.f, 0.f), acc1 = pack2(0.f, 0.f);
#pragma unroll
    for (int c = 0; c < CHUNK; c += 2) {
        float z0, z1;
        unpack2(fma2(pack2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), sc2, bo2), z0, z1);
        const uint32_t p0 = __float_as_uint(fast_exp2(z0)), p1 = __float_as_uint(fast_exp2(z1));
        const uint64_t p = pack2(__uint_as_float(p0), __uint_as_float(p1));
        if ((c >> 1) & 1) acc1 = add2(acc1, p);
        else acc0 = add2(acc0, p);
        r[c / 2] = __byte_perm(p0, p1, 0x7632);
        unpack2(fma2(pack2(__uint_as_float(p0 & 0xffff0000u), __uint_as_float(p1 & 0xffff0000u)), minus, p), z0, z1);
        rest[c / 2] = pack_bf16(z0, z1);
    }
    float a0, a1, b0, b1;
    unpack2(acc0, a0, a1);
    unpack2(acc1, b0, b1);
    return (a0 + a1) + (b0 + b1);
}

// The block's keys: n_cached of the band, from position lo on, which are known before the tree is; its nodes; the skips.
struct Keys {
    int n_cached, n_band, n_keys;  // the band's cached keys; these and the nodes; all
    int lo, first;                 // first band key of a root; lowest position of the queries
    int spread;                    // keys of a skip window
};

template <int D, int KV>
__global__ void __launch_bounds__(THREADS, 2) tree_tc_kernel(const __grid_constant__ Args args) {
    using C = Cfg<D, KV>;
    constexpr int ST = C::ST, NB = C::NB;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
    Meta &m = *reinterpret_cast<Meta *>(smem + C::META_OFF);
    const uint32_t sbase = smem_u32(smem), sBar = smem_u32(m.bars);
    auto bar = [&](int i) -> uint32_t { return sBar + i * 8; };
    static_assert(C::NBARS <= 32, "barriers");
    const ExtendArgs &e = args.t.e;
    const Shape &s = e.s;
    const PagedCache &c = e.cache;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int id = args.div_ngrp.div(blockIdx.x), h0 = (blockIdx.x - id * args.ngrp) * args.GP, kvh = args.div_G.div(h0);

    if (warp == MMA_WARP) {
        if (lane < C::NBARS) mbar_init(bar(lane), (uint32_t)C::arrivals(lane));
        fence_barrier_init();
    }
    if (tid < kTreeMax / 32) m.depths[tid] = 0u;
    if (tid == 0) {
        m.abort = 0u;
        m.n = m.taken = m.broken = 0;
    }
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // ---- which block this is
    {
        const int B = e.batch.B, R = args.R;
        // sequence b, whose first block has the number `first`
        auto of = [&](int b, int t0, int t1, int ctx, long long first) {
            const long long x = (id - first) * R;
            if (x < 0 || x >= (long long)t1 - t0) return;
            if (atomicExch(&m.taken, 1)) return;  // (offsets that decrease: another one's, too)
            m.b = b; m.t0 = t0; m.n = t1 - t0; m.ctx = ctx; m.x0 = (int)x;
        };
        auto fits = [&](int t0, int t1, int ctx) -> bool {
            const bool in = sequence_ok(c, e.batch, t0, t1, ctx) && t1 - t0 <= kTreeMax;
            if (!in && blockIdx.x == 0) record_index(e.index_word);
            return in;
        };
        if (B <= SCANNED) {  // the sequences' blocks counted: those that exist have the lowest numbers
            long long base = 0;
            for (int b0 = 0; b0 < B; b0 += THREADS) {
                const int b = b0 + tid;
                int u0 = 0, u1 = 0, x = 0;
                if (b < B) {
                    u0 = ld_now(e.batch.cu + b);
                    u1 = ld_now(e.batch.cu + b + 1);
                    x = ld_now(e.batch.ctx + b);
                    if (!fits(u0, u1, x)) u1 = u0;
                }
                const int blocks = (u1 - u0 + R - 1) / R;
                int upto = blocks;
#pragma unroll
                for (int w = 1; w < 32; w <<= 1) {
                    const int y = __shfl_up_sync(kFull, upto, w);
                    if (lane >= w) upto += y;
                }
                if (b0 > 0) __syncthreads();
                if (lane == 31) m.sums[warp] = upto;
                __syncthreads();
                int all = 0;
#pragma unroll
                for (int w = 0; w < THREADS / 32; ++w) {
                    const int y = m.sums[w];
                    if (w < warp) upto += y;
                    all += y;
                }
                of(b, u0, u1, x, base + upto - blocks);
                base += all;
            }
        } else {  // numbered with room between the sequences, searched
            if (blockIdx.x == 0)  // offsets that decrease may hide their sequence from the search
                for (int b = tid; b < B; b += THREADS)
                    if (ld_now(e.batch.cu + b) > ld_now(e.batch.cu + b + 1)) record_index(e.index_word);
            if (warp == 0) {
                const int b = find_sequence(B, [&](int j) { return plan::group_start(j, ld_now(e.batch.cu + j), R) <= id; });
                if (b < B && lane == 0) {
                    const int u0 = ld_now(e.batch.cu + b), u1 = ld_now(e.batch.cu + b + 1), x = ld_now(e.batch.ctx + b);
                    if (sequence_ok(c, e.batch, u0, u1, x) && u1 - u0 <= kTreeMax) of(b, u0, u1, x, plan::group_start(b, u0, R));
                    else record_index(e.index_word);
                }
            }
        }
    }
    __syncthreads();
    const int n = m.n, t0 = m.t0, ctx = m.ctx, x0 = m.x0, R = args.R, nr = min(R, n - x0);
    if (n == 0) return;
    const WaitCtx wc{&m.abort, e.status, e.timeout_ns};
    Keys k{};
    k.lo = band_lo(ctx, s.mode, s.k_local);
    k.n_cached = ctx - k.lo;

    // ---- producers: a key's cache row, and (bf16) the tiles that need nothing of the tree
    const int *table = e.batch.table + (long long)m.b * c.width;
    const int pw = warp - 4;
    int early = 0, bad_at = -1;  // tiles under way; the highest position whose page was out of range among them
    auto row_at = [&](int pos) -> int {  // (-2: a page out of range)
        const int pg = page_of(c, table, 0, pos);
        return pg < 0 ? -2 : row_in_page(c, pg, kvh, pos);
    };
    auto free_stage = [&](int t) -> bool {  // the stage of tile t: its last tile's products done, the queries in TMEM
        bool w = true;
        if (t >= ST) w = wait_bar(bar(C::B_EMPTY + t % ST), (t / ST - 1) & 1, wc);
        else if (t >= ST - 2) w = wait_bar(bar(C::B_QT), 0, wc);
        return __all_sync(kFull, w);
    };
    auto copy_tile = [&](int t, int row) {  // bf16: the rows that the lanes hold
        constexpr int PER = D / 8, AT_ONCE = 32 / PER;  // pieces of a row; rows at a time
        const int piece = lane % PER;
        const uint32_t sk = sbase + C::k_at(t % ST), sv = sbase + C::v_at(t % ST);
#pragma unroll
        for (int i = 0; i < 8; i += AT_ONCE) {
            const int r = 8 * pw + i + lane / PER, rr = __shfl_sync(kFull, row, r);
            const long long at = (long long)max(rr, 0) * D + piece * 8;
            const uint32_t to = piece_at(r, piece, C::DBLK);
            cp_async16(sk + to, static_cast<const __nv_bfloat16 *>(c.k) + at, rr >= 0);
            cp_async16(sv + to, static_cast<const __nv_bfloat16 *>(c.v) + at, rr >= 0);
        }
        cp_async_arrive(bar(C::B_FULL + t % ST));
    };
    auto copy_raw = [&](int t, int row) {  // 8 bits: the rows that the lanes hold, as they are (each warp converts its own)
        constexpr int PER = D / 16, AT_ONCE = 32 / PER;
        const int piece = lane % PER;
        const uint32_t raw = sbase + C::RAW_OFF + (t % C::RAW) * C::RAW_BYTES;
#pragma unroll
        for (int i = 0; i < 8; i += AT_ONCE) {
            const int r = 8 * pw + i + lane / PER, rr = __shfl_sync(kFull, row, r);
            const long long at = (long long)max(rr, 0) * D + piece * 16;
            cp_async16(raw + r * D + piece * 16, static_cast<const uint8_t *>(c.k) + at, rr >= 0);
            cp_async16(raw + (CHUNK + r) * D + piece * 16, static_cast<const uint8_t *>(c.v) + at, rr >= 0);
        }
        {  // scales: 4 bytes of a row, or of two (d = 64)
            const int r = 8 * pw + (lane & 7), rr = __shfl_sync(kFull, row, r);
            const long long at = (long long)max(rr, 0) * (D / kScaleBlock) & ~3ll;
            if (lane < 16) cp_async4(raw + C::RAW_SCALES + ((lane >> 3) * CHUNK + r) * 4, (lane < 8 ? c.k_scale : c.v_scale) + at, rr >= 0);
            const unsigned odd = __ballot_sync(kFull, rr >= 0 && (rr & 1));
            if (D == 64 && lane == 0) m.odd[t % C::RAW][pw] = odd;
        }
        cp_async_commit();
    };
    if (warp >= 4 && warp < 8) {
        {
            const int tiles = min(k.n_cached / CHUNK, KV == kKvBf16 ? ST - 2 : C::RAW);
            int rw = tiles > 0 ? row_at(k.lo + lane) : 0;
            for (; early < tiles; ++early) {
                const int row = rw, pos = k.lo + early * CHUNK + lane;
                if (early + 1 < tiles) rw = row_at(pos + CHUNK);
                if (row < 0) bad_at = pos;
                if constexpr (KV == kKvBf16) copy_tile(early, row);
                else copy_raw(early, row);
            }
        }
    } else if (warp == MMA_WARP) {
        tmem_alloc(smem_u32(&m.tmem), TMEM_COLS);
    } else {
        // ---- the queries on their way; the tree
        for (int j = tid; j < n; j += PRODUCERS) {
            const int p = ld_now(args.t.parent + t0 + j);
            m.parent[j] = p;
            if (p < -1 || p >= j) m.broken = 1;
        }
        constexpr int PER = D / 8, AT_ONCE = PRODUCERS / PER;  // pieces of a row; rows at a time
        const int piece = tid % PER;
#pragma unroll 4
        for (int r = tid / PER; r < BM; r += AT_ONCE) {
            const int node = r & (R - 1), h = h0 + (r >> args.R_log2);
            const bool in = node < nr;
            const __nv_bfloat16 *src = e.q + (long long)(t0 + x0 + (in ? node : 0)) * e.q_stride + (long long)h * D + piece * 8;
            cp_async16(sbase + piece_at(r, piece, C::Q_DBLK), src, in);
        }
        cp_async_arrive(bar(C::B_Q));
        const int words = (x0 + nr + 31) / 32;  // (words of nodes past the block's are not read)
        if (tid < nr)
            for (int w = 0; w < words; ++w) m.band[w][tid] = m.skip[w][tid] = 0u;
        named_bar_sync(1, PRODUCERS);
        if (!m.broken && tid < nr) {
            int deep = 0, reach = s.k_local;  // the farthest back of the band
            if (s.mode == kModeEcp) {
                for (int at = m.parent[x0 + tid]; at >= 0; at = m.parent[at]) ++deep;
                reach = ctx + deep - band_lo(ctx + deep, s.mode, s.k_local);
            }
            deep = -1;
            for (int at = x0 + tid; at >= 0; at = m.parent[at]) {
                const int gap = ++deep;
                if (gap <= reach) m.band[at >> 5][tid] |= 1u << (at & 31);
                else if (s.mode != kModeEcp && s.S > 0 && gap % s.period == 0 && gap / s.period <= s.S) m.skip[at >> 5][tid] |= 1u << (at & 31);
            }
            m.pos[tid] = ctx + deep;
            atomicOr(&m.depths[deep >> 5], 1u << (deep & 31));
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = m.tmem;
    const bool run = !m.broken;
    if (!run && tid == 0) record_index(e.index_word);
    int n_tiles = 0;
    if (run) {
        int lo = kTreeMax, hi = 0;
#pragma unroll
        for (int w = 0; w < kTreeMax / 32; ++w) {
            const unsigned bits = m.depths[w];
            if (bits) {
                lo = min(lo, 32 * w + __ffs(bits) - 1);
                hi = 32 * w + 31 - __clz(bits);
            }
        }
        k.first = ctx + lo;
        k.spread = hi - lo + 1;
        k.n_band = k.n_cached + x0 + nr;
        k.n_keys = k.n_band;
        if (s.mode != kModeEcp && s.S > 0) k.n_keys += k.spread * max(0, min(s.S, (ctx + hi) / s.period) - args.m_first + 1);
        n_tiles = (k.n_keys + CHUNK - 1) / CHUNK;
    }

    if (!run) {
    } else if (warp >= 4 && warp < 8) {
        // ================= producers
        const int lowest = band_lo(k.first, s.mode, s.k_local);  // (below it a page may be gone)
        if (bad_at >= lowest) record_index(e.index_word);
        auto row_of = [&](int t) -> int {  // this lane's key of tile t: its cache row, or negative
            const int kk = t * CHUNK + lane;
            if (kk >= k.n_keys) return -1;
            int pos;
            if (kk < k.n_cached) {
                pos = k.lo + kk;
                if (pos < lowest) return -1;
            } else if (kk < k.n_band) {
                pos = ctx + kk - k.n_cached;
            } else {
                const int x = kk - k.n_band, w = x / k.spread, u = x - w * k.spread, deep = k.first - ctx + u;
                pos = k.first + u - (args.m_first + w) * s.period;
                if (pos < 0 || pos >= ctx || !(m.depths[deep >> 5] >> (deep & 31) & 1)) return -1;
            }
            const int row = row_at(pos);
            if (row < 0) record_index(e.index_word);
            return row;
        };
        if constexpr (KV == kKvBf16) {
            int rw = row_of(early);
            for (int t = early; t < n_tiles; ++t) {
                const int row = rw;
                if (t + 1 < n_tiles) rw = row_of(t + 1);
                if (!free_stage(t)) break;
                copy_tile(t, row);
            }
        } else {
            constexpr int PER = D / 16, AT_ONCE = 32 / PER;  // 16-code pieces of a row; rows at a time
            const int piece = lane % PER;
            int rw = row_of(early);
            auto ahead = [&](int t) {  // tile t, the rows of the next one looked up (past the last one: an empty group)
                const int row = rw;
                if (t + 1 < n_tiles) rw = row_of(t + 1);
                if (t < n_tiles) copy_raw(t, row);
                else cp_async_commit();
            };
            for (int t = early; t < C::RAW; ++t) ahead(t);
            for (int t = 0; t < n_tiles; ++t) {
                cp_async_wait<C::RAW - 1>();
                __syncwarp();
                if (!free_stage(t)) break;
                const uint8_t *raw = smem + C::RAW_OFF + (t % C::RAW) * C::RAW_BYTES;
                uint8_t *sk = smem + C::k_at(t % ST), *sv = smem + C::v_at(t % ST);
                const unsigned odd = D == 64 ? m.odd[t % C::RAW][pw] : 0u;
#pragma unroll
                for (int i = 0; i < 8; i += AT_ONCE) {
                    const int x = i + lane / PER, r = 8 * pw + x;
                    auto convert = [&](uint8_t *to, int which) {
                        const uint4 w = *reinterpret_cast<const uint4 *>(raw + (which * CHUNK + r) * D + piece * 16);
                        const uint32_t sc4 = *reinterpret_cast<const uint32_t *>(raw + C::RAW_SCALES + (which * CHUNK + r) * 4);
                        const Scale2<KV> s2 = scale_same<KV>(sc4 >> (8 * (piece >> 1) + (odd >> x & 1) * 16) & 0xffu);
                        uint4 a, b;
                        codes_to_bf16<KV>(w.x, s2, s2.big, a.x, a.y);
                        codes_to_bf16<KV>(w.y, s2, s2.big, a.z, a.w);
                        codes_to_bf16<KV>(w.z, s2, s2.big, b.x, b.y);
                        codes_to_bf16<KV>(w.w, s2, s2.big, b.z, b.w);
                        *reinterpret_cast<uint4 *>(to + piece_at(r, 2 * piece, C::DBLK)) = a;
                        *reinterpret_cast<uint4 *>(to + piece_at(r, 2 * piece + 1, C::DBLK)) = b;
                    };
                    convert(sk, 0);
                    convert(sv, 1);
                }
                fence_proxy_async_smem();
                mbar_arrive(bar(C::B_FULL + t % ST));
                __syncwarp();
                ahead(t + C::RAW);
            }
        }
    } else if (warp == MMA_WARP) {
        // ================= the products
        const uint32_t aQ = tbase + C::Q_COL, is = idesc_bf16(BM, CHUNK, 0, 0), io = idesc_bf16(BM, D, 0, 1);
        bool fine = __all_sync(kFull, wait_bar(bar(C::B_Q), 0, wc));
        if (fine) {
            fence_proxy_async_smem();
            tc_fence_after();
            if (elect_one()) {
                const uint64_t q0 = sdesc(sbase, 16, 1024);
#pragma unroll
                for (int dc = 0; dc < C::KD; ++dc)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) tmem_cp_128x256b(aQ + (dc * 4 + ks) * 8, q0 + (uint64_t)((dc * C::Q_DBLK + ks * 32) >> 4));
                tc_commit(bar(C::B_QT));
            }
            __syncwarp();
        }
        for (int t = 0; fine && t < n_tiles + NB - 1; ++t) {
            if (t < n_tiles) {
                fine = __all_sync(kFull, wait_bar(bar(C::B_FULL + t % ST), (t / ST) & 1, wc));
                if (!fine) break;
                fence_proxy_async_smem();
                tc_fence_after();
                const uint64_t b0 = sdesc(sbase + C::k_at(t % ST), 16, 1024);
                if (elect_one()) {
#pragma unroll
                    for (int dc = 0; dc < C::KD; ++dc)
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_ts(tbase + (t % NB) * CHUNK, aQ + (dc * 4 + ks) * 8, b0 + (uint64_t)((dc * C::DBLK + ks * 32) >> 4), is, (dc | ks) != 0);
                    tc_commit(bar(C::B_SF + t % NB));
                }
                __syncwarp();
            }
            const int u = t - (NB - 1);
            if (u >= 0) {
                fine = __all_sync(kFull, wait_bar(bar(C::B_PR + u % NB), (u / NB) & 1, wc));
                if (!fine) break;
                tc_fence_after();
                const uint64_t b0 = sdesc(sbase + C::v_at(u % ST), C::DBLK, 1024);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)  // the weights' first terms, then the second ones
                        mma_ts(tbase + C::O_COL, tbase + (u % NB) * CHUNK + kk * 8, b0 + (uint64_t)(((kk & 1) * 16 * ROW_BYTES) >> 4), io, (u > 0 || kk > 0) ? 1u : 0u);
                    tc_commit(bar(C::B_EMPTY + u % ST));
                    if (u == n_tiles - 1) tc_commit(bar(C::B_OF));
                }
                __syncwarp();
            }
        }
        if (elect_one()) tc_commit(bar(C::B_DR));
        __syncwarp();
        volatile uint32_t zero = 0;
        WaitCtx w2{&zero, e.status, e.timeout_ns};
        wait_bar(bar(C::B_DR), 0, w2);
    } else {
        // ================= softmax and epilogue: one thread per row
        const int r = tid, node = r & (R - 1), h = h0 + (r >> args.R_log2), mine = min(node, nr - 1);  // (a row without a node: dropped)
        const bool row_ok = node < nr;
        const long long at = (long long)(t0 + x0 + mine) * s.H + h;
        const float al = e.alpha ? ld_now(e.alpha + at) : 1.f;
        const float off_band = e.alpha ? log2f(al) : 0.f, off_skip = log2f(1.f - al), sc = s.scale_log2;
        const uint32_t tl = tbase + ((uint32_t)(warp * 32) << 16);
        const int i = m.pos[mine];
        // the list's place of the row's first cached band key, and of its key in the first skip window
        const int first = band_lo(i, s.mode, s.k_local) - k.lo, in_window = k.n_band + i - k.first;
        float m_ref = -INFINITY, l = 0.f;
        bool fine = true;
        for (int t = 0; t < n_tiles; ++t) {
            // which of the tile's keys are in the row's band, which its skips
            unsigned mb = 0u, ms = 0u;
            const int base = t * CHUNK;
            {
                const int a = max(first - base, 0), b = min(k.n_cached - base, 32);
                if (a < b) mb = (b == 32 ? kFull : (1u << b) - 1u) & (kFull << a);
            }
            if (base + CHUNK > k.n_cached && base < k.n_band) {  // the nodes' bits, moved to where the list has them
                const int w = (base - k.n_cached) >> 5, by = k.n_cached & 31;  // word w starts in the tile before, or with it
                const bool lo_in = w >= 0, hi_in = by > 0 && 32 * (w + 1) < x0 + nr;
                const unsigned b0 = lo_in ? m.band[w][mine] : 0u, b1 = hi_in ? m.band[w + 1][mine] : 0u;
                const unsigned s0 = lo_in ? m.skip[w][mine] : 0u, s1 = hi_in ? m.skip[w + 1][mine] : 0u;
                mb |= by ? b0 >> (32 - by) | b1 << by : b0;
                ms |= by ? s0 >> (32 - by) | s1 << by : s0;
            }
            if (base + CHUNK > k.n_band) {
                int w = max(0, base - in_window + k.spread - 1) / k.spread;  // the first window whose key lies in the tile, or after
                for (int x = in_window + w * k.spread; x < min(base + CHUNK, k.n_keys); x += k.spread, ++w) {
                    const int pos = i - (args.m_first + w) * s.period;
                    if (pos >= 0 && pos < ctx) ms |= 1u << (x - base);
                }
            }
            fine = __all_sync(kFull, wait_bar(bar(C::B_SF + t % NB), (t / NB) & 1, wc));
            if (!fine) break;
            tc_fence_after();
            __syncwarp();
            const uint32_t tS = tl + (t % NB) * CHUNK;
            uint32_t ra[CHUNK];
            tmem_ld32(tS, ra);
            tmem_wait_ld(ra);
            float bo, scale = sc;
            const bool plain = __all_sync(kFull, mb == kFull);
            float mt;
            if (plain) {
                mt = fmaf(tile_raw_max(ra), sc, off_band);
                bo = off_band;
            } else {  // logits in place
#pragma unroll
                for (int x = 0; x < CHUNK; ++x) {
                    const float z = __uint_as_float(ra[x]);
                    const float y = fmaf(z, sc, mb >> x & 1 ? off_band : off_skip);
                    ra[x] = __float_as_uint((mb | ms) >> x & 1 ? y : -INFINITY);
                }
                mt = tile_raw_max(ra);
                bo = 0.f;
                scale = 1.f;
            }
            float corr = 1.f;
            bool need_o = false;
            if (mt > m_ref) {
                const float m_new = mt + kHeadroom;
                if (m_ref != -INFINITY) {
                    corr = fast_exp2(m_ref - m_new);
                    need_o = true;
                }
                m_ref = m_new;
            }
            const float mu = m_ref == -INFINITY ? 0.f : m_ref;
            uint32_t rest[CHUNK / 2];
            const float sum = tile_exp_terms(ra, rest, scale, bo - mu);
            l = fmaf(l, corr, sum);
            tmem_st16(tS, ra);
            tmem_st16(tS + CHUNK / 2, rest);
            __syncwarp();
            if (__any_sync(kFull, need_o)) {  // O moves with the reference; the last P V must be done
                fine = __all_sync(kFull, wait_bar(bar(C::B_EMPTY + (t - 1) % ST), ((t - 1) / ST) & 1, wc));
                if (!fine) break;
                tc_fence_after();
#pragma unroll 1
                for (int oc = 0; oc < D / 16; ++oc) {
                    uint32_t x[16];
                    tmem_ld16(tl + C::O_COL + oc * 16, x);
                    tmem_wait_ld(x);
#pragma unroll
                    for (int y = 0; y < 16; ++y) x[y] = __float_as_uint(__uint_as_float(x[y]) * corr);
                    tmem_st16(tl + C::O_COL + oc * 16, x);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(bar(C::B_PR + t % NB));
        }
        if (fine) fine = __all_sync(kFull, wait_bar(bar(C::B_OF), 0, wc));
        uint32_t seen[4] = {};
        if (fine) {
            tc_fence_after();
            __syncwarp();
            const float inv = l == 0.f ? 0.f : 1.f / l;
            // through the warp's part of the tiles' space (every product is done), so that rows go out whole
            uint8_t *stage = smem + warp * (32 * D * 2);
            constexpr int PER = D / 8;
#pragma unroll 1
            for (int oc = 0; oc < D / 32; oc += 2) {
                uint32_t x[64];
                tmem_ld32(tl + C::O_COL + oc * 32, x);
                tmem_ld32(tl + C::O_COL + oc * 32 + 32, x + 32);
                tmem_wait_ld(x);
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    const float *f = reinterpret_cast<const float *>(x) + 8 * w;
                    const uint4 val = l == 0.f ? make_uint4(0u, 0u, 0u, 0u)
                                               : make_uint4(pack_bf16(f[0] * inv, f[1] * inv), pack_bf16(f[2] * inv, f[3] * inv),
                                                            pack_bf16(f[4] * inv, f[5] * inv), pack_bf16(f[6] * inv, f[7] * inv));
                    watch(seen, val);
                    *reinterpret_cast<uint4 *>(stage + lane * (D * 2) + (((4 * oc + w) ^ (lane & 7)) << 4)) = val;
                }
            }
            __syncwarp();
#pragma unroll 4
            for (int y = lane / PER; y < 32; y += 32 / PER) {
                const int rr = warp * 32 + y, p = lane % PER;
                if ((rr & (R - 1)) < nr)
                    *reinterpret_cast<uint4 *>(e.out + ((long long)(t0 + x0 + (rr & (R - 1))) * s.H + h0 + (rr >> args.R_log2)) * D + p * 8) =
                        *reinterpret_cast<const uint4 *>(stage + y * (D * 2) + ((p ^ (y & 7)) << 4));
            }
            if (row_ok) e.lse[at] = l == 0.f ? -INFINITY : (m_ref + log2f(l)) * kLn2;
        }
        const unsigned bad = __ballot_sync(kFull, row_ok && went_bad(seen) && l == l);
        if (lane == 0) m.bad[warp] = bad;
    }

    // ---- teardown
    cp_async_wait_all();  // (a tree that is left out: the queries)
    tc_fence_before();
    __syncthreads();
    if (warp == MMA_WARP) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tbase, TMEM_COLS);
    }
    // ---- rows that a value of another row's key made non-finite: once more, by themselves (pi_row.cuh)
    if (!run || m.abort) return;
    for (int r = warp; r < BM; r += THREADS / 32) {
        if (!(m.bad[r >> 5] >> (r & 31) & 1)) continue;
        const int node = x0 + (r & (R - 1)), h = h0 + (r >> args.R_log2);
        const long long at = (long long)(t0 + node) * s.H + h;
        RowKeys keys = row_keys(s, m.pos[r & (R - 1)], kvh, args.m_first, e.q + (long long)(t0 + node) * e.q_stride + (long long)h * D,
                                e.batch.table + (long long)m.b * c.width, e.alpha ? e.alpha + at : nullptr);
        keys.parent = args.t.parent + t0;
        keys.ctx = ctx;
        keys.node = node;
        attend_row<D, KV, true>(c, keys, e.out + at * D);
    }
}

template <int D, int KV>
static cudaError_t launch(const Args &a, long long blocks, cudaStream_t st) {
    auto *kernel = tree_tc_kernel<D, KV>;
    static PerDeviceOnce configured;
    int dev = 0;
    cudaGetDevice(&dev);
    if (configured.needed(dev)) {
        const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<D, KV>());
        if (err != cudaSuccess) return err;
        configured.mark(dev);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = (size_t)smem_bytes<D, KV>();
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace ttc

cudaError_t launch_tree_tc(const ExtendTreeArgs &t, cudaStream_t st) {
    using namespace ttc;
    const ExtendArgs &e = t.e;
    const Shape &s = e.s;
    const int G = s.H / s.Hkv;
    const int GP = tree_heads(G), log2 = GP == 1 ? 7 : GP == 2 ? 6 : GP == 4 ? 5 : GP == 8 ? 4 : 3;
    const int R = BM / GP, ngrp = s.H / GP;
    const Args a{t, GP, R, log2, ngrp, s.mode != kModeEcp && s.S > 0 ? first_skip_multiple(s) : 1, tc::make_fastdiv(ngrp), tc::make_fastdiv(G)};
    const long long blocks = (e.batch.T + e.batch.B * (long long)(R - 1)) / R * ngrp;
    switch (e.cache.kv_type) {
        case kKvBf16: return s.d == 64 ? launch<64, kKvBf16>(a, blocks, st) : launch<128, kKvBf16>(a, blocks, st);
        case kKvE4m3: return s.d == 64 ? launch<64, kKvE4m3>(a, blocks, st) : launch<128, kKvE4m3>(a, blocks, st);
        default: return s.d == 64 ? launch<64, kKvInt8>(a, blocks, st) : launch<128, kKvInt8>(a, blocks, st);
    }
}

}  // namespace pi
