// pi_extend_tc.cu -- pi-Attention / ECP attention of a chunk of new tokens per sequence over a paged
// key/value cache, on sm_103a tensor cores.
//
// What it computes: for the token at position i of its sequence, row i of the causal forward ("pi-Attention:
// Periodic Sparse Transformers for Efficient Long-Context Modeling", section 2.1-2.3; ECP page, section 2):
// one softmax over the band and the skip keys i - m*period with the gate's log-priors.
//
// How: the forward's pipeline (128 query rows = GP heads of one KV group x R consecutive positions as the M of
// every MMA, 32-key tiles, Q and P as TMEM operands, S and O accumulated in TMEM, one softmax thread
// per row, two persistent CTAs per SM), with what a batch of ragged, paged sequences asks for:
//   * A plan kernel turns the batch's offsets and contexts into a list of position blocks; it and the
//     checks run on the device, so that a captured graph follows its inputs.  The attention kernel starts
//     beside it (programmatic launch) and waits for it once its barriers and TMEM are set up.
//   * A sequence's blocks lie on multiples of R positions (a chunk of at most R tokens is one block where it
//     starts), and key tiles on multiples of 32, so that a tile lies inside one page (page 16: two) and is one
//     TMA box per 64 columns.  With period % 32 = 0 a skip window falls on whole tiles too; any other
//     period costs one tile more per window.
//   * The lanes of a producer warp look up the page-table entries of 32 tiles at once, a block ahead.
//   * Queries are loaded from [T, H, d] through a map whose rows are tokens.  A block that is not full (a
//     sequence's first or last) loads rows of its neighbours too; their rows are computed and dropped:
//     its output goes from registers to the valid rows only, a full block's through shared memory and TMA.
//   * Rows of V that no query of the block attends may hold anything (evicted or unwritten rows, NaN among them):
//     they are zeroed in shared memory before the product, since 0 * NaN is not 0.  Scores of K rows outside
//     a row's range are replaced before they are used.
//   * 8-bit caches: a producer warp brings codes and scale bytes into a ring of raw tiles, and four more
//     warps turn them into the bf16 tiles of the pipeline (exact, see pi_paged.cuh).  One lane takes 16 codes
//     of a row; raw and converted tiles are both swizzled, so that neither side has bank conflicts.
#include <cuda.h>

#include "pi_launch.h"
#include "pi_mma.cuh"
#include "pi_paged.cuh"
#include "pi_tc_ptx.cuh"
#include "pi_tile.cuh"

namespace pi {
namespace ext {

using namespace tc;

constexpr int BM = 128;         // rows per block (MMA M)
constexpr int TMEM_COLS = 256;  // per CTA, two CTAs per SM
constexpr int ROW_BYTES = 128;  // one 64-element bf16 swizzle row

// ------------------------------------------------------------------ the plan

// A position block of one sequence: positions first .. last hold its queries, row 0 is position p0 and packed
// token tq (possibly before the sequence's own).
struct PlanBlock {
    int b, p0, tq, first, last, pad[3];
};
constexpr int PLAN_HEAD = 32;  // bytes before the blocks: [0] their number

__host__ __device__ __forceinline__ long long max_blocks(long long T, long long B, int R) {
    // n tokens lie in at most floor(n / R) + 2 blocks, and a sequence without tokens in none
    return T / R + 2 * (B < T ? B : T);
}

constexpr int PLAN_THREADS = 1024;

__global__ void __launch_bounds__(PLAN_THREADS) plan_kernel(PagedCache c, PagedBatch bt, int R, int *plan, int *index_word) {
    __shared__ int upto[PLAN_THREADS];  // blocks of the round's sequences up to and including each
    __shared__ int warp_sum[PLAN_THREADS / 32];
    asm volatile("griddepcontrol.launch_dependents;");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    PlanBlock *blocks = reinterpret_cast<PlanBlock *>(reinterpret_cast<char *>(plan) + PLAN_HEAD);
    // Offsets that decrease would let sequences overlap and their blocks outgrow the plan: nothing is planned.
    bool sorted = true;
    for (int b = tid; b < bt.B; b += PLAN_THREADS) sorted = sorted && bt.cu[b] <= bt.cu[b + 1];
    if (!__syncthreads_and(sorted)) {
        if (tid == 0) {
            record_index(index_word);
            plan[0] = 0;
        }
        return;
    }
    // n tokens at ctx ..: blocks at multiples of R, or one where a short chunk starts
    auto start = [&](int n, int ctx) { return n <= R ? ctx : ctx / R * R; };
    int base = 0;
    for (int b0 = 0; b0 < bt.B; b0 += PLAN_THREADS) {
        const int b = b0 + tid;
        int cnt = 0;
        if (b < bt.B) {
            const int t0 = bt.cu[b], t1 = bt.cu[b + 1], ctx = bt.ctx[b];
            if (!sequence_ok(c, bt, t0, t1, ctx)) record_index(index_word);
            else if (t1 > t0) cnt = (ctx + (t1 - t0) - 1 - start(t1 - t0, ctx)) / R + 1;
        }
        int sum = cnt;
#pragma unroll
        for (int w = 1; w < 32; w <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, sum, w);
            if (lane >= w) sum += x;
        }
        if (lane == 31) warp_sum[warp] = sum;
        __syncthreads();
        int before = 0;
        for (int w = 0; w < warp; ++w) before += warp_sum[w];
        upto[tid] = sum + before;
        __syncthreads();
        const int total = upto[PLAN_THREADS - 1];
        for (int x = tid; x < total; x += PLAN_THREADS) {
            int lo = 0, hi = PLAN_THREADS - 1;  // first sequence of the round with more than x blocks up to it
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (upto[mid] > x) hi = mid;
                else lo = mid + 1;
            }
            const int t0 = bt.cu[b0 + lo], n = bt.cu[b0 + lo + 1] - t0, ctx = bt.ctx[b0 + lo];
            const int p0 = start(n, ctx) + (x - (lo > 0 ? upto[lo - 1] : 0)) * R;
            const int4 d = make_int4(b0 + lo, p0, t0 + p0 - ctx, max(p0, ctx));
            *reinterpret_cast<int4 *>(&blocks[base + x]) = d;
            blocks[base + x].last = min(p0 + R, ctx + n) - 1;
        }
        base += total;
        __syncthreads();
    }
    if (tid == 0) plan[0] = base;
}

// ------------------------------------------------------------------ shared memory, TMEM, barriers

template <int D, int KV>
struct Cfg {
    static constexpr bool QUANT = KV != kKvBf16;
    static constexpr int NB = D == 64 ? 4 : 2;  // S buffers; TMEM columns as in the forward
    static constexpr int O_COL = 128, Q_COL = D == 128 ? 64 : 192;
    static constexpr int KD = D / 64;
    static constexpr int Q_BYTES = BM * D * 2, Q_DBLK = BM * ROW_BYTES;
    static constexpr int KV_STAGE = CHUNK * D * 2, KV_DBLK = CHUNK * ROW_BYTES;
    static constexpr int KSTAGES = (QUANT ? 24576 : 49152) / KV_STAGE;
    static constexpr int VSTAGES = (QUANT ? 24576 : 32768) / KV_STAGE;
    static constexpr int RSTAGES = QUANT ? 24576 / (2 * CHUNK * D) : 0;  // raw tiles: K then V codes
    static constexpr int RAW = CHUNK * D;                                // bytes of one tile's codes
    static constexpr int SCALES = CHUNK * (D / kScaleBlock);             // bytes of one tile's scales
    static constexpr int Q_OFF = 0;
    static constexpr int K_OFF = Q_OFF + Q_BYTES;
    static constexpr int V_OFF = K_OFF + KSTAGES * KV_STAGE;
    static constexpr int R_OFF = V_OFF + VSTAGES * KV_STAGE;
    static constexpr int SC_OFF = R_OFF + RSTAGES * 2 * RAW;
    static constexpr int DATA_BYTES = SC_OFF + RSTAGES * 2 * SCALES;
    // barriers; tiles are counted across the blocks a CTA processes, block k completes the per-block
    // ones in phase k
    static constexpr int B_Q = 0;                 // Q tile landed
    static constexpr int B_KF = 1;                // K tile in its bf16 stage
    static constexpr int B_KE = B_KF + KSTAGES;   // that stage free
    static constexpr int B_VF = B_KE + KSTAGES;
    static constexpr int B_VE = B_VF + VSTAGES;
    static constexpr int B_SF = B_VE + VSTAGES;   // [NB] S in TMEM
    static constexpr int B_PR = B_SF + NB;        // [NB] P written over it (128)
    static constexpr int B_PV = B_PR + NB;        // [NB] its PV product done
    static constexpr int B_OF = B_PV + NB;        // O of the block complete
    static constexpr int B_QT = B_OF + 1;         // Q copied into TMEM
    static constexpr int B_STF = B_QT + 1;        // output staged, or stored (128)
    static constexpr int B_STR = B_STF + 1;       // staged output read by its store
    static constexpr int B_DR = B_STR + 1;        // drains of the two MMA issuers
    static constexpr int B_DR2 = B_DR + 1;
    static constexpr int B_SD = B_DR2 + 1;        // S products of the block done
    static constexpr int B_RF = B_SD + 1;         // [RSTAGES] raw tile landed
    static constexpr int B_RE = B_RF + RSTAGES;   // [RSTAGES] raw tile read (4 warps)
    static constexpr int NBARS = B_RE + RSTAGES;
    static constexpr int arrivals(int idx) {
        if ((idx >= B_PR && idx < B_PR + NB) || idx == B_STF) return 128;
        if (QUANT && ((idx >= B_KF && idx < B_KF + KSTAGES) || (idx >= B_VF && idx < B_VF + VSTAGES) || idx >= B_RE)) return 4;
        return 1;
    }
    static constexpr int BAR_BYTES = NBARS * 8 + 16;
    static_assert(BAR_BYTES <= 512, "barriers must fit the alignment gap or its complement");
    static constexpr int SMEM_BYTES = DATA_BYTES + 1024;  // data from a 1024-byte boundary; barriers in the gap or behind
    static_assert(SMEM_BYTES <= 115712, "two CTAs per SM");
    static constexpr int THREADS = QUANT ? 384 : 256;
};

struct Args {
    ExtendArgs a;
    const int *plan;
    int GP, R, R_log2, ngrp;
    int m_first;
    int aligned;  // period % 32 == 0: every skip window has the same place in its tiles
    int box;      // rows of a TMA box: min(32, page)
    FastDiv div_ngrp, div_G, div_period;
};

// One block: a plan block x one group of GP heads, and its key tiles.
struct Block {
    int b, p0, tq, first, last, h0, g;
    int lo, n_band;       // first band key of the first query; tiles from lo rounded down to 32
    int cpb;              // tiles per skip window
    uint32_t inv_cpb;     // ceil(2^32 / cpb)
    int n_tiles;
    int full_lo, full_hi; // tiles inside the band of every query
};

__device__ __forceinline__ PlanBlock load_plan(const Args &a, int L) {
    const int4 *p = reinterpret_cast<const int4 *>(reinterpret_cast<const char *>(a.plan) + PLAN_HEAD) + 2 * a.div_ngrp.div(L);
    const int4 x = p[0];
    PlanBlock d;
    d.b = x.x; d.p0 = x.y; d.tq = x.z; d.first = x.w;
    d.last = *reinterpret_cast<const int *>(p + 1);
    return d;
}

__device__ __forceinline__ void describe(const Args &a, const PlanBlock &d, int L, Block &k) {
    const Shape &s = a.a.s;
    k.b = d.b; k.p0 = d.p0; k.tq = d.tq; k.first = d.first; k.last = d.last;
    k.h0 = (L - a.div_ngrp.div(L) * a.ngrp) * a.GP;
    k.g = a.div_G.div(k.h0);
    k.lo = band_lo(d.first, s.mode, s.k_local);
    const int key0 = k.lo & ~(CHUNK - 1);
    k.n_band = (d.last - key0) / CHUNK + 1;
    int windows = 0;
    if (s.mode != kModeEcp && s.S > 0) windows = max(0, min(s.S, a.div_period.div(d.last)) - a.m_first + 1);
    k.cpb = a.aligned ? (d.last >> 5) - (d.first >> 5) + 1 : ((d.last - d.first) >> 5) + 2;
    k.inv_cpb = 0xffffffffu / (uint32_t)k.cpb + 1u;  // 0 for one tile per window
    k.n_tiles = k.n_band + windows * k.cpb;
    const int lo_last = band_lo(d.last, s.mode, s.k_local);
    k.full_lo = (lo_last - key0 + CHUNK - 1) / CHUNK;
    const int span = d.first - (CHUNK - 1) - key0;
    k.full_hi = span >= 0 ? span / CHUNK : -1;
}

// Tile ti of a block: its first key (negative: a tile wholly before the sequence), whether it is a skip tile,
// and its skip distance.
__device__ __forceinline__ int tile_key0(const Args &a, const Block &k, int ti, int &back, bool &skip) {
    skip = ti >= k.n_band;
    if (!skip) {
        back = 0;
        return (k.lo & ~(CHUNK - 1)) + ti * CHUNK;
    }
    const uint32_t x = (uint32_t)(ti - k.n_band);
    const uint32_t w = k.inv_cpb ? __umulhi(x, k.inv_cpb) : x;
    back = (a.m_first + (int)w) * a.a.s.period;
    return ((k.first - back) & ~(CHUNK - 1)) + (int)(x - w * (uint32_t)k.cpb) * CHUNK;
}

// Keys of tile ti that some query of the block attends or may attend: lo .. hi (empty: lo > hi).
__device__ __forceinline__ int tile_range(const Args &a, const Block &k, int ti, int &lo, int &hi) {
    int back;
    bool skip;
    const int key0 = tile_key0(a, k, ti, back, skip);
    lo = max(key0, skip ? max(0, k.first - back) : k.lo);
    hi = min(key0 + CHUNK - 1, k.last - back);
    return key0;
}

constexpr int NO_PAGE = -2;  // a box without an attended row

template <int D, int KV>
__global__ void __launch_bounds__(Cfg<D, KV>::THREADS, 2)
extend_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO, const Args args) {
    using C = Cfg<D, KV>;
    constexpr int KST = C::KSTAGES, VST = C::VSTAGES, NB = C::NB;
    constexpr int RST = C::QUANT ? C::RSTAGES : 1;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
    uint8_t *smem = smem_raw + pad;
    const uint32_t sbase = raw_addr + pad;
    const uint32_t bar_off = (pad >= (uint32_t)C::BAR_BYTES) ? 0u : pad + C::DATA_BYTES;
    const uint32_t sQ = sbase + C::Q_OFF, sK = sbase + C::K_OFF, sV = sbase + C::V_OFF;
    const uint32_t sBar = raw_addr + bar_off;
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem_raw + bar_off + C::NBARS * 8);
    uint32_t *tmem_slot = misc;
    volatile uint32_t *abort_flag = misc + 1;
    auto bar = [&](int idx) -> uint32_t { return sBar + idx * 8; };

    const ExtendArgs &ea = args.a;
    const Shape &s = ea.s;
    const PagedCache &cache = ea.cache;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const WaitCtx wc{abort_flag, ea.status, ea.timeout_ns};

    if (warp == 0) {
        for (int idx = lane; idx < C::NBARS; idx += 32) mbar_init(bar(idx), (uint32_t)C::arrivals(idx));
        if (lane == 0) *abort_flag = 0u;
        fence_barrier_init();
        __syncwarp();
        tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
    }
    if (threadIdx.x == 32) {
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
        prefetch_tmap(&tmO);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_slot;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan is written

    const int n_blocks = args.plan[0] * args.ngrp;
    const int L0 = blockIdx.x, LS = gridDim.x;
    auto next_block = [&](int L) -> int { return (L < n_blocks - LS) ? L + LS : n_blocks; };

    // ---- page lookup of a producer warp: lane x holds the page-table entries of tile t0 + x (page 16: of
    // both halves), NO_PAGE where a box has no attended row
    auto lookup = [&](const Block &k, int t0, int &e0, int &e1) {
        e0 = e1 = NO_PAGE;
        if (t0 + lane >= k.n_tiles) return;
        int lo, hi;
        const int key0 = tile_range(args, k, t0 + lane, lo, hi);
        const int *row = ea.batch.table + (long long)k.b * cache.width;
        if (args.box == CHUNK) {
            if (lo <= hi) e0 = __ldg(row + (key0 >> cache.page_log2));
        } else {
            if (lo <= min(hi, key0 + 15)) e0 = __ldg(row + (key0 >> cache.page_log2));
            if (max(lo, key0 + 16) <= hi) e1 = __ldg(row + ((key0 + 16) >> cache.page_log2));
        }
    };
    // page-table entry -> plane of the page maps (one past the last, which reads as zeros, where there is no page)
    auto plane = [&](const Block &k, int e) -> int {
        if ((unsigned)e < (unsigned)cache.n_pages) return e * cache.Hkv + k.g;
        if (e != NO_PAGE) record_index(ea.index_word);
        return cache.n_pages * cache.Hkv;
    };
    // Walks the tiles of every block of the CTA: issue(block, tile, number, z0, z1, row) by the whole warp, with the
    // entries of a block's first 32 tiles requested a block ahead.  before/after a block: hooks.
    auto walk_tiles = [&](auto &&issue, auto &&block_end) {
        if (L0 >= n_blocks) return true;
        Block k;
        int e0, e1;
        describe(args, load_plan(args, L0), L0, k);
        lookup(k, 0, e0, e1);
        PlanBlock pn = load_plan(args, min(L0 + LS, n_blocks - 1));
        uint32_t n = 0;
        for (int L = L0, kb = 0;; ++kb) {
            const int Ln = next_block(L);
            Block kn = k;
            int n0 = NO_PAGE, n1 = NO_PAGE;
            if (Ln < n_blocks) {
                describe(args, pn, Ln, kn);
                lookup(kn, 0, n0, n1);
                const int Lnn = next_block(Ln);
                if (Lnn < n_blocks) pn = load_plan(args, Lnn);
            }
            int z0 = 0, z1 = 0;
            for (int t = 0; t < k.n_tiles; ++t, ++n) {
                if ((t & 31) == 0) {
                    if (t) lookup(k, t, e0, e1);
                    z0 = plane(k, e0);
                    z1 = plane(k, e1);
                }
                if (!issue(k, t, n, __shfl_sync(0xffffffffu, z0, t & 31), __shfl_sync(0xffffffffu, z1, t & 31))) return false;
            }
            if (!block_end(k, kn, kb, Ln < n_blocks)) return false;
            if (Ln >= n_blocks) return true;
            L = Ln;
            k = kn;
            e0 = n0;
            e1 = n1;
        }
    };
    // one lane: a tile's boxes of bf16 rows
    auto load_tile = [&](const CUtensorMap *tm, uint32_t dst, uint32_t full, int row, int z0, int z1, uint64_t policy) {
        mbar_expect_tx(full, C::KV_STAGE);
        for (int dc = 0; dc < C::KD; ++dc) {
            tma_load_3d_hint(dst + dc * C::KV_DBLK, tm, dc * 64, row, z0, full, policy);
            if (args.box != CHUNK)
                tma_load_3d_hint(dst + dc * C::KV_DBLK + 16 * ROW_BYTES, tm, dc * 64, 0, z1, full, policy);
        }
    };
    auto page_row = [&](const Block &k, int t) -> int {
        int back;
        bool skip;
        return tile_key0(args, k, t, back, skip) & (cache.page - 1);
    };
    auto issue_q = [&](const Block &k) {  // one lane
        mbar_expect_tx(bar(C::B_Q), C::Q_BYTES);
        for (int dc = 0; dc < C::KD; ++dc)
            tma_load_3d_hint(sQ + dc * C::Q_DBLK, &tmQ, dc * 64, k.tq, k.h0, bar(C::B_Q), policy_evict_first());
    };
    auto is_whole = [&](const Block &k) -> bool { return k.first == k.p0 && k.last == k.p0 + args.R - 1; };
    // The staged output of block kb (one lane): stored if the block is full (else its rows went out from registers).
    auto store_out = [&](const Block &k, int kb) -> bool {
        if (!wait_bar(bar(C::B_STF), (uint32_t)(kb & 1), wc)) return false;
        if (is_whole(k)) {
            for (int dc = 0; dc < C::KD; ++dc)
                tma_store_3d(&tmO, sQ + dc * C::Q_DBLK, dc * 64, k.tq, k.h0, policy_evict_first());
            tma_store_commit_and_wait();
        }
        mbar_arrive(bar(C::B_STR));
        return true;
    };
    // After a producer gave up: its loads in flight land before the CTA leaves.
    auto drain = [&](int full, int stages, uint32_t issued) {
        volatile uint32_t zero = 0;
        WaitCtx w2{&zero, nullptr, 20000000ull};
        for (uint32_t x = (issued > (uint32_t)stages ? issued - stages : 0); x < issued; ++x)
            wait_bar(bar(full + (int)(x % stages)), (x / stages) & 1, w2);
    };

    if (warp == 0) {
        // ================= producer: K tiles (bf16), or the raw K and V tiles with their scales (8 bits)
        const uint64_t reused = policy_evict_last();
        uint32_t issued = 0;
        auto issue = [&](const Block &k, int t, uint32_t n, int z0, int z1) -> bool {
            const int stages = C::QUANT ? RST : KST, full = C::QUANT ? C::B_RF : C::B_KF, empty = C::QUANT ? C::B_RE : C::B_KE;
            const int st = (int)(n % stages);
            const uint32_t round = n / stages;
            const bool ok = round == 0 || wait_bar(bar(empty + st), (round - 1) & 1, wc);
            if (!__all_sync(0xffffffffu, ok)) return false;
            issued = n + 1;
            if (lane == 0) {
                const int row = page_row(k, t);
                if constexpr (!C::QUANT) {
                    load_tile(&tmK, sK + st * C::KV_STAGE, bar(full + st), row, z0, z1, reused);
                } else {
                    // codes by TMA (zeros where there is no page), scales as contiguous bytes: where there is no page
                    // the converters take any scale (a code of zero, or a masked row)
                    const uint32_t dst = sbase + C::R_OFF + st * 2 * C::RAW, sc = sbase + C::SC_OFF + st * 2 * C::SCALES;
                    const int none = cache.n_pages * cache.Hkv, halves = args.box == CHUNK ? 1 : 2;
                    const uint32_t bytes = C::SCALES / halves;
                    uint32_t total = 2 * C::RAW;
                    for (int h = 0; h < halves; ++h) total += (h ? z1 : z0) != none ? 2 * bytes : 0;
                    mbar_expect_tx(bar(full + st), total);
                    for (int h = 0; h < halves; ++h) {
                        const int z = h ? z1 : z0, r = h ? 0 : row;
                        tma_load_3d_hint(dst + h * 16 * D, &tmK, 0, r, z, bar(full + st), reused);
                        tma_load_3d_hint(dst + C::RAW + h * 16 * D, &tmV, 0, r, z, bar(full + st), reused);
                        if (z == none) continue;
                        const long long at = (((long long)z << cache.page_log2) + r) * (D / kScaleBlock);
                        bulk_load(sc + h * bytes, cache.k_scale + at, bytes, bar(full + st));
                        bulk_load(sc + C::SCALES + h * bytes, cache.v_scale + at, bytes, bar(full + st));
                    }
                }
            }
            __syncwarp();
            return true;
        };
        walk_tiles(issue, [](const Block &, const Block &, int, bool) { return true; });
        if (*abort_flag && lane == 0) drain(C::QUANT ? C::B_RF : C::B_KF, C::QUANT ? RST : KST, issued);
        __syncwarp();
    } else if (warp == 2) {
        // ================= Q tiles, the stores of staged output, and (bf16) the V tiles.  At V tile t_st of block k
        // the output of block k-1 has been staged; once its store has read the buffer, the Q tile of block
        // k+1 takes its place (that of block k is in TMEM by then).
        const uint64_t reused = policy_evict_last();
        uint32_t issued = 0;
        int q_loads = 0;
        Block prev, nx;
        bool have_next = false;
        int kb_now = 0;
        auto turn = [&](int kb) -> bool {  // the whole warp: store block kb-1, load block kb+1's queries
            bool ok = true;
            if (lane == 0) {
                if (kb > 0) ok = store_out(prev, kb - 1);
                if (ok && have_next) {
                    ok = wait_bar(bar(C::B_QT), (uint32_t)(kb & 1), wc);
                    if (ok) issue_q(nx);
                }
            }
            ok = __all_sync(0xffffffffu, ok);
            if (ok && have_next) ++q_loads;
            return ok;
        };
        bool ok = true;
        if (L0 < n_blocks) {
            Block k;
            describe(args, load_plan(args, L0), L0, k);
            if (lane == 0) issue_q(k);
            q_loads = 1;
            __syncwarp();
        }
        if constexpr (!C::QUANT) {
            int L = L0;
            auto issue = [&](const Block &k, int t, uint32_t n, int z0, int z1) -> bool {
                if (t == 0) {
                    const int Ln = next_block(L);
                    have_next = Ln < n_blocks;
                    if (have_next) describe(args, load_plan(args, Ln), Ln, nx);
                }
                const int st = (int)(n % VST);
                const uint32_t round = n / VST;
                const bool w = round == 0 || wait_bar(bar(C::B_VE + st), (round - 1) & 1, wc);
                if (!__all_sync(0xffffffffu, w)) return false;
                issued = n + 1;
                if (lane == 0) load_tile(&tmV, sV + st * C::KV_STAGE, bar(C::B_VF + st), page_row(k, t), z0, z1, reused);
                __syncwarp();
                return t != min(4, k.n_tiles - 1) || turn(kb_now);
            };
            ok = walk_tiles(issue, [&](const Block &k, const Block &, int kb, bool) {
                prev = k;
                kb_now = kb + 1;
                L = next_block(L);
                return true;
            });
        } else {
            for (int L = L0; ok && L < n_blocks; L = next_block(L), ++kb_now) {
                Block k;
                describe(args, load_plan(args, L), L, k);
                const int Ln = next_block(L);
                have_next = Ln < n_blocks;
                if (have_next) describe(args, load_plan(args, Ln), Ln, nx);
                ok = turn(kb_now);
                prev = k;
            }
        }
        if (ok && kb_now > 0 && lane == 0) ok = store_out(prev, kb_now - 1);  // the CTA's last block
        __syncwarp();
        if (*abort_flag && lane == 0) {
            volatile uint32_t zero = 0;
            WaitCtx w2{&zero, nullptr, 20000000ull};
            if (q_loads > 0) wait_bar(bar(C::B_Q), (uint32_t)((q_loads - 1) & 1), w2);
            if (!C::QUANT) drain(C::B_VF, VST, issued);
            tma_store_commit_and_wait();
        }
        __syncwarp();
    } else if (warp == 1) {
        // ================= S issuer: S = Q K^T into the tile's TMEM buffer, Q from TMEM (whole warp, one elected
        // lane issuing); it runs ahead of the PV issuer
        const uint32_t aQ = tbase + C::Q_COL;
        const uint32_t idesc = idesc_bf16(BM, CHUNK, 0, 0);
        uint32_t gs = 0;
        int kb = 0;
        bool ok = true;
        PlanBlock pd{};
        if (L0 < n_blocks) pd = load_plan(args, L0);
        for (int L = L0; ok && L < n_blocks; L = next_block(L), ++kb) {
            Block k;
            describe(args, pd, L, k);
            if (next_block(L) < n_blocks) pd = load_plan(args, next_block(L));
            bool w = (kb == 0) || wait_bar(bar(C::B_SD), (uint32_t)((kb - 1) & 1), wc);
            if (w) w = wait_bar(bar(C::B_Q), (uint32_t)(kb & 1), wc);
            ok = __all_sync(0xffffffffu, w);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                const uint64_t q0 = sdesc(sQ, 16, 1024);
#pragma unroll
                for (int dc = 0; dc < C::KD; ++dc)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        tmem_cp_128x256b(aQ + (dc * 4 + ks) * 8, q0 + (uint64_t)((dc * C::Q_DBLK + ks * 32) >> 4));
                tc_commit(bar(C::B_QT));
            }
            __syncwarp();
            for (int t = 0; t < k.n_tiles; ++t, ++gs) {
                const int st = (int)(gs % KST), buf = (int)(gs % NB);
                bool r = wait_bar(bar(C::B_KF + st), (gs / KST) & 1, wc);
                if (r && gs >= NB) r = wait_bar(bar(C::B_PV + buf), ((gs - NB) / NB) & 1, wc);
                if (!__all_sync(0xffffffffu, r)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t b0 = sdesc(sK + st * C::KV_STAGE, 16, 1024);
                if (elect_one()) {
#pragma unroll
                    for (int dc = 0; dc < C::KD; ++dc)
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_ts(tbase + buf * CHUNK, aQ + (dc * 4 + ks) * 8, b0 + (uint64_t)((dc * C::KV_DBLK + ks * 32) >> 4),
                                   idesc, (dc | ks) != 0);
                    tc_commit(bar(C::B_SF + buf));
                    tc_commit(bar(C::B_KE + st));
                    if (t == k.n_tiles - 1) tc_commit(bar(C::B_SD));
                }
                __syncwarp();
            }
        }
        if (elect_one()) tc_commit(bar(C::B_DR));
        __syncwarp();
        volatile uint32_t zero = 0;
        WaitCtx w2{&zero, ea.status, ea.timeout_ns};
        wait_bar(bar(C::B_DR), 0, w2);
    } else if (warp == 3) {
        // ================= PV issuer: O += P V with P from TMEM
        const uint32_t idesc = idesc_bf16(BM, D, 0, 1);
        uint32_t gp = 0;
        bool ok = true;
        PlanBlock pd{};
        if (L0 < n_blocks) pd = load_plan(args, L0);
        for (int L = L0; ok && L < n_blocks; L = next_block(L)) {
            Block k;
            describe(args, pd, L, k);
            if (next_block(L) < n_blocks) pd = load_plan(args, next_block(L));
            for (int t = 0; t < k.n_tiles; ++t, ++gp) {
                const int buf = (int)(gp % NB), st = (int)(gp % VST);
                bool w = wait_bar(bar(C::B_VF + st), (gp / VST) & 1, wc);
                if (!C::QUANT && w) {
                    // rows of V that no query attends: zero (the converters do this for 8-bit tiles)
                    int lo, hi;
                    const int key0 = tile_range(args, k, t, lo, hi);
                    if (lo > key0 || hi < key0 + CHUNK - 1) {  // the same for the warp
                        if (key0 + lane < lo || key0 + lane > hi) {
                            uint8_t *row = smem + C::V_OFF + st * C::KV_STAGE + lane * ROW_BYTES;
#pragma unroll
                            for (int x = 0; x < C::KD * 8; ++x)
                                *reinterpret_cast<uint4 *>(row + (x >> 3) * C::KV_DBLK + (x & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                }
                if (w) w = wait_bar(bar(C::B_PR + buf), (gp / NB) & 1, wc);
                if (!__all_sync(0xffffffffu, w)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t b0 = sdesc(sV + st * C::KV_STAGE, C::KV_DBLK, 1024);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk)
                        mma_ts(tbase + C::O_COL, tbase + buf * CHUNK + kk * 8, b0 + (uint64_t)((kk * 16 * ROW_BYTES) >> 4), idesc,
                               (t > 0 || kk > 0) ? 1u : 0u);
                    tc_commit(bar(C::B_PV + buf));
                    tc_commit(bar(C::B_VE + st));
                    if (t == k.n_tiles - 1) tc_commit(bar(C::B_OF));
                }
                __syncwarp();
            }
        }
        if (elect_one()) tc_commit(bar(C::B_DR2));
        __syncwarp();
        volatile uint32_t zero = 0;
        WaitCtx w2{&zero, ea.status, ea.timeout_ns};
        wait_bar(bar(C::B_DR2), 0, w2);
    } else if (warp < 8) {
        // ================= softmax and epilogue: one thread per row
        const int q4 = warp & 3;
        const int r = q4 * 32 + lane;
        const int R = args.R;
        const int hh = r >> args.R_log2, trow = r & (R - 1);
        const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
        const float sc = s.scale_log2;
        auto alpha_of = [&](const PlanBlock &d, int L) -> float {
            const int i = d.p0 + trow;
            if (!ea.alpha || i < d.first || i > d.last) return 1.f;
            const int h0 = (L - args.div_ngrp.div(L) * args.ngrp) * args.GP;
            return __ldg(ea.alpha + (long long)(d.tq + trow) * s.H + h0 + hh);
        };
        bool ok = true;
        uint32_t gsm = 0;
        int kb = 0;
        PlanBlock pd{}, pn{};
        float al_next = 1.f;
        if (L0 < n_blocks) {
            pd = load_plan(args, L0);
            al_next = alpha_of(pd, L0);
        }
        for (int L = L0; ok && L < n_blocks; ++kb) {
            Block k;
            describe(args, pd, L, k);
            const int Ln = next_block(L);
            const bool has_next = Ln < n_blocks;
            if (has_next) pn = load_plan(args, Ln);
            const float al = al_next;
            const float off_band = ea.alpha ? log2f(al) : 0.f, off_skip = log2f(1.f - al);
            // a row without a query takes the part of the nearest one; its result is dropped
            const int i = min(max(k.p0 + trow, k.first), k.last), h = k.h0 + hh;
            const bool row_ok = i == k.p0 + trow;
            const int lo_i = band_lo(i, s.mode, s.k_local);

            float m_ref = -INFINITY, l = 0.f;
            for (int t = 0; t < k.n_tiles; ++t, ++gsm) {
                const int buf = (int)(gsm % NB);
                ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_SF + buf), (gsm / NB) & 1, wc));
                if (!ok) break;
                tc_fence_after();
                __syncwarp();
                const uint32_t tS = tbase + lane_base + buf * CHUNK;
                uint32_t ra[CHUNK];
                tmem_ld32(tS, ra);
                tmem_wait_ld();
                // Tiles inside every query's band: P with the running reference; the maximum only once some P
                // exceeds 2^8, which a sum above 2^8 is the first sign of.
                const bool fast = t >= k.full_lo && t <= k.full_hi && __all_sync(0xffffffffu, m_ref != -INFINITY);
                float corr = 1.f, lsum, bo;
                bool need_o = false, diag = false;
                int clo = 0;
                float zdiag = 0.f, mu = 0.f;
                if (fast) {
                    bo = off_band - m_ref;
                } else {
                    int back, chi;
                    bool sk;
                    const int key0 = tile_key0(args, k, t, back, sk);
                    float off;
                    if (!sk) {
                        clo = max(lo_i - key0, 0);
                        chi = min(i - key0, CHUNK - 1);
                        off = off_band;
                    } else {
                        const int jk = i - back, c = jk - key0;
                        if (jk >= 0 && c >= 0 && c < CHUNK) { clo = c; chi = c; }
                        else { clo = CHUNK; chi = -1; }
                        off = off_skip;
                    }
                    const float mt = tile_max(reinterpret_cast<float *>(ra), clo, chi, sk, sc, off);
                    if (mt > m_ref + kRescaleThreshold) {
                        if (m_ref != -INFINITY) {
                            corr = fast_exp2(m_ref - mt);
                            need_o = t > 0;
                        }
                        m_ref = mt;
                    }
                    l *= corr;
                    mu = (m_ref == -INFINITY) ? 0.f : m_ref;
                    bo = off - mu;
                    diag = sk;
                    zdiag = mt;
                }
                if (diag) {
                    lsum = tile_exp_diag(ra, clo, zdiag, mu);
                } else {
#pragma unroll 1
                    for (int pass = 0;; ++pass) {
                        lsum = tile_exp(ra, sc, bo);
                        if (!fast || pass > 0 || !__any_sync(0xffffffffu, !(lsum <= 256.f))) break;
                        tmem_ld32(tS, ra);
                        tmem_wait_ld();
                        const float mt = fmaf(tile_raw_max(ra), sc, off_band);
                        if (mt > m_ref + kRescaleThreshold) {
                            corr = fast_exp2(m_ref - mt);
                            need_o = true;
                            m_ref = mt;
                        }
                        l *= corr;
                        bo = off_band - m_ref;
                    }
                }
                tmem_st16(tS, ra);  // P as bf16 pairs (half a step of 2^-7 relative; l sums the unrounded values)
                l += lsum;
                __syncwarp();
                // O is rescaled where the reference moved; PV of the previous tile must be done (its phase is the
                // barrier's last: the next PV waits for this thread's P)
                if (__any_sync(0xffffffffu, need_o)) {
                    const bool r_ = wait_bar(bar(C::B_PV + (int)((gsm - 1) % NB)), ((gsm - 1) / NB) & 1, wc);
                    if (!__all_sync(0xffffffffu, r_)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const float f = need_o ? corr : 1.f;
#pragma unroll 1
                    for (int oc = 0; oc < D / 16; ++oc) {
                        uint32_t x[16];
                        tmem_ld16(tbase + lane_base + C::O_COL + oc * 16, x);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 16; ++c) x[c] = __float_as_uint(__uint_as_float(x[c]) * f);
                        tmem_st16(tbase + lane_base + C::O_COL + oc * 16, x);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(bar(C::B_PR + buf));
            }
            if (ok && has_next) al_next = alpha_of(pn, Ln);  // used after the epilogue

            // ---- epilogue: O / l as bf16, staged in shared memory for its TMA store, or (a block that is not full)
            // straight to the rows that hold queries
            const bool whole = is_whole(k);
            if (ok) ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_OF), (uint32_t)(kb & 1), wc));
            if (ok && kb > 0) ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_STR), (uint32_t)((kb - 1) & 1), wc));
            if (ok && has_next) ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_QT), (uint32_t)((kb + 1) & 1), wc));
            if (!ok) break;
            const float inv_l = (l > 0.f) ? 1.f / l : 0.f;
            tc_fence_after();
            __syncwarp();
            const long long row_g = (long long)(k.tq + trow) * s.H + h;
            __nv_bfloat16 *orow = ea.out + row_g * D;
#pragma unroll 1
            for (int oh = 0; oh < D / 32; oh += 2) {
                uint32_t x[64];
                tmem_ld32(tbase + lane_base + C::O_COL + oh * 32, x);
                tmem_ld32(tbase + lane_base + C::O_COL + oh * 32 + 32, x + 32);
                tmem_wait_ld();
                uint8_t *rowp = smem + C::Q_OFF + (oh >> 1) * C::Q_DBLK + r * ROW_BYTES;
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    const float *f = reinterpret_cast<const float *>(x) + 8 * w;
                    const uint4 val = make_uint4(pack_bf16(f[0] * inv_l, f[1] * inv_l), pack_bf16(f[2] * inv_l, f[3] * inv_l),
                                                 pack_bf16(f[4] * inv_l, f[5] * inv_l), pack_bf16(f[6] * inv_l, f[7] * inv_l));
                    if (whole) *reinterpret_cast<uint4 *>(rowp + ((w ^ (r & 7)) << 4)) = val;
                    else if (row_ok) *reinterpret_cast<uint4 *>(orow + oh * 32 + w * 8) = val;
                }
            }
            fence_proxy_async_smem();
            tc_fence_before();
            mbar_arrive(bar(C::B_STF));
            if (row_ok) ea.lse[row_g] = (l > 0.f) ? (m_ref + log2f(l)) * kLn2 : -INFINITY;
            L = Ln;
            pd = pn;
        }
    } else if constexpr (C::QUANT) {
        // ================= converters (warps 8-11): raw tiles -> bf16 tiles.  Lane = row of the tile; warp w takes
        // the codes of columns (D / 4) w ... (D / 4) w + D / 4 - 1, which share a scale block.
        const int w = warp - 8;
        constexpr int CH = D / 64;  // 16-code chunks per lane and tile
        uint32_t n = 0;
        bool ok = true;
        PlanBlock pd{};
        if (L0 < n_blocks) pd = load_plan(args, L0);
        for (int L = L0; ok && L < n_blocks; L = next_block(L)) {
            Block k;
            describe(args, pd, L, k);
            if (next_block(L) < n_blocks) pd = load_plan(args, next_block(L));
            for (int t = 0; t < k.n_tiles; ++t, ++n) {
                const int rs = (int)(n % RST);
                int lo, hi;
                const int key0 = tile_range(args, k, t, lo, hi);
                const bool used = key0 + lane >= lo && key0 + lane <= hi;
                ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_RF + rs), (n / RST) & 1, wc));
                if (!ok) break;
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const uint8_t *raw = smem + C::R_OFF + rs * 2 * C::RAW + kv * C::RAW + lane * D;
                    uint4 x[CH];
#pragma unroll
                    for (int u = 0; u < CH; ++u) {
                        // raw rows of 128 bytes are swizzled over 8 rows, rows of 64 bytes over pairs of rows
                        const int chunk = w * CH + u;
                        x[u] = *reinterpret_cast<const uint4 *>(raw + ((D == 128 ? chunk ^ (lane & 7) : chunk ^ ((lane >> 1) & 3)) << 4));
                    }
                    const uint32_t sb = smem[C::SC_OFF + (rs * 2 + kv) * C::SCALES + lane * (D / kScaleBlock) + w * (D / 4) / kScaleBlock];
                    const Scale2 s2 = scale_same(sb);
                    if (kv == 1) {  // both raw tiles are read
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(C::B_RE + rs));
                    }
                    const int stages = kv ? VST : KST, st = (int)(n % stages);
                    const uint32_t round = n / stages;
                    if (round > 0) ok = __all_sync(0xffffffffu, wait_bar(bar((kv ? C::B_VE : C::B_KE) + st), (round - 1) & 1, wc));
                    if (!ok) break;
                    uint8_t *out = smem + (kv ? C::V_OFF : C::K_OFF) + st * C::KV_STAGE + lane * ROW_BYTES;
#pragma unroll
                    for (int u = 0; u < CH; ++u) {
                        uint32_t o[8];
                        const uint32_t c4[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
                        for (int y = 0; y < 4; ++y) codes_to_bf16<KV>(c4[y], s2, o[2 * y], o[2 * y + 1]);
                        if (!used) {  // may hold anything: zero for the PV product, any score is masked
#pragma unroll
                            for (int y = 0; y < 8; ++y) o[y] = 0u;
                        }
                        const int col = (w * CH + u) * 16, c16 = (col & 63) >> 3;  // 16-byte pieces c16, c16 + 1 of the row
                        uint8_t *blk = out + (col >> 6) * C::KV_DBLK;
                        *reinterpret_cast<uint4 *>(blk + ((c16 ^ (lane & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4 *>(blk + (((c16 + 1) ^ (lane & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar((kv ? C::B_VF : C::B_KF) + st));
                }
                if (!ok) break;
            }
        }
    }

    // ---- teardown
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tbase, TMEM_COLS);
    }
}

// ------------------------------------------------------------------ host side

// 3-D map of 16-bit (bf16) or 8-bit elements: [n2][n1][n0] with strides in bytes and a box (b0, b1, b2).
static bool encode(CUtensorMap *m, const void *ptr, bool bf16, int n0, long long n1, long long n2, long long st1, long long st2,
                   int b0, int b1, int b2, CUtensorMapSwizzle swizzle) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)n0, (cuuint64_t)n1, (cuuint64_t)n2};
    const cuuint64_t strides[2] = {(cuuint64_t)st1, (cuuint64_t)st2};
    const cuuint32_t box[3] = {(cuuint32_t)b0, (cuuint32_t)b1, (cuuint32_t)b2};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(ptr), dims, strides,
              box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int KV>
static cudaError_t launch(const Args &a, cudaStream_t st) {
    using C = Cfg<D, KV>;
    const ExtendArgs &e = a.a;
    const PagedCache &c = e.cache;
    const long long planes = (long long)c.n_pages * c.Hkv, row = (long long)D * (C::QUANT ? 1 : 2);
    const CUtensorMapSwizzle page_swizzle = !C::QUANT || D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    CUtensorMap mq, mk, mv, mo;
    if (!encode(&mq, e.q, true, D, e.batch.T, e.s.H, e.q_stride * 2, D * 2, 64, a.R, a.GP, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode(&mo, e.out, true, D, e.batch.T, e.s.H, (long long)e.s.H * D * 2, D * 2, 64, a.R, a.GP, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode(&mk, c.k, !C::QUANT, D, c.page, planes, row, row * c.page, C::QUANT ? D : 64, a.box, 1, page_swizzle) ||
        !encode(&mv, c.v, !C::QUANT, D, c.page, planes, row, row * c.page, C::QUANT ? D : 64, a.box, 1, page_swizzle))
        return cudaErrorNotSupported;
    static PerDeviceOnce configured;
    int dev = 0;
    cudaGetDevice(&dev);
    if (configured.needed(dev)) {
        const cudaError_t err = cudaFuncSetAttribute(extend_tc_kernel<D, KV>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
        if (err != cudaSuccess) return err;
        configured.mark(dev);
    }
    const long long most = max_blocks(e.batch.T, e.batch.B, a.R) * a.ngrp;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min<long long>(most, 2LL * pi::sm_count()), 1, 1);
    cfg.blockDim = dim3(C::THREADS, 1, 1);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, extend_tc_kernel<D, KV>, mq, mk, mv, mo, a);
}

static int packed_heads(int G) { return G % 4 == 0 ? 4 : G % 2 == 0 ? 2 : 1; }

}  // namespace ext

size_t extend_workspace_bytes(long long B, long long T) {
    // blocks of at least 32 positions
    return (size_t)(ext::PLAN_HEAD + ext::max_blocks(T, B, ext::BM / 4) * (long long)sizeof(ext::PlanBlock));
}

cudaError_t launch_extend(const ExtendArgs &e, cudaStream_t st) {
    using namespace ext;
    const Shape &s = e.s;
    const int G = s.H / s.Hkv, GP = packed_heads(G), R = BM / GP, ngrp = s.H / GP;
    if (max_blocks(e.batch.T, e.batch.B, R) * ngrp > 0x7fffffffLL - 1024) return cudaErrorInvalidConfiguration;
    const bool skips = s.mode != kModeEcp && s.S > 0;
    Args a{e, e.workspace, GP, R, R == 32 ? 5 : R == 64 ? 6 : 7, ngrp, skips ? first_skip_multiple(s) : 1,
           skips && s.period % CHUNK == 0, std::min(CHUNK, e.cache.page), make_fastdiv(ngrp), make_fastdiv(G),
           make_fastdiv(skips ? s.period : 1)};
    plan_kernel<<<1, PLAN_THREADS, 0, st>>>(e.cache, e.batch, R, e.workspace, e.index_word);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    const bool d64 = s.d == 64;
    switch (e.cache.kv_type) {
        case kKvBf16: return d64 ? launch<64, kKvBf16>(a, st) : launch<128, kKvBf16>(a, st);
        case kKvE4m3: return d64 ? launch<64, kKvE4m3>(a, st) : launch<128, kKvE4m3>(a, st);
        default: return d64 ? launch<64, kKvInt8>(a, st) : launch<128, kKvInt8>(a, st);
    }
}

}  // namespace pi
