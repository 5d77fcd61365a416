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
//   * A plan kernel (over 8-bit caches the converting one, see below) turns the batch's offsets and contexts into a list of
//     position blocks; it and the checks run on the device, so that a captured graph follows its inputs.  The attention
//     kernel starts beside it (programmatic launch) and waits for it once its barriers and TMEM are set up.
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
//     a row's range are replaced before they are used.  Where a row that some of the block's queries attend holds a
//     non-finite value, the others' products are NaN too: such output rows are computed again (pi_row.cuh).
//   * 8-bit caches: the 32-key tiles that the chunk attends are first turned into bf16 tiles in the workspace (exact,
//     see pi_paged.cuh), which the same kernel then reads instead of pages.  A key tile serves up to a dozen blocks,
//     and each of them converting its own (four converter warps per CTA between a ring of raw tiles and the pipeline)
//     put so much into the SM's instruction stream that a 65536-token chunk (16 heads on 4, d = 128, band 256,
//     4 skips of 1024) took 512-640 us; converted beforehand it takes 264 us, and 233 us over bf16 pages.
#include <cuda.h>

#include <type_traits>

#include "pi_launch.h"
#include "pi_mma.cuh"
#include "pi_paged.cuh"
#include "pi_plan.cuh"
#include "pi_row.cuh"
#include "pi_tc_ptx.cuh"
#include "pi_tile.cuh"

namespace pi {
namespace ext {

using namespace tc;
using namespace plan;
static_assert(TILE == CHUNK, "one size of tile");

constexpr int BM = 128;         // rows per block (MMA M)
constexpr int TMEM_COLS = 256;  // per CTA, two CTAs per SM
constexpr int ROW_BYTES = 128;  // one 64-element bf16 swizzle row
constexpr int THREADS = 256;

// ------------------------------------------------------------------ the plan

constexpr int PLAN_THREADS = 256, PLAN_CTAS = 8;  // each makes the same sums and writes its share

struct PlanArgs {
    Shape s;
    PagedCache c;
    PagedBatch bt;
    int R, m_first;
    int *plan, *index_word;
    int2 *slots;  // 8-bit caches: [slot] sequence and tile (negative: before the sequence); else null
};

__device__ __forceinline__ PlanBlock *plan_blocks(const PlanArgs &a) {
    return reinterpret_cast<PlanBlock *>(reinterpret_cast<char *>(a.plan) + PLAN_HEAD);
}

// Block `x` of the plan: the one at `place` of sequence b, whose bf16 tiles (8-bit caches) are in slot and the following.
__device__ __forceinline__ void write_block(const PlanArgs &a, int x, int b, int t0, int n, int ctx, int place, int slot) {
    PlanBlock *to = plan_blocks(a) + x;
    PlanBlock k = plan_block(a.s, a.m_first, a.R, b, t0, n, ctx, first_block(n, ctx, a.R) + place * a.R);
    int4 *out = reinterpret_cast<int4 *>(to);
    out[0] = make_int4(k.p0, k.tq, k.first, k.last);
    out[1] = make_int4(k.b, k.lo, k.n_band, k.n_tiles);
    out[2] = make_int4(k.cpb, (int)k.inv_cpb, k.full_lo, k.full_hi);
    if (!a.slots) return;
    place_slots(k, seq_tiles(a.s, a.m_first, n, ctx), slot, ctx);
    out[3] = make_int4(k.slot, k.slot_lo, k.slot_windows, k.ctx);
    to->per_window = k.per_window;
}

// A warp's view of a batch of at most 32 sequences, one to a lane.
struct Lanes {
    int t0, n, ctx, slots_upto;  // n = 0: none, or out of range; slots of the sequences up to and including this one
    SeqTiles q;
    bool sorted;  // the warp's: offsets do not decrease

    __device__ __forceinline__ Lanes() : t0(0), n(0), ctx(0), slots_upto(0), q{}, sorted(true) {}
    __device__ __forceinline__ Lanes(const PlanArgs &a, bool record) : t0(0), n(0), ctx(0), slots_upto(0), q{} {
        const int lane = threadIdx.x & 31;
        sorted = true;
        if (lane < a.bt.B) {
            const int t1 = a.bt.cu[lane + 1];
            t0 = a.bt.cu[lane];
            ctx = a.bt.ctx[lane];
            sorted = t0 <= t1;
            if (sequence_ok(a.c, a.bt, t0, t1, ctx)) n = t1 - t0;
            else if (record) record_index(a.index_word);
        }
        sorted = __all_sync(0xffffffffu, sorted);
        if (a.slots) {
            if (n > 0) q = seq_tiles(a.s, a.m_first, n, ctx);
            slots_upto = sums(q.slots);
        }
    }
    static __device__ __forceinline__ int sums(int x) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int w = 1; w < 32; w <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, w);
            if (lane >= w) x += y;
        }
        return x;
    }
};

// What CTA `part` of PLAN_CTAS does for the plan of at most 32 sequences: one round of loads, no barrier (with make_plan
// below a 1024-token chunk over bf16 pages takes 13.4 us instead of 12.6).  The kernels that use it need no list of slots.
__device__ __forceinline__ void make_short_plan(const PlanArgs &a, int part) {
    const int lane = threadIdx.x & 31, wid = part * (PLAN_THREADS / 32) + (threadIdx.x >> 5);
    const Lanes v(a, wid == 0);
    const int cnt = v.n > 0 ? count_blocks(v.n, v.ctx, a.R) : 0, upto = Lanes::sums(cnt);
    const int total = v.sorted ? __shfl_sync(0xffffffffu, upto, 31) : 0;
    for (int x0 = wid * 32; x0 < total; x0 += PLAN_CTAS * PLAN_THREADS) {
        const int x = x0 + lane;
        int o = 0;  // the sequence of block x: as many have ended before
#pragma unroll
        for (int step = 16; step > 0; step >>= 1)
            if (__shfl_sync(0xffffffffu, upto, o + step - 1) <= x) o += step;
        auto of = [&](int y) { return __shfl_sync(0xffffffffu, y, o); };
        const int t0 = of(v.t0), n = of(v.n), ctx = of(v.ctx), place = x - of(upto - cnt), slot = of(v.slots_upto - v.q.slots);
        if (x < total) write_block(a, x, o, t0, n, ctx, place, slot);
    }
    if (wid == 0 && lane == 31) {
        a.plan[0] = total;
        a.plan[1] = v.sorted ? v.slots_upto : 0;
        if (!v.sorted) record_index(a.index_word);
    }
}

// (for the conversion, whose registers it would crowd; in the plan's own kernel a call costs 0.7 us)
__device__ __noinline__ void make_short_plan_apart(const PlanArgs &a, int part) { make_short_plan(a, part); }

// The same for any number of sequences, PLAN_THREADS at a time; with the list of slots.
__device__ __forceinline__ void make_plan(const PlanArgs &a, int part) {
    const PagedCache &c = a.c;
    const PagedBatch &bt = a.bt;
    const int R = a.R;
    int *plan = a.plan, *index_word = a.index_word;
    __shared__ int upto[PLAN_THREADS];  // blocks of the round's sequences up to and including each
    __shared__ int slots_upto[PLAN_THREADS];
    __shared__ int warp_sum[PLAN_THREADS / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // Offsets that decrease would let sequences overlap and their blocks outgrow the plan: nothing is planned.
    bool sorted = true;
    for (int b = tid; b < bt.B; b += PLAN_THREADS) sorted = sorted && bt.cu[b] <= bt.cu[b + 1];
    if (!__syncthreads_and(sorted)) {
        if (tid == 0 && part == 0) {
            record_index(index_word);
            plan[0] = plan[1] = 0;
        }
        return;
    }
    // inclusive sums over the CTA's threads into buf; returns the total
    auto scan = [&](int x, int *buf) -> int {
        int sum = x;
#pragma unroll
        for (int w = 1; w < 32; w <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, w);
            if (lane >= w) sum += y;
        }
        __syncthreads();  // warp_sum and buf are free
        if (lane == 31) warp_sum[warp] = sum;
        __syncthreads();
        for (int w = 0; w < warp; ++w) sum += warp_sum[w];
        buf[tid] = sum;
        __syncthreads();
        return buf[PLAN_THREADS - 1];
    };
    // the thread whose share of the sums holds item x, and the item's place in it
    auto owner = [&](const int *buf, int x, int &place) -> int {
        int lo = 0, hi = PLAN_THREADS - 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (buf[mid] > x) hi = mid;
            else lo = mid + 1;
        }
        place = x - (lo > 0 ? buf[lo - 1] : 0);
        return lo;
    };
    int base = 0, slot_base = 0;
    for (int b0 = 0; b0 < bt.B; b0 += PLAN_THREADS) {
        const int b = b0 + tid;
        int cnt = 0, slots = 0;
        if (b < bt.B) {
            const int t0 = bt.cu[b], t1 = bt.cu[b + 1], ctx = bt.ctx[b];
            if (!sequence_ok(c, bt, t0, t1, ctx)) record_index(index_word);
            else if (t1 > t0) {
                cnt = count_blocks(t1 - t0, ctx, R);
                if (a.slots) slots = seq_tiles(a.s, a.m_first, t1 - t0, ctx).slots;
            }
        }
        const int total = scan(cnt, upto);
        const int total_slots = a.slots ? scan(slots, slots_upto) : 0;
        for (int x = part * PLAN_THREADS + tid; x < total; x += PLAN_CTAS * PLAN_THREADS) {
            int place;
            const int o = owner(upto, x, place);
            const int t0 = bt.cu[b0 + o], n = bt.cu[b0 + o + 1] - t0, ctx = bt.ctx[b0 + o];
            write_block(a, base + x, b0 + o, t0, n, ctx, place, a.slots ? slot_base + (o > 0 ? slots_upto[o - 1] : 0) : 0);
        }
        for (int x = part * PLAN_THREADS + tid; x < total_slots; x += PLAN_CTAS * PLAN_THREADS) {
            int place;
            const int o = owner(slots_upto, x, place);
            const int n = bt.cu[b0 + o + 1] - bt.cu[b0 + o], ctx = bt.ctx[b0 + o];
            const SeqTiles q = seq_tiles(a.s, a.m_first, n, ctx);
            a.slots[slot_base + x] = make_int2(b0 + o, slot_tile(a.s, a.m_first, q, n, ctx, place));
        }
        base += total;
        slot_base += total_slots;
    }
    if (tid == 0 && part == 0) {
        plan[0] = base;
        plan[1] = slot_base;
    }
}

__global__ void __launch_bounds__(PLAN_THREADS) plan_kernel(const __grid_constant__ PlanArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    if (a.bt.B <= 32) make_short_plan(a, blockIdx.x);
    else make_plan(a, blockIdx.x);
}

// ------------------------------------------------------------------ 8-bit tiles to bf16

struct ConvertArgs {
    PlanArgs p;
    __nv_bfloat16 *k, *v;  // [slots, Hkv, 32, d]
};

constexpr int CONVERT_WARPS = 8;

__device__ __forceinline__ void st_keep(uint4 *p, const uint4 &x, uint64_t policy) {
    asm volatile("st.global.L2::cache_hint.v4.u32 [%0], {%1, %2, %3, %4}, %5;" ::"l"(p), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w),
                 "l"(policy)
                 : "memory");
}

// Whether some query of the chunk attends a key in x .. y of its sequence.
__device__ __forceinline__ bool attended(const PlanArgs &a, int b, int x, int y) {
    const int t0 = a.bt.cu[b], n = a.bt.cu[b + 1] - t0, ctx = a.bt.ctx[b], last = ctx + n - 1;
    if (y >= band_lo(ctx, a.s.mode, a.s.k_local) && x <= last) return true;
    if (a.s.mode == kModeEcp || a.s.S == 0 || x > last) return false;
    // a window's keys are ctx - m * period .. last - m * period
    const int m_hi = min(a.s.S, (last - x) / a.s.period);
    const int m_lo = max(a.m_first, ctx > y ? (ctx - y - 1) / a.s.period + 1 : 0);
    return m_lo <= m_hi;
}

// One warp per (slot, KV head, K or V): 32 rows of codes, all of them in flight at once, to 32 rows of bf16.  Rows of a page
// out of range become zeros.
// LANES (at most 32 sequences): the kernel makes the plan too, in its first CTAs, and the others find their slots' sequences
// themselves, one sequence to a lane, instead of waiting for a plan kernel.
template <int D, int KV, bool LANES>
__global__ void __launch_bounds__(CONVERT_WARPS * 32, D == 64 ? 4 : 3) convert_kernel(const __grid_constant__ ConvertArgs args) {
    const PlanArgs &a = args.p;
    static_assert(CONVERT_WARPS * 32 == PLAN_THREADS, "a CTA of the plan");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    if (LANES && blockIdx.x < PLAN_CTAS) {
        make_short_plan_apart(a, blockIdx.x);
        return;
    }
    const int cta = blockIdx.x - (LANES ? PLAN_CTAS : 0), ctas = gridDim.x - (LANES ? PLAN_CTAS : 0);
    const PagedCache &c = a.c;
    const int lane = threadIdx.x & 31;
    constexpr int PER_ROW = D / 8, ITER = CHUNK * PER_ROW / 32;  // pieces of 8 codes (16 bytes of bf16); pieces per lane
    constexpr int SB = D / kScaleBlock;                          // scale bytes of a row
    const Lanes v = LANES ? Lanes(a, false) : Lanes();  // (the plan records what is out of range)
    if (LANES && !v.sorted) return;
    const int upto = v.slots_upto;
    const int heads = c.Hkv * 2, items = (LANES ? __shfl_sync(0xffffffffu, upto, 31) : a.plan[1]) * heads, step = ctas * CONVERT_WARPS;
    const int half = c.page < CHUNK ? lane >> 4 : 0;
    // an item's sequence, tile and page (page 16: of the lane's half): requested an item ahead
    auto slot_of = [&](int x) -> int2 {
        if (x >= items) return make_int2(0, -1);
        const int slot = x / heads;
        if (!LANES) return ld_now(a.slots + slot);
        const int b = __ffs(__ballot_sync(0xffffffffu, upto > slot)) - 1;
        auto of = [&](int y) { return __shfl_sync(0xffffffffu, y, b); };
        const SeqTiles qb{of(v.q.lo), of(v.q.band_tiles), of(v.q.per_window), of(v.q.slots)};
        return make_int2(b, slot_tile(a.s, a.m_first, qb, of(v.n), of(v.ctx), slot - of(upto) + qb.slots));
    };
    auto page = [&](int2 st) -> int {
        const int pos = st.y * CHUNK + half * 16;
        return st.y >= 0 && pos < c.width << c.page_log2 ? ld_now(a.bt.table + (long long)st.x * c.width + (pos >> c.page_log2)) : -1;
    };
    int x = cta * CONVERT_WARPS + (threadIdx.x >> 5);
    int2 st = slot_of(x), st_next = slot_of(x + step);
    int pg = page(st);
    uint64_t keep;  // the tiles are read again soon, by the attention kernel
    asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(keep));
    for (; x < items; x += step) {
        const int2 now = st;
        int p_now = pg;
        st = st_next;
        pg = page(st);
        st_next = slot_of(x + 2 * step);
        if (now.y < 0) continue;
        const bool val = x & 1;
        const int slot = x / heads, g = (x - slot * heads) >> 1, pos = now.y * CHUNK;
        if ((unsigned)p_now >= (unsigned)c.n_pages) {
            p_now = -1;
            if ((lane & 15) == 0 && attended(a, now.x, pos + half * 16, pos + (c.page < CHUNK ? half * 16 + 15 : CHUNK - 1)))
                record_index(a.index_word);
        }
        const long long sh = (long long)slot * c.Hkv + g;
        // A tile's 32 rows (page 16: each half's 16) are contiguous: a lane's pieces lie 256 bytes apart, and lane r holds the
        // scale bytes of row r.
        const uint8_t *codes = static_cast<const uint8_t *>(val ? c.v : c.k), *scales = val ? c.v_scale : c.k_scale;
        const int p0 = __shfl_sync(0xffffffffu, p_now, 0), p1 = __shfl_sync(0xffffffffu, p_now, 16);
        const int at = pos & (c.page - 1), at1 = c.page < CHUNK ? -16 : at;  // first row of the second half less 16
        const uint2 *c0 = reinterpret_cast<const uint2 *>(codes + (long long)row_in_page(c, max(p0, 0), g, at) * D) + lane;
        const uint2 *c1 = reinterpret_cast<const uint2 *>(codes + (long long)(row_in_page(c, max(p1, 0), g, 0) + at1) * D) + lane;
        uint2 w[ITER];
#pragma unroll
        for (int u = 0; u < ITER; ++u) {
            const bool in = (u < ITER / 2 ? p0 : p1) >= 0;
            w[u] = in ? ld_now((u < ITER / 2 ? c0 : c1) + u * 32) : make_uint2(0u, 0u);
        }
        uint32_t sc = 0u;
        const int p = lane < 16 ? p0 : p1;
        if (p >= 0) {
            const long long row = row_in_page(c, p, g, 0) + (lane < 16 ? at : at1) + lane;
            sc = SB == 4 ? ld_now(reinterpret_cast<const uint32_t *>(scales) + row) : ld_now(reinterpret_cast<const uint16_t *>(scales) + row);
        }
        uint4 *out = reinterpret_cast<uint4 *>((val ? args.v : args.k) + sh * (CHUNK * D)) + lane;
        auto piece = [&](const uint2 &x, int u, bool big) {
            const uint32_t s4 = __shfl_sync(0xffffffffu, sc, u * (32 / PER_ROW) + lane / PER_ROW);
            const Scale2<KV> s2 = scale_same<KV>(s4 >> (8 * (lane % PER_ROW / 4)) & 0xffu);
            uint4 o;
            codes_to_bf16<KV>(x.x, s2, big, o.x, o.y);
            codes_to_bf16<KV>(x.y, s2, big, o.z, o.w);
            st_keep(out + u * 32, o, keep);
        };
        // e4m3: scales above 2^7 need a second factor (rare)
        const bool big = KV == kKvE4m3 && __any_sync(0xffffffffu, __vcmpgtu4(sc, 0x86868686u) != 0u);
        if (!big) {
#pragma unroll
            for (int u = 0; u < ITER; ++u) piece(w[u], u, false);
        } else {
#pragma unroll
            for (int u = 0; u < ITER; ++u) piece(w[u], u, true);
        }
    }
}

// ------------------------------------------------------------------ shared memory, TMEM, barriers

template <int D>
struct Cfg {
    static constexpr int NB = D == 64 ? 4 : 2;  // S buffers; TMEM columns as in the forward
    static constexpr int O_COL = 128, Q_COL = D == 128 ? 64 : 192;
    static constexpr int KD = D / 64;
    static constexpr int Q_BYTES = BM * D * 2, Q_DBLK = BM * ROW_BYTES;
    static constexpr int KV_STAGE = CHUNK * D * 2, KV_DBLK = CHUNK * ROW_BYTES;
    static constexpr int KSTAGES = 49152 / KV_STAGE;
    static constexpr int VSTAGES = 32768 / KV_STAGE;
    static constexpr int Q_OFF = 0;
    static constexpr int K_OFF = Q_OFF + Q_BYTES;
    static constexpr int V_OFF = K_OFF + KSTAGES * KV_STAGE;
    static constexpr int DATA_BYTES = V_OFF + VSTAGES * KV_STAGE;
    // barriers; tiles are counted across the blocks a CTA processes, block k completes the per-block
    // ones in phase k
    static constexpr int B_Q = 0;                 // Q tile landed
    static constexpr int B_KF = 1;                // K tile landed
    static constexpr int B_KE = B_KF + KSTAGES;   // its stage free
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
    static constexpr int NBARS = B_SD + 1;
    static constexpr int arrivals(int idx) {
        if ((idx >= B_PR && idx < B_PR + NB) || idx == B_STF) return 128;
        return 1;
    }
    static constexpr int BAR_BYTES = NBARS * 8 + 16;
    static_assert(BAR_BYTES <= 512, "barriers must fit the alignment gap or its complement");
    static constexpr int SMEM_BYTES = DATA_BYTES + 1024;  // data from a 1024-byte boundary; barriers in the gap or behind
    static_assert(SMEM_BYTES <= 115712, "two CTAs per SM");
};

struct Args {
    ExtendArgs a;
    const int *plan;
    int GP, R, R_log2, ngrp;
    int m_first;
    int aligned;  // skips_aligned()
    int box;      // rows of a TMA box: min(32, page)
    int n_planes; // pages, or slots of converted tiles
    FastDiv div_ngrp, div_G;
};

// One block: a plan block x one group of GP heads.
struct Block : PlanBlock {
    int h0, g;
};

__device__ __forceinline__ const int4 *plan_at(const Args &a, int L) {
    return reinterpret_cast<const int4 *>(reinterpret_cast<const char *>(a.plan) + PLAN_HEAD) + 5 * a.div_ngrp.div(L);
}
__device__ __forceinline__ void load_rows(const Args &a, int L, PlanBlock &k) {  // the block's rows only
    const int4 x = plan_at(a, L)[0];
    k.p0 = x.x; k.tq = x.y; k.first = x.z; k.last = x.w;
}
__device__ __forceinline__ void load_tiles(const Args &a, int L, PlanBlock &k) {  // the rest
    const int4 *p = plan_at(a, L);
    const int4 y = p[1], z = p[2];
    k.b = y.x; k.lo = y.y; k.n_band = y.z; k.n_tiles = y.w;
    k.cpb = z.x; k.inv_cpb = (uint32_t)z.y; k.full_lo = z.z; k.full_hi = z.w;
}
__device__ __forceinline__ void load_slots(const Args &a, int L, PlanBlock &k) {  // where its converted tiles are
    const int4 *p = plan_at(a, L);
    const int4 x = p[3];
    k.slot = x.x; k.slot_lo = x.y; k.slot_windows = x.z; k.ctx = x.w;
    k.per_window = reinterpret_cast<const int *>(p + 4)[0];
}
__device__ __forceinline__ int first_head(const Args &a, int L) { return (L - a.div_ngrp.div(L) * a.ngrp) * a.GP; }
template <bool CONVERTED>
__device__ __forceinline__ void load_block(const Args &a, int L, Block &k) {
    load_rows(a, L, k);
    load_tiles(a, L, k);
    if (CONVERTED) load_slots(a, L, k);
    k.h0 = first_head(a, L);
    k.g = a.div_G.div(k.h0);
}

// The non-finite rows of the CTA's blocks, each by a warp.
template <int D, bool CONVERTED>
__device__ __noinline__ void again(const Args &args, int L0, int n_blocks) {
    const ExtendArgs &ea = args.a;
    const Shape &s = ea.s;
    const PagedCache &cache = ea.cache;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, LS = gridDim.x;
    for (int L = L0; L < n_blocks; L = L < n_blocks - LS ? L + LS : n_blocks) {
        Block k;
        load_block<false>(args, L, k);
#pragma unroll 1
        for (int r = warp; r < BM; r += THREADS / 32) {
            const int t = r & (args.R - 1), i = k.p0 + t, h = k.h0 + (r >> args.R_log2);
            if (i < k.first || i > k.last) continue;
            const long long row = (long long)(k.tq + t) * s.H + h;
            __nv_bfloat16 *out = ea.out + row * D;
            uint32_t seen[4] = {};
            if (lane < D / 8) {
                const uint4 x = *reinterpret_cast<const uint4 *>(out + 8 * lane);
                watch(seen, x);
            }
            const float lse = ea.lse[row];
            if (!__any_sync(0xffffffffu, went_bad(seen)) || lse != lse) continue;  // (a NaN among the row's own scores)
            const RowKeys keys = row_keys(s, i, k.g, args.m_first, ea.q + (long long)(k.tq + t) * ea.q_stride + (long long)h * D,
                                          ea.batch.table + (long long)k.b * cache.width, ea.alpha ? ea.alpha + row : nullptr);
            if (!CONVERTED) attend_row<D, kKvBf16>(cache, keys, out);
            else if (cache.kv_type == kKvE4m3) attend_row<D, kKvE4m3>(cache, keys, out);
            else attend_row<D, kKvInt8>(cache, keys, out);
        }
    }
}

constexpr int NO_PAGE = -2;  // a box without an attended row

// CONVERTED: key and value tiles from the workspace (8-bit caches) instead of pages.
template <int D, bool CONVERTED>
__global__ void __launch_bounds__(THREADS, 2)
extend_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO, const __grid_constant__ Args args) {
    using C = Cfg<D>;
    constexpr int KST = C::KSTAGES, VST = C::VSTAGES, NB = C::NB;
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
    volatile uint32_t *abort_flag = misc + 1, *bad_flag = misc + 2;  // bad: a non-finite output seen
    auto bar = [&](int idx) -> uint32_t { return sBar + idx * 8; };

    const ExtendArgs &ea = args.a;
    const Shape &s = ea.s;
    const PagedCache &cache = ea.cache;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const WaitCtx wc{abort_flag, ea.status, ea.timeout_ns};

    if (warp == 0) {
        for (int idx = lane; idx < C::NBARS; idx += 32) mbar_init(bar(idx), (uint32_t)C::arrivals(idx));
        if (lane == 0) *abort_flag = *bad_flag = 0u;
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
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan is written, and the tiles are converted

    // (The first block's entry of the plan is loaded beside the number of blocks: the grid is no larger than the plan's room.)
    const int n_blocks = args.plan[0] * args.ngrp;
    const int L0 = blockIdx.x, LS = gridDim.x;
    auto next_block = [&](int L) -> int { return (L < n_blocks - LS) ? L + LS : n_blocks; };

    // ---- page lookup of a producer warp: lane x holds the page-table entries of tile t0 + x (page 16: of
    // both halves; NO_PAGE where a box has no attended row) and the tile's first row in its page
    auto lookup = [&](const Block &k, int t0, int &e0, int &e1, int &row) {
        e0 = e1 = NO_PAGE;
        row = 0;
        if (t0 + lane >= k.n_tiles) return;
        int lo, hi;
        const int key0 = tile_range(args.m_first, args.a.s.period, k, t0 + lane, lo, hi);
        if (CONVERTED) {
            if (lo > hi) return;
            int back;
            bool skip;
            tile_key0(args.m_first, args.a.s.period, k, t0 + lane, back, skip);
            e0 = tile_slot(args.m_first, s.period, k, key0, back, skip);
            return;
        }
        const int *table = ea.batch.table + (long long)k.b * cache.width;
        row = key0 & (cache.page - 1);
        if (args.box == CHUNK) {
            if (lo <= hi) e0 = ld_now(table + (key0 >> cache.page_log2));
        } else {
            if (lo <= min(hi, key0 + 15)) e0 = ld_now(table + (key0 >> cache.page_log2));
            if (max(lo, key0 + 16) <= hi) e1 = ld_now(table + ((key0 + 16) >> cache.page_log2));
        }
    };
    // page-table entry (or slot) -> plane of the page maps (one past the last, which reads as zeros, where there is no page)
    auto plane = [&](const Block &k, int e) -> int {
        if ((unsigned)e < (unsigned)args.n_planes) return e * cache.Hkv + k.g;
        if (e != NO_PAGE) record_index(ea.index_word);
        return args.n_planes * cache.Hkv;
    };
    // Walks the tiles of every block of the CTA: issue(block, the next one, is there one, tile, tiles so far, planes and
    // row) by the whole warp, with the entries of a block's first 32 tiles requested a block ahead.
    auto walk_tiles = [&](auto &&issue) {
        Block k, kn;
        int e0, e1, row;
        load_block<CONVERTED>(args, L0, k);
        if (L0 >= n_blocks) return true;
        lookup(k, 0, e0, e1, row);
        uint32_t n = 0;
        for (int L = L0;;) {
            const int Ln = next_block(L);
            int n0 = NO_PAGE, n1 = NO_PAGE, nrow = 0;
            if (Ln < n_blocks) {
                load_block<CONVERTED>(args, Ln, kn);
                lookup(kn, 0, n0, n1, nrow);
            }
            int z0 = 0, z1 = 0;
            for (int t = 0; t < k.n_tiles; ++t, ++n) {
                if ((t & 31) == 0) {
                    if (t) lookup(k, t, e0, e1, row);
                    z0 = plane(k, e0);
                    z1 = plane(k, e1);
                }
                if (!issue(k, kn, Ln < n_blocks, t, n, __shfl_sync(0xffffffffu, z0, t & 31), __shfl_sync(0xffffffffu, z1, t & 31),
                           __shfl_sync(0xffffffffu, row, t & 31)))
                    return false;
            }
            if (Ln >= n_blocks) return true;
            L = Ln;
            k = kn;
            e0 = n0;
            e1 = n1;
            row = nrow;
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
    auto issue_q = [&](const Block &k) {  // one lane
        mbar_expect_tx(bar(C::B_Q), C::Q_BYTES);
        for (int dc = 0; dc < C::KD; ++dc)
            tma_load_3d_hint(sQ + dc * C::Q_DBLK, &tmQ, dc * 64, k.tq, k.h0, bar(C::B_Q), policy_evict_first());
    };
    auto is_whole = [&](const PlanBlock &k) -> bool { return k.first == k.p0 && k.last == k.p0 + args.R - 1; };
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
        // ================= producer: K tiles
        const uint64_t reused = policy_evict_last();
        uint32_t issued = 0;
        auto issue = [&](const Block &, const Block &, bool, int, uint32_t n, int z0, int z1, int row) -> bool {
            const int st = (int)(n % KST);
            const uint32_t round = n / KST;
            const bool ok = round == 0 || wait_bar(bar(C::B_KE + st), (round - 1) & 1, wc);
            if (!__all_sync(0xffffffffu, ok)) return false;
            issued = n + 1;
            if (lane == 0) load_tile(&tmK, sK + st * C::KV_STAGE, bar(C::B_KF + st), row, z0, z1, reused);
            __syncwarp();
            return true;
        };
        walk_tiles(issue);
        if (*abort_flag && lane == 0) drain(C::B_KF, KST, issued);
        __syncwarp();
    } else if (warp == 2) {
        // ================= Q tiles, the stores of staged output, and the V tiles.  At V tile t_st of block k
        // the output of block k-1 has been staged; once its store has read the buffer, the Q tile of block
        // k+1 takes its place (that of block k is in TMEM by then).
        const uint64_t reused = policy_evict_last();
        uint32_t issued = 0;
        int q_loads = 0;
        Block prev;
        int kb = 0;
        auto turn = [&](const Block &nx, bool have_next) -> bool {  // the whole warp: store block kb-1, load block kb+1's queries
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
        Block k0;
        load_block<CONVERTED>(args, L0, k0);
        if (L0 < n_blocks) {
            if (lane == 0) issue_q(k0);
            q_loads = 1;
            __syncwarp();
        }
        auto issue = [&](const Block &k, const Block &nx, bool have_next, int t, uint32_t n, int z0, int z1, int row) -> bool {
            const int st = (int)(n % VST);
            const uint32_t round = n / VST;
            const bool w = round == 0 || wait_bar(bar(C::B_VE + st), (round - 1) & 1, wc);
            if (!__all_sync(0xffffffffu, w)) return false;
            issued = n + 1;
            if (lane == 0) load_tile(&tmV, sV + st * C::KV_STAGE, bar(C::B_VF + st), row, z0, z1, reused);
            __syncwarp();
            if (t == min(4, k.n_tiles - 1) && !turn(nx, have_next)) return false;
            if (t == k.n_tiles - 1) {
                prev = k;
                ++kb;
            }
            return true;
        };
        ok = walk_tiles(issue);
        if (ok && kb > 0 && lane == 0) ok = store_out(prev, kb - 1);  // the CTA's last block
        __syncwarp();
        if (*abort_flag && lane == 0) {
            volatile uint32_t zero = 0;
            WaitCtx w2{&zero, nullptr, 20000000ull};
            if (q_loads > 0) wait_bar(bar(C::B_Q), (uint32_t)((q_loads - 1) & 1), w2);
            drain(C::B_VF, VST, issued);
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
        int n_next = plan_at(args, L0)[1].w;
        for (int L = L0; ok && L < n_blocks; L = next_block(L), ++kb) {
            const int n_tiles = n_next;
            if (next_block(L) < n_blocks) n_next = plan_at(args, next_block(L))[1].w;
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
            for (int t = 0; t < n_tiles; ++t, ++gs) {
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
                    if (t == n_tiles - 1) tc_commit(bar(C::B_SD));
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
        PlanBlock kn{};
        auto load = [&](int L) {
            load_rows(args, L, kn);
            load_tiles(args, L, kn);
        };
        load(L0);
        for (int L = L0; ok && L < n_blocks; L = next_block(L)) {
            const PlanBlock k = kn;
            if (next_block(L) < n_blocks) load(next_block(L));
            // (otherwise every tile's rows are all attended, or all before the sequence and loaded as zeros)
            const bool ragged = ((k.lo | k.first | (k.last + 1)) & (CHUNK - 1)) != 0 || (k.n_tiles > k.n_band && !args.aligned);
            for (int t = 0; t < k.n_tiles; ++t, ++gp) {
                const int buf = (int)(gp % NB), st = (int)(gp % VST);
                bool w = wait_bar(bar(C::B_VF + st), (gp / VST) & 1, wc);
                if (w && ragged) {
                    // rows of V that no query attends: zero
                    int lo, hi;
                    const int key0 = tile_range(args.m_first, args.a.s.period, k, t, lo, hi);
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
    } else {
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
            return ld_now(ea.alpha + (long long)(d.tq + trow) * s.H + first_head(args, L) + hh);
        };
        bool ok = true;
        uint32_t gsm = 0;
        int kb = 0;
        PlanBlock k{}, kn{};  // this block and the next one (its rows; its tiles are loaded before the epilogue)
        float al_next = 1.f;
        load_rows(args, L0, k);
        load_tiles(args, L0, k);
        if (L0 < n_blocks) {
            if (next_block(L0) < n_blocks) load_rows(args, next_block(L0), kn);
            al_next = alpha_of(k, L0);
        }
        for (int L = L0; ok && L < n_blocks; ++kb) {
            const int Ln = next_block(L);
            const bool has_next = Ln < n_blocks;
            const float al = al_next;
            if (has_next) al_next = alpha_of(kn, Ln);  // requested now, used after this block
            const float off_band = ea.alpha ? log2f(al) : 0.f, off_skip = log2f(1.f - al);
            // a row without a query takes the part of the nearest one; its result is dropped
            const int i = min(max(k.p0 + trow, k.first), k.last), h = first_head(args, L) + hh;
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
                tmem_wait_ld(ra);
                // Tiles inside every query's band: P with the running reference; the maximum only once some P
                // exceeds 1, which a sum above 1 is the first sign of.
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
                    const int key0 = tile_key0(args.m_first, args.a.s.period, k, t, back, sk);
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
                    if (mt > m_ref) {
                        const float m_new = mt + kHeadroom;
                        if (m_ref != -INFINITY) {
                            corr = fast_exp2(m_ref - m_new);
                            need_o = t > 0;
                        }
                        m_ref = m_new;
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
                        if (!fast || pass > 0 || !__any_sync(0xffffffffu, !(lsum <= kRescaleSum))) break;
                        tmem_ld32(tS, ra);
                        tmem_wait_ld(ra);
                        const float mt = fmaf(tile_raw_max(ra), sc, off_band);
                        if (mt > m_ref) {
                            const float m_new = mt + kHeadroom;
                            corr = fast_exp2(m_ref - m_new);
                            need_o = true;
                            m_ref = m_new;
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
                        tmem_wait_ld(x);
#pragma unroll
                        for (int c = 0; c < 16; ++c) x[c] = __float_as_uint(__uint_as_float(x[c]) * f);
                        tmem_st16(tbase + lane_base + C::O_COL + oc * 16, x);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(bar(C::B_PR + buf));
            }

            // ---- epilogue: O / l as bf16, staged in shared memory for its TMA store, or (a block that is not full)
            // straight to the rows that hold queries
            const bool whole = is_whole(k);
            if (has_next) load_tiles(args, Ln, kn);
            if (ok) ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_OF), (uint32_t)(kb & 1), wc));
            if (ok && kb > 0) ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_STR), (uint32_t)((kb - 1) & 1), wc));
            if (ok && has_next) ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_QT), (uint32_t)((kb + 1) & 1), wc));
            if (!ok) break;
            const float inv_l = l == 0.f ? 0.f : 1.f / l;
            uint32_t seen[4] = {};
            tc_fence_after();
            __syncwarp();
            const long long row_g = (long long)(k.tq + trow) * s.H + h;
            __nv_bfloat16 *orow = ea.out + row_g * D;
#pragma unroll 1
            for (int oh = 0; oh < D / 32; oh += 2) {
                uint32_t x[64];
                tmem_ld32(tbase + lane_base + C::O_COL + oh * 32, x);
                tmem_ld32(tbase + lane_base + C::O_COL + oh * 32 + 32, x + 32);
                tmem_wait_ld(x);
                uint8_t *rowp = smem + C::Q_OFF + (oh >> 1) * C::Q_DBLK + r * ROW_BYTES;
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    const float *f = reinterpret_cast<const float *>(x) + 8 * w;
                    const uint4 val = make_uint4(pack_bf16(f[0] * inv_l, f[1] * inv_l), pack_bf16(f[2] * inv_l, f[3] * inv_l),
                                                 pack_bf16(f[4] * inv_l, f[5] * inv_l), pack_bf16(f[6] * inv_l, f[7] * inv_l));
                    watch(seen, val);
                    if (whole) *reinterpret_cast<uint4 *>(rowp + ((w ^ (r & 7)) << 4)) = val;
                    else if (row_ok) *reinterpret_cast<uint4 *>(orow + oh * 32 + w * 8) = val;
                }
            }
            fence_proxy_async_smem();
            tc_fence_before();
            mbar_arrive(bar(C::B_STF));
            if (row_ok) ea.lse[row_g] = l == 0.f ? -INFINITY : (m_ref + log2f(l)) * kLn2;
            if (row_ok && went_bad(seen) && l == l) *bad_flag = 1u;
            k = kn;
            L = Ln;
            if (L < n_blocks && next_block(L) < n_blocks) load_rows(args, next_block(L), kn);
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
    // ---- rows that a value of another row's key made non-finite: once more, by themselves (pi_row.cuh)
    if (!*bad_flag || *abort_flag) return;
    if (warp == 2 && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // this thread's stores are done
    __syncthreads();
    again<D, CONVERTED>(args, L0, n_blocks);
}

// ------------------------------------------------------------------ host side

// 3-D bf16 map [n2][n1][d] with strides in bytes and a box (64, b1, b2), 128-byte swizzle.
static bool encode(CUtensorMap *m, const void *ptr, int d, long long n1, long long n2, long long st1, long long st2, int b1, int b2) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)n1, (cuuint64_t)n2};
    const cuuint64_t strides[2] = {(cuuint64_t)st1, (cuuint64_t)st2};
    const cuuint32_t box[3] = {64u, (cuuint32_t)b1, (cuuint32_t)b2};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The workspace: the plan; for an 8-bit cache the slots' list and the converted tiles.
struct Layout {
    size_t slots, k, v, bytes;  // offsets
    long long n_slots;
};
static Layout layout(const Shape &s, int kv_type, long long B, long long T, long long cap) {
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    Layout l{};
    const int GP = packed_heads(s.H / s.Hkv);
    l.bytes = l.slots = up((size_t)(PLAN_HEAD + max_blocks(T, B, BM / GP) * (long long)sizeof(PlanBlock)));
    if (kv_type == kKvBf16) return l;
    l.n_slots = most_slots(s, B, T, cap);
    const size_t tiles = up((size_t)l.n_slots * s.Hkv * CHUNK * s.d * 2);
    l.k = l.slots + up((size_t)l.n_slots * sizeof(int2));
    l.v = l.k + tiles;
    l.bytes = l.v + tiles;
    return l;
}

// Launches a kernel that may start while the one before it on the stream still runs (it waits for it itself).
template <typename K, typename... A>
static cudaError_t launch_dependent(K kernel, long long grid, int threads, int smem, cudaStream_t st, const A &...a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a...);
}

template <int D, bool CONVERTED>
static cudaError_t launch(const Args &a, const void *k, const void *v, cudaStream_t st) {
    const ExtendArgs &e = a.a;
    const PagedCache &c = e.cache;
    const long long planes = (long long)a.n_planes * c.Hkv, rows = CONVERTED ? CHUNK : c.page;
    CUtensorMap mq, mk, mv, mo;
    if (!encode(&mq, e.q, D, e.batch.T, e.s.H, e.q_stride * 2, D * 2, a.R, a.GP) ||
        !encode(&mo, e.out, D, e.batch.T, e.s.H, (long long)e.s.H * D * 2, D * 2, a.R, a.GP) ||
        !encode(&mk, k, D, rows, planes, D * 2, D * 2 * rows, a.box, 1) || !encode(&mv, v, D, rows, planes, D * 2, D * 2 * rows, a.box, 1))
        return cudaErrorNotSupported;
    constexpr int smem = Cfg<D>::SMEM_BYTES;
    static PerDeviceOnce configured;
    int dev = 0;
    cudaGetDevice(&dev);
    if (configured.needed(dev)) {
        const cudaError_t err = cudaFuncSetAttribute(extend_tc_kernel<D, CONVERTED>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (err != cudaSuccess) return err;
        configured.mark(dev);
    }
    const long long most = max_blocks(e.batch.T, e.batch.B, a.R) * a.ngrp;
    return launch_dependent(extend_tc_kernel<D, CONVERTED>, std::min<long long>(most, 2LL * pi::sm_count()), THREADS, smem, st, mq, mk, mv,
                            mo, a);
}

}  // namespace ext

bool extend_workspace(const ExtendArgs &e, size_t &bytes) {
    const Shape &s = e.s;
    const PagedCache &c = e.cache;
    const long long T = e.batch.T, B = e.batch.B, cap = (long long)c.width << c.page_log2;
    bytes = 0;
    if (T * s.H > 0x7fffffffLL) return false;  // rows of lse
    if (extend_few_rows(e)) return true;
    const int GP = packed_heads(s.H / s.Hkv);
    if (ext::max_blocks(T, B, ext::BM / GP) * (s.H / GP) > 0x7fffffffLL - 1024) return false;
    if (c.kv_type != kKvBf16 && ext::most_slots(s, B, T, cap) > 0x7fffffffLL / (2 * ext::CHUNK) / s.Hkv) return false;
    bytes = ext::layout(s, c.kv_type, B, T, cap).bytes;
    return true;
}

cudaError_t launch_extend(const ExtendArgs &e, cudaStream_t st) {
    using namespace ext;
    if (extend_few_rows(e)) return launch_extend_few(e, st);
    const Shape &s = e.s;
    const PagedCache &c = e.cache;
    const int G = s.H / s.Hkv, GP = packed_heads(G), R = BM / GP, ngrp = s.H / GP;
    const bool quant = c.kv_type != kKvBf16, skips = s.mode != kModeEcp && s.S > 0;
    const Layout l = layout(s, c.kv_type, e.batch.B, e.batch.T, (long long)c.width << c.page_log2);
    char *ws = reinterpret_cast<char *>(e.workspace);
    int2 *slots = quant ? reinterpret_cast<int2 *>(ws + l.slots) : nullptr;
    Args a{e, e.workspace, GP, R, R == 32 ? 5 : R == 64 ? 6 : 7, ngrp, skips ? first_skip_multiple(s) : 1,
           skips_aligned(s), quant ? CHUNK : std::min(CHUNK, c.page), quant ? (int)l.n_slots : c.n_pages,
           make_fastdiv(ngrp), make_fastdiv(G)};
    const PlanArgs pa{s, c, e.batch, R, a.m_first, e.workspace, e.index_word, slots};
    cudaError_t err = cudaSuccess;
    const bool lanes = e.batch.B <= 32;
    if (!quant || !lanes) {
        err = launch_dependent(plan_kernel, PLAN_CTAS, PLAN_THREADS, 0, st, pa);
        if (err != cudaSuccess) return err;
    }
    if (!quant) return s.d == 64 ? launch<64, false>(a, c.k, c.v, st) : launch<128, false>(a, c.k, c.v, st);
    __nv_bfloat16 *k = reinterpret_cast<__nv_bfloat16 *>(ws + l.k), *v = reinterpret_cast<__nv_bfloat16 *>(ws + l.v);
    const long long items = l.n_slots * s.Hkv * 2;
    const long long grid = std::min<long long>((items + CONVERT_WARPS - 1) / CONVERT_WARPS, 4LL * pi::sm_count());
    auto convert = [&](auto in_lanes) {
        constexpr bool L = decltype(in_lanes)::value;
        auto kernel = s.d == 64 ? (c.kv_type == kKvE4m3 ? convert_kernel<64, kKvE4m3, L> : convert_kernel<64, kKvInt8, L>)
                                : (c.kv_type == kKvE4m3 ? convert_kernel<128, kKvE4m3, L> : convert_kernel<128, kKvInt8, L>);
        return launch_dependent(kernel, grid + (L ? PLAN_CTAS : 0), CONVERT_WARPS * 32, 0, st, ConvertArgs{pa, k, v});
    };
    err = lanes ? convert(std::true_type{}) : convert(std::false_type{});
    if (err != cudaSuccess) return err;
    return s.d == 64 ? launch<64, true>(a, k, v, st) : launch<128, true>(a, k, v, st);
}

}  // namespace pi
