// pi_plan.cuh -- the arithmetic of a paged batch's work lists: a chunk's position blocks, their key tiles, the bf16 tiles of an 8-bit
// cache and their bound, the token groups of short chunks, and the narrowing of the sequence search.  All of it is integer
// work on sizes, for the host as for the device.
#pragma once

#include <algorithm>
#include <cstdint>

#include "pi_common.cuh"

namespace pi {
namespace plan {

constexpr int TILE = 32;  // keys per tile

// Whether every skip window has the same place in its tiles.
__host__ __device__ __forceinline__ bool skips_aligned(const Shape &s) { return s.mode != kModeEcp && s.S > 0 && s.period % TILE == 0; }

// A position block of one sequence and its key tiles, the same for every group of heads.
struct PlanBlock {
    int p0, tq, first, last;  // positions first .. last hold queries; row 0 is position p0 and packed token tq
                              // (possibly before the sequence's own)
    int b, lo, n_band, n_tiles;  // sequence; first band key of the first query; tiles from lo rounded down to 32, and all
    int cpb;                     // tiles per skip window
    uint32_t inv_cpb;            // ceil(2^32 / cpb), 0 for one tile
    int full_lo, full_hi;        // tiles inside the band of every query
    int slot, slot_lo, slot_windows, ctx;  // 8-bit caches: where the sequence's bf16 tiles are (SeqTiles);
    int per_window, pad[3];                // slot_windows < 0: all in one run
};
static_assert(sizeof(PlanBlock) == 80, "16-byte loads");

// The bf16 tiles of a sequence over an 8-bit cache, `slots` of them from slot on: either all tiles from its first
// attended key to its last (band_tiles = 0: tile x, keys 32 x ..., in slot + x - lo), or the band's tiles followed by
// `per_window` for each skip window, whichever is fewer (a long chunk's windows overlap).
struct SeqTiles {
    int lo;          // first tile of all, or of the band
    int band_tiles;
    int per_window;
    int slots;
};

__host__ __device__ __forceinline__ SeqTiles seq_tiles(const Shape &s, int m_first, int n, int ctx) {
    const int last = ctx + n - 1, band0 = band_lo(ctx, s.mode, s.k_local);
    int windows = 0;
    if (s.mode != kModeEcp && s.S > 0) {
        const int m_last = last / s.period < s.S ? last / s.period : s.S;
        windows = m_last >= m_first ? m_last - m_first + 1 : 0;
    }
    SeqTiles q;
    q.lo = band0 >> 5;
    q.band_tiles = (last >> 5) - q.lo + 1;
    q.per_window = ((n - 1) >> 5) + 2;
    q.slots = q.band_tiles;
    if (windows > 0) {
        const long long far = (long long)ctx - (long long)(m_first + windows - 1) * s.period;
        int lo = far > 0 ? (int)(far >> 5) : 0;
        if (q.lo < lo) lo = q.lo;
        const long long each = q.band_tiles + (long long)windows * q.per_window;
        const int all = (last >> 5) - lo + 1;
        if (all <= each) {
            q.lo = lo;
            q.band_tiles = 0;
            q.slots = all;
        } else {
            q.slots = (int)each;
        }
    }
    return q;
}

// The tile in a sequence's slot `place` (negative: none).
__host__ __device__ __forceinline__ int slot_tile(const Shape &s, int m_first, const SeqTiles &q, int n, int ctx, int place) {
    if (!q.band_tiles || place < q.band_tiles) return q.lo + place;
    const int w = (place - q.band_tiles) / q.per_window, back = (m_first + w) * s.period;
    const int tile = ((ctx - back) >> 5) + (place - q.band_tiles) % q.per_window;
    // the window's last tile may lie past it, and a whole tile before the sequence
    return tile > (ctx + n - 1 - back) >> 5 ? -1 : tile;
}

// Most slots that a batch can take, from its sizes alone (cap: positions a page table reaches); below 2^60 for any that the
// C ABI lets through.
inline long long most_slots(const Shape &s, long long B, long long T, long long cap) {
    const long long seqs = std::min(B, T);
    const long long band = std::min<long long>(cap, s.mode == kModeEcp ? 2LL * s.k_local : s.k_local);
    long long windows = 0, reach = band;
    if (s.mode != kModeEcp && s.S > 0) {
        windows = std::min<long long>(s.S, cap / s.period);
        reach = std::min<long long>(cap, std::max(band, windows * s.period));
    }
    const long long each = (T + seqs * band) / 32 + 2 * seqs + windows * (T / 32 + 2 * seqs);
    const long long all = (T + seqs * reach) / 32 + 2 * seqs;
    return std::min(each, all);
}
constexpr int PLAN_HEAD = 32;  // bytes before the blocks: [0] their number, [1] the slots used

__host__ __device__ __forceinline__ long long max_blocks(long long T, long long B, int R) {
    // n tokens lie in at most floor(n / R) + 2 blocks, and a sequence without tokens in none
    return T / R + 2 * (B < T ? B : T);
}

// n tokens at ctx ..: blocks at multiples of R, or one where a short chunk starts
__host__ __device__ __forceinline__ int first_block(int n, int ctx, int R) { return n <= R ? ctx : ctx / R * R; }
__host__ __device__ __forceinline__ int count_blocks(int n, int ctx, int R) { return (ctx + n - 1 - first_block(n, ctx, R)) / R + 1; }

// The block of n tokens at ctx .. whose row 0 is position p0.
__host__ __device__ __forceinline__ PlanBlock plan_block(const Shape &s, int m_first, int R, int b, int t0, int n, int ctx, int p0) {
    PlanBlock k;
    k.p0 = p0;
    k.tq = t0 + p0 - ctx;
    k.first = max(p0, ctx);
    k.last = min(p0 + R, ctx + n) - 1;
    k.b = b;
    k.lo = band_lo(k.first, s.mode, s.k_local);
    const int key0 = k.lo & ~(TILE - 1);
    k.n_band = (k.last - key0) / TILE + 1;
    int windows = 0;
    if (s.mode != kModeEcp && s.S > 0) windows = max(0, min(s.S, k.last / s.period) - m_first + 1);
    k.cpb = skips_aligned(s) ? (k.last >> 5) - (k.first >> 5) + 1 : ((k.last - k.first) >> 5) + 2;
    k.inv_cpb = 0xffffffffu / (uint32_t)k.cpb + 1u;
    k.n_tiles = k.n_band + windows * k.cpb;
    k.full_lo = (band_lo(k.last, s.mode, s.k_local) - key0 + TILE - 1) / TILE;
    const int span = k.first - (TILE - 1) - key0;
    k.full_hi = span >= 0 ? span / TILE : -1;
    return k;
}

// Tile ti of a block: its first key (negative: a tile wholly before the sequence), whether it is a skip tile,
// and its skip distance.
__host__ __device__ __forceinline__ int tile_key0(int m_first, int period, const PlanBlock &k, int ti, int &back, bool &skip) {
    skip = ti >= k.n_band;
    if (!skip) {
        back = 0;
        return (k.lo & ~(TILE - 1)) + ti * TILE;
    }
    const uint32_t x = (uint32_t)(ti - k.n_band);
    const uint32_t w = k.inv_cpb ? (uint32_t)(((uint64_t)x * k.inv_cpb) >> 32) : x;
    back = (m_first + (int)w) * period;
    return ((k.first - back) & ~(TILE - 1)) + (int)(x - w * (uint32_t)k.cpb) * TILE;
}

// Where the bf16 tiles of the block's sequence are, the first of its slots being `slot`.
__host__ __device__ __forceinline__ void place_slots(PlanBlock &k, const SeqTiles &q, int slot, int ctx) {
    k.slot = slot;
    k.slot_lo = q.lo;
    k.slot_windows = q.band_tiles ? slot + q.band_tiles : -1;
    k.ctx = ctx;
    k.per_window = q.per_window;
}

// The slot of the block's tile with first key key0 (not before the sequence), of the band or of the skips at distance back.
__host__ __device__ __forceinline__ int tile_slot(int m_first, int period, const PlanBlock &k, int key0, int back, bool skip) {
    if (skip && k.slot_windows >= 0)
        return k.slot_windows + (back / period - m_first) * k.per_window + (key0 >> 5) - ((k.ctx - back) >> 5);
    return k.slot + (key0 >> 5) - k.slot_lo;
}

// Keys of tile ti that some query of the block attends or may attend: lo .. hi (empty: lo > hi).
__host__ __device__ __forceinline__ int tile_range(int m_first, int period, const PlanBlock &k, int ti, int &lo, int &hi) {
    int back;
    bool skip;
    const int key0 = tile_key0(m_first, period, k, ti, back, skip);
    lo = max(key0, skip ? max(0, k.first - back) : k.lo);
    hi = min(key0 + TILE - 1, k.last - back);
    return key0;
}

// Short chunks: the first of sequence j's token groups, `at` being its first packed token.  Numbered from (at + j (group - 1)) / group
// on, a sequence of n tokens has the ceil(n / group) numbers that it needs before the next one's.
__host__ __device__ __forceinline__ long long group_start(int j, int at, int group) { return ((long long)at + (long long)j * (group - 1)) / group; }

}  // namespace plan

// The range that a search over 1 .. B still covers, with 32 probes to a round: probe x is place(x) if it lies inside, and after a
// round c of them were below.
struct SearchRange {
    int lo, len, step;
    __host__ __device__ __forceinline__ explicit SearchRange(int B) : lo(0), len(B), step((B + 31) >> 5) {}
    __host__ __device__ __forceinline__ bool inside(int x) const { return (x + 1) * step <= len; }
    __host__ __device__ __forceinline__ int place(int x) const { return lo + (x + 1) * step; }
    __host__ __device__ __forceinline__ void narrow(int c) {
        lo += c * step;
        len = len - c * step < step - 1 ? len - c * step : step - 1;
        step = (len + 31) >> 5;
    }
};

}  // namespace pi
