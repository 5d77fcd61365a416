// The paged kernels' work-list arithmetic (csrc/pi_plan.cuh) behind plain functions, for the host tests.
#include "pi_plan.cuh"

using namespace pi;
using namespace pi::plan;

static Shape shape(int k_local, int period, int S, int ecp) {
    Shape s{};
    s.k_local = k_local;
    s.period = period;
    s.S = S;
    s.mode = ecp ? kModeEcp : 0;
    return s;
}
static int first_multiple(const Shape &s) { return s.mode != kModeEcp && s.S > 0 ? first_skip_multiple(s) : 1; }

extern "C" {

int n_blocks(int n, int ctx, int R) { return count_blocks(n, ctx, R); }
long long block_bound(long long T, long long B, int R) { return max_blocks(T, B, R); }

// Block `x` of a chunk of n tokens at ctx: out = p0, tq, first, last, tiles, band tiles, and the band tiles without masks.
void block(int k_local, int period, int S, int ecp, int R, int t0, int n, int ctx, int x, int *out) {
    const Shape s = shape(k_local, period, S, ecp);
    const PlanBlock k = plan_block(s, first_multiple(s), R, 0, t0, n, ctx, first_block(n, ctx, R) + x * R);
    const int v[8] = {k.p0, k.tq, k.first, k.last, k.n_tiles, k.n_band, k.full_lo, k.full_hi};
    for (int i = 0; i < 8; ++i) out[i] = v[i];
}

// Its tile `ti`: out = first key, skip distance (0: band), lowest and highest key that may be attended, and its slot where the
// sequence's slots start at `slot`.
void tile(int k_local, int period, int S, int ecp, int R, int n, int ctx, int x, int ti, int slot, int *out) {
    const Shape s = shape(k_local, period, S, ecp);
    const int m = first_multiple(s);
    PlanBlock k = plan_block(s, m, R, 0, 0, n, ctx, first_block(n, ctx, R) + x * R);
    place_slots(k, seq_tiles(s, m, n, ctx), slot, ctx);
    bool skip;
    out[0] = tile_key0(m, period, k, ti, out[1], skip);
    tile_range(m, period, k, ti, out[2], out[3]);
    out[4] = tile_slot(m, period, k, out[0], out[1], skip);
}

int n_slots(int k_local, int period, int S, int ecp, int n, int ctx) {
    const Shape s = shape(k_local, period, S, ecp);
    return seq_tiles(s, first_multiple(s), n, ctx).slots;
}
int tile_of_slot(int k_local, int period, int S, int ecp, int n, int ctx, int place) {
    const Shape s = shape(k_local, period, S, ecp);
    const int m = first_multiple(s);
    return slot_tile(s, m, seq_tiles(s, m, n, ctx), n, ctx, place);
}
long long slot_bound(int k_local, int period, int S, int ecp, long long B, long long T, long long cap) {
    return most_slots(shape(k_local, period, S, ecp), B, T, cap);
}

long long token_group(int j, int at, int group) { return group_start(j, at, group); }

// The search for the number of j in 1 .. B with cu[j] <= t, its 32 probes one after the other; counts probes outside 1 .. B.
int search(const int *cu, int B, int t, int *outside) {
    SearchRange r(B);
    *outside = 0;
    while (r.len > 0) {
        int c = 0;
        for (int x = 0; x < 32; ++x) {
            if (!r.inside(x)) continue;
            const int j = r.place(x);
            if (j < 1 || j > B) ++*outside;
            else c += cu[j] <= t;
        }
        r.narrow(c);
    }
    return r.lo;
}

}  // extern "C"
