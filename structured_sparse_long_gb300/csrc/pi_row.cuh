// pi_row.cuh -- one row of the paged attention by one warp, over the keys that this row attends and no others.
//
// The tiled kernels multiply a tile's values by P = 0 where a row does not attend a key that other rows of its block do, and 0 * NaN
// or 0 * infinity is NaN.  They look at their results (one multiplication by zero per pair of outputs, 69.1 -> 69.7 us for the
// 16384-token chunk below) and compute the rows that came out non-finite again here, after the CTA's last block, so that no
// wait of the pipeline spans it.  Bound by latency, a row at a time per warp (some 40 us at 260 keys): a 16384-token chunk
// over bf16 pages, 16 heads on 4, d = 128, takes 0.7 to 0.9 ms with one NaN among its attended values.
#pragma once

#include "pi_mma.cuh"
#include "pi_paged.cuh"
#include "pi_quant.cuh"

namespace pi {

// A query row and its keys: the band lo .. i, then i - m * period for m = m_first .. m_first + n_skip - 1.
struct RowKeys {
    const __nv_bfloat16 *q;  // [d]
    const int *table;        // its sequence's pages
    int kvh, lo, i, m_first, n_skip, period;
    float scale_log2, off_band, off_skip;
    // a drafted tree's node: its sequence's parents, the positions from which on a key is an ancestor, and its own number
    const int *parent;
    int ctx, node;
};

__device__ __forceinline__ RowKeys row_keys(const Shape &s, int i, int kvh, int m_first, const __nv_bfloat16 *q, const int *table,
                                            const float *alpha) {
    const int n_skip = s.mode != kModeEcp && s.S > 0 ? max(0, min(s.S, i / s.period) - m_first + 1) : 0;
    const float al = alpha ? *alpha : 1.f;
    return RowKeys{q, table, kvh, band_lo(i, s.mode, s.k_local), i, m_first, n_skip, s.period, s.scale_log2, alpha ? log2f(al) : 0.f,
                   log2f(1.f - al), nullptr, 0, 0};
}

// The row, to out[d].  For the whole warp.
template <int D, int KV, bool TREE = false>
__device__ __forceinline__ void attend_row(const PagedCache &c, const RowKeys &k, __nv_bfloat16 *out) {
    constexpr int NC = D / 64;
    const int lane = threadIdx.x & 31, col = 8 * (lane & 7);
    const int n_band = k.i - k.lo + 1, n = n_band + k.n_skip;
    float m = -INFINITY, l = 0.f, o[NC][8] = {};
    for (int k0 = 0; k0 < n; k0 += 32) {  // a key per lane for the scores
        const int kk = k0 + lane;
        int row = -1;
        float z = -INFINITY;
        if (kk < n) {
            int pos = kk < n_band ? k.lo + kk : k.i - (k.m_first + kk - n_band) * k.period;
            if (TREE && pos >= k.ctx) {
                int at = k.node;
                for (int up = k.i - pos; up > 0; --up) at = ld_now(k.parent + at);
                pos = k.ctx + at;
            }
            const int pg = page_of(c, k.table, 0, pos);
            if (pg >= 0) row = row_in_page(c, pg, k.kvh, pos);
        }
        if (row >= 0) {
            float dot = 0.f;
#pragma unroll 8
            for (int x = 0; x < D / 8; ++x) {
                float a[8], b[8];
                unpack8(get8<KV>(c, c.k, c.k_scale, row, 8 * x), a);
                unpack8(ld_now(reinterpret_cast<const uint4 *>(k.q) + x), b);
#pragma unroll
                for (int e = 0; e < 8; ++e) dot = fmaf(a[e], b[e], dot);
            }
            z = fmaf(dot, k.scale_log2, kk < n_band ? k.off_band : k.off_skip);
        }
        float mx = z;
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
        const float mn = fmaxf(m, mx), ref = mn == -INFINITY ? 0.f : mn, corr = exp2f(m - ref), p = exp2f(z - ref);
        m = mn;
        l = fmaf(l, corr, p);
#pragma unroll
        for (int e = 0; e < 8 * NC; ++e) o[e >> 3][e & 7] *= corr;
#pragma unroll 4
        for (int x = 0; x < 32; x += 4) {  // a key per eight lanes for the values
            const int r = __shfl_sync(0xffffffffu, row, x + (lane >> 3));
            const float w = __shfl_sync(0xffffffffu, p, x + (lane >> 3));
#pragma unroll
            for (int y = 0; y < NC; ++y) {
                float v[8] = {};
                if (r >= 0) unpack8(get8<KV>(c, c.v, c.v_scale, r, col + 64 * y), v);
#pragma unroll
                for (int e = 0; e < 8; ++e) o[y][e] = fmaf(r >= 0 ? w : 0.f, v[e], o[y][e]);
            }
        }
    }
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int y = 0; y < NC; ++y) {
        float *x = o[y];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] += __shfl_xor_sync(0xffffffffu, x[e], 8);
            x[e] += __shfl_xor_sync(0xffffffffu, x[e], 16);
            x[e] = l == 0.f ? 0.f : x[e] * inv;  // (no finite logit: 0, whatever the values are)
        }
        if (lane < 8)
            *reinterpret_cast<uint4 *>(out + col + 64 * y) =
                make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
}

// A NaN in `sum` (0 before the first pair of bf16) once some pair held a NaN or an infinity.
__device__ __forceinline__ void watch(uint32_t &sum, uint32_t pair) {
    const __nv_bfloat162 r = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&pair), __nv_bfloat162(__ushort_as_bfloat16(0), __ushort_as_bfloat16(0)),
                                     *reinterpret_cast<const __nv_bfloat162 *>(&sum));
    sum = *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ bool went_bad(uint32_t sum) { return (sum & 0x7fff7fffu) != 0u; }
// The same of 16 bytes, in four sums that do not wait for each other.
__device__ __forceinline__ void watch(uint32_t (&sum)[4], const uint4 &x) {
    watch(sum[0], x.x);
    watch(sum[1], x.y);
    watch(sum[2], x.z);
    watch(sum[3], x.w);
}
__device__ __forceinline__ bool went_bad(const uint32_t (&sum)[4]) { return went_bad(sum[0] | sum[1] | sum[2] | sum[3]); }

}  // namespace pi
