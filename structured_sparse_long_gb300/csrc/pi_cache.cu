// pi_cache.cu -- writing new rows into the paged key/value cache, quantised where it holds 8 bits,
// and reading rows back.
//
// Both move each element once: a new row's 2 d bytes are read and 2 d (bf16) or d + d/32 (8 bits)
// written, or the other way round, so HBM bandwidth bounds long calls and the chain of dependent
// loads (sequence, page, row) the short ones.
//
// One warp per packed token: its lanes take the token's Hkv * d elements eight at a time (16 bytes
// of bf16), K and V together, so that a block of 32 elements lies in four neighbouring lanes and
// its largest magnitude takes two shuffles.  The token's sequence is searched by the whole warp
// (two rounds of probes for up to 1024 sequences) while its first elements are in flight.
#include "pi_paged.cuh"

namespace pi {
namespace cache {

constexpr int WARPS = 8;
constexpr int PRE = 2;  // element groups per lane and tensor in flight before the row is known

__device__ __forceinline__ float absmax8(const uint4 &x) {
    // bf16 magnitudes compare like their bits; infinities and NaN come out at 0x7f80 or above
    uint32_t m = 0;
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    m = max(m >> 16, m & 0xffffu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    return __uint_as_float(m << 16);
}

// Eight elements to eight codes, given the block's scale exponent.
template <int KV>
__device__ __forceinline__ uint2 encode8(const uint4 &x, int e) {
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);  // 2^-e, -e in [-122, 120]
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t o[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float y[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            y[2 * j] = __uint_as_float(w[2 * i + j] << 16) * inv;
            y[2 * j + 1] = __uint_as_float(w[2 * i + j] & 0xffff0000u) * inv;
        }
        if (KV == kKvE4m3) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2], y[3]), __NV_SATFINITE, __NV_E4M3);
            o[i] = lo | hi << 16;
        } else {
            o[i] = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i] |= ((uint32_t)__float2int_rn(y[j]) & 0xffu) << (8 * j);
        }
    }
    return make_uint2(o[0], o[1]);
}

// Eight elements of a row into the cache (`in`: this lane has some; the others of the warp take part
// in the block maxima only).
template <int KV>
__device__ __forceinline__ void put8(const PagedCache &c, void *pages, uint8_t *scales, const uint4 &x, long long row, int col,
                                     bool in) {
    if (KV == kKvBf16) {
        if (in) *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(pages) + row * c.d + col) = x;
        return;
    }
    const float amax = absmax8(x);
    const bool finite = __float_as_uint(amax) < 0x7f800000u;
    const int e = finite ? scale_exp<KV>(amax) : 0;
    const uint2 codes = finite ? encode8<KV>(x, e) : make_uint2(0u, 0u);
    if (!in) return;
    *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(pages) + row * c.d + col) = codes;
    if ((col & (kScaleBlock - 1)) == 0)
        scales[row * (c.d / kScaleBlock) + col / kScaleBlock] = (uint8_t)(finite ? e + 127 : kScaleNan);
}

template <int KV>
__global__ void __launch_bounds__(WARPS * 32) append_kernel(const AppendArgs a) {
    const int t = blockIdx.x * WARPS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (t >= a.batch.T) return;
    const PagedCache &c = a.cache;
    const int n = c.Hkv << (c.d_log2 - 3);  // groups of eight elements: a multiple of 8
    const uint4 *pk = reinterpret_cast<const uint4 *>(a.k + (long long)t * a.k_stride);
    const uint4 *pv = reinterpret_cast<const uint4 *>(a.v + (long long)t * a.v_stride);
    uint4 xk[PRE], xv[PRE];
    auto load = [&](int g0) {
#pragma unroll
        for (int u = 0; u < PRE; ++u) {
            const int j = g0 + lane + 32 * u;
            xk[u] = j < n ? __ldg(pk + j) : make_uint4(0u, 0u, 0u, 0u);
            xv[u] = j < n ? __ldg(pv + j) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    load(0);
    int b;
    const int pos = locate(c, a.batch, t, b, a.index_word);
    if (pos < 0) return;
    const int pg = page_of(c, a.batch.table, b, pos);
    if (pg < 0) {
        record_index(a.index_word);
        return;
    }
    for (int g0 = 0;;) {
#pragma unroll
        for (int u = 0; u < PRE; ++u) {
            const int j = g0 + lane + 32 * u, col = j * 8 & (c.d - 1), head = j >> (c.d_log2 - 3);
            const long long row = row_in_page(c, pg, head, pos);
            put8<KV>(c, c.k, c.k_scale, xk[u], row, col, j < n);
            put8<KV>(c, c.v, c.v_scale, xv[u], row, col, j < n);
        }
        g0 += 32 * PRE;
        if (g0 >= n) break;
        load(g0);
    }
}

template <int KV>
__global__ void __launch_bounds__(WARPS * 32) read_kernel(const ReadArgs a) {
    const int t = blockIdx.x * WARPS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (t >= a.batch.T) return;
    const PagedCache &c = a.cache;
    const int n = c.Hkv << (c.d_log2 - 3);
    int b;
    const int pos = locate(c, a.batch, t, b, a.index_word);
    if (pos < 0) return;
    const int pg = page_of(c, a.batch.table, b, pos);
    if (pg < 0) {
        record_index(a.index_word);
        return;
    }
    uint4 *ok = reinterpret_cast<uint4 *>(a.k) + (long long)t * n, *ov = reinterpret_cast<uint4 *>(a.v) + (long long)t * n;
    for (int g0 = 0; g0 < n; g0 += 32 * PRE) {
        uint4 xk[PRE], xv[PRE];
#pragma unroll
        for (int u = 0; u < PRE; ++u) {
            const int j = g0 + lane + 32 * u, col = j * 8 & (c.d - 1), head = j >> (c.d_log2 - 3);
            if (j >= n) continue;
            const long long row = row_in_page(c, pg, head, pos);
            xk[u] = get8<KV>(c, c.k, c.k_scale, row, col);
            xv[u] = get8<KV>(c, c.v, c.v_scale, row, col);
        }
#pragma unroll
        for (int u = 0; u < PRE; ++u) {
            const int j = g0 + lane + 32 * u;
            if (j >= n) continue;
            ok[j] = xk[u];
            ov[j] = xv[u];
        }
    }
}

}  // namespace cache

cudaError_t launch_append(const AppendArgs &a, cudaStream_t st) {
    using namespace cache;
    const unsigned grid = (unsigned)((a.batch.T + WARPS - 1) / WARPS);
    if (a.cache.kv_type == kKvBf16) append_kernel<kKvBf16><<<grid, WARPS * 32, 0, st>>>(a);
    else if (a.cache.kv_type == kKvE4m3) append_kernel<kKvE4m3><<<grid, WARPS * 32, 0, st>>>(a);
    else append_kernel<kKvInt8><<<grid, WARPS * 32, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_cache_read(const ReadArgs &a, cudaStream_t st) {
    using namespace cache;
    const unsigned grid = (unsigned)((a.batch.T + WARPS - 1) / WARPS);
    if (a.cache.kv_type == kKvBf16) read_kernel<kKvBf16><<<grid, WARPS * 32, 0, st>>>(a);
    else if (a.cache.kv_type == kKvE4m3) read_kernel<kKvE4m3><<<grid, WARPS * 32, 0, st>>>(a);
    else read_kernel<kKvInt8><<<grid, WARPS * 32, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace pi
