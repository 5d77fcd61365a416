// pi_cache.cu -- writing new rows into the paged key/value cache, quantised where it holds 8 bits,
// and reading rows back.
//
// Both move each element once: a new row's 2 d bytes are read and 2 d (bf16) or d + d/32 (8 bits)
// written, or the other way round, so HBM bandwidth bounds long calls and the chain of dependent
// loads (sequence, page, row) the short ones.
//
// A warp takes a packed token (long reads: four neighbouring ones): its lanes take the token's Hkv * d elements K and V
// together, 8 at a time, or 16 where they are quantised, so that a block of 32 elements lies in two neighbouring lanes and
// its largest magnitude takes one shuffle.  The tokens' sequence is searched by the whole warp (two rounds of probes for up
// to 1024 sequences) while their elements are in flight.
#include "pi_mma.cuh"
#include "pi_paged.cuh"
#include "pi_quant.cuh"

namespace pi {
namespace cache {

constexpr int WARPS = 8;
constexpr unsigned kFull = 0xffffffffu;

// A lane's share of a row: 16 elements, or 8 that stay bf16.
template <int KV>
struct Piece {
    static constexpr int N = KV == kKvBf16 ? 1 : 2;  // 16-byte pieces of bf16
    static constexpr int E = 8 * N;
    uint4 x[N];
};

// Largest magnitude of the 32 elements that this lane and the next hold.
__device__ __forceinline__ float absmax32(const Piece<kKvE4m3> &p) {
    // bf16 magnitudes compare like their bits; infinities and NaN come out at 0x7f80 or above
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t w[4] = {p.x[i].x, p.x[i].y, p.x[i].z, p.x[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) m = __vmaxu2(m, w[j] & 0x7fff7fffu);
    }
    m = max(m >> 16, m & 0xffffu);
    m = max(m, __shfl_xor_sync(kFull, m, 1));
    return __uint_as_float(m << 16);
}

// Eight elements to eight codes, given the block's scale exponent.
template <int KV>
__device__ __forceinline__ uint2 encode8(const uint4 &x, int e) {
    float y[8];
    unpack8(x, y);
    return encode_codes<KV>(y, e);
}

// A piece into the cache (`in`: this lane has one; the others of the warp take part in the block maxima only).
template <int KV>
__device__ __forceinline__ void put(const PagedCache &c, void *pages, uint8_t *scales, const Piece<KV> &p, long long row, int col,
                                    bool in) {
    if constexpr (KV == kKvBf16) {
        if (in) *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(pages) + row * c.d + col) = p.x[0];
    } else {
        const float amax = absmax32(reinterpret_cast<const Piece<kKvE4m3> &>(p));
        const bool finite = __float_as_uint(amax) < 0x7f800000u;
        const int e = finite ? scale_exp<KV>(amax) : 0;
        const uint2 lo = encode8<KV>(p.x[0], e), hi = encode8<KV>(p.x[1], e);
        if (!in) return;
        *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(pages) + row * c.d + col) =
            finite ? make_uint4(lo.x, lo.y, hi.x, hi.y) : make_uint4(0u, 0u, 0u, 0u);
        if ((col & (kScaleBlock - 1)) == 0)
            scales[row * (c.d / kScaleBlock) + col / kScaleBlock] = (uint8_t)(finite ? e + 127 : kScaleNan);
    }
}

// Position and page of packed tokens t .. t + TOK - 1, in lanes 0 .. TOK - 1 (page -1: the token has no row).
template <int TOK>
__device__ __forceinline__ void locate_run(const PagedCache &c, const PagedBatch &bt, int t, int &pos, int &pg, int *index_word) {
    const int lane = threadIdx.x & 31;
    int b;
    pos = locate(c, bt, t, b, index_word);
    const bool first = pos >= 0;
    const int end = first ? ld_now(bt.cu + b + 1) : t + 1;  // tokens of the first one's sequence end here
    if (lane > 0) pos = first && lane < TOK && t + lane < end ? pos + lane : -1;
    int seq = b;
#pragma unroll 1
    for (int i = max(1, end - t); i < TOK && t + i < bt.T; ++i) {  // the others: searched one by one
        const int p = locate(c, bt, t + i, b, index_word);
        if (lane == i) {
            pos = p;
            seq = b;
        }
    }
    pg = -1;
    if (lane < TOK && pos >= 0) {
        pg = page_of(c, bt.table, seq, pos);
        if (pg < 0) record_index(index_word);
    }
}

// The warp's token (or run of tokens) and its 32 pieces of it; a token's warps are neighbours.
template <typename A>
__device__ __forceinline__ int token_of(const A &a, int &chunk) {
    const unsigned w = blockIdx.x * WARPS + (threadIdx.x >> 5), t = w / (unsigned)a.chunks;
    chunk = (int)(w - t * (unsigned)a.chunks);
    return (int)t;
}

template <int KV>
__global__ void __launch_bounds__(WARPS * 32) append_kernel(const AppendArgs a) {
    int chunk;
    const int t = token_of(a, chunk), lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (t >= a.batch.T) return;
    const PagedCache &c = a.cache;
    constexpr int E = Piece<KV>::E, N = Piece<KV>::N;
    const int n = (c.Hkv << c.d_log2) / E;  // pieces of a token: an even number
    const int j = chunk * 32 + lane, col = j * E & (c.d - 1), head = j * E >> c.d_log2;
    const uint4 *pk = reinterpret_cast<const uint4 *>(a.k + (long long)t * a.k_stride) + j * N;
    const uint4 *pv = reinterpret_cast<const uint4 *>(a.v + (long long)t * a.v_stride) + j * N;
    Piece<KV> k, v;
#pragma unroll
    for (int x = 0; x < N; ++x) {
        k.x[x] = j < n ? ld_now(pk + x) : make_uint4(0u, 0u, 0u, 0u);
        v.x[x] = j < n ? ld_now(pv + x) : make_uint4(0u, 0u, 0u, 0u);
    }
    int pos, pg;
    locate_run<1>(c, a.batch, t, pos, pg, a.index_word);
    pos = __shfl_sync(kFull, pos, 0);
    pg = __shfl_sync(kFull, pg, 0);
    const long long row = row_in_page(c, pg, head, pos);
    put<KV>(c, c.k, c.k_scale, k, row, col, j < n && pg >= 0);
    put<KV>(c, c.v, c.v_scale, v, row, col, j < n && pg >= 0);
}

template <int KV, int TOK>
__global__ void __launch_bounds__(WARPS * 32) read_kernel(const ReadArgs a) {
    int chunk;
    const int t = token_of(a, chunk) * TOK, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (t >= a.batch.T) return;
    const PagedCache &c = a.cache;
    const int n = c.Hkv << (c.d_log2 - 3);  // groups of eight elements
    int pos, pg;
    locate_run<TOK>(c, a.batch, t, pos, pg, a.index_word);
    const int j = chunk * 32 + lane, col = j * 8 & (c.d - 1), head = j >> (c.d_log2 - 3);
#pragma unroll 2
    for (int i = 0; i < TOK; ++i) {
        const int p = __shfl_sync(kFull, pos, i), g = __shfl_sync(kFull, pg, i);
        if (g < 0 || j >= n) continue;
        const long long row = row_in_page(c, g, head, p), at = (long long)(t + i) * n + j;
        const uint4 k = get8<KV>(c, c.k, c.k_scale, row, col), v = get8<KV>(c, c.v, c.v_scale, row, col);
        reinterpret_cast<uint4 *>(a.k)[at] = k;
        reinterpret_cast<uint4 *>(a.v)[at] = v;
    }
}

template <typename K, typename A>
static cudaError_t launch(K kernel, int tokens, int piece, A a, cudaStream_t st) {
    a.chunks = (a.cache.Hkv * a.cache.d / piece + 31) / 32;
    const long long warps = ((long long)a.batch.T + tokens - 1) / tokens * a.chunks;  // (fits: rows_fit)
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((warps + WARPS - 1) / WARPS), 1, 1);
    cfg.blockDim = dim3(WARPS * 32, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];  // it may start while the kernel before it on the stream ends (and waits for it)
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace cache

cudaError_t launch_append(const AppendArgs &a, cudaStream_t st) {
    using namespace cache;
    // a token per warp (65536 tokens of 4 heads, d = 128, int8: 32.9 us; two per warp 34.3, four 39.9)
    switch (a.cache.kv_type) {
        case kKvBf16: return launch(append_kernel<kKvBf16>, 1, 8, a, st);
        case kKvE4m3: return launch(append_kernel<kKvE4m3>, 1, 16, a, st);
        default: return launch(append_kernel<kKvInt8>, 1, 16, a, st);
    }
}

cudaError_t launch_cache_read(const ReadArgs &a, cudaStream_t st) {
    using namespace cache;
    // four tokens per warp, two of them in flight, once that leaves the SMs full of warps (65536 tokens of 4 e4m3 heads, d = 128:
    // 35.0 us; one token per warp 38.6, two 35.9, eight 36.4; a tenth as many of 16 int8 heads, d = 64: one 7.2, four 8.4)
    const bool run = (long long)a.batch.T * a.cache.Hkv * a.cache.d >= (128LL << 10) * sm_count();
    switch (a.cache.kv_type) {
        case kKvBf16: return run ? launch(read_kernel<kKvBf16, 4>, 4, 8, a, st) : launch(read_kernel<kKvBf16, 1>, 1, 8, a, st);
        case kKvE4m3: return run ? launch(read_kernel<kKvE4m3, 4>, 4, 8, a, st) : launch(read_kernel<kKvE4m3, 1>, 1, 8, a, st);
        default: return run ? launch(read_kernel<kKvInt8, 4>, 4, 8, a, st) : launch(read_kernel<kKvInt8, 1>, 1, 8, a, st);
    }
}

}  // namespace pi
