// pi_paged.h -- host-side launch descriptors of the paged key/value cache's operators, shared by the
// C ABI and the kernel files.
#pragma once

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "pi_common.cuh"

namespace pi {

constexpr int kStatusIndex = -8;  // a device-side index out of range (PI_ERR_INDEX)

// What the pages of a paged cache hold (pi_kv_type_t).
constexpr int kKvBf16 = 0, kKvE4m3 = 1, kKvInt8 = 2;

// A paged key/value cache and the width of its users' page tables; sizes are checked on the host
// (page a power of two, d 64 or 128, n_pages * Hkv * page < 2^31 rows).
struct PagedCache {
    void *k, *v;                 // [n_pages, Hkv, page, d] bf16 or 8-bit codes
    uint8_t *k_scale, *v_scale;  // [n_pages, Hkv, page, d / 32], 8 bits only
    int kv_type, n_pages, Hkv, page, page_log2, d, d_log2;
    int width;                   // page-table entries per sequence
};

// A packed batch: sequence b has the tokens cu[b] .. cu[b+1]-1 of T, at positions ctx[b] ...
struct PagedBatch {
    const int *table;  // [B, width]
    const int *cu;     // [B + 1]
    const int *ctx;    // [B]
    int B, T;
};

struct AppendArgs {
    const __nv_bfloat16 *k, *v;     // [T, Hkv, d], tokens k_stride and v_stride elements apart
    long long k_stride, v_stride;
    PagedCache cache;
    PagedBatch batch;
    int *index_word;
    int chunks;  // warps per token, set at the launch
};

// Warps of a token in append and read, of 256 elements each or more, and whether a launch holds those of T tokens.
inline bool rows_fit(const PagedCache &c, long long T) { return T * ((c.Hkv * (long long)c.d + 255) / 256) <= 0x7fffffffLL; }

struct ReadArgs {
    __nv_bfloat16 *k, *v;  // [T, Hkv, d]
    PagedCache cache;
    PagedBatch batch;
    int *index_word;
    int chunks;
};

struct ExtendArgs {
    const __nv_bfloat16 *q;  // [T, H, d], tokens q_stride elements apart
    long long q_stride;
    const float *alpha;      // [T, H] or null (ECP)
    __nv_bfloat16 *out;      // [T, H, d]
    float *lse;              // [T, H]
    Shape s;                 // H, Hkv, d, k_local, period, S, mode, scale_log2
    PagedCache cache;
    PagedBatch batch;
    int *workspace;          // extend_workspace()
    int *status, *index_word;
    uint64_t timeout_ns;
};

struct DecodePagedArgs {
    const __nv_bfloat16 *q;  // [B, H, d], sequences q_stride elements apart
    long long q_stride;
    const float *alpha;      // [B, H] or null (ECP)
    const int *table;        // [B, width]
    const int *lens;         // [B] rows of the cache, the new token's among them
    __nv_bfloat16 *out;      // [B, H, d]
    float *lse;              // [B, H]
    Shape s;
    PagedCache cache;
    int *index_word;
};

// Query heads of a KV group in one 128-row block of the chunk attention: the largest of 4, 2, 1 that divides the group.
inline int packed_heads(int G) { return G % 4 == 0 ? 4 : G % 2 == 0 ? 2 : 1; }

// rows into and out of a paged cache (pi_cache.cu)
cudaError_t launch_append(const AppendArgs &a, cudaStream_t st);
cudaError_t launch_cache_read(const ReadArgs &a, cudaStream_t st);

// attention over a paged cache: a chunk of new tokens per sequence (pi_extend_tc.cu), one new token per
// sequence (pi_decode_paged.cu)
// the workspace of a call; false where its kernels cannot number the rows, blocks or tiles of its sizes
bool extend_workspace(const ExtendArgs &a, size_t &bytes);
cudaError_t launch_extend(const ExtendArgs &a, cudaStream_t st);
// the same for few tokens per sequence (pi_decode_paged.cu), and whether a call is one of those
cudaError_t launch_extend_few(const ExtendArgs &a, cudaStream_t st);
bool extend_few_rows(const ExtendArgs &a);
cudaError_t launch_decode_paged(const DecodePagedArgs &a, cudaStream_t st);

// Device words of the current device, looked up once per device (api.cu): the status word of the
// bounded waits, and the one that out-of-range indexes are recorded in.  Null on a CUDA error.
int *status_word();
int *index_word();

// Streaming multiprocessors of the current device (1 on a CUDA error).
inline int sm_count() {
    constexpr int kMaxDev = 64;
    static std::atomic<int> cache[kMaxDev];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return 1;
    n = cache[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 1;
        cache[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

}  // namespace pi
