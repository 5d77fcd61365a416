// pi_keep.cu -- the rows of an accepted path moved together in the paged cache, in all layers at once.
//
// Row path[j] of a sequence's tree goes to row j, in ascending order.  A row's 16-byte pieces are independent of each other, so a thread
// owns one piece (a layer, keys or values, a head, 16 bytes; over 8-bit caches also the row's scale bytes) of all of the
// path's rows and moves them in order: with path[j] ascending a row is overwritten only after it was read, and no
// barrier is needed.  Eight rows are in flight at a time.  The call is bound by the latency of its dependent loads (offsets, path,
// page table, rows) unless hundreds of layers' rows move.
#include "pi_mma.cuh"
#include "pi_paged.cuh"
#include "pi_step.h"

namespace pi {
namespace keep {

constexpr int THREADS = 256;
constexpr int ROWS = 8;  // rows in flight

template <typename T>
__device__ __forceinline__ void move(T *pages, const int2 *rows, int n, long long offset, long long stride) {
    // row r's piece lies at pages[offset + r * stride]
    for (int j0 = 0; j0 < n; j0 += ROWS) {
        T x[ROWS];
#pragma unroll
        for (int j = 0; j < ROWS; ++j)
            if (j0 + j < n && rows[j0 + j].x != rows[j0 + j].y) x[j] = pages[offset + rows[j0 + j].x * stride];
#pragma unroll
        for (int j = 0; j < ROWS; ++j)
            if (j0 + j < n && rows[j0 + j].x != rows[j0 + j].y) pages[offset + rows[j0 + j].y * stride] = x[j];
    }
}

__global__ void __launch_bounds__(THREADS) keep_kernel(const __grid_constant__ KeepArgs a) {
    __shared__ int2 rows[THREADS];  // source and place of the path's rows, for head 0 (both 0: not moved)
    const PagedCache &c = a.cache;
    const int b = blockIdx.x / (unsigned)a.chunks, chunk = blockIdx.x - b * a.chunks, tid = threadIdx.x;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int t0 = ld_now(a.batch.cu + b), t1 = ld_now(a.batch.cu + b + 1), ctx = ld_now(a.batch.ctx + b), n = ld_now(a.count + b);
    bool ok = sequence_ok(c, a.batch, t0, t1, ctx) && n >= 0 && n <= t1 - t0;
    // row j of the path: whether it follows the one before it, and (place) where it lies
    auto look = [&](int j, bool place) -> bool {
        const int x = ld_now(a.path + t0 + j), before = j > 0 ? ld_now(a.path + t0 + j - 1) : -1;
        if (x <= before || x >= t1 - t0) return false;
        if (place) {
            int2 r = make_int2(0, 0);
            if (x != j) {
                const int from = page_of(c, a.batch.table, b, ctx + x), to = page_of(c, a.batch.table, b, ctx + j);
                if (from < 0 || to < 0) record_index(a.index_word);
                else r = make_int2(row_in_page(c, from, 0, ctx + x), row_in_page(c, to, 0, ctx + j));
            }
            rows[tid] = r;
        }
        return true;
    };
    for (int j = tid; ok && j < n; j += THREADS) ok = look(j, j < THREADS);
    if (!__syncthreads_and(ok)) {
        if (tid == 0) record_index(a.index_word);
        return;
    }
    const bool quant = c.kv_type != kKvBf16;
    const int row16 = quant ? c.d / 16 : c.d / 8, per_head = row16 + quant, item = chunk * THREADS + tid, per_layer = 2 * c.Hkv * per_head;
    const int layer = item / per_layer, piece = item - layer * per_layer;
    const int col = piece % per_head, head = (piece / per_head) % c.Hkv, val = piece / per_head / c.Hkv;
    const long long first = (long long)head << c.page_log2;
    for (int j0 = 0;;) {
        const int m = min(THREADS, n - j0);
        if (layer < a.layers) {
            if (col < row16) {
                move(static_cast<uint4 *>(val ? a.v[layer] : a.k[layer]), rows, m, first * row16 + col, row16);
            } else if (c.d == 128) {
                move(reinterpret_cast<uint32_t *>(val ? a.v_scale[layer] : a.k_scale[layer]), rows, m, first, 1);
            } else {
                move(reinterpret_cast<uint16_t *>(val ? a.v_scale[layer] : a.k_scale[layer]), rows, m, first, 1);
            }
        }
        j0 += THREADS;
        if (j0 >= n) break;
        __syncthreads();
        if (j0 + tid < n) look(j0 + tid, true);
        __syncthreads();
    }
}

}  // namespace keep

cudaError_t launch_keep(const KeepArgs &args, cudaStream_t st) {
    using namespace keep;
    KeepArgs a = args;
    a.chunks = (int)(((long long)keep_pieces(a.cache) * a.layers + THREADS - 1) / THREADS);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.batch.B * a.chunks), 1, 1);  // (fits: keep_fits)
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];  // it may start while the kernel before it on the stream ends (and waits for it)
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, keep_kernel, a);
}

}  // namespace pi
