// api_paged.cu -- the C ABI of the paged key/value cache (include/pi_attn.h): validation of every
// argument the host can see, then one launch on the caller's stream.  What only the device can see
// (page-table entries, offsets, lengths) is checked by the kernels, which record PI_ERR_INDEX and leave
// the work concerned out.
#include <cstdint>

#include "api_checks.h"
#include "pi_attn.h"
#include "pi_paged.h"

using namespace pi::api;

extern "C" {

int pi_attn_cache_append(const void *k, const void *v, long long k_stride, long long v_stride,
                         const pi_attn_cache_t *cache, const pi_attn_batch_t *batch, void *stream) {
    if (!k || !v || !batch) return PI_ERR_NULL;
    pi::AppendArgs a{};
    int rc = make_cache(cache, batch->width, a.cache);
    if (rc == PI_OK) rc = make_batch(batch, a.batch);
    if (rc == PI_OK) rc = check_stride(k_stride, cache->Hkv, cache->d);
    if (rc == PI_OK) rc = check_stride(v_stride, cache->Hkv, cache->d);
    if (rc != PI_OK) return rc;
    if (!pi::rows_fit(a.cache, batch->T)) return PI_ERR_UNSUPPORTED;
    if (!aligned(k, 16) || !aligned(v, 16)) return PI_ERR_ALIGN;
    a.k = static_cast<const __nv_bfloat16 *>(k);
    a.v = static_cast<const __nv_bfloat16 *>(v);
    a.k_stride = k_stride; a.v_stride = v_stride;
    if (!(a.index_word = pi::index_word())) return PI_ERR_CUDA;
    return map_cuda(pi::launch_append(a, static_cast<cudaStream_t>(stream)));
}

int pi_attn_cache_read(const pi_attn_cache_t *cache, const pi_attn_batch_t *batch, void *k, void *v, void *stream) {
    if (!k || !v || !batch) return PI_ERR_NULL;
    pi::ReadArgs a{};
    int rc = make_cache(cache, batch->width, a.cache);
    if (rc == PI_OK) rc = make_batch(batch, a.batch);
    if (rc != PI_OK) return rc;
    if (!pi::rows_fit(a.cache, batch->T)) return PI_ERR_UNSUPPORTED;
    if (!aligned(k, 16) || !aligned(v, 16)) return PI_ERR_ALIGN;
    a.k = static_cast<__nv_bfloat16 *>(k);
    a.v = static_cast<__nv_bfloat16 *>(v);
    if (!(a.index_word = pi::index_word())) return PI_ERR_CUDA;
    return map_cuda(pi::launch_cache_read(a, static_cast<cudaStream_t>(stream)));
}

size_t pi_attn_extend_workspace_size(const pi_attn_cache_t *cache, int B, int T, int width, int H, int k_local, int period, int S,
                                     int mode) {
    static const float some_alpha = 0.f;
    pi::ExtendArgs a{};
    if (B <= 0 || T <= 0 || B > kMaxSequences || make_cache(cache, width, a.cache) != PI_OK ||
        make_attention(a.cache, H, k_local, period, S, mode, &some_alpha, a.s) != PI_OK)
        return 0;
    a.batch.B = B;
    a.batch.T = T;
    size_t bytes;
    return pi::extend_workspace(a, bytes) ? bytes : 0;
}

int pi_attn_extend(const void *q, long long q_stride, const pi_attn_cache_t *cache, const pi_attn_batch_t *batch,
                   const float *alpha, int H, int k_local, int period, int S, int mode, void *out, float *lse,
                   void *workspace, size_t workspace_bytes, void *stream) {
    if (!q || !batch || !out || !lse) return PI_ERR_NULL;
    pi::ExtendArgs a{};
    int rc = make_cache(cache, batch->width, a.cache);
    if (rc == PI_OK) rc = make_batch(batch, a.batch);
    if (rc == PI_OK) rc = make_attention(a.cache, H, k_local, period, S, mode, alpha, a.s);
    if (rc == PI_OK) rc = check_stride(q_stride, H, cache->d);
    if (rc != PI_OK) return rc;
    size_t need;
    if (!pi::extend_workspace(a, need)) return PI_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || (alpha && !aligned(alpha, 4))) return PI_ERR_ALIGN;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.q_stride = q_stride;
    a.alpha = mode != PI_MODE_ECP ? alpha : nullptr;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse;
    if (need > 0 && (!workspace || workspace_bytes < need)) return PI_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return PI_ERR_ALIGN;
    a.workspace = static_cast<int *>(workspace);
    a.timeout_ns = kWaitTimeoutNs;
    if (!(a.status = pi::status_word()) || !(a.index_word = pi::index_word())) return PI_ERR_CUDA;
    return map_cuda(pi::launch_extend(a, static_cast<cudaStream_t>(stream)));
}

int pi_attn_decode_paged(const void *q, long long q_stride, const pi_attn_cache_t *cache, const int *table, const int *lens,
                         int B, int width, const float *alpha, int H, int k_local, int period, int S, int mode, void *out,
                         float *lse, void *stream) {
    if (!q || !table || !lens || !out || !lse) return PI_ERR_NULL;
    pi::DecodePagedArgs a{};
    int rc = make_cache(cache, width, a.cache);
    if (rc == PI_OK) rc = make_attention(a.cache, H, k_local, period, S, mode, alpha, a.s);
    if (rc != PI_OK) return rc;
    if (B <= 0) return PI_ERR_SHAPE;
    if (H / cache->Hkv > 16 || B > 65535) return PI_ERR_UNSUPPORTED;
    rc = check_stride(q_stride, H, cache->d);
    if (rc != PI_OK) return rc;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || (alpha && !aligned(alpha, 4)) || !aligned(table, 4) ||
        !aligned(lens, 4))
        return PI_ERR_ALIGN;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.q_stride = q_stride;
    a.alpha = mode != PI_MODE_ECP ? alpha : nullptr;
    a.table = table;
    a.lens = lens;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse;
    a.s.B = B;
    if (!(a.index_word = pi::index_word())) return PI_ERR_CUDA;
    return map_cuda(pi::launch_decode_paged(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
