// api_paged.cu -- the C ABI of the paged key/value cache (include/pi_attn.h): validation of every
// argument the host can see, then one launch on the caller's stream.  What only the device can see
// (page-table entries, offsets, lengths) is checked by the kernels, which record PI_ERR_INDEX and leave
// the work concerned out.
#include <cstdint>

#include "pi_attn.h"
#include "pi_paged.h"

namespace {

constexpr int kMaxSequences = 1 << 30;              // what the search of a token's sequence numbers in an int
constexpr uint64_t kWaitTimeoutNs = 2000000000ull;  // bound on every device-side wait

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int ilog2(int x) {
    int l = 0;
    while ((1 << l) < x) ++l;
    return l;
}

int make_cache(const pi_attn_cache_t *c, int width, pi::PagedCache &out) {
    if (!c || !c->k || !c->v) return PI_ERR_NULL;
    if (c->kv_type != PI_KV_BF16 && c->kv_type != PI_KV_E4M3 && c->kv_type != PI_KV_INT8) return PI_ERR_UNSUPPORTED;
    const bool quant = c->kv_type != PI_KV_BF16;
    if (quant && (!c->k_scale || !c->v_scale)) return PI_ERR_NULL;
    if (c->n_pages <= 0 || c->Hkv <= 0 || width <= 0) return PI_ERR_SHAPE;
    if (c->Hkv > 65535) return PI_ERR_UNSUPPORTED;
    if (c->d != 64 && c->d != 128) return PI_ERR_UNSUPPORTED;
    if (c->page < 16 || c->page > 256 || (c->page & (c->page - 1))) return PI_ERR_UNSUPPORTED;
    if ((long long)c->n_pages * c->Hkv > 0x7fffffffLL / c->page) return PI_ERR_UNSUPPORTED;
    if ((long long)width * c->page > 0x7fff0000LL) return PI_ERR_UNSUPPORTED;  // positions and a few tiles fit int
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return PI_ERR_ALIGN;
    if (quant && (!aligned(c->k_scale, 16) || !aligned(c->v_scale, 16))) return PI_ERR_ALIGN;
    out.k = c->k; out.v = c->v;
    out.k_scale = static_cast<uint8_t *>(c->k_scale);
    out.v_scale = static_cast<uint8_t *>(c->v_scale);
    out.kv_type = c->kv_type; out.n_pages = c->n_pages; out.Hkv = c->Hkv;
    out.page = c->page; out.page_log2 = ilog2(c->page);
    out.d = c->d; out.d_log2 = ilog2(c->d);
    out.width = width;
    return PI_OK;
}

int make_batch(const pi_attn_batch_t *b, pi::PagedBatch &out) {
    if (!b->table || !b->cu || !b->ctx) return PI_ERR_NULL;
    if (b->B <= 0 || b->T <= 0) return PI_ERR_SHAPE;
    if (b->B > kMaxSequences) return PI_ERR_UNSUPPORTED;
    if (!aligned(b->table, 4) || !aligned(b->cu, 4) || !aligned(b->ctx, 4)) return PI_ERR_ALIGN;
    out.table = b->table; out.cu = b->cu; out.ctx = b->ctx; out.B = b->B; out.T = b->T;
    return PI_OK;
}

// A token's rows lie `heads * d` elements one after the other; tokens are `stride` elements apart.
int check_stride(long long stride, int heads, int d) {
    if (stride < (long long)heads * d || stride >= (1LL << 38) || stride % 8) return PI_ERR_SHAPE;
    return PI_OK;
}

int make_attention(const pi::PagedCache &c, int H, int k_local, int period, int S, int mode, const float *alpha, pi::Shape &s) {
    if (mode != PI_MODE_PI && mode != PI_MODE_ECP) return PI_ERR_UNSUPPORTED;
    if (mode != PI_MODE_ECP && !alpha) return PI_ERR_NULL;
    if (H <= 0 || H % c.Hkv != 0 || k_local < 0 || S < 0) return PI_ERR_SHAPE;
    if (mode != PI_MODE_ECP && S > 0 && period <= 0) return PI_ERR_SHAPE;
    if (mode == PI_MODE_ECP && (k_local <= 0 || S != 0)) return PI_ERR_SHAPE;
    // key lists and tile counts fit int
    const long long positions = (long long)c.width * c.page;
    if (mode != PI_MODE_ECP && S > 0 && std::min<long long>(S, positions / period) > (1LL << 27)) return PI_ERR_UNSUPPORTED;
    s = pi::Shape{};
    s.H = H; s.Hkv = c.Hkv; s.d = c.d;
    s.k_local = k_local; s.period = period; s.S = S; s.mode = mode;
    s.scale_log2 = (float)(1.4426950408889634 / __builtin_sqrt((double)c.d));
    return PI_OK;
}

int map_cuda(cudaError_t e) { return e == cudaSuccess ? PI_OK : PI_ERR_CUDA; }

}  // namespace

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
