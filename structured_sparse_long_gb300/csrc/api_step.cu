// api_step.cu -- the C ABI of rotary positions and of a speculative serving step (include/pi_attn.h): validation of every argument
// that the host can see, then one launch on the caller's stream (pi_attn_cache_keep: one per 64 layers).  Offsets, parents, tokens and page-table
// entries are checked by the kernels.
#include <algorithm>
#include <cstdint>

#include "api_checks.h"
#include "pi_attn.h"
#include "pi_step.h"

using namespace pi::api;

namespace {

int make_rotary(const pi_attn_rotary_t *r, int d, pi::Rotary &out) {
    if (!r || !r->step) return PI_ERR_NULL;
    if (r->rot <= 0 || r->rot > d || r->rot % 16 || !(r->scale - r->scale == 0.f)) return PI_ERR_SHAPE;
    if (!aligned(r->step, 8)) return PI_ERR_ALIGN;
    out = pi::Rotary{r->step, r->rot, r->interleaved != 0, r->scale};
    return PI_OK;
}

// {batch, head, position} strides of a tensor of these sizes; one of a dimension of size 1 is not used.
int check_strides(const long long *s, int B, int heads, int N, int per16, long long least, long long *out) {
    const int size[3] = {B, heads, N};
    for (int i = 0; i < 3; ++i) {
        out[i] = size[i] > 1 ? s[i] : 0;
        if (size[i] > 1 && (s[i] < least || s[i] >= (1LL << 38) || s[i] % per16)) return PI_ERR_SHAPE;
    }
    return PI_OK;
}

int make_tensor(const void *x, const long long *xs, void *y, const long long *ys, int B, int heads, int N, int d, int f32, pi::RotaryTensor &t) {
    if (!x || !xs || !y || !ys) return PI_ERR_NULL;
    long long a[3], b[3];
    int rc = check_strides(xs, B, heads, N, f32 ? 4 : 8, 0, a);
    if (rc == PI_OK) rc = check_strides(ys, B, heads, N, f32 ? 4 : 8, d, b);
    if (rc != PI_OK) return rc;
    for (const long long *s : {a, b})  // offsets in bytes fit 63 bits
        if ((double)s[0] * B + (double)s[1] * heads + (double)s[2] * N >= 0x1p60) return PI_ERR_UNSUPPORTED;
    if (!aligned(x, 16) || !aligned(y, 16)) return PI_ERR_ALIGN;
    if (x == y && (a[0] != b[0] || a[1] != b[1] || a[2] != b[2])) return PI_ERR_SHAPE;
    t = pi::RotaryTensor{x, y, a[0], a[1], a[2], b[0], b[1], b[2], heads};
    return PI_OK;
}

// Whether pages of these caches, each `rows` rows of d elements, lie in the same memory.
bool pages_overlap(const pi::KeepArgs &a) {
    const pi::PagedCache &c = a.cache;
    const bool quant = c.kv_type != pi::kKvBf16;
    const size_t rows = (size_t)c.n_pages * c.Hkv * c.page, bytes = rows * c.d * (quant ? 1 : 2), scales = rows * (c.d / 32);  // (a byte per 32 elements)
    struct Range {
        uintptr_t at;
        size_t bytes;
    } r[4 * pi::kKeepLayers];
    int n = 0;
    for (int i = 0; i < a.layers; ++i) {
        for (const void *p : {a.k[i], a.v[i]}) r[n++] = Range{reinterpret_cast<uintptr_t>(p), bytes};
        if (quant)
            for (const void *p : {a.k_scale[i], a.v_scale[i]}) r[n++] = Range{reinterpret_cast<uintptr_t>(p), scales};
    }
    std::sort(r, r + n, [](const Range &x, const Range &y) { return x.at < y.at; });
    for (int i = 1; i < n; ++i)
        if (r[i].at - r[i - 1].at < r[i - 1].bytes) return true;
    return false;
}

}  // namespace

extern "C" {

int pi_attn_rotary(const void *q, const long long *q_strides, const void *k, const long long *k_strides, const pi_attn_rotary_t *rotary,
                   const int *pos, int start, int B, int H, int Hkv, int N, int d, int f32, int back, void *q_out,
                   const long long *q_out_strides, void *k_out, const long long *k_out_strides, void *stream) {
    pi::RotaryArgs a{};
    if (B <= 0 || H <= 0 || Hkv < 0 || N <= 0 || start < 0) return PI_ERR_SHAPE;
    if (d != 32 && d != 64 && d != 128) return PI_ERR_UNSUPPORTED;
    if (H > 65535 || Hkv > 65535 || (long long)B * N > 0x7fffffffLL || (long long)B * N * ((long long)H + Hkv) * d >= 1LL << 45 ||
        (H + 3) / 4 + (Hkv + 3) / 4 > 65535)
        return PI_ERR_UNSUPPORTED;
    if (!pos && (long long)start + N > 1LL << 31) return PI_ERR_SHAPE;
    int rc = make_rotary(rotary, d, a.r);
    if (rc == PI_OK) rc = make_tensor(q, q_strides, q_out, q_out_strides, B, H, N, d, f32, a.t[0]);
    if (rc == PI_OK && Hkv > 0) rc = make_tensor(k, k_strides, k_out, k_out_strides, B, Hkv, N, d, f32, a.t[1]);
    if (rc != PI_OK) return rc;
    if (!aligned(pos, 4)) return PI_ERR_ALIGN;
    a.pos = pos;
    a.start = start;
    a.B = B; a.N = N; a.d = d;
    a.f32 = f32 != 0;
    a.back = back != 0;
    return map_cuda(pi::launch_rotary(a, static_cast<cudaStream_t>(stream)));
}

int pi_attn_rotary_append(const void *q, long long q_stride, const void *k, long long k_stride, const void *v, long long v_stride,
                          const pi_attn_rotary_t *rotary, const pi_attn_cache_t *cache, const pi_attn_batch_t *batch, const int *parent,
                          int H, void *q_out, long long q_out_stride, void *stream) {
    if (!q || !k || !v || !q_out || !batch) return PI_ERR_NULL;
    pi::RotaryAppendArgs g{};
    int rc = make_cache(cache, batch->width, g.a.cache);
    if (rc == PI_OK) rc = make_batch(batch, g.a.batch);
    if (rc == PI_OK) rc = make_rotary(rotary, cache->d, g.r);
    if (rc != PI_OK) return rc;
    if (H <= 0) return PI_ERR_SHAPE;
    if (H > 65535) return PI_ERR_UNSUPPORTED;
    rc = check_stride(q_stride, H, cache->d);
    if (rc == PI_OK) rc = check_stride(q_out_stride, H, cache->d);
    if (rc == PI_OK) rc = check_stride(k_stride, cache->Hkv, cache->d);
    if (rc == PI_OK) rc = check_stride(v_stride, cache->Hkv, cache->d);
    if (rc != PI_OK) return rc;
    if (q == q_out && q_stride != q_out_stride) return PI_ERR_SHAPE;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(parent, 4)) return PI_ERR_ALIGN;
    g.q = static_cast<const __nv_bfloat16 *>(q);
    g.a.k = static_cast<const __nv_bfloat16 *>(k);
    g.a.v = static_cast<const __nv_bfloat16 *>(v);
    g.q_out = static_cast<__nv_bfloat16 *>(q_out);
    g.q_stride = q_stride; g.q_out_stride = q_out_stride;
    g.a.k_stride = k_stride; g.a.v_stride = v_stride;
    g.parent = parent;
    g.H = H;
    if (!pi::rotary_append_fits(g)) return PI_ERR_UNSUPPORTED;
    if (!(g.a.index_word = pi::index_word())) return PI_ERR_CUDA;
    return map_cuda(pi::launch_rotary_append(g, static_cast<cudaStream_t>(stream)));
}

int pi_attn_extend_tree(const void *q, long long q_stride, const pi_attn_cache_t *cache, const pi_attn_batch_t *batch, const int *parent,
                        const float *alpha, int H, int k_local, int period, int S, int mode, void *out, float *lse, void *stream) {
    if (!q || !batch || !parent || !out || !lse) return PI_ERR_NULL;
    pi::ExtendTreeArgs t{};
    pi::ExtendArgs &a = t.e;
    int rc = make_cache(cache, batch->width, a.cache);
    if (rc == PI_OK) rc = make_batch(batch, a.batch);
    if (rc == PI_OK) rc = make_attention(a.cache, H, k_local, period, S, mode, alpha, a.s);
    if (rc == PI_OK) rc = check_stride(q_stride, H, cache->d);
    if (rc != PI_OK) return rc;
    if ((long long)batch->T * H > 0x7fffffffLL) return PI_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(alpha, 4) || !aligned(parent, 4)) return PI_ERR_ALIGN;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.q_stride = q_stride;
    a.alpha = mode != PI_MODE_ECP ? alpha : nullptr;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse;
    t.parent = parent;
    bool fits;
    t.few = pi::tree_few(t, fits);
    if (!fits) return PI_ERR_UNSUPPORTED;
    a.timeout_ns = kWaitTimeoutNs;
    if (!(a.status = pi::status_word()) || !(a.index_word = pi::index_word())) return PI_ERR_CUDA;
    return map_cuda(pi::launch_extend_tree(t, static_cast<cudaStream_t>(stream)));
}

int pi_attn_verify_tree(const float *target, long long target_stride, const float *draft, long long draft_stride, const int *tokens,
                        const int *cu, const int *parent, const float *u, const float *u_next, int B, int T, int V, int *path,
                        int *count, int *next, void *stream) {
    if (!target || !tokens || !cu || !parent || !u || !u_next || !path || !count || !next) return PI_ERR_NULL;
    if (B <= 0 || T <= 0 || V <= 0) return PI_ERR_SHAPE;
    if (B > 65535 || V > 1 << 30) return PI_ERR_UNSUPPORTED;
    if (target_stride < V || target_stride >= 1LL << 38 || (draft && (draft_stride < V || draft_stride >= 1LL << 38))) return PI_ERR_SHAPE;
    if ((double)T * (double)std::max(target_stride, draft ? draft_stride : 0LL) >= 0x1p60) return PI_ERR_UNSUPPORTED;  // offsets in bytes fit 63 bits
    for (const void *p : {(const void *)target, (const void *)draft, (const void *)tokens, (const void *)cu, (const void *)parent, (const void *)u,
                          (const void *)u_next, (const void *)path, (const void *)count, (const void *)next})
        if (!aligned(p, 4)) return PI_ERR_ALIGN;
    pi::VerifyArgs a{target, draft, target_stride, draft_stride, tokens, cu, parent, u, u_next, B, T, V, path, count, next, nullptr};
    if (!(a.index_word = pi::index_word())) return PI_ERR_CUDA;
    return map_cuda(pi::launch_verify(a, static_cast<cudaStream_t>(stream)));
}

int pi_attn_cache_keep(const pi_attn_cache_t *caches, int n_caches, const pi_attn_batch_t *batch, const int *path, const int *count,
                       void *stream) {
    if (!caches || !batch || !path || !count) return PI_ERR_NULL;
    if (n_caches <= 0) return PI_ERR_SHAPE;
    pi::KeepArgs a{};
    int rc = make_batch(batch, a.batch);
    if (rc != PI_OK) return rc;
    for (int i = 0; i < n_caches; ++i) {
        const pi_attn_cache_t &c = caches[i], &d = caches[0];
        rc = make_cache(&c, batch->width, a.cache);
        if (rc != PI_OK) return rc;
        if (c.kv_type != d.kv_type || c.n_pages != d.n_pages || c.Hkv != d.Hkv || c.page != d.page || c.d != d.d) return PI_ERR_SHAPE;
    }
    if (!pi::keep_fits(a.cache, batch->B, std::min(n_caches, pi::kKeepLayers))) return PI_ERR_UNSUPPORTED;
    if (!aligned(path, 4) || !aligned(count, 4)) return PI_ERR_ALIGN;
    a.path = path;
    a.count = count;
    auto take = [&](int first) {  // a launch's layers
        a.layers = std::min(n_caches - first, pi::kKeepLayers);
        for (int i = 0; i < a.layers; ++i) {
            const pi_attn_cache_t &c = caches[first + i];
            a.k[i] = c.k; a.v[i] = c.v;
            a.k_scale[i] = static_cast<uint8_t *>(c.k_scale);
            a.v_scale[i] = static_cast<uint8_t *>(c.v_scale);
        }
    };
    for (int first = 0; first < n_caches; first += pi::kKeepLayers) {
        take(first);
        if (pages_overlap(a)) return PI_ERR_SHAPE;
    }
    if (!(a.index_word = pi::index_word())) return PI_ERR_CUDA;
    for (int first = 0; first < n_caches; first += pi::kKeepLayers) {
        if (n_caches > pi::kKeepLayers) take(first);
        rc = map_cuda(pi::launch_keep(a, static_cast<cudaStream_t>(stream)));
        if (rc != PI_OK) return rc;
    }
    return PI_OK;
}

int pi_attn_debug_tree_kernel(const pi_attn_cache_t *cache, int B, int T, int width, int H, int k_local, int period, int S, int mode) {
    const int any = 0;
    const float alpha = 0.f;
    const pi_attn_batch_t batch{&any, &any, &any, B, T, width};  // (not read)
    pi::ExtendTreeArgs t{};
    int rc = make_cache(cache, width, t.e.cache);
    if (rc == PI_OK) rc = make_batch(&batch, t.e.batch);
    if (rc == PI_OK) rc = make_attention(t.e.cache, H, k_local, period, S, mode, &alpha, t.e.s);
    if (rc != PI_OK) return rc;
    bool fits = (long long)T * H <= 0x7fffffffLL;
    const bool few = fits && pi::tree_few(t, fits);
    return !fits ? PI_ERR_UNSUPPORTED : few ? 0 : 1;
}

}  // extern "C"
