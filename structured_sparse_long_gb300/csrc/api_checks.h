// api_checks.h -- checks of the arguments that the paged cache's entry points share, and the kernels' descriptors made of them.
#pragma once

#include <cstdint>

#include "pi_attn.h"
#include "pi_paged.h"

namespace pi {
namespace api {

constexpr int kMaxSequences = 1 << 30;              // what the search of a token's sequence numbers in an int
constexpr uint64_t kWaitTimeoutNs = 2000000000ull;  // bound on every device-side wait

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int ilog2(int x) {
    int l = 0;
    while ((1 << l) < x) ++l;
    return l;
}

inline int make_cache(const pi_attn_cache_t *c, int width, pi::PagedCache &out) {
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

inline int make_batch(const pi_attn_batch_t *b, pi::PagedBatch &out) {
    if (!b->table || !b->cu || !b->ctx) return PI_ERR_NULL;
    if (b->B <= 0 || b->T <= 0) return PI_ERR_SHAPE;
    if (b->B > kMaxSequences) return PI_ERR_UNSUPPORTED;
    if (!aligned(b->table, 4) || !aligned(b->cu, 4) || !aligned(b->ctx, 4)) return PI_ERR_ALIGN;
    out.table = b->table; out.cu = b->cu; out.ctx = b->ctx; out.B = b->B; out.T = b->T;
    return PI_OK;
}

// A token's rows lie `heads * d` elements one after the other; tokens are `stride` elements apart.
inline int check_stride(long long stride, int heads, int d) {
    if (stride < (long long)heads * d || stride >= (1LL << 38) || stride % 8) return PI_ERR_SHAPE;
    return PI_OK;
}

inline int make_attention(const pi::PagedCache &c, int H, int k_local, int period, int S, int mode, const float *alpha, pi::Shape &s) {
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

inline int map_cuda(cudaError_t e) { return e == cudaSuccess ? PI_OK : PI_ERR_CUDA; }


}  // namespace api
}  // namespace pi
