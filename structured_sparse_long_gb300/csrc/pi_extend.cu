// pi_extend.cu -- pi-Attention / ECP attention of new tokens over a paged key/value cache, on CUDA
// cores: one warp per (token, head).  Lane j of a 32-key chunk scores key j; the warp keeps one online
// softmax and every lane d / 32 output columns.
#include "pi_paged.cuh"

namespace pi {
namespace ext {

constexpr int WARPS = 4;
constexpr unsigned kFull = 0xffffffffu;

struct Row {
    int b, pos;  // sequence and position of the query
};

template <int D, int KV>
__device__ __forceinline__ void attend(const PagedCache &c, const Shape &s, const int *table, const __nv_bfloat16 *q, float al,
                                       bool has_alpha, int b, int i, int g, __nv_bfloat16 *out, float *lse, int *index_word) {
    const int lane = threadIdx.x & 31;
    constexpr int RC = D / 32;
    float o[RC], m = -INFINITY, l = 0.f;
    for (int r = 0; r < RC; ++r) o[r] = 0.f;
    const float off_b = has_alpha ? log2f(al) : 0.f, off_s = log2f(1.f - al);
    auto chunk = [&](int j, bool valid, float off) {
        float z = -INFINITY;
        int pg = valid ? page_of(c, table, b, j) : 0;
        if (pg < 0) {
            record_index(index_word);
            valid = false;
        }
        const long long row = valid ? row_in_page(c, pg, g, j) : 0;
        if (valid) {
            float acc = 0.f;
            for (int x = 0; x < D; x += 8) {
                const uint4 u = get8<KV>(c, c.k, c.k_scale, row, x);
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
                float t[8];
                load8(q + x, t);
                for (int e = 0; e < 4; ++e) {
                    acc = fmaf(t[2 * e], __uint_as_float(w[e] << 16), acc);
                    acc = fmaf(t[2 * e + 1], __uint_as_float(w[e] & 0xffff0000u), acc);
                }
            }
            z = fmaf(acc, s.scale_log2, off);
        }
        float mx = z;
        for (int w = 16; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, w));
        const float mn = fmaxf(m, mx);
        if (mn == -INFINITY) return;
        const float corr = exp2f(m - mn), p = exp2f(z - mn);
        float ps = p;
        for (int w = 16; w; w >>= 1) ps += __shfl_xor_sync(kFull, ps, w);
        l = l * corr + ps;
        m = mn;
        for (int r = 0; r < RC; ++r) o[r] *= corr;
        for (int k = 0; k < 32; ++k) {
            const float pk = __shfl_sync(kFull, p, k);
            const long long rk = __shfl_sync(kFull, row, k);
            if (pk == 0.f) continue;
            for (int r = 0; r < RC; ++r) {
                const int col = lane + 32 * r;
                float x;
                if (KV == kKvBf16) x = __bfloat162float(static_cast<const __nv_bfloat16 *>(c.v)[rk * D + col]);
                else {
                    const uint8_t code = static_cast<const uint8_t *>(c.v)[rk * D + col];
                    const float sc = scale_of(c.v_scale[rk * RC + r]);
                    x = KV == kKvInt8 ? (float)(int8_t)code * sc
                                      : __half2float(__half(__nv_cvt_fp8_to_halfraw(code, __NV_E4M3))) * sc;
                }
                o[r] = fmaf(pk, x, o[r]);
            }
        }
    };
    if (i >= 0) {
        const int lo = band_lo(i, s.mode, s.k_local);
        for (int j0 = lo; j0 <= i; j0 += 32) chunk(j0 + lane, j0 + lane <= i, off_b);
        if (s.mode != kModeEcp)
            for (int m0 = 1; m0 <= s.S; m0 += 32) {
                const long long back = (long long)(m0 + lane) * s.period;
                const bool valid = m0 + lane <= s.S && back > s.k_local && back <= i;
                chunk(valid ? i - (int)back : 0, valid, off_s);
            }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    for (int r = 0; r < RC; ++r) out[lane + 32 * r] = __float2bfloat16_rn(o[r] * inv);
    if (lane == 0) *lse = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

template <int D, int KV>
__global__ void __launch_bounds__(WARPS * 32) extend_kernel(const ExtendArgs a) {
    const long long w = (long long)blockIdx.x * WARPS + (threadIdx.x >> 5);
    if (w >= (long long)a.batch.T * a.s.H) return;
    const int t = (int)(w / a.s.H), h = (int)(w % a.s.H);
    int b;
    const int pos = locate(a.cache, a.batch, t, b, a.index_word);
    if (pos < 0) return;
    attend<D, KV>(a.cache, a.s, a.batch.table, a.q + t * a.q_stride + h * D, a.alpha ? a.alpha[w] : 1.f, a.alpha != nullptr, b,
                  pos, h / (a.s.H / a.s.Hkv), a.out + w * D, a.lse + w, a.index_word);
}

template <int D, int KV>
__global__ void __launch_bounds__(WARPS * 32) decode_kernel(const DecodePagedArgs a) {
    const int w = blockIdx.x * WARPS + (threadIdx.x >> 5);
    if (w >= a.s.B * a.s.H) return;
    const int b = w / a.s.H, h = w % a.s.H;
    int n = a.lens[b];
    if (n < 0 || n > (long long)a.cache.width << a.cache.page_log2) {
        record_index(a.index_word);
        n = 0;
    }
    attend<D, KV>(a.cache, a.s, a.table, a.q + b * a.q_stride + h * D, a.alpha ? a.alpha[w] : 1.f, a.alpha != nullptr, b, n - 1,
                  h / (a.s.H / a.s.Hkv), a.out + (long long)w * D, a.lse + w, a.index_word);
}

}  // namespace ext

cudaError_t launch_extend(const ExtendArgs &a, cudaStream_t st) {
    using namespace ext;
    const long long n = (long long)a.batch.T * a.s.H;
    const unsigned grid = (unsigned)((n + WARPS - 1) / WARPS);
#define PI_GO(D, KV) \
    if (a.s.d == D && a.cache.kv_type == KV) extend_kernel<D, KV><<<grid, WARPS * 32, 0, st>>>(a);
    PI_GO(64, 0) PI_GO(64, 1) PI_GO(64, 2) PI_GO(128, 0) PI_GO(128, 1) PI_GO(128, 2)
#undef PI_GO
    return cudaGetLastError();
}

cudaError_t launch_decode_paged(const DecodePagedArgs &a, cudaStream_t st) {
    using namespace ext;
    const unsigned grid = (unsigned)((a.s.B * a.s.H + WARPS - 1) / WARPS);
#define PI_GO(D, KV) \
    if (a.s.d == D && a.cache.kv_type == KV) decode_kernel<D, KV><<<grid, WARPS * 32, 0, st>>>(a);
    PI_GO(64, 0) PI_GO(64, 1) PI_GO(64, 2) PI_GO(128, 0) PI_GO(128, 1) PI_GO(128, 2)
#undef PI_GO
    return cudaGetLastError();
}

}  // namespace pi
