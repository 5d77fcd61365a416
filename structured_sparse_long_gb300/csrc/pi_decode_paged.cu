// pi_decode_paged.cu -- one decode step of pi-Attention / ECP attention against a paged key/value cache:
// for sequence b with n = lens[b] cached rows and query head h, row n - 1 of the forward.
//
// The neighbour rows of a (sequence, KV head) -- the band, then the skips -- form a key list that is cut
// into tiles of 16 keys.  Every warp of a CTA (and of its cluster, where few sequences leave SMs idle)
// takes tiles of its own and needs nothing from the others until the end:
//   * The tile's rows are looked up by one lane each (a page-table load per key), then all of the
//     tile's K and V bytes are requested at once, straight into registers and straight into the layout
//     of the warp's matrix products, so that no shared memory and no barrier lies between HBM and
//     the arithmetic, and a warp has 8 KB (bf16, d = 128) in flight.
//   * S^T = K Q^T by mma.m16n8k16 (16 keys x 8 heads): the head group's queries are the 8 columns, so
//     grouped heads cost nothing.  A contraction may take its elements in any order as long as both
//     operands agree: lane 4 g + t holds 16 contiguous bytes of key rows g and g + 8, whose elements
//     are its share of the k steps, and the queries are loaded the same way.
//   * The softmax keeps a running maximum and sum per head in 32 bits: a lane holds heads 2t, 2t+1 of keys g,
//     g + 8, so a tile's maximum takes three shuffles per head; the sums stay per lane until the end.
//   * O^T += V^T P^T (16 elements of d x 8 heads): P^T is S^T's accumulator rounded to bf16 (half a step
//     of 2^-7 relative, as in the forward) and transposed by movmatrix; lane 4 g + t holds 16 (8-bit
//     cache: 16 or 8) contiguous bytes of V rows 2t, 2t+1, 2t+8, 2t+9, which two byte permutes per word
//     turn into the pairs of keys that the product wants.
//   * 8-bit codes become bf16 in registers (exact, see pi_paged.cuh).
// The partial states (m, l, o) meet in shared memory, and across a cluster through distributed shared
// memory.  With a few hundred keys per sequence the step is bound by the latency of its dependent
// loads (length, page table, rows) for small batches and by HBM for large ones.
#include "pi_mma.cuh"
#include "pi_paged.cuh"

#include "pi_launch.h"

namespace pi {
namespace decp {

constexpr int MAX_P = 8;   // CTAs per cluster (portable limit)
constexpr int KEYS = 16;   // keys per tile: the rows of S^T
constexpr unsigned kFull = 0xffffffffu;

struct Args {
    DecodePagedArgs a;
    int m_first;
};

// ---- what a lane holds of a tile -------------------------------------------------------------

// K: 16 bytes each of rows g and g + 8, C chunks per row; V: C chunks of VB bytes each of rows 2t, 2t+1,
// 2t+8, 2t+9.  Registers are 32-bit words.
template <int D, int KV>
struct Frag;

template <int D>
struct Frag<D, kKvBf16> {
    static constexpr int C = D / 32;       // 16-byte chunks of a K row per lane: elements 32 c + 8 t ...
    static constexpr int CV = D / 64;      // 16-byte chunks of a V row per lane: elements 64 c + 8 g ...
    uint4 k[2][C], v[4][CV];
};
template <int D>
struct Frag8 {
    static constexpr int C = D / 64;       // 16-byte chunks of a K row: elements 64 c + 16 t ...
    static constexpr int VW = D / 32;      // words of a V row: elements (D / 8) g ... : 4 (d = 128) or 2
    uint4 k[2][C];
    uint32_t v[4][VW];
    uint32_t ks[2], vs[4];                 // scale bytes of the lane's K rows (all), of its V elements
};
template <int D> struct Frag<D, kKvE4m3> : Frag8<D> {};
template <int D> struct Frag<D, kKvInt8> : Frag8<D> {};

template <int D, int KV>
__device__ __forceinline__ void load_k(Frag<D, KV> &f, const PagedCache &c, int half, int row, int t) {
    // a row of -1 (no key, or a page out of range) reads as zeros; its score is masked
    if constexpr (KV == kKvBf16) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(c.k) + (long long)row * D) + t;
#pragma unroll
        for (int x = 0; x < f.C; ++x) f.k[half][x] = row >= 0 ? ldg_stream(p + 4 * x) : make_uint4(0u, 0u, 0u, 0u);
    } else {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(c.k) + (long long)row * D) + t;
#pragma unroll
        for (int x = 0; x < f.C; ++x) f.k[half][x] = row >= 0 ? ldg_stream(p + 4 * x) : make_uint4(0u, 0u, 0u, 0u);
        if (D == 128) f.ks[half] = row >= 0 ? __ldg(reinterpret_cast<const uint32_t *>(c.k_scale) + row) : 0u;
        else f.ks[half] = row >= 0 ? __ldg(reinterpret_cast<const uint16_t *>(c.k_scale) + row) : 0u;
    }
}

template <int D, int KV>
__device__ __forceinline__ void load_v(Frag<D, KV> &f, const PagedCache &c, int which, int row, int g) {
    if constexpr (KV == kKvBf16) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(c.v) + (long long)row * D) + g;
#pragma unroll
        for (int x = 0; x < f.CV; ++x) f.v[which][x] = row >= 0 ? ldg_stream(p + 8 * x) : make_uint4(0u, 0u, 0u, 0u);
    } else {
        const uint8_t *p = static_cast<const uint8_t *>(c.v) + (long long)row * D + g * (D / 8);
        if constexpr (D == 128) {
            const uint4 x = row >= 0 ? ldg_stream(reinterpret_cast<const uint4 *>(p)) : make_uint4(0u, 0u, 0u, 0u);
            f.v[which][0] = x.x; f.v[which][1] = x.y; f.v[which][2] = x.z; f.v[which][3] = x.w;
        } else {
            const uint2 x = row >= 0 ? __ldg(reinterpret_cast<const uint2 *>(p)) : make_uint2(0u, 0u);
            f.v[which][0] = x.x; f.v[which][1] = x.y;
        }
        // elements (D / 8) g ... lie in one block of 32
        f.vs[which] = row >= 0 ? __ldg(c.v_scale + (long long)row * (D / kScaleBlock) + g * (D / 8) / kScaleBlock) : 0u;
    }
}

// ---- the two products ----------------------------------------------------------------------

// s[nh] += K (16 keys) . Q (heads 8 nh ...): q[nh][k step] from load_q
template <int D, int KV, int NH>
__device__ __forceinline__ void scores(const Frag<D, KV> &f, const uint2 (&q)[NH][D / 16], float (&s)[NH][4], int t) {
    if constexpr (KV == kKvBf16) {
#pragma unroll
        for (int x = 0; x < f.C; ++x) {
#pragma unroll
            for (int nh = 0; nh < NH; ++nh) {
                mma_bf16(s[nh], f.k[0][x].x, f.k[1][x].x, f.k[0][x].y, f.k[1][x].y, q[nh][2 * x].x, q[nh][2 * x].y);
                mma_bf16(s[nh], f.k[0][x].z, f.k[1][x].z, f.k[0][x].w, f.k[1][x].w, q[nh][2 * x + 1].x, q[nh][2 * x + 1].y);
            }
        }
    } else {
#pragma unroll
        for (int x = 0; x < f.C; ++x) {
            // elements 64 x + 16 t ... of a row lie in block 2 x + t / 2
            const Scale2<KV> s0 = scale_same<KV>(f.ks[0] >> (8 * (2 * x + (t >> 1))) & 0xffu);
            const Scale2<KV> s1 = scale_same<KV>(f.ks[1] >> (8 * (2 * x + (t >> 1))) & 0xffu);
            const uint32_t w0[4] = {f.k[0][x].x, f.k[0][x].y, f.k[0][x].z, f.k[0][x].w};
            const uint32_t w1[4] = {f.k[1][x].x, f.k[1][x].y, f.k[1][x].z, f.k[1][x].w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {  // one k step per word: four elements of each row
                uint32_t a0, a2, a1, a3;
                codes_to_bf16<KV>(w0[w], s0, s0.big, a0, a2);
                codes_to_bf16<KV>(w1[w], s1, s1.big, a1, a3);
#pragma unroll
                for (int nh = 0; nh < NH; ++nh) mma_bf16(s[nh], a0, a1, a2, a3, q[nh][4 * x + w].x, q[nh][4 * x + w].y);
            }
        }
    }
}

// The queries of head 8 nh + g in the k order of scores().
template <int D, int KV>
__device__ __forceinline__ void load_q(uint2 (&q)[D / 16], const __nv_bfloat16 *row, bool ok, int t) {
    const uint4 *p = reinterpret_cast<const uint4 *>(row);
#pragma unroll
    for (int x = 0; x < D / 32; ++x) {
        // bf16 cache: elements 32 x + 8 t ...; 8 bits: halves of 64 (x / 2) + 16 t ...
        const int at = KV == kKvBf16 ? 4 * x + t : 8 * (x >> 1) + 2 * t + (x & 1);
        const uint4 u = ok ? __ldg(p + at) : make_uint4(0u, 0u, 0u, 0u);
        q[2 * x] = make_uint2(u.x, u.y);
        q[2 * x + 1] = make_uint2(u.z, u.w);
    }
}

// o[nh][j] += V^T P^T; accumulator j holds elements elem(j, g), elem(j, g) + 1 of heads 2t, 2t + 1
template <int D, int KV>
__device__ __forceinline__ int elem(int j, int g) {
    return KV == kKvBf16 ? 64 * (j >> 2) + 8 * g + 2 * (j & 3) : (D / 8) * g + 2 * j;
}
template <int D, int KV, int NH>
__device__ __forceinline__ void accumulate(const Frag<D, KV> &f, const uint32_t (&p)[NH][2], float (&o)[NH][D / 16][4]) {
    if constexpr (KV == kKvBf16) {
#pragma unroll
        for (int x = 0; x < f.CV; ++x) {
            const uint32_t r[4][4] = {{f.v[0][x].x, f.v[0][x].y, f.v[0][x].z, f.v[0][x].w},
                                      {f.v[1][x].x, f.v[1][x].y, f.v[1][x].z, f.v[1][x].w},
                                      {f.v[2][x].x, f.v[2][x].y, f.v[2][x].z, f.v[2][x].w},
                                      {f.v[3][x].x, f.v[3][x].y, f.v[3][x].z, f.v[3][x].w}};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t a0 = __byte_perm(r[0][w], r[1][w], 0x5410), a1 = __byte_perm(r[0][w], r[1][w], 0x7632);
                const uint32_t a2 = __byte_perm(r[2][w], r[3][w], 0x5410), a3 = __byte_perm(r[2][w], r[3][w], 0x7632);
#pragma unroll
                for (int nh = 0; nh < NH; ++nh) mma_bf16(o[nh][4 * x + w], a0, a1, a2, a3, p[nh][0], p[nh][1]);
            }
        }
    } else {
        const Scale2<KV> s01 = scale_pair<KV>(f.vs[0], f.vs[1]), s23 = scale_pair<KV>(f.vs[2], f.vs[3]);
#pragma unroll
        for (int w = 0; w < f.VW; ++w) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // codes 2h, 2h + 1 of the word, each with its pair of keys
                const uint32_t sel = h ? 0x7362 : 0x5140;
                uint32_t a0, a1, a2, a3;
                codes_to_bf16<KV>(__byte_perm(f.v[0][w], f.v[1][w], sel), s01, s01.big, a0, a1);
                codes_to_bf16<KV>(__byte_perm(f.v[2][w], f.v[3][w], sel), s23, s23.big, a2, a3);
#pragma unroll
                for (int nh = 0; nh < NH; ++nh) mma_bf16(o[nh][2 * w + h], a0, a1, a2, a3, p[nh][0], p[nh][1]);
            }
        }
    }
}

// NH: groups of 8 query heads (1 or 2); WARPS per CTA
template <int D, int KV, int NH, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, NH == 1 ? 2 : 1) decode_paged_kernel(const Args args) {
    const DecodePagedArgs &a = args.a;
    const Shape &s = a.s;
    const PagedCache &c = a.cache;
    constexpr int PART = D + 4;  // floats of a head's partial state: o[D], m, l, padding to 16 bytes
    extern __shared__ __align__(16) float part[];  // [WARPS][G][PART]
    const int P = gridDim.x, rank = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int G = s.H / s.Hkv, h0 = kvh * G;

    int n = __ldg(a.lens + b);
    uint2 q[NH][D / 16];
    float offb[NH][2], offs[NH][2];
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
        load_q<D, KV>(q[nh], a.q + (long long)b * a.q_stride + (h0 + 8 * nh + g) * D, 8 * nh + g < G, t);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int hh = 8 * nh + 2 * t + e;
            const float al = a.alpha && hh < G ? __ldg(a.alpha + (long long)b * s.H + h0 + hh) : 1.f;
            offb[nh][e] = a.alpha ? log2f(al) : 0.f;
            offs[nh][e] = log2f(1.f - al);
        }
    }
    if (n < 0 || n > (long long)c.width << c.page_log2) {
        if (threadIdx.x == 0) record_index(a.index_word);
        n = 0;
    }
    // the key list: band lo .. n-1, then the skips n-1 - m * period, m = m_first ...
    const int i = n - 1;
    const int lo = n > 0 ? band_lo(i, s.mode, s.k_local) : 0, n_band = n - lo;
    int n_keys = n_band;
    if (n > 0 && s.mode != kModeEcp && s.S > 0) n_keys += max(0, min(s.S, i / s.period) - args.m_first + 1);
    const int n_tiles = (n_keys + KEYS - 1) / KEYS;

    float m[NH][2], l[NH][2], o[NH][D / 16][4];
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
#pragma unroll
        for (int e = 0; e < 2; ++e) { m[nh][e] = -INFINITY; l[nh][e] = 0.f; }
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nh][j][e] = 0.f;
    }
    const int step = P * WARPS;
    for (int tile = rank * WARPS + warp; tile < n_tiles; tile += 2 * step) {
        // rows of this tile (lanes 0-15) and of the warp's next one (16-31)
        const int kk = (tile + (lane < KEYS ? 0 : step)) * KEYS + (lane & (KEYS - 1));
        int row = -1;
        if (kk < n_keys) {
            const int pos = kk < n_band ? lo + kk : i - (args.m_first + kk - n_band) * s.period;
            const int pg = page_of(c, a.table, b, pos);
            if (pg >= 0) row = row_in_page(c, pg, kvh, pos);
            else record_index(a.index_word);
        }
#pragma unroll 1
        for (int u = 0; u < 2; ++u) {
            const int t0 = (tile + u * step) * KEYS;
            if (t0 >= n_keys) break;
            Frag<D, KV> f;
#pragma unroll
            for (int x = 0; x < 2; ++x) load_k<D, KV>(f, c, x, __shfl_sync(kFull, row, u * KEYS + g + 8 * x), t);
#pragma unroll
            for (int x = 0; x < 4; ++x)
                load_v<D, KV>(f, c, x, __shfl_sync(kFull, row, u * KEYS + 2 * t + (x & 1) + 8 * (x >> 1)), g);
            const bool has0 = __shfl_sync(kFull, row, u * KEYS + g) >= 0, has1 = __shfl_sync(kFull, row, u * KEYS + g + 8) >= 0;
            float sc[NH][4] = {};
            scores<D, KV, NH>(f, q, sc, t);
            uint32_t p[NH][2];
#pragma unroll
            for (int nh = 0; nh < NH; ++nh) {
                const bool b0 = t0 + g < n_band, b1 = t0 + g + 8 < n_band;
                float pr[4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float z0 = has0 ? fmaf(sc[nh][e], s.scale_log2, b0 ? offb[nh][e] : offs[nh][e]) : -INFINITY;
                    const float z1 = has1 ? fmaf(sc[nh][2 + e], s.scale_log2, b1 ? offb[nh][e] : offs[nh][e]) : -INFINITY;
                    float mx = fmaxf(z0, z1);
                    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
                    const float mn = fmaxf(m[nh][e], mx), ref = mn == -INFINITY ? 0.f : mn;
                    const float corr = exp2f(m[nh][e] - ref);
                    pr[e] = exp2f(z0 - ref);
                    pr[2 + e] = exp2f(z1 - ref);
                    l[nh][e] = fmaf(l[nh][e], corr, pr[e] + pr[2 + e]);
                    m[nh][e] = mn;
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        o[nh][j][e] *= corr;
                        o[nh][j][2 + e] *= corr;
                    }
                }
                p[nh][0] = transpose8(pack_bf16x2(pr[0], pr[1]));
                p[nh][1] = transpose8(pack_bf16x2(pr[2], pr[3]));
            }
            accumulate<D, KV, NH>(f, p, o);
        }
    }

    // ---- the warps' partial states to shared memory
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float sum = l[nh][e];
            sum += __shfl_xor_sync(kFull, sum, 4);
            sum += __shfl_xor_sync(kFull, sum, 8);
            sum += __shfl_xor_sync(kFull, sum, 16);
            const int hh = 8 * nh + 2 * t + e;
            if (hh < G) {
                float *ps = part + (warp * G + hh) * PART;
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
                    *reinterpret_cast<float2 *>(ps + elem<D, KV>(j, g)) = make_float2(o[nh][j][e], o[nh][j][2 + e]);
                if (g == 0) *reinterpret_cast<float2 *>(ps + D) = make_float2(m[nh][e], sum);
            }
        }
    __syncthreads();

    // merge of `cnt` states `stride` floats apart: columns col, col + 1 of a head
    auto finish = [&](int hh, int col, float mt, float lt, float x, float y) {
        const float inv = lt > 0.f ? 1.f / lt : 0.f;
        const long long at = (long long)b * s.H + h0 + hh;
        *reinterpret_cast<uint32_t *>(a.out + at * D + col) = pack_bf16x2(x * inv, y * inv);
        if (col == 0) a.lse[at] = lt > 0.f ? (mt + log2f(lt)) * kLn2 : -INFINITY;
    };
    const int pairs = G * (D / 2);
    for (int w = threadIdx.x; w < pairs; w += WARPS * 32) {
        const int hh = w / (D / 2), col = 2 * (w % (D / 2));
        float2 ml[WARPS], ov[WARPS];
#pragma unroll
        for (int x = 0; x < WARPS; ++x) {
            const float *ps = part + (x * G + hh) * PART;
            ml[x] = *reinterpret_cast<const float2 *>(ps + D);
            ov[x] = *reinterpret_cast<const float2 *>(ps + col);
        }
        float mt = -INFINITY;
#pragma unroll
        for (int x = 0; x < WARPS; ++x) mt = fmaxf(mt, ml[x].x);
        float lt = 0.f, x0 = 0.f, x1 = 0.f;
        const float ref = mt == -INFINITY ? 0.f : mt;
#pragma unroll
        for (int x = 0; x < WARPS; ++x) {
            const float e = exp2f(ml[x].x - ref);
            lt = fmaf(e, ml[x].y, lt);
            x0 = fmaf(e, ov[x].x, x0);
            x1 = fmaf(e, ov[x].y, x1);
        }
        if (P == 1) {
            finish(hh, col, mt, lt, x0, x1);
        } else {  // the CTA's state, behind the warps'
            float *ps = part + (WARPS * G + hh) * PART;
            *reinterpret_cast<float2 *>(ps + col) = make_float2(x0, x1);
            if (col == 0) *reinterpret_cast<float2 *>(ps + D) = make_float2(mt, lt);
        }
    }
    if (P == 1) return;
    cluster_sync();
    const uint32_t base = smem_addr(part + WARPS * G * PART);
    for (int w = rank * WARPS * 32 + threadIdx.x; w < pairs; w += P * WARPS * 32) {
        const int hh = w / (D / 2), col = 2 * (w % (D / 2));
        float2 ml[MAX_P], ov[MAX_P];
#pragma unroll
        for (int x = 0; x < MAX_P; ++x)
            if (x < P) {
                const uint32_t at = peer_addr(base + (uint32_t)(hh * PART) * 4u, x);
                ml[x] = ld_peer2(at + D * 4);
                ov[x] = ld_peer2(at + col * 4);
            }
        float mt = -INFINITY;
#pragma unroll
        for (int x = 0; x < MAX_P; ++x)
            if (x < P) mt = fmaxf(mt, ml[x].x);
        float lt = 0.f, x0 = 0.f, x1 = 0.f;
        const float ref = mt == -INFINITY ? 0.f : mt;
#pragma unroll
        for (int x = 0; x < MAX_P; ++x)
            if (x < P) {
                const float e = exp2f(ml[x].x - ref);
                lt = fmaf(e, ml[x].y, lt);
                x0 = fmaf(e, ov[x].x, x0);
                x1 = fmaf(e, ov[x].y, x1);
            }
        finish(hh, col, mt, lt, x0, x1);
    }
    cluster_sync();  // every CTA's shared memory stays until the others have read it
}

template <int D, int KV, int NH>
static cudaError_t launch(const Args &a, int P, cudaStream_t st) {
    constexpr int WARPS = 8;
    const int G = a.a.s.H / a.a.s.Hkv;
    const int smem = (WARPS + 1) * G * (D + 4) * 4;
    auto *kernel = decode_paged_kernel<D, KV, NH, WARPS>;
    static PerDeviceOnce configured;  // shared memory above the 48 KB default
    int dev = 0;
    cudaGetDevice(&dev);
    if (configured.needed(dev)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (WARPS + 1) * 8 * NH * (D + 4) * 4);
        if (e != cudaSuccess) return e;
        configured.mark(dev);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)P, (unsigned)a.a.s.Hkv, (unsigned)a.a.s.B);
    cfg.blockDim = dim3(WARPS * 32, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)P;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = P > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int D, int KV>
static cudaError_t launch_heads(const Args &a, int P, cudaStream_t st) {
    return a.a.s.H / a.a.s.Hkv <= 8 ? launch<D, KV, 1>(a, P, st) : launch<D, KV, 2>(a, P, st);
}

}  // namespace decp

cudaError_t launch_decode_paged(const DecodePagedArgs &a, cudaStream_t st) {
    using namespace decp;
    const Shape &s = a.s;
    Args args{a, s.mode != kModeEcp && s.S > 0 ? first_skip_multiple(s) : 1};
    // tiles of the longest key list, and CTAs per (sequence, KV head): one tile per warp while the
    // grid stays within about two CTAs per SM
    const long long cap = (long long)a.cache.width << a.cache.page_log2;
    const long long keys = std::min<long long>(cap, s.mode == kModeEcp ? 2LL * s.k_local : (long long)s.k_local + 1 + s.S);
    const long long tiles = (keys + KEYS - 1) / KEYS, pairs = (long long)s.B * s.Hkv;
    const int P = (int)std::max<long long>(1, std::min<long long>({(long long)MAX_P, (tiles + 7) / 8, 2LL * sm_count() / pairs}));
    const bool d64 = s.d == 64;
    switch (a.cache.kv_type) {
        case kKvBf16: return d64 ? launch_heads<64, kKvBf16>(args, P, st) : launch_heads<128, kKvBf16>(args, P, st);
        case kKvE4m3: return d64 ? launch_heads<64, kKvE4m3>(args, P, st) : launch_heads<128, kKvE4m3>(args, P, st);
        default: return d64 ? launch_heads<64, kKvInt8>(args, P, st) : launch_heads<128, kKvInt8>(args, P, st);
    }
}

}  // namespace pi
