// pi_rotary.cu -- rotary positions: queries and keys (or their gradients) of a training layer turned on the way between the
// projection's layout and the attention's, and a serving step's new queries and keys turned as the keys and values go into
// the paged cache.
//
// An angle is a position times turns per position in 64-bit fixed point, whose product wraps as turns do: two integer
// multiplications reduce it, exactly, however far the position is.  What is left of a turn, as fp32, goes to sincospi.
// Every element is read once and written once, so HBM bounds long calls.  The sines of a position are the same for all of its heads:
//   * rotary_kernel: a thread has 8 pairs (16 elements) of a row and walks over heads with the same 8 sines and cosines.
//   * append_kernel: a CTA puts its tokens' sines into shared memory, since a cache row's 8-bit blocks of 32 elements do not fall
//     on the pairs' halves: a lane has 16 contiguous elements of a key row and reads their partners once more (from L1).
#include "pi_mma.cuh"
#include "pi_paged.cuh"
#include "pi_quant.cuh"
#include "pi_step.h"
#include "pi_tree.cuh"

namespace pi {
namespace rot {

constexpr int THREADS = 256;
constexpr unsigned kFull = 0xffffffffu;

// (cos, sin) of pos * step[j] turns, times the scale.
__device__ __forceinline__ float2 turn(const Rotary &r, int j, int pos) {
    const uint2 w = ld_now(reinterpret_cast<const uint2 *>(r.step + j));
    const unsigned long long step = (unsigned long long)w.y << 32 | w.x;
    const int part = (int)(((unsigned long long)(long long)pos * step) >> 32);  // of a turn, in 2^-32: -1/2 .. 1/2
    float s, c;
    sincospif((float)part * 0x1p-31f, &s, &c);
    return make_float2(c * r.scale, s * r.scale);
}

// Eight elements of a row.
template <typename T>
struct Eight {
    uint4 w[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = ld_stream(reinterpret_cast<const uint4 *>(p) + i);
    }
    __device__ __forceinline__ void store(T *p) const {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4 *>(p)[i] = w[i];
    }
    __device__ __forceinline__ void unpack(float (&f)[8]) const {
        if constexpr (sizeof(T) == 2) {
            unpack8(w[0], f);
        } else {
            const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(u[j]);
        }
    }
    __device__ __forceinline__ void pack(const float (&f)[8]) {
        if constexpr (sizeof(T) == 2) {
            w[0] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                w[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3]));
        }
    }
};

// The 8 pairs of 16 elements a, b: (a[j], b[j]), or neighbours within each.
template <bool INTER>
__device__ __forceinline__ void turn_pairs(float (&a)[8], float (&b)[8], const float2 (&cs)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float &x = INTER ? (j < 4 ? a[2 * j] : b[2 * j - 8]) : a[j], &y = INTER ? (j < 4 ? a[2 * j + 1] : b[2 * j - 7]) : b[j];
        const float x0 = x;
        x = fmaf(x0, cs[j].x, -y * cs[j].y);
        y = fmaf(x0, cs[j].y, y * cs[j].x);
    }
}

// blockIdx.y: a share of `per` heads of the queries or of the keys.
template <typename T, bool INTER>
__global__ void __launch_bounds__(THREADS) rotary_kernel(const __grid_constant__ RotaryArgs g, int per, int q_shares) {
    constexpr int AHEAD = sizeof(T) == 2 ? 4 : 2;  // heads whose elements are in flight
    const int units = g.d / 16, u = threadIdx.x % units;
    const unsigned row = blockIdx.x * (THREADS / units) + threadIdx.x / units;  // (B * N < 2^31)
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (row >= (unsigned)g.B * g.N) return;
    const int b = (int)(row / (unsigned)g.N), n = (int)(row - (unsigned)b * g.N);
    const bool keys = (int)blockIdx.y >= q_shares;
    const RotaryTensor &t = g.t[keys];
    const int h0 = ((int)blockIdx.y - (keys ? q_shares : 0)) * per, h1 = min(h0 + per, t.heads);
    const bool turns = u < g.r.rot / 16;
    const int at_a = turns && !INTER ? 8 * u : 16 * u, at_b = turns && !INTER ? at_a + g.r.rot / 2 : at_a + 8;
    const T *x = static_cast<const T *>(t.x) + b * t.x_batch + n * t.x_pos;
    T *y = static_cast<T *>(t.y) + b * t.y_batch + n * t.y_pos;
    Eight<T> ea[AHEAD], eb[AHEAD];
    auto load = [&](int h) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (h + i < h1) {
                const T *p = x + (h + i) * t.x_head;
                ea[i].load(p + at_a);
                eb[i].load(p + at_b);
            }
    };
    load(h0);
    float2 cs[8];
    if (turns) {
        const int pos = g.pos ? ld_now(g.pos + row) : g.start + n;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            cs[j] = turn(g.r, 8 * u + j, pos);
            if (g.back) cs[j].y = -cs[j].y;
        }
    }
#pragma unroll 1
    for (int h = h0; h < h1; h += AHEAD) {
        if (h > h0) load(h);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (h + i < h1) {
                if (turns) {
                    float fa[8], fb[8];
                    ea[i].unpack(fa);
                    eb[i].unpack(fb);
                    turn_pairs<INTER>(fa, fb, cs);
                    ea[i].pack(fa);
                    eb[i].pack(fb);
                }
                T *p = y + (h + i) * t.y_head;
                ea[i].store(p + at_a);
                eb[i].store(p + at_b);
            }
    }
}

// ------------------------------------------------------------------ a serving step's new tokens

struct Place {
    int line, pg;  // cache position of the token's row, and its page (-1: the token is left out)
};

// 16 elements of a key or value row into the cache, 32 a block of two lanes.  For the whole warp.
template <int KV>
__device__ __forceinline__ void put16(const PagedCache &c, void *pages, uint8_t *scales, const float (&lo)[8], const float (&hi)[8],
                                      long long row, int col, bool in) {
    if constexpr (KV == kKvBf16) {
        Eight<__nv_bfloat16> x, y;
        x.pack(lo);
        y.pack(hi);
        __nv_bfloat16 *p = static_cast<__nv_bfloat16 *>(pages) + row * c.d + col;
        if (in) {
            x.store(p);
            y.store(p + 8);
        }
    } else {
        uint32_t m = 0;  // magnitudes compare like their bits; infinities and NaN come out on top
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, max(__float_as_uint(lo[j]) & 0x7fffffffu, __float_as_uint(hi[j]) & 0x7fffffffu));
        m = max(m, __shfl_xor_sync(kFull, m, 1));
        const bool finite = m < 0x7f800000u;
        const int e = finite ? scale_exp<KV>(__uint_as_float(m)) : 0;
        const uint2 x = encode_codes<KV>(lo, e), y = encode_codes<KV>(hi, e);
        if (!in) return;
        *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(pages) + row * c.d + col) =
            finite ? make_uint4(x.x, x.y, y.x, y.y) : make_uint4(0u, 0u, 0u, 0u);
        if ((col & (kScaleBlock - 1)) == 0)
            scales[row * (c.d / kScaleBlock) + col / kScaleBlock] = (uint8_t)(finite ? e + 127 : kScaleNan);
    }
}

// TOK tokens per CTA.  A token's work comes in pieces of 16 elements, those of its queries, keys and values each padded to
// whole warps.
template <int KV, bool INTER, int TOK>
__global__ void __launch_bounds__(THREADS) append_kernel(const __grid_constant__ RotaryAppendArgs g) {
    extern __shared__ float2 turns[];  // [TOK][rot / 2]
    __shared__ Place place[TOK];
    static_assert(TOK <= THREADS / 32, "a warp per token");
    const PagedCache &c = g.a.cache;
    const PagedBatch &bt = g.a.batch;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rot = g.r.rot, half = rot / 2;
    const int per_row = c.d / 16, row_log2 = c.d_log2 - 4;
    const int nq = (g.H * per_row + 31) & ~31, nk = (c.Hkv * per_row + 31) & ~31, n = nq + 2 * nk;
    const int first = blockIdx.x * TOK, tokens = min(TOK, bt.T - first), items = tokens * n;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // piece `it`: its token, what it is (0: queries, 1: keys, 2: values), head and first element
    struct Piece {
        int tok, kind, head, col;
        bool in;
    };
    auto piece = [&](int it) {
        Piece p;
        p.tok = it / n;
        int x = it - p.tok * n;
        p.kind = x < nq ? 0 : x < nq + nk ? 1 : 2;
        x -= p.kind == 0 ? 0 : p.kind == 1 ? nq : nq + nk;
        p.head = x >> row_log2;
        p.col = 16 * (x & (per_row - 1));
        p.in = p.head < (p.kind == 0 ? g.H : c.Hkv);
        return p;
    };
    using Row = Eight<__nv_bfloat16>;
    Row x0, x1, y0, y1;  // the elements, and (keys, pairs in halves) their partners
    auto load = [&](const Piece &p) {
        if (!p.in) {
            x0.w[0] = x1.w[0] = y0.w[0] = y1.w[0] = make_uint4(0u, 0u, 0u, 0u);
            return;
        }
        const long long t = first + p.tok;
        const __nv_bfloat16 *r = p.kind == 0 ? g.q + t * g.q_stride : p.kind == 1 ? g.a.k + t * g.a.k_stride : g.a.v + t * g.a.v_stride;
        r += (long long)p.head * c.d;
        if (p.kind == 0) {  // 8 pairs, in halves from both of them
            const bool halves = !INTER && p.col < rot;
            x0.load(r + (halves ? p.col / 2 : p.col));
            x1.load(r + (halves ? p.col / 2 + half : p.col + 8));
        } else {
            x0.load(r + p.col);
            x1.load(r + p.col + 8);
            if (!INTER && p.kind == 1) {
                const int e0 = p.col, e1 = p.col + 8;
                y0.load(r + (e0 < half ? e0 + half : e0 < rot ? e0 - half : e0));
                y1.load(r + (e1 < half ? e1 + half : e1 < rot ? e1 - half : e1));
            }
        }
    };
    Piece p = piece(threadIdx.x);
    p.in = p.in && (int)threadIdx.x < items;
    load(p);

    if (warp < tokens) {  // where the token's row goes, and its sines
        const int t = first + warp;
        int b, line = locate(c, bt, t, b, g.a.index_word), pos = line, pg = -1;
        if (line >= 0) {
            if (g.parent) {
                const int t0 = ld_now(bt.cu + b), deep = tree_depth(g.parent, t0, ld_now(bt.cu + b + 1) - t0, t - t0);
                pos = deep < 0 ? -1 : line - (t - t0) + deep;
            }
            if (pos >= 0) pg = page_of(c, bt.table, b, line);
            if (pg < 0 && lane == 0) record_index(g.a.index_word);
        }
        if (lane == 0) place[warp] = Place{line, pg};
        for (int j = lane; j < half; j += 32) turns[warp * half + j] = turn(g.r, j, pos);
    }
    __syncthreads();

    for (int it = threadIdx.x; it < items; it += THREADS) {  // (whole warps)
        if (it >= THREADS) {
            p = piece(it);
            load(p);
        }
        const Place pl = place[p.tok];
        const float2 *cs = turns + p.tok * half;
        p.in = p.in && pl.pg >= 0;
        if (p.kind == 0) {
            const bool halves = !INTER && p.col < rot;
            if (p.col < rot) {
                float a[8], b[8];
                float2 w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = cs[p.col / 2 + j];
                x0.unpack(a);
                x1.unpack(b);
                turn_pairs<INTER>(a, b, w);
                x0.pack(a);
                x1.pack(b);
            }
            if (p.in) {
                __nv_bfloat16 *r = g.q_out + (first + p.tok) * g.q_out_stride + (long long)p.head * c.d;
                x0.store(r + (halves ? p.col / 2 : p.col));
                x1.store(r + (halves ? p.col / 2 + half : p.col + 8));
            }
            continue;
        }
        float a[8], b[8];
        x0.unpack(a);
        x1.unpack(b);
        if (p.kind == 1 && p.col < rot) {
            if constexpr (INTER) {
                float2 w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = cs[p.col / 2 + j];
                turn_pairs<true>(a, b, w);
            } else {
                auto eight = [&](float (&x)[8], const Row &partner, int e) {  // (rot / 2 is a multiple of 8: on one side of it)
                    float y[8];
                    partner.unpack(y);
                    const bool low = e < half;
                    const float2 *w = cs + (low ? e : e - half);
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = fmaf(x[j], w[j].x, low ? -y[j] * w[j].y : y[j] * w[j].y);
                };
                eight(a, y0, p.col);
                eight(b, y1, p.col + 8);
            }
        }
        const long long row = row_in_page(c, max(pl.pg, 0), p.head, max(pl.line, 0));
        if (KV == kKvBf16 && (p.kind == 2 || p.col >= rot)) {  // as they are
            __nv_bfloat16 *r = static_cast<__nv_bfloat16 *>(p.kind == 1 ? c.k : c.v) + row * c.d + p.col;
            if (p.in) {
                x0.store(r);
                x1.store(r + 8);
            }
        } else if (p.kind == 1) {
            put16<KV>(c, c.k, c.k_scale, a, b, row, p.col, p.in);
        } else {
            put16<KV>(c, c.v, c.v_scale, a, b, row, p.col, p.in);
        }
    }
}

// A launch that may start while the kernel before it on the stream ends (and waits for it).
template <typename K, typename... A>
static cudaError_t launch(K kernel, dim3 grid, size_t smem, cudaStream_t st, const A &...a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a...);
}

template <int KV, int TOK>
static cudaError_t launch_append(const RotaryAppendArgs &g, cudaStream_t st) {
    const dim3 grid((unsigned)((g.a.batch.T - 1) / TOK + 1), 1, 1);
    const size_t smem = (size_t)TOK * (g.r.rot / 2) * sizeof(float2);
    return g.r.interleaved ? launch(append_kernel<KV, true, TOK>, grid, smem, st, g) : launch(append_kernel<KV, false, TOK>, grid, smem, st, g);
}
template <int KV>
static cudaError_t launch_append(const RotaryAppendArgs &g, cudaStream_t st) {
    return g.a.batch.T >= 16 * sm_count() ? launch_append<KV, 8>(g, st) : launch_append<KV, 1>(g, st);
}

}  // namespace rot

cudaError_t launch_rotary(const RotaryArgs &a, cudaStream_t st) {
    using namespace rot;
    const int per = 4, q_shares = (a.t[0].heads + per - 1) / per, k_shares = (a.t[1].heads + per - 1) / per;
    const long long rows = (long long)a.B * a.N, of = THREADS / (a.d / 16);
    const dim3 grid((unsigned)((rows + of - 1) / of), (unsigned)(q_shares + k_shares), 1);
    auto kernel = a.f32 ? (a.r.interleaved ? rotary_kernel<float, true> : rotary_kernel<float, false>)
                        : (a.r.interleaved ? rotary_kernel<__nv_bfloat16, true> : rotary_kernel<__nv_bfloat16, false>);
    return launch(kernel, grid, 0, st, a, per, q_shares);
}

cudaError_t launch_rotary_append(const RotaryAppendArgs &a, cudaStream_t st) {
    using namespace rot;
    switch (a.a.cache.kv_type) {
        case kKvBf16: return launch_append<kKvBf16>(a, st);
        case kKvE4m3: return launch_append<kKvE4m3>(a, st);
        default: return launch_append<kKvInt8>(a, st);
    }
}

}  // namespace pi
