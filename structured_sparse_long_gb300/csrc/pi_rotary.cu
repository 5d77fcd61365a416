// pi_rotary.cu -- rotary positions: queries and keys (or their gradients) of a training layer turned on the way between the
// projection's layout and the attention's, and a serving step's new queries and keys turned as the keys and values go into
// the paged cache.
//
// An angle is a position times turns per position in 64-bit fixed point, whose product wraps as turns do: two integer
// multiplications reduce it, exactly, however far the position is.  What is left of a turn, as fp32, goes to sincospi.
// Every element is read once and written once, so HBM bounds long calls.  The sines of a position are the same for all of its heads:
//   * rotary_kernel: a thread has 8 pairs (16 elements) of a row and walks over heads with the same 8 sines and cosines.
//   * append_kernel: every warp is on its own.  One takes four heads of neighbouring tokens' queries, in the same way; another a token's keys
//     and values.  A cache row's 8-bit blocks of 32 elements do not fall on the pairs' halves, so there a lane has 16 contiguous
//     elements of a key row, reads their partners once more (from L1), and the warp's sines lie in shared memory.
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

// The 8 pairs of 16 elements a, b: (a[j], b[j]), or neighbours within each; two pairs to an instruction.
template <bool INTER>
__device__ __forceinline__ void turn_pairs(float (&a)[8], float (&b)[8], const float2 (&cs)[8]) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        float *p = INTER ? (j < 4 ? a + 2 * j : b + 2 * j - 8) : a + j, *q = INTER ? p + 1 : b + j;
        constexpr int step = INTER ? 2 : 1;
        const uint64_t x = tc::pack2(p[0], p[step]), y = tc::pack2(q[0], q[step]);
        const uint64_t c = tc::pack2(cs[j].x, cs[j + 1].x), s = tc::pack2(cs[j].y, cs[j + 1].y), m = tc::pack2(-cs[j].y, -cs[j + 1].y);
        tc::unpack2(tc::fma2(x, c, tc::mul2(y, m)), p[0], p[step]);
        tc::unpack2(tc::fma2(x, s, tc::mul2(y, c)), q[0], q[step]);
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

constexpr int QH = 4;  // heads of a warp's queries at a time

// How a launch is cut: heads of a warp's queries, CTAs for the queries, and for the keys and values.
struct append_size {
    int q_heads;
    long long queries, rows;
};
static append_size append_blocks(const RotaryAppendArgs &g) {
    const PagedCache &c = g.a.cache;
    const long long T = g.a.batch.T, per_warp = 512 / c.d, warps = THREADS / 32, groups = (T + per_warp - 1) / per_warp;
    // two rounds of heads with the same sines, where that leaves 12 warps per SM (16 heads, d = 128: 4000 tokens 10.5 us, one round 11.4; 2000
    // tokens 9.2 and 7.4)
    const int q_heads = groups * ((g.H + 2 * QH - 1) / (2 * QH)) >= 12LL * sm_count() ? 2 * QH : QH;
    const long long q = groups * ((g.H + q_heads - 1) / q_heads), kv = T * ((c.Hkv * (long long)c.d + 511) / 512);
    return append_size{q_heads, (q + warps - 1) / warps, (kv + warps - 1) / warps};
}

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
        float m = 0.f;  // (a NaN stays one)
#pragma unroll
        for (int j = 0; j < 8; ++j) asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(fabsf(lo[j])), "f"(fabsf(hi[j])));
        const float other = __shfl_xor_sync(kFull, m, 1);
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(other));
        const bool finite = m < INFINITY;
        const int e = finite ? scale_exp<KV>(m) : 0;
        const uint2 x = encode_codes<KV>(lo, e), y = encode_codes<KV>(hi, e);
        if (!in) return;
        *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(pages) + row * c.d + col) =
            finite ? make_uint4(x.x, x.y, y.x, y.y) : make_uint4(0u, 0u, 0u, 0u);
        if ((col & (kScaleBlock - 1)) == 0)
            scales[row * (c.d / kScaleBlock) + col / kScaleBlock] = (uint8_t)(finite ? e + 127 : kScaleNan);
    }
}

// Where packed tokens t .. t + n - 1 go (n <= 31), in lanes 0 .. n - 1: the position of each in its text and its row's place.  For the whole
// warp.  The first one's sequence is searched; the others' is one of the next 31, whose offsets one round of loads brings (so that a
// step of single tokens costs no search for each), or, with more empty ones in between, searched too.
__device__ __forceinline__ void look_up(const RotaryAppendArgs &g, int t, int n, int &pos, Place &place) {
    const PagedCache &c = g.a.cache;
    const PagedBatch &bt = g.a.batch;
    const int lane = threadIdx.x & 31, B = bt.B;
    pos = -1;
    place = Place{0, -1};
    const int b0 = find_sequence(B, [&](int j) { return ld_now(bt.cu + j) <= t; });
    if (b0 >= B) return;
    const int start = ld_now(bt.cu + min(b0 + lane, B)), at = ld_now(bt.ctx + min(b0 + lane, B - 1));
    int b = B, t0 = 0, t1 = 0, ctx = 0;  // of the lane's token
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        const int on = __popc(__ballot_sync(kFull, lane > 0 && b0 + lane <= B && start <= t + i));
        int bi = b0 + on, u0 = __shfl_sync(kFull, start, on & 31), u1 = __shfl_sync(kFull, start, (on + 1) & 31), x = __shfl_sync(kFull, at, on & 31);
        if (on == 31) {
            bi = find_sequence(B, [&](int j) { return ld_now(bt.cu + j) <= t + i; });
            u0 = ld_now(bt.cu + min(bi, B - 1));
            u1 = ld_now(bt.cu + min(bi, B - 1) + 1);
            x = ld_now(bt.ctx + min(bi, B - 1));
        }
        if (lane == i) {
            b = bi; t0 = u0; t1 = u1; ctx = x;
        }
    }
    const bool mine = lane < n && t + lane < bt.T && b < B;
    const bool ok = mine && sequence_ok(c, bt, t0, t1, ctx) && t + lane >= t0 && t + lane < t1;
    int deep = t + lane - t0;
    if (g.parent) {
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            if (!__shfl_sync(kFull, ok, i)) continue;
            const int u0 = __shfl_sync(kFull, t0, i), u1 = __shfl_sync(kFull, t1, i), d = tree_depth(g.parent, u0, u1 - u0, t + i - u0);
            if (lane == i) deep = d;
        }
    }
    if (ok && deep >= 0) {
        pos = ctx + deep;
        place.line = ctx + t + lane - t0;
        place.pg = page_of(c, bt.table, b, place.line);
    }
    if (mine && place.pg < 0) record_index(g.a.index_word);
}

// The sines of 8 pairs, group g of a token's: in four quarters of two pairs, quarter by quarter for all groups, so that lanes with
// neighbouring groups read neighbouring 16 bytes of shared memory.
__device__ __forceinline__ void read_turns(float2 (&cs)[8], const float4 *turns, int groups, int g) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float4 x = turns[q * groups + g];
        cs[2 * q] = make_float2(x.x, x.y);
        cs[2 * q + 1] = make_float2(x.z, x.w);
    }
}

// The first q_blocks CTAs' warps turn queries, q_heads of neighbouring tokens each, the others keys.
template <int KV, bool INTER>
__global__ void __launch_bounds__(THREADS, 4) append_kernel(const __grid_constant__ RotaryAppendArgs g, int q_blocks, int q_heads) {
    extern __shared__ float4 all_turns[];  // [warps][4][rot / 16]
    const PagedCache &c = g.a.cache;
    const int lane = threadIdx.x & 31, rot = g.r.rot, half = rot / 2;
    const int units = c.d / 16, units_log2 = c.d_log2 - 4;
    using Row = Eight<__nv_bfloat16>;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if ((int)blockIdx.x < q_blocks) {  // ---- queries: 32 / units neighbouring tokens, QH heads, 8 pairs to a lane
        const unsigned w = blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5), shares = (g.H + q_heads - 1) / q_heads;
        const int share = w % shares, n = 32 >> units_log2, u = lane & (units - 1);
        const long long t0 = (long long)(w / shares) * n;
        if (t0 >= g.a.batch.T) return;
        const int mine = lane >> units_log2, t = (int)t0 + mine, h0 = share * q_heads, h1 = min(h0 + q_heads, g.H);
        const bool turns = u < rot / 16;
        const int at_a = turns && !INTER ? 8 * u : 16 * u, at_b = turns && !INTER ? at_a + half : at_a + 8;
        const bool there = t < g.a.batch.T;
        const __nv_bfloat16 *x = g.q + (long long)(there ? t : 0) * g.q_stride;
        Row qa[QH], qb[QH];
        auto load = [&](int h) {
#pragma unroll
            for (int i = 0; i < QH; ++i)
                if (there && h + i < h1) {
                    qa[i].load(x + (h + i) * c.d + at_a);
                    qb[i].load(x + (h + i) * c.d + at_b);
                }
        };
        load(h0);
        int pos;
        Place place;
        look_up(g, (int)t0, n, pos, place);
        pos = __shfl_sync(kFull, pos, mine);
        if (__shfl_sync(kFull, place.pg, mine) < 0) return;
        float2 cs[8];
        if (turns)
#pragma unroll
            for (int j = 0; j < 8; ++j) cs[j] = turn(g.r, 8 * u + j, pos);
        __nv_bfloat16 *y = g.q_out + (long long)t * g.q_out_stride;
#pragma unroll 1
        for (int h = h0; h < h1; h += QH) {
            if (h > h0) load(h);
#pragma unroll
            for (int i = 0; i < QH; ++i)
                if (h + i < h1) {
                    if (turns) {
                        float fa[8], fb[8];
                        qa[i].unpack(fa);
                        qb[i].unpack(fb);
                        turn_pairs<INTER>(fa, fb, cs);
                        qa[i].pack(fa);
                        qb[i].pack(fb);
                    }
                    qa[i].store(y + (h + i) * c.d + at_a);
                    qb[i].store(y + (h + i) * c.d + at_b);
                }
        }
        return;
    }
    // ---- a token's keys and values, 16 neighbouring elements of each to a lane, and (keys, pairs in halves) the partners of their two eights
    const unsigned w = (blockIdx.x - q_blocks) * (THREADS / 32) + (threadIdx.x >> 5);
    const int t = (int)(w / (unsigned)g.a.chunks), chunk = (int)(w - t * (unsigned)g.a.chunks);
    if (t >= g.a.batch.T) return;
    const int j = chunk * 32 + lane, head = j >> units_log2, col = 16 * (j & (units - 1)), groups = rot / 16;
    const bool some = head < c.Hkv;
    const __nv_bfloat16 *pk = g.a.k + (long long)t * g.a.k_stride + (long long)j * 16, *pv = g.a.v + (long long)t * g.a.v_stride + (long long)j * 16;
    Row k0, k1, y0, y1, v0, v1;
    k0.w[0] = k1.w[0] = y0.w[0] = y1.w[0] = v0.w[0] = v1.w[0] = make_uint4(0u, 0u, 0u, 0u);
    if (some) {
        auto partner = [&](int e) -> int { return e < half ? half : e < rot ? -half : 0; };
        k0.load(pk);
        k1.load(pk + 8);
        v0.load(pv);
        v1.load(pv + 8);
        if (!INTER) {
            y0.load(pk + partner(col));
            y1.load(pk + 8 + partner(col + 8));
        }
    }
    int pos;
    Place place;
    look_up(g, t, 1, pos, place);
    pos = __shfl_sync(kFull, pos, 0);
    const int pg = __shfl_sync(kFull, place.pg, 0), line = __shfl_sync(kFull, place.line, 0);
    if (pg < 0) return;
    const long long row = row_in_page(c, pg, min(head, c.Hkv - 1), line);
    if constexpr (KV == kKvBf16) {  // values as they are
        __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(c.v) + row * c.d + col;
        if (some) {
            v0.store(to);
            v1.store(to + 8);
        }
    } else {
        float a[8], b[8];
        v0.unpack(a);
        v1.unpack(b);
        put16<KV>(c, c.v, c.v_scale, a, b, row, col, some);
    }
    float4 *turns = all_turns + (threadIdx.x >> 5) * 4 * groups;
    for (int i = lane; i < half; i += 32) reinterpret_cast<float2 *>(turns)[2 * ((i >> 1 & 3) * groups + (i >> 3)) + (i & 1)] = turn(g.r, i, pos);
    __syncwarp();
    const bool turned = col < rot;  // (rot is a multiple of 16)
    if (KV == kKvBf16 && !turned) {
        __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(c.k) + row * c.d + col;
        if (some) {
            k0.store(to);
            k1.store(to + 8);
        }
        return;
    }
    float a[8], b[8];
    k0.unpack(a);
    k1.unpack(b);
    if (turned) {
        float2 cs[8];
        if constexpr (INTER) {
            read_turns(cs, turns, groups, col / 16);
            turn_pairs<true>(a, b, cs);
        } else {
            auto eight = [&](float (&x)[8], const Row &other, int e) {  // (rot / 2 is a multiple of 8: on one side of it)
                const float sign = e < half ? -1.f : 1.f;
                const uint64_t sign2 = tc::pack2(sign, sign);
                read_turns(cs, turns, groups, (e < half ? e : e - half) / 8);
                float y[8];
                other.unpack(y);
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const uint64_t part = tc::mul2(tc::mul2(tc::pack2(y[i], y[i + 1]), tc::pack2(cs[i].y, cs[i + 1].y)), sign2);
                    tc::unpack2(tc::fma2(tc::pack2(x[i], x[i + 1]), tc::pack2(cs[i].x, cs[i + 1].x), part), x[i], x[i + 1]);
                }
            };
            eight(a, y0, col);
            eight(b, y1, col + 8);
        }
    }
    put16<KV>(c, c.k, c.k_scale, a, b, row, col, some);
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

template <int KV>
static cudaError_t launch_append(const RotaryAppendArgs &args, cudaStream_t st) {
    RotaryAppendArgs g = args;
    const PagedCache &c = g.a.cache;
    const append_size n = append_blocks(g);
    g.a.chunks = (c.Hkv * c.d + 511) / 512;
    const dim3 grid((unsigned)(n.queries + n.rows), 1, 1);  // (fits: rotary_append_fits)
    const size_t smem = (size_t)(THREADS / 32) * (g.r.rot / 2) * sizeof(float2);
    return g.r.interleaved ? launch(append_kernel<KV, true>, grid, smem, st, g, (int)n.queries, n.q_heads)
                           : launch(append_kernel<KV, false>, grid, smem, st, g, (int)n.queries, n.q_heads);
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

bool rotary_append_fits(const RotaryAppendArgs &a) {
    const rot::append_size n = rot::append_blocks(a);
    return n.queries + n.rows <= 0x7fffffffLL && n.queries < (1LL << 28) && n.rows < (1LL << 28);  // warps are numbered in 32 bits
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
