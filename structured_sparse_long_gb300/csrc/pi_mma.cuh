// pi_mma.cuh -- warp-level building blocks of the paged cache's attention: the 16 x 8 x 16 bf16 matrix
// product, 8-bit codes to bf16 pairs, a cache row's elements, and loads across a cluster.
#pragma once

#include <cstdint>

#include "pi_paged.cuh"
#include "pi_tc_ptx.cuh"

namespace pi {

// d (16 x 8, fp32) += a (16 x 16, bf16) b (16 x 8, bf16).  Lane 4 g + t holds rows g, g + 8 of a
// at columns 2t, 2t+1 (a0, a1) and 2t+8, 2t+9 (a2, a3), rows 2t, 2t+1 (b0) and 2t+8, 2t+9 (b1) of
// b at column g, and rows g (d[0], d[1]), g + 8 (d[2], d[3]) of d at columns 2t, 2t+1.
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The transpose of an 8 x 8 matrix of 16-bit values, lane 4 g + t holding columns 2t, 2t+1 of row g.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&t);
}

// 16 bytes that are read once: past L1 (coherent, see ld_now).
__device__ __forceinline__ uint4 ld_stream(const uint4 *p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}

// Scales of the two codes of a pair, from their bytes, as codes_to_bf16 takes them.
//   int8: as fp32.
//   e4m3: as a bf16 pair of factors 2^120 s; what of 2^120 s exceeds 2^127 is in a second pair.
template <int KV>
struct Scale2;
template <>
struct Scale2<kKvInt8> {
    uint64_t s;
    bool big;  // not used
};
template <>
struct Scale2<kKvE4m3> {
    uint32_t f, more;
    bool big;
};

template <int KV>
__device__ __forceinline__ Scale2<KV> scale_pair(uint32_t lo, uint32_t hi) {
    Scale2<KV> r;
    if constexpr (KV == kKvInt8) {
        r.s = tc::pack2(scale_of((int)lo), scale_of((int)hi));
        r.big = false;
    } else {
        // byte b: 2^120 * 2^(b - 127) has the bf16 exponent field b + 120, at most 254; 255 is a NaN
        auto factor = [](uint32_t b) -> uint32_t { return b == (uint32_t)kScaleNan ? 0x7fffu : min(b + 120u, 254u) << 7; };
        auto rest = [](uint32_t b) -> uint32_t { return (b > 134u ? b - 134u + 127u : 127u) << 7; };
        r.f = factor(lo) | factor(hi) << 16;
        r.big = max(lo, hi) > 134u;
        r.more = rest(lo) | rest(hi) << 16;
    }
    return r;
}
template <int KV>
__device__ __forceinline__ Scale2<KV> scale_same(uint32_t b) { return scale_pair<KV>(b, b); }

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// The four codes of a word to two bf16 pairs: codes 0, 1 to `a` and 2, 3 to `b`, the even ones times the
// pair's low scale, the odd ones times the high one.
//   e4m3: the code's sign, exponent and fraction moved to bf16's places are the value times 2^-120 (both formats hold
//   their subnormals alike), which the factor makes up for: exact, five instructions per pair.
//   int8: code + 128 as the low byte of an fp32 number 2^23 + code + 128, less 2^23 + 128, times s.
// `big`: whether the second factors are needed (some scale above 2^7; a caller may ask once for a whole tile).
template <int KV>
__device__ __forceinline__ void codes_to_bf16(uint32_t w, const Scale2<KV> &s, bool big, uint32_t &a, uint32_t &b) {
    if constexpr (KV == kKvE4m3) {
        const uint32_t x = __byte_perm(w, 0u, 0x1404), y = __byte_perm(w, 0u, 0x3424);  // code << 8 per half
        a = mul_bf16x2((x & 0x7f007f00u) >> 4 | (x & 0x80008000u), s.f);
        b = mul_bf16x2((y & 0x7f007f00u) >> 4 | (y & 0x80008000u), s.f);
        if (big) {
            a = mul_bf16x2(a, s.more);
            b = mul_bf16x2(b, s.more);
        }
    } else {
        const uint32_t u = w ^ 0x80808080u;
        float f[4];
        const uint64_t off = tc::pack2(-8388736.f, -8388736.f);
        auto two = [&](uint32_t sel0, uint32_t sel1) {
            return tc::mul2(tc::add2(tc::pack2(__uint_as_float(__byte_perm(u, 0x4b000000u, sel0)),
                                               __uint_as_float(__byte_perm(u, 0x4b000000u, sel1))), off), s.s);
        };
        tc::unpack2(two(0x7440, 0x7441), f[0], f[1]);
        tc::unpack2(two(0x7442, 0x7443), f[2], f[3]);
        a = pack_bf16x2(f[0], f[1]);
        b = pack_bf16x2(f[2], f[3]);
    }
}

// Eight elements of a cache row as bf16.  (16 per lane would be wider loads, but each of a lane's two 16-byte stores would then
// fill half of its 32-byte sectors: 46.6 us where this takes 38.5, for 65536 tokens of 4 e4m3 heads, d = 128.)
template <int KV>
__device__ __forceinline__ uint4 get8(const PagedCache &c, const void *pages, const uint8_t *scales, long long row, int col) {
    if constexpr (KV == kKvBf16) {
        return ld_now(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(pages) + row * c.d + col));
    } else {
        const uint2 w = ld_now(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(pages) + row * c.d + col));
        const Scale2<KV> s = scale_same<KV>(ld_now(scales + row * (c.d / kScaleBlock) + col / kScaleBlock));
        uint4 x;
        codes_to_bf16<KV>(w.x, s, s.big, x.x, x.y);
        codes_to_bf16<KV>(w.y, s, s.big, x.z, x.w);
        return x;
    }
}

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Until all CTAs of the cluster run: before one writes into another's shared memory (no memory is handed over).
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
// Before a CTA ends whose shared memory others read: past it, all have (their values were used; no writes need to be seen).
__device__ __forceinline__ void cluster_leave() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// Address of another CTA's copy of a shared-memory location, and a load from there.
__device__ __forceinline__ uint32_t peer_addr(uint32_t local, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}
__device__ __forceinline__ float2 ld_peer2(uint32_t addr) {
    float2 f;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(f.x), "=f"(f.y) : "r"(addr));
    return f;
}
__device__ __forceinline__ float4 ld_peer4(uint32_t addr) {
    float4 f;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w) : "r"(addr));
    return f;
}

// Two numbers into another CTA's shared memory (seen there past the next cluster_sync()).
__device__ __forceinline__ void st_peer2(uint32_t addr, float2 f) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(f.x), "f"(f.y) : "memory");
}

}  // namespace pi
