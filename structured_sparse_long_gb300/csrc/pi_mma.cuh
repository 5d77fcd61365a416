// pi_mma.cuh -- warp-level building blocks of the paged cache's attention: the 16 x 8 x 16 bf16 matrix
// product, 8-bit codes to bf16 pairs, and loads across a cluster.
#pragma once

#include <cstdint>

#include "pi_paged.cuh"

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

// 16 bytes that are read once: past L1.
__device__ __forceinline__ uint4 ldg_stream(const uint4 *p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}

// Scales of the two codes of a pair, from their bytes.
struct Scale2 {
    float lo, hi;
};
__device__ __forceinline__ Scale2 scale_pair(uint32_t lo, uint32_t hi) { return Scale2{scale_of((int)lo), scale_of((int)hi)}; }
__device__ __forceinline__ Scale2 scale_same(uint32_t b) { return scale_pair(b, b); }

// The four codes of a word to two bf16 pairs: codes 0, 1 to `a` and 2, 3 to `b`, the even ones times
// s.lo, the odd ones times s.hi.
template <int KV>
__device__ __forceinline__ void codes_to_bf16(uint32_t w, const Scale2 &s, uint32_t &a, uint32_t &b) {
    float f[4];
    if (KV == kKvE4m3) {
        const __half2_raw h0 = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
        const __half2_raw h1 = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
        const float2 x = __half22float2(__half2(h0)), y = __half22float2(__half2(h1));
        f[0] = x.x; f[1] = x.y; f[2] = y.x; f[3] = y.y;
    } else {
        // 2^23 + (code + 128) from its bits, less 2^23 + 128
        const uint32_t u = w ^ 0x80808080u;
        const float off = 8388608.f + 128.f;
        f[0] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440)) - off;
        f[1] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7441)) - off;
        f[2] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7442)) - off;
        f[3] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7443)) - off;
    }
    a = pack_bf16x2(f[0] * s.lo, f[1] * s.hi);
    b = pack_bf16x2(f[2] * s.lo, f[3] * s.hi);
}

// Contiguous bytes (a multiple of 16, both addresses 16-byte aligned) into shared memory, counted on an mbarrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
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

}  // namespace pi
