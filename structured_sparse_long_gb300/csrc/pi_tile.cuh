// pi_tile.cuh -- a softmax row's work on one 32-key tile, and launch-constant division: shared by the
// tensor-core forwards.
#pragma once

#include <cstdint>

#include "pi_tc_ptx.cuh"

namespace pi {
namespace tc {

constexpr int CHUNK = 32;                 // keys per tile (TMA box rows; the N of the S products)
// A row's reference m is set this much (log2 units) above its largest logit so far, and moves, with O rescaled, once a logit exceeds
// it.  P is then at most 1, so that the unnormalised O is at most the sum of the values' magnitudes: it overflows only where
// values reach fp32's largest over the row's number of keys.  (Set to the maximum and left to lag behind by as much, P reached
// 2^12, and a band of 300 values of 2^112 overflowed.)  A relative weight is lost below 2^-114 at the latest, 2^-126 being
// the smallest P.  A row's first tile may hold a single key, so a smaller distance makes rescales common: 8 took C4
// 242 us, the fused gate C8 270 us and a 16384-token chunk over bf16 pages 76 us, 12 takes 237, 254 and 70 us, 16 and 24 the
// same.
constexpr float kHeadroom = 12.f;
constexpr float kRescaleSum = 1.f;  // a tile's sum of P above this is the first sign of a logit above the reference

// Phase 1 of a tile for one row (general path): mask the scores outside [clo, chi] and return
// the tile's largest logit in log2 units (prior included).  A skip tile holds at most one
// valid column per row (its diagonal), read with a select tree instead of a full pass.
__device__ __forceinline__ float tile_max(float *f, int clo, int chi, bool skip, float sc, float off) {
    if (skip) {
        if (clo > chi) return -INFINITY;
        return fmaf(select32(f, clo), sc, off);
    }
    if (!__all_sync(0xffffffffu, clo <= 0 && chi >= 31)) {
#pragma unroll
        for (int c = 0; c < 32; ++c) f[c] = (c >= clo && c <= chi) ? f[c] : -INFINITY;
    }
    // four independent partial maxima: a short dependency chain
    float m0 = max3(f[0], f[1], f[2]), m1 = max3(f[3], f[4], f[5]);
    float m2 = max3(f[6], f[7], f[8]), m3 = max3(f[9], f[10], f[11]);
#pragma unroll
    for (int c = 12; c < 28; c += 8) {
        m0 = max3(m0, f[c], f[c + 1]);
        m1 = max3(m1, f[c + 2], f[c + 3]);
        m2 = max3(m2, f[c + 4], f[c + 5]);
        m3 = max3(m3, f[c + 6], f[c + 7]);
    }
    m0 = max3(m0, f[28], f[29]);
    m1 = max3(m1, f[30], f[31]);
    const float mx = fmaxf(max3(m0, m1, m2), m3);
    return (mx == -INFINITY) ? -INFINITY : fmaf(mx, sc, off);
}

// P = exp2(s * sc + bo) for a tile's 32 raw scores, packed as 16 bf16 pairs in place (word
// c/2 is written after scores c and c+1 were read); returns the sum of the fp32 values.
// Masked scores (-inf) give exactly 0.
__device__ __forceinline__ float tile_exp(uint32_t *r, float sc, float bo) {
    const uint64_t sc2 = pack2(sc, sc), bo2 = pack2(bo, bo);
    uint64_t acc0 = pack2(0.f, 0.f), acc1 = pack2(0.f, 0.f);  // two independent sums
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
        float z0, z1;
        unpack2(fma2(pack2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), sc2, bo2), z0, z1);
        const float p0 = fast_exp2(z0);
        const float p1 = fast_exp2(z1);
        if ((c >> 1) & 1) acc1 = add2(acc1, pack2(p0, p1));
        else acc0 = add2(acc0, pack2(p0, p1));
        r[c / 2] = pack_bf16(p0, p1);
    }
    float a0, a1, b0, b1;
    unpack2(acc0, a0, a1);
    unpack2(acc1, b0, b1);
    return (a0 + a1) + (b0 + b1);
}

// Skip tile: P is zero except column clo, exp2(zdiag - mu); packed into words 0-15.
__device__ __forceinline__ float tile_exp_diag(uint32_t *r, int clo, float zdiag, float mu) {
    const float p = (clo < CHUNK) ? fast_exp2(zdiag - mu) : 0.f;
    __nv_bfloat16 hb = __float2bfloat16_rn(p);
    const uint32_t bits = (uint32_t)(*reinterpret_cast<uint16_t *>(&hb));
    const uint32_t word = (clo & 1) ? (bits << 16) : bits;
#pragma unroll
    for (int w = 0; w < 16; ++w) r[w] = (w == (clo >> 1)) ? word : 0u;
    return p;
}

// Largest of a tile's 32 raw scores (four independent chains).
__device__ __forceinline__ float tile_raw_max(const uint32_t *r) {
    float m[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) m[k] = max3(__uint_as_float(r[k]), __uint_as_float(r[k + 4]), __uint_as_float(r[k + 8]));
#pragma unroll
    for (int c = 12; c < 28; c += 8) {
#pragma unroll
        for (int k = 0; k < 4; ++k) m[k] = max3(m[k], __uint_as_float(r[c + k]), __uint_as_float(r[c + 4 + k]));
    }
    m[0] = max3(m[0], __uint_as_float(r[28]), __uint_as_float(r[29]));
    m[1] = max3(m[1], __uint_as_float(r[30]), __uint_as_float(r[31]));
    return fmaxf(max3(m[0], m[1], m[2]), m[3]);
}

// Division by a divisor fixed for the launch, as a multiply and a shift (Granlund and
// Montgomery, "Division by invariant integers using multiplication", 1994: with
// l = ceil(log2 d) and m = floor(2^(32+l) / d) + 1, floor(n / d) = floor(n m / 2^(32+l)) for
// every 32-bit n).  The dividends here are below 2^31, so n * m (m < 2^33) fits 64 bits.
struct FastDiv {
    uint64_t m;
    int sh;
    __device__ __forceinline__ int div(int n) const {
        return (int)(((unsigned long long)(unsigned)n * m) >> sh);
    }
};
static inline FastDiv make_fastdiv(int d) {
    int l = 0;
    while ((1LL << l) < (long long)d) ++l;
    const unsigned __int128 num = (unsigned __int128)1 << (32 + l);
    FastDiv f;
    f.m = (uint64_t)(num / (unsigned)d) + 1;
    f.sh = 32 + l;
    return f;
}

}  // namespace tc
}  // namespace pi
