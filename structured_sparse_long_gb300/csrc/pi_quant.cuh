// pi_quant.cuh -- elements to the codes of an 8-bit cache row (pi_paged.cuh has the format), and bf16 to fp32.
#pragma once

#include "pi_paged.cuh"

namespace pi {

__device__ __forceinline__ void unpack8(const uint4 &x, float (&f)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
}

// Eight elements to eight codes, given the block's scale exponent: each is rounded once.
template <int KV>
__device__ __forceinline__ uint2 encode_codes(const float (&x)[8], int e) {
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);  // 2^-e, -e in [-122, 120]
    uint32_t o[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float *y = x + 4 * i;
        if (KV == kKvE4m3) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0] * inv, y[1] * inv), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2] * inv, y[3] * inv), __NV_SATFINITE, __NV_E4M3);
            o[i] = lo | hi << 16;
        } else {
            // in 2^23 .. 2^24 the step is 1: the sum's rounding is the code's, and its low byte the code
            uint32_t c[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) c[j] = __float_as_uint(fmaf(y[j], inv, 12582912.f));
            o[i] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
        }
    }
    return make_uint2(o[0], o[1]);
}

}  // namespace pi
