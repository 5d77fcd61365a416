// pi_paged.cuh -- the paged key/value cache: where a position's row is, and what an 8-bit row holds.
//
// Position p of sequence b is row p % page of page table[b][p / page]; a page holds, per KV head,
// `page` rows of d elements ([n_pages][Hkv][page][d]).  An 8-bit row keeps, per block of 32
// elements, codes c and one byte s standing for the scale 2^(s - 127): element = c * 2^(s - 127).
// The scale is the smallest power of two, at least 2^-120, that brings the block's largest
// magnitude to at most 448 (e4m3) or 127 (int8).  A power of two scales exactly, so a code is the
// element rounded once (half a step of the code's own grid), and c * 2^(s - 127) is a bf16 number:
// an e4m3 code has 4 significant bits and an int8 code at most 7, and with scales of 2^-120 or more the
// smallest code, 2^-9 * 2^-120, is still a multiple of bf16's smallest 2^-133 (an element above
// 0.96 * 2^128 may round up to 2^128, which reads as an infinity).  A block with an
// infinity or a NaN gets the byte 255 (NaN) and reads back as NaN.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "pi_common.cuh"
#include "pi_paged.h"
#include "pi_plan.cuh"

namespace pi {

constexpr int kScaleBlock = 32;       // elements per scale byte
constexpr int kScaleNan = 255;        // byte of a block with a non-finite element
constexpr int kMinScaleExp = -120;

// A load of what the kernel before this one may have written.  These kernels start before that one ends (programmatic launch, and
// griddepcontrol.wait before the first load), so nothing is constant for a kernel's life, as the non-coherent loads of __ldg
// want it; those could also be moved above the wait.  (Written out: as C++ loads, single tokens over int8 caches, d = 64, take
// 4 % longer.)
template <typename T>
__device__ __forceinline__ T ld_now(const T *p) {
    static_assert(sizeof(T) == 1 || sizeof(T) == 2 || sizeof(T) == 4 || sizeof(T) == 8 || sizeof(T) == 16, "one load");
    if constexpr (sizeof(T) <= 4) {
        uint32_t x;
        if constexpr (sizeof(T) == 1) asm volatile("ld.global.u8 %0, [%1];" : "=r"(x) : "l"(p));
        else if constexpr (sizeof(T) == 2) asm volatile("{.reg .u16 t; ld.global.u16 t, [%1]; cvt.u32.u16 %0, t;}" : "=r"(x) : "l"(p));
        else asm volatile("ld.global.u32 %0, [%1];" : "=r"(x) : "l"(p));
        if constexpr (sizeof(T) == 4) return *reinterpret_cast<T *>(&x);
        else return (T)x;
    } else if constexpr (sizeof(T) == 8) {
        T r;
        asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(*reinterpret_cast<uint32_t *>(&r.x)), "=r"(*reinterpret_cast<uint32_t *>(&r.y)) : "l"(p));
        return r;
    } else {
        T r;
        asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
        return r;
    }
}

__device__ __forceinline__ void record_index(int *word) { atomicCAS(word, kStatusOk, kStatusIndex); }

// Row of the cache (of the [n_pages * Hkv * page] rows) that holds position pos of sequence b for
// KV head 0, or -1 for a page-table entry outside the pool.  pos must be inside [0, width * page).
__device__ __forceinline__ int page_of(const PagedCache &c, const int *table, long long b, int pos) {
    const int pg = ld_now(table + b * c.width + (pos >> c.page_log2));
    return (unsigned)pg < (unsigned)c.n_pages ? pg : -1;
}
__device__ __forceinline__ int row_in_page(const PagedCache &c, int pg, int g, int pos) {
    return ((pg * c.Hkv + g) << c.page_log2) + (pos & (c.page - 1));
}

// 2^(byte - 127) as fp32 (255: NaN).
__device__ __forceinline__ float scale_of(int byte) {
    return byte == kScaleNan ? __int_as_float(0x7fffffff) : __int_as_float(byte << 23);
}

// Exponent e of a block's scale 2^e from its largest magnitude (finite, >= 0): the smallest
// e >= kMinScaleExp with amax <= Q * 2^e.  448 = 1.75 * 2^8 and 127 = 1.984375 * 2^6, so e follows
// from amax's exponent and from whether its significand exceeds Q's.
template <int KV>
__device__ __forceinline__ int scale_exp(float amax) {
    const uint32_t u = __float_as_uint(amax);
    constexpr uint32_t kTop = KV == kKvE4m3 ? 0x600000u : 0x7e0000u;  // fraction bits of 1.75, 1.984375
    constexpr int kUp = KV == kKvE4m3 ? 8 : 6;
    const int e = (int)(u >> 23) - 127 - kUp + ((u & 0x7fffffu) > kTop ? 1 : 0);
    return max(e, kMinScaleExp);  // subnormal amax: far below the floor of the scales
}

// The number of j in [1, B] with below(j), which holds up to some j and for none after: with below(j) = (cu[j] <= t)
// the sequence of packed token t (B: t is behind the last one).  Searched by the whole warp, 32 probes at a time; ends, with
// every probe in [1, B], whatever below() answers.
template <typename F>
__device__ __forceinline__ int find_sequence(int B, F below) {
    const int lane = threadIdx.x & 31;
    SearchRange r(B);
    while (r.len > 0) r.narrow(__popc(__ballot_sync(0xffffffffu, r.inside(lane) && below(r.place(lane)))));
    return r.lo;
}

// Whether a sequence's offsets and context are in range: its tokens inside the batch, its rows inside
// its page table.
__device__ __forceinline__ bool sequence_ok(const PagedCache &c, const PagedBatch &bt, int t0, int t1, int ctx) {
    return t0 >= 0 && t0 <= t1 && t1 <= bt.T && ctx >= 0 && (long long)ctx + (t1 - t0) <= (long long)c.width << c.page_log2;
}

// Position of packed token t in its sequence b, or -1 (t behind the last sequence, or an index out of
// range, which is recorded).  For the whole warp.
__device__ __forceinline__ int locate(const PagedCache &c, const PagedBatch &bt, int t, int &b, int *index_word) {
    b = find_sequence(bt.B, [&](int j) { return ld_now(bt.cu + j) <= t; });
    if (b >= bt.B) return -1;
    const int t0 = ld_now(bt.cu + b), t1 = ld_now(bt.cu + b + 1), ctx = ld_now(bt.ctx + b);
    if (!sequence_ok(c, bt, t0, t1, ctx) || t < t0 || t >= t1) {
        record_index(index_word);
        return -1;
    }
    return ctx + t - t0;
}

}  // namespace pi
