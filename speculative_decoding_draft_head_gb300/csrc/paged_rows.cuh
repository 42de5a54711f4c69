// Packed rows, pages and 8-bit codes: device helpers of the cache and the
// attention kernels.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "device_common.cuh"
#include "internal.h"

namespace dspark {

// The request of packed row r: the largest b with row0[b] <= r, found by the
// whole warp (32 probes a round, so two rounds up to 1024 requests); -1 when
// row r belongs to none.  Reads row0[0 .. B] only, whatever its values.
__device__ __forceinline__ int find_request(const int64_t *__restrict__ row0, int B, int64_t r, int lane) {
    int lo = 0, n = B;
    while (true) {
        const int step = (n + 31) / 32;
        const int i = lane * step;
        const bool at_or_before = i < n && row0[lo + i] <= r;
        const unsigned hits = __ballot_sync(0xffffffffu, at_or_before);
        if (hits == 0) return -1;
        const int k = 31 - __clz(hits);
        lo += k * step;
        n = min(step, n - k * step);
        if (step == 1) break;
    }
    return (r < row0[lo + 1]) ? lo : -1;
}

// Where a token's codes are, in units of head rows: head h of the token is
// head row place + h * page_size of the cache's arrays.  -1 - flag when it has
// no place.
__device__ __forceinline__ int64_t find_place(const PagedRows &p, int b, int64_t pos, int n_pages, int n_kv_heads,
                                              int page_size) {
    if (pos < 0 || pos >= (int64_t)p.max_pages * page_size) return -1 - (int64_t)kFlagBadLength;
    const int slot = (int)pos / page_size;
    const int page = p.block_table[(int64_t)b * p.max_pages + slot];
    if (page < 0 || page >= n_pages) return -1 - (int64_t)kFlagBadPage;
    return (int64_t)page * n_kv_heads * page_size + ((int)pos - slot * page_size);
}

// ------------------------------------------------------------ 8-bit codes --
// Four codes to two pairs of fp16, exactly.
template <int kFormat>
__device__ __forceinline__ void decode4(uint32_t c, __half2 &a, __half2 &b) {
    if constexpr (kFormat == DSPARK_KV_E4M3) {
        uint32_t x, y;
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
            : "=r"(x), "=r"(y)
            : "r"(c));
        a = *reinterpret_cast<__half2 *>(&x);
        b = *reinterpret_cast<__half2 *>(&y);
    } else {
        // the byte u = code + 128 under the fp16 bits 0x64.. is 1024 + u
        c ^= 0x80808080u;
        uint32_t x = __byte_perm(c, 0x64646464u, 0x4140), y = __byte_perm(c, 0x64646464u, 0x4342);
        const __half2 off = __float2half2_rn(1152.f);
        a = __hsub2(*reinterpret_cast<__half2 *>(&x), off);
        b = __hsub2(*reinterpret_cast<__half2 *>(&y), off);
    }
}

// Four values, already scaled into [-Q, Q], to four codes (nearest, ties to
// even).
template <int kFormat>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    if constexpr (kFormat == DSPARK_KV_E4M3) {
        uint32_t r;
        asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
            : "=r"(r)
            : "f"(a), "f"(b), "f"(c), "f"(d));
        return r;
    } else {
        // at 1.5 * 2^23 a float's steps are 1, and the low byte of its bits is
        // the rounded value's (|x| stays below 127.5: x * (127 / amax) is off
        // by less than 127 * 2^-23)
        const float off = 0x1.8p23f;
        const uint32_t x = __float_as_uint(__fadd_rn(a, off)), y = __float_as_uint(__fadd_rn(b, off));
        const uint32_t z = __float_as_uint(__fadd_rn(c, off)), w = __float_as_uint(__fadd_rn(d, off));
        return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
    }
}

template <typename T>
__device__ __forceinline__ float2 pair_to_float(uint32_t w);
template <>
__device__ __forceinline__ float2 pair_to_float<__nv_bfloat16>(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 pair_to_float<__half>(uint32_t w) {
    return __half22float2(*reinterpret_cast<__half2 *>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t float_to_pair(float a, float b);
template <>
__device__ __forceinline__ uint32_t float_to_pair<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t float_to_pair<__half>(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// The largest of top[j] over a head row's lanes, for the head row j = sub % 4:
// the first two exchanges halve what a lane holds, the others join the rest.
template <int kLanes>
__device__ __forceinline__ uint32_t top_of_row(const uint32_t (&top)[4], int sub) {
    const bool b0 = sub & 1, b1 = sub & 2;
    uint32_t lo = b0 ? top[1] : top[0], hi = b0 ? top[3] : top[2];
    lo = max(lo, __shfl_xor_sync(0xffffffffu, b0 ? top[0] : top[1], 1));
    hi = max(hi, __shfl_xor_sync(0xffffffffu, b0 ? top[2] : top[3], 1));
    uint32_t t = max(b1 ? hi : lo, __shfl_xor_sync(0xffffffffu, b1 ? lo : hi, 2));
#pragma unroll
    for (int d = 4; d < kLanes; d *= 2) t = max(t, __shfl_xor_sync(0xffffffffu, t, d));
    return t;
}

}  // namespace dspark
