// What the attention kernels over the quantised cache share: a request's rows
// and lengths, and the arithmetic of a softmax in powers of two whose reference
// follows each row's largest term with its value's scale.
#pragma once

#include "paged_rows.cuh"

namespace dspark {

constexpr float kVUp = 0x1p12f, kVDown = 0x1p-12f;   // what value scales are multiplied by, and its inverse
constexpr float kVLeast = -88.f;           // log2 of the least of these that the reference counts: value scales
                                           // below 2^-100 lose precision, not range
constexpr float kPeak = 7.f;               // log2 of P's largest bound when the reference moves ...
constexpr uint32_t kPast = 0x7c00u;        // ... which it does when a P reaches these bits, fp16's infinity,
constexpr float kSumMost = 0x1p105f;       // or when 32 terms of l sum to more than this

struct Request {
    int64_t first;
    int n, len;
    bool rows_ok, len_ok;
};

__device__ __forceinline__ Request load_request(const AttentionArgs &a, int b) {
    Request q;
    const int64_t lo = a.rows.row0[b], hi = a.rows.row0[b + 1];
    q.first = lo;
    q.rows_ok = lo >= 0 && hi >= lo && hi <= a.rows.n_rows;
    q.n = q.rows_ok ? (int)(hi - lo) : 0;
    q.len = a.rows.start[b];
    q.len_ok = q.len >= q.n && (int64_t)q.len <= (int64_t)a.rows.max_pages * a.cache.page_size &&
               !(a.row_mask && q.n > 64);
    return q;
}

// ---------------------------------------------------------- packed fp32 pairs --
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &x, float &y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ uint32_t half_pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}
// x * 2^d for a whole d <= 0 (or -inf), in two steps: references lie up to some 200 apart, and what is far
// below a new one can be of any size in l
__device__ __forceinline__ float scale_down(float x, float d) {
    const float a = fmaxf(d, -120.f);
    return x * fast_exp2(a) * fast_exp2(d - a);
}

}  // namespace dspark
