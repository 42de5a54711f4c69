// The quantised key/value cache: writing new rows and reading rows back.
//
// Both kernels move bytes: 2 D elements in and 2 D codes out per (token, kv
// head), or the reverse, with a handful of instructions per element, so what
// bounds a large call is the memory and what bounds a small one is the chain
// row -> request -> page -> token.  A block takes kRows packed rows: its warps
// look the rows' places up once, then groups of lanes take one head row each
// (8 elements a lane: 16-byte loads of bf16/fp16, 8-byte stores of codes, both
// whole lines per head row) with several head rows in flight.
#include "paged_rows.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

// places of the block's rows: smem[i] for row r0 + i (see find_place), or
// kNoRow when the row belongs to no request
constexpr int64_t kNoRow = INT64_MIN;
template <int kRows>
__device__ __forceinline__ void block_places(int64_t *place, const PagedRows &p, int r0, int n_pages, int n_kv_heads,
                                             int page_size, uint32_t *flags) {
    const int lane = threadIdx.x & 31;
    for (int i = threadIdx.x >> 5; i < kRows; i += kThreads / 32) {
        const int r = r0 + i;
        int64_t at = kNoRow;
        if (r < p.n_rows) {
            const int b = find_request(p.row0, p.B, r, lane);
            if (b >= 0) {
                const int64_t pos = (int64_t)p.start[b] + (r - p.row0[b]);
                at = p.start[b] < 0 ? -1 - (int64_t)kFlagBadLength
                                    : find_place(p, b, pos, n_pages, n_kv_heads, page_size);
                if (at < 0 && lane == 0) atomicOr(flags, (uint32_t)(-1 - at));
            }
        }
        if (lane == 0) place[i] = at;
    }
    __syncthreads();
}

// 8 consecutive elements as fp32
template <typename T>
struct Eight {
    uint4 w;
    __device__ __forceinline__ void load(const T *p) { w = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = pair_to_float<T>(u[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
};
template <>
struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = __ldg(reinterpret_cast<const float4 *>(p));
        b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
};

// kLanes lanes per head row: 8 (D <= 64) or 16 (D <= 128)
template <typename T, int kFormat, int kLanes, int kRows>
__global__ void __launch_bounds__(kThreads)
kv_append_kernel(dspark_kv_cache c, PagedRows p, const T *__restrict__ k, const T *__restrict__ v, int64_t k_stride,
                 int64_t v_stride) {
    constexpr float kTop = kFormat == DSPARK_KV_E4M3 ? 448.f : 127.f;
    __shared__ int64_t place[kRows];
    const int r0 = blockIdx.x * kRows;
    block_places<kRows>(place, p, r0, c.n_pages, c.n_kv_heads, c.page_size, c.flags);

    const int sub = threadIdx.x % kLanes, D = c.head_dim;
    const int units = kRows * c.n_kv_heads * 2;
    constexpr int kGroups = kThreads / kLanes;
    bool nonfinite = false;
    for (int u0 = threadIdx.x / kLanes; u0 < units; u0 += kGroups * kUnroll) {
        Eight<T> in[kUnroll];
        int64_t at[kUnroll];
        int kv[kUnroll];
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            const int u = u0 + j * kGroups;
            const int i = u % kRows, hk = u / kRows, h = hk >> 1;
            kv[j] = hk & 1;
            at[j] = u < units ? place[i] : -1;
            if (at[j] < 0) continue;
            at[j] += (int64_t)h * c.page_size;
            if (sub * 8 < D)
                in[j].load((kv[j] ? v + (r0 + i) * v_stride : k + (r0 + i) * k_stride) + (int64_t)h * D + sub * 8);
        }
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            float x[8] = {};
            uint32_t top = 0;  // the bits of |x| order like the values, NaN above inf
            if (at[j] >= 0 && sub * 8 < D) {
                in[j].get(x);
#pragma unroll
                for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
            }
#pragma unroll
            for (int d = kLanes / 2; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
            if (at[j] < 0) continue;
            const bool good = top < 0x7f800000u;
            const float amax = fmaxf(__uint_as_float(top), 0x1p-100f);
            const float mul = good ? __fdiv_rn(kTop, amax) : 0.f;
            nonfinite |= !good;
            if (sub * 8 < D) {
                uint2 w = make_uint2(0u, 0u);
                if (good) {
                    w.x = encode2<kFormat>(x[0] * mul, x[1] * mul) | (encode2<kFormat>(x[2] * mul, x[3] * mul) << 16);
                    w.y = encode2<kFormat>(x[4] * mul, x[5] * mul) | (encode2<kFormat>(x[6] * mul, x[7] * mul) << 16);
                }
                unsigned char *codes = static_cast<unsigned char *>(kv[j] ? c.v : c.k);
                *reinterpret_cast<uint2 *>(codes + at[j] * D + sub * 8) = w;
            }
            if (sub == 0)
                (kv[j] ? c.v_scale : c.k_scale)[at[j]] = good ? __fdiv_rn(amax, kTop) : __int_as_float(0x7fffffff);
        }
    }
    if (nonfinite) atomicOr(c.flags, kFlagNonfinite);
}

template <typename T, int kFormat, int kLanes, int kRows>
__global__ void __launch_bounds__(kThreads)
kv_read_kernel(dspark_kv_cache c, PagedRows p, T *__restrict__ k_out, T *__restrict__ v_out) {
    __shared__ int64_t place[kRows];
    const int r0 = blockIdx.x * kRows;
    block_places<kRows>(place, p, r0, c.n_pages, c.n_kv_heads, c.page_size, c.flags);

    const int sub = threadIdx.x % kLanes, D = c.head_dim;
    const int units = kRows * c.n_kv_heads * 2;
    constexpr int kGroups = kThreads / kLanes;
    for (int u0 = threadIdx.x / kLanes; u0 < units; u0 += kGroups * kUnroll) {
        uint2 in[kUnroll];
        float scale[kUnroll];
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            const int u = u0 + j * kGroups;
            const int i = u % kRows, hk = u / kRows, h = hk >> 1;
            in[j] = make_uint2(0u, 0u);
            scale[j] = __int_as_float(0x7fffffff);
            if (u >= units || place[i] < 0 || sub * 8 >= D) continue;
            const int64_t at = place[i] + (int64_t)h * c.page_size;
            const unsigned char *codes = static_cast<const unsigned char *>((hk & 1) ? c.v : c.k);
            in[j] = __ldg(reinterpret_cast<const uint2 *>(codes + at * D + sub * 8));
            scale[j] = __ldg(((hk & 1) ? c.v_scale : c.k_scale) + at);
        }
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            const int u = u0 + j * kGroups;
            const int i = u % kRows, hk = u / kRows, h = hk >> 1;
            T *out = (hk & 1) ? v_out : k_out;
            if (u >= units || place[i] == kNoRow || sub * 8 >= D || !out) continue;
            out += ((int64_t)(r0 + i) * c.n_kv_heads + h) * D + sub * 8;
            __half2 g[4];
            decode4<kFormat>(in[j].x, g[0], g[1]);
            decode4<kFormat>(in[j].y, g[2], g[3]);
            float x[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = __half22float2(g[e]);
                x[2 * e] = f.x * scale[j];
                x[2 * e + 1] = f.y * scale[j];
            }
            if constexpr (sizeof(T) == 4) {
                reinterpret_cast<float4 *>(out)[0] = make_float4(x[0], x[1], x[2], x[3]);
                reinterpret_cast<float4 *>(out)[1] = make_float4(x[4], x[5], x[6], x[7]);
            } else {
                *reinterpret_cast<uint4 *>(out) =
                    make_uint4(float_to_pair<T>(x[0], x[1]), float_to_pair<T>(x[2], x[3]),
                               float_to_pair<T>(x[4], x[5]), float_to_pair<T>(x[6], x[7]));
            }
        }
    }
}

// Rows a block takes: 8 once that still gives every SM a few blocks, else 1 so
// that a small call spreads over the SMs.
constexpr int kManyRows = 8;
bool many_rows(int n_rows) { return n_rows >= 4 * kManyRows * kNumSMs; }

template <typename T, int kFormat, int kLanes>
void append_rows(const dspark_kv_cache &c, const PagedRows &p, const void *k, const void *v, int64_t ks, int64_t vs,
                 cudaStream_t s) {
    const T *kt = static_cast<const T *>(k), *vt = static_cast<const T *>(v);
    if (many_rows(p.n_rows))
        kv_append_kernel<T, kFormat, kLanes, kManyRows>
            <<<(p.n_rows + kManyRows - 1) / kManyRows, kThreads, 0, s>>>(c, p, kt, vt, ks, vs);
    else
        kv_append_kernel<T, kFormat, kLanes, 1><<<p.n_rows, kThreads, 0, s>>>(c, p, kt, vt, ks, vs);
}

template <typename T, int kFormat, int kLanes>
void read_rows(const dspark_kv_cache &c, const PagedRows &p, void *k, void *v, cudaStream_t s) {
    T *kt = static_cast<T *>(k), *vt = static_cast<T *>(v);
    if (many_rows(p.n_rows))
        kv_read_kernel<T, kFormat, kLanes, kManyRows>
            <<<(p.n_rows + kManyRows - 1) / kManyRows, kThreads, 0, s>>>(c, p, kt, vt);
    else
        kv_read_kernel<T, kFormat, kLanes, 1><<<p.n_rows, kThreads, 0, s>>>(c, p, kt, vt);
}

template <typename T>
void append_t(const dspark_kv_cache &c, const PagedRows &p, const void *k, const void *v, int64_t ks, int64_t vs,
              cudaStream_t s) {
    const bool e4m3 = c.format == DSPARK_KV_E4M3, narrow = c.head_dim <= 64;
    if (e4m3 && narrow) append_rows<T, DSPARK_KV_E4M3, 8>(c, p, k, v, ks, vs, s);
    else if (e4m3) append_rows<T, DSPARK_KV_E4M3, 16>(c, p, k, v, ks, vs, s);
    else if (narrow) append_rows<T, DSPARK_KV_INT8, 8>(c, p, k, v, ks, vs, s);
    else append_rows<T, DSPARK_KV_INT8, 16>(c, p, k, v, ks, vs, s);
}

template <typename T>
void read_t(const dspark_kv_cache &c, const PagedRows &p, void *k, void *v, cudaStream_t s) {
    const bool e4m3 = c.format == DSPARK_KV_E4M3, narrow = c.head_dim <= 64;
    if (e4m3 && narrow) read_rows<T, DSPARK_KV_E4M3, 8>(c, p, k, v, s);
    else if (e4m3) read_rows<T, DSPARK_KV_E4M3, 16>(c, p, k, v, s);
    else if (narrow) read_rows<T, DSPARK_KV_INT8, 8>(c, p, k, v, s);
    else read_rows<T, DSPARK_KV_INT8, 16>(c, p, k, v, s);
}

}  // namespace

cudaError_t launch_kv_append(const dspark_kv_cache &c, const PagedRows &p, const void *k, const void *v,
                             int64_t k_stride, int64_t v_stride, dspark_dtype dt, cudaStream_t s) {
    if (dt == DSPARK_BF16) append_t<__nv_bfloat16>(c, p, k, v, k_stride, v_stride, s);
    else if (dt == DSPARK_F16) append_t<__half>(c, p, k, v, k_stride, v_stride, s);
    else append_t<float>(c, p, k, v, k_stride, v_stride, s);
    return cudaGetLastError();
}

cudaError_t launch_kv_read(const dspark_kv_cache &c, const PagedRows &p, dspark_dtype dt, void *k_out, void *v_out,
                           cudaStream_t s) {
    if (dt == DSPARK_BF16) read_t<__nv_bfloat16>(c, p, k_out, v_out, s);
    else if (dt == DSPARK_F16) read_t<__half>(c, p, k_out, v_out, s);
    else read_t<float>(c, p, k_out, v_out, s);
    return cudaGetLastError();
}

}  // namespace dspark
