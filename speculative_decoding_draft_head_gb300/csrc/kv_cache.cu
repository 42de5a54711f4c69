// The quantised key/value cache: writing new rows and reading rows back.
//
// Both kernels move bytes: 2 D elements in and 2 D codes out per (token, kv
// head), or the reverse.  What bounds a large call is the memory, as long as an
// element costs few instructions; what bounds a small one is its launch and the
// chain row -> request -> page -> token (append of 32 tokens: 3.1 us on the
// device, of a Python call's 7.5 us).  A block takes some packed rows: its warps look
// the rows' places up once, then groups of lanes take one head row each (8
// elements a lane: 16-byte loads of bf16/fp16, 8-byte stores of codes, both
// whole lines per head row) with several head rows in flight.
#include "paged_rows.cuh"

namespace dspark {
namespace {

// Threads a block (the kernels alone, on the prompts and contexts below): writing
// takes 128 us with 128 and 136 us with 256; reading is as fast with either, 116
// us with 256 and 114 us with 128.
constexpr int kAppendThreads = 128;
constexpr int kReadThreads = 256;

// places of the block's rows: smem[i] for row r0 + i (see find_place), or
// kNoRow when the row belongs to no request
constexpr int64_t kNoRow = INT64_MIN;
template <int kRows, int kThreads>
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

// 8 consecutive elements; top() is the largest |x| as the bits of a float:
// those order like the values, with infinities and NaN above all numbers
template <typename T>
struct Eight {
    uint4 w;
    __device__ __forceinline__ void clear() { w = make_uint4(0u, 0u, 0u, 0u); }
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
    __device__ __forceinline__ uint32_t top() const {
        // two values a word: the 16-bit types' bits order like their values too
        const uint32_t m = 0x7fff7fffu;
        const uint32_t t = __vmaxu2(__vmaxu2(w.x & m, w.y & m), __vmaxu2(w.z & m, w.w & m));
        const float2 f = pair_to_float<T>(t);
        return max(__float_as_uint(f.x), __float_as_uint(f.y));
    }
};
template <>
struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void load(const float *p) {
        a = __ldg(reinterpret_cast<const float4 *>(p));
        b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    __device__ __forceinline__ uint32_t top() const {
        float x[8];
        get(x);
        uint32_t t = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) t = max(t, __float_as_uint(x[e]) & 0x7fffffffu);
        return t;
    }
};

// Writing.  A group of kLanes lanes (8 for D <= 64, 16 for D <= 128) takes four
// head rows at a time, 8 elements a lane: with kMany the same head of four
// rows, else four heads of the block's only row.  The next four are loaded as
// each is done with, the first while the places are looked up.
//
// What bounds a large call after the memory is the issue of instructions, so
// the work that is one a head row, its maximum's exchange and two divisions,
// is done for four head rows at once, by a lane each: 125,000 tokens of 8 heads
// of 128 bf16 elements take 130 us a call (6.0 TB/s, 88% of a copy's rate) and took
// 220 us with that work done by every lane; fp32 elements 184 us (7.0 TB/s).
template <typename T, int kFormat, int kLanes, bool kMany>
__global__ void __launch_bounds__(kAppendThreads)
kv_append_kernel(dspark_kv_cache c, PagedRows p, const T *__restrict__ k, const T *__restrict__ v, int64_t k_stride,
                 int64_t v_stride) {
    constexpr float kTop = kFormat == DSPARK_KV_E4M3 ? 448.f : 127.f;
    constexpr int kGroups = 32 / kLanes, kRows = kMany ? 4 * kGroups : 1;
    __shared__ int64_t place[kRows];
    const int r0 = blockIdx.x * kRows, warp = threadIdx.x >> 5;
    const int sub = threadIdx.x % kLanes, group = threadIdx.x % 32 / kLanes;
    const int D = c.head_dim, H = c.n_kv_heads;
    const bool in_row = sub * 8 < D;
    // head row j of a step is head hk(j) (keys' heads, then values') of row i(j)
    const int step = kAppendThreads / 32 * (kMany ? 1 : 4 * kGroups);
    auto row = [&](int j) { return kMany ? j * kGroups + group : 0; };
    auto head = [&](int at, int j) { return kMany ? at : at + j * kGroups + group; };
    Eight<T> in[4];
    auto load = [&](int at, int j) {
        const int hk = head(at, j), r = r0 + row(j);
        in[j].clear();
        if (hk < 2 * H && r < p.n_rows && in_row)
            in[j].load((hk < H ? k + r * k_stride + (int64_t)hk * D : v + r * v_stride + (int64_t)(hk - H) * D) + sub * 8);
    };
    int at = warp * (kMany ? 1 : 4 * kGroups);
#pragma unroll
    for (int j = 0; j < 4; ++j) load(at, j);
    block_places<kRows, kAppendThreads>(place, p, r0, c.n_pages, H, c.page_size, c.flags);

    bool nonfinite = false;
    for (; at < 2 * H; at += step) {
        uint32_t tops[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) tops[j] = in[j].top();
        const uint32_t top = top_of_row<kLanes>(tops, sub);
        const bool good = top < 0x7f800000u;
        const float amax = fmaxf(__uint_as_float(top), 0x1p-100f);
        const float mul_of = good ? __fdiv_rn(kTop, amax) : 0.f;
        if (sub < 4) {
            const int hk = head(at, sub);
            const int64_t to = place[row(sub)];
            if (hk < 2 * H && to >= 0) {
                nonfinite |= !good;
                (hk < H ? c.k_scale : c.v_scale)[to + (int64_t)(hk < H ? hk : hk - H) * c.page_size] =
                    good ? __fdiv_rn(amax, kTop) : __int_as_float(0x7fffffff);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float mul = __shfl_sync(0xffffffffu, mul_of, j, kLanes);
            const int hk = head(at, j);
            const int64_t to = place[row(j)];
            float x[8];
            in[j].get(x);
            load(at + step, j);
            if (hk >= 2 * H || to < 0 || !in_row) continue;
            uint2 w;
            w.x = encode4<kFormat>(x[0] * mul, x[1] * mul, x[2] * mul, x[3] * mul);
            w.y = encode4<kFormat>(x[4] * mul, x[5] * mul, x[6] * mul, x[7] * mul);
            if (mul == 0.f) w = make_uint2(0u, 0u);  // 0 * inf is NaN
            unsigned char *codes = static_cast<unsigned char *>(hk < H ? c.k : c.v);
            *reinterpret_cast<uint2 *>(codes + (to + (int64_t)(hk < H ? hk : hk - H) * c.page_size) * D + sub * 8) = w;
        }
    }
    if (nonfinite) atomicOr(c.flags, kFlagNonfinite);
}

// Reading.  A group of lanes takes kUnroll head rows at a time; 119,000 tokens
// of 8 heads of 128 elements to bf16 take 119 us a call (6.2 TB/s, 91% of a copy's
// rate; the kernel alone 116 us with 16 rows a block and 8 in flight, 120 us with
// 8 and 4).  125,000 tokens to fp32 take 238 us (5.4 TB/s): four of the five bytes
// that such a call moves are written.
constexpr int kUnroll = 8;
template <typename T, int kFormat, int kLanes, int kRows>
__global__ void __launch_bounds__(kReadThreads)
kv_read_kernel(dspark_kv_cache c, PagedRows p, T *__restrict__ k_out, T *__restrict__ v_out) {
    __shared__ int64_t place[kRows];
    const int r0 = blockIdx.x * kRows;
    block_places<kRows, kReadThreads>(place, p, r0, c.n_pages, c.n_kv_heads, c.page_size, c.flags);

    const int sub = threadIdx.x % kLanes, D = c.head_dim;
    const int units = kRows * c.n_kv_heads * 2;
    constexpr int kGroups = kReadThreads / kLanes;
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

// Several rows a block, or one so that a small call spreads over the SMs.  A block of several rows works through
// its heads one after the other, so that the crossing lies the higher the wider a row is.  Measured, cold caches
// (one / several rows a block, us):
//   writing bf16  D = 128, 1 head: 1,200 rows 5.2 / 5.0, 4,864 rows 11.2 / 5.8
//                 D = 128, 8 heads: 2,400 rows 8.4 / 9.6, 4,864 rows 13.3 / 10.9
//                 D = 128, 32 heads: 4,864 rows 26.5 / 30.0, 9,728 rows 48.2 / 42.3
//                 D = 64: 1 head 2,400 rows 7.5 / 6.7, 8 heads 4,864 rows 11.7 / 10.1, 32 heads 9,728 rows 30.0 / 31.0
//   writing fp32  D = 128, 8 heads: 1,200 rows 8.2 / 9.9, 2,400 rows 11.6 / 10.3
//   reading bf16  D = 128: 1 head 300 rows 5.1 / 5.2, 8 heads 600 rows 8.0 / 7.8, 32 heads 1,200 rows 12.1 / 19.1 and
//                 2,400 rows 19.4 / 18.9;  D = 64: 8 heads 600 rows 7.7 / 6.3, 32 heads 1,200 rows 10.8 / 10.8
//   reading fp32  D = 128, 8 heads: 600 rows 8.2 / 10.1, 1,200 rows 11.0 / 10.1
constexpr int kReadRows = 16;
template <typename T>
bool append_many(int n_rows, int rows, int heads) {     // `rows`: of a block
    return (int64_t)n_rows * (sizeof(T) == 4 ? 6 : 4) >= (int64_t)(3 * rows + 6 * heads) * kNumSMs;
}
template <typename T>
bool read_many(int n_rows, int heads, int D) {
    return (int64_t)n_rows * 1024 >= (1536 + 2 * (int64_t)heads * D * (int64_t)sizeof(T)) * kNumSMs;
}

template <typename T, int kFormat, int kLanes>
void append_rows(const dspark_kv_cache &c, const PagedRows &p, const void *k, const void *v, int64_t ks, int64_t vs,
                 cudaStream_t s) {
    const T *kt = static_cast<const T *>(k), *vt = static_cast<const T *>(v);
    constexpr int kRows = 128 / kLanes;
    if (append_many<T>(p.n_rows, kRows, c.n_kv_heads))
        kv_append_kernel<T, kFormat, kLanes, true>
            <<<(p.n_rows + kRows - 1) / kRows, kAppendThreads, 0, s>>>(c, p, kt, vt, ks, vs);
    else
        kv_append_kernel<T, kFormat, kLanes, false><<<p.n_rows, kAppendThreads, 0, s>>>(c, p, kt, vt, ks, vs);
}

template <typename T, int kFormat, int kLanes>
void read_rows(const dspark_kv_cache &c, const PagedRows &p, void *k, void *v, cudaStream_t s) {
    T *kt = static_cast<T *>(k), *vt = static_cast<T *>(v);
    if (read_many<T>(p.n_rows, c.n_kv_heads, c.head_dim))
        kv_read_kernel<T, kFormat, kLanes, kReadRows>
            <<<(p.n_rows + kReadRows - 1) / kReadRows, kReadThreads, 0, s>>>(c, p, kt, vt);
    else
        kv_read_kernel<T, kFormat, kLanes, 1><<<p.n_rows, kReadThreads, 0, s>>>(c, p, kt, vt);
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
