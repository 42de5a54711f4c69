// Rotary positions: rows turned by the angles of their positions, alone or on
// the way into the quantised cache.
//
// Mathematics.  Pair i of a head, (a, b), at position p of its axis becomes
// (a cos t - b sin t, b cos t + a sin t) with t = p w_i.  Only t modulo a full
// turn counts, so an angle is kept in turns as a 64-bit fraction: the step of
// one position, w_i / 2 pi in units of 2^-64 turns, times the position, modulo
// 2^64, is one integer product that wraps where the angle does.  Its error is
// |p| 2^-65 turns, so 2^-34 turns at the last 31-bit position, where the fp32
// product p w_i would be off by hundreds of radians.  What is left after the
// nearest quarter turn, in [-1/8, 1/8] of a turn, goes to sincospi in fp32: sine and
// cosine are off by a few 2^-25, the turned values by that times their pair's
// size, in fp32; keys are rounded once, to their codes, other rows once, to
// their type.
//
// What bounds it: memory, when large (see the figures at the launches); the
// launch and the chain row -> request -> page and position -> angle -> store
// when small.  A block takes a few rows; its threads make each row's sines and
// cosines once, in shared memory, for all heads.  A lane takes four pairs, so
// that both halves of a pair are in its registers: two groups of four elements,
// which lie half the turned width apart (halves) or side by side (adjacent).
#include "paged_rows.cuh"

namespace dspark {
namespace {

// cosine and sine of a 64-bit fraction of a turn
__device__ __forceinline__ void turn(uint64_t phase, float &c, float &s) {
    const uint32_t hi = (uint32_t)(phase >> 32);
    const uint32_t quarter = (hi + 0x20000000u) >> 30;            // to the nearest
    float c0, s0;
    sincospif((float)(int)(hi - (quarter << 30)) * 0x1p-31f, &s0, &c0);
    const float x = (quarter & 1) ? s0 : c0, y = (quarter & 1) ? c0 : s0;
    c = (quarter == 1 || quarter == 2) ? -x : x;
    s = quarter >= 2 ? -y : y;
}

// A lane's eight elements of a head row: four first and four second partners
// (or, beyond the turned width, eight that pass), as two groups of four at
// off[0] and off[1].
struct Eighth {
    int off0, off1, pair;     // pair: the first of the four, -1: none
    __device__ __forceinline__ Eighth(int i, int n_pairs, bool adjacent) {
        const bool turned = i < n_pairs / 4;
        pair = turned ? 4 * i : -1;
        off0 = adjacent ? 8 * i : turned ? 4 * i : 2 * n_pairs + 8 * (i - n_pairs / 4);
        off1 = turned && !adjacent ? n_pairs + 4 * i : off0 + 4;
    }
};

template <typename T>
struct Four {
    uint2 w;
    __device__ __forceinline__ void load(const T *p) { w = __ldg(reinterpret_cast<const uint2 *>(p)); }
    __device__ __forceinline__ void get(float *x) const {
        const float2 a = pair_to_float<T>(w.x), b = pair_to_float<T>(w.y);
        x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
    }
    static __device__ __forceinline__ void store(T *p, const float *x) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(float_to_pair<T>(x[0], x[1]), float_to_pair<T>(x[2], x[3]));
    }
};
template <>
struct Four<float> {
    float4 w;
    __device__ __forceinline__ void load(const float *p) { w = __ldg(reinterpret_cast<const float4 *>(p)); }
    __device__ __forceinline__ void get(float *x) const { x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w; }
    static __device__ __forceinline__ void store(float *p, const float *x) {
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    }
};

// eight elements in the order of memory, their pairs turned
template <bool kAdjacent>
__device__ __forceinline__ void turn8(float (&x)[8], const float *cos, const float *sin) {
    const float4 c4 = *reinterpret_cast<const float4 *>(cos), s4 = *reinterpret_cast<const float4 *>(sin);
    const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int ia = kAdjacent ? 2 * i : i, ib = kAdjacent ? 2 * i + 1 : i + 4;
        const float a = x[ia], b = x[ib];
        x[ia] = a * c[i] - b * s[i];
        x[ib] = b * c[i] + a * s[i];
    }
}

__device__ __forceinline__ int axis_of(const dspark_rotary &z, int pair) {
    return z.axis ? min(max(z.axis[pair], 0), z.n_axes - 1) : 0;
}

// ---------------------------------------------------------------- rows alone --
// A block takes `rows` consecutive rows of every head.  Its items, eight elements
// each, lie in the order of memory: by head inside a row, or by row inside a head.
constexpr int kRowThreads = 256;
constexpr int kRowUnroll = 4;

struct TurnRows {
    dspark_rotary z;
    int64_t row_stride, head_stride, out_row_stride, out_head_stride;
    const int32_t *positions;
    int n_rows, n_heads, head_dim, rows;
    bool inverse, rows_inside;      // rows_inside: a head's rows lie closer than a row's heads
};

template <typename T, bool kAdjacent>
__global__ void __launch_bounds__(kRowThreads)
rotary_rows_kernel(const __grid_constant__ TurnRows a, const T *x, T *out) {     // (may be the same rows)
    extern __shared__ __align__(16) float table[];      // [rows][n_pairs] cosines, then sines
    const int n_pairs = a.z.n_pairs, r0 = blockIdx.x * a.rows, rows = min(a.rows, a.n_rows - r0);
    float *cos = table, *sin = table + a.rows * n_pairs;
    for (int i = threadIdx.x; i < rows * n_pairs; i += kRowThreads) {
        const int row = i / n_pairs, pair = i - row * n_pairs;
        const int p = a.positions[(int64_t)axis_of(a.z, pair) * a.n_rows + r0 + row];
        float c, s;
        turn((uint64_t)(int64_t)p * a.z.step[pair], c, s);
        cos[i] = c;
        sin[i] = a.inverse ? -s : s;
    }
    __syncthreads();
    const int eighths = a.head_dim / 8, inner = a.rows_inside ? rows : a.n_heads;
    const int items = rows * a.n_heads * eighths;
    for (int i0 = threadIdx.x; i0 < items; i0 += kRowThreads * kRowUnroll) {
        Four<T> in[kRowUnroll][2];
        int64_t to[kRowUnroll];
        int at[kRowUnroll];             // of the cosines, -1: the elements pass
        int apart[kRowUnroll];
#pragma unroll
        for (int j = 0; j < kRowUnroll; ++j) {
            const int i = i0 + j * kRowThreads;
            if (i >= items) continue;
            const int hr = i / eighths, outer = hr / inner, in_at = hr - outer * inner;
            const int row = a.rows_inside ? in_at : outer, head = a.rows_inside ? outer : in_at;
            const Eighth e(i - hr * eighths, n_pairs, kAdjacent);
            const T *from = x + (r0 + row) * a.row_stride + head * a.head_stride + e.off0;
            to[j] = (r0 + row) * a.out_row_stride + head * a.out_head_stride + e.off0;
            apart[j] = e.off1 - e.off0;
            at[j] = e.pair < 0 ? -1 : row * n_pairs + e.pair;
            in[j][0].load(from);
            in[j][1].load(from + apart[j]);
        }
#pragma unroll
        for (int j = 0; j < kRowUnroll; ++j) {
            if (i0 + j * kRowThreads >= items) continue;
            float y[8];
            in[j][0].get(y);
            in[j][1].get(y + 4);
            if (at[j] >= 0) turn8<kAdjacent>(y, cos + at[j], sin + at[j]);
            Four<T>::store(out + to[j], y);
            Four<T>::store(out + to[j] + apart[j], y + 4);
        }
    }
}

// ------------------------------------------------------------ into the cache --
// A block takes `rows` packed rows.  A warp takes steps of four head rows a group
// of kLanes lanes (8 for D <= 64, 16 for D <= 128): of the queries, turned and
// written; of the keys, turned and quantised; of the values, quantised.  The
// one-off work of a quantised head row, its maximum's exchange and two divisions, is
// done for four at once, by a lane each.
constexpr int kAppendThreads = 128;
constexpr int kAppendRows = 4;          // most rows a block

struct AppendRotary {
    dspark_kv_cache c;
    PagedRows p;
    dspark_rotary z;
    int64_t q_stride, k_stride, v_stride, q_out_stride, offset;
    const int32_t *positions;
    int n_q_heads, rows;
};

template <typename T, int kFormat, int kLanes, bool kAdjacent>
__global__ void __launch_bounds__(kAppendThreads)
kv_append_rotary_kernel(const __grid_constant__ AppendRotary a, const T *q, const T *__restrict__ k,
                        const T *__restrict__ v, T *q_out) {
    constexpr float kTop = kFormat == DSPARK_KV_E4M3 ? 448.f : 127.f;
    constexpr int kGroups = 32 / kLanes, kPairs = kLanes * 4;     // pairs at most
    __shared__ __align__(16) float cos[kAppendRows * kPairs], sin[kAppendRows * kPairs];
    __shared__ int64_t place[kAppendRows], position[kAppendRows];
    __shared__ int known[kAppendRows];                            // the row belongs to a request
    const dspark_kv_cache &c = a.c;
    const int r0 = blockIdx.x * a.rows, rows = min(a.rows, a.p.n_rows - r0), lane = threadIdx.x & 31;
    const int D = c.head_dim, H = c.n_kv_heads, n_pairs = a.z.n_pairs;
    for (int i = threadIdx.x >> 5; i < rows; i += kAppendThreads / 32) {
        const int r = r0 + i, b = find_request(a.p.row0, a.p.B, r, lane);
        int64_t at = -1, pos = 0;
        if (b >= 0) {
            const int start = a.p.start[b];
            pos = (int64_t)start + (r - a.p.row0[b]);
            at = start < 0 ? -1 - (int64_t)kFlagBadLength : find_place(a.p, b, pos, c.n_pages, H, c.page_size);
            if (at < 0 && lane == 0) atomicOr(c.flags, (uint32_t)(-1 - at));
        }
        if (lane == 0) place[i] = at, position[i] = pos + a.offset, known[i] = b >= 0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < rows * n_pairs; i += kAppendThreads) {
        const int row = i / n_pairs, pair = i - row * n_pairs;
        int64_t at = position[row];
        if (a.positions) at = a.positions[(int64_t)axis_of(a.z, pair) * a.p.n_rows + r0 + row];
        turn((uint64_t)at * a.z.step[pair], cos[row * kPairs + pair], sin[row * kPairs + pair]);
    }
    __syncthreads();

    const int sub = lane % kLanes, group = lane / kLanes;
    const bool in_row = sub * 8 < D;
    const Eighth e(sub, n_pairs, kAdjacent);
    const int Hq = a.n_q_heads;
    constexpr int kStep = 4 * kGroups;                            // head rows of a warp's step
    const int steps_q = (rows * Hq + kStep - 1) / kStep, steps_kv = (rows * H + kStep - 1) / kStep;
    bool nonfinite = false;
    for (int step = threadIdx.x >> 5; step < steps_q + 2 * steps_kv; step += kAppendThreads / 32) {
        const bool is_q = step < steps_q, is_v = step >= steps_q + steps_kv;
        const int heads = is_q ? Hq : H, first = (step - (is_q ? 0 : is_v ? steps_q + steps_kv : steps_q)) * kStep;
        const float per_head = 1.f / (float)heads;
        const T *from = is_q ? q : is_v ? v : k;
        const int64_t stride = is_q ? a.q_stride : is_v ? a.v_stride : a.k_stride;
        int row[4], head[4];
        Four<T> in[4][2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = first + j * kGroups + group;
            row[j] = (int)(((float)i + 0.5f) * per_head);         // exact: i is far below 2^22
            head[j] = i - row[j] * heads;
            if (row[j] >= rows) row[j] = -1;
            if (row[j] < 0 || !in_row) continue;
            const T *at = from + (r0 + row[j]) * stride + (int64_t)head[j] * D;
            in[j][0].load(at + e.off0);
            in[j][1].load(at + e.off1);
        }
        float x[4][8];
        uint32_t tops[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            tops[j] = 0;
            if (row[j] < 0 || !in_row) continue;
            in[j][0].get(x[j]);
            in[j][1].get(x[j] + 4);
            if (!is_v && e.pair >= 0) turn8<kAdjacent>(x[j], cos + row[j] * kPairs + e.pair, sin + row[j] * kPairs + e.pair);
#pragma unroll
            for (int i = 0; i < 8; ++i) tops[j] = max(tops[j], __float_as_uint(x[j][i]) & 0x7fffffffu);
        }
        if (is_q) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (row[j] < 0 || !in_row || !known[row[j]]) continue;
                T *to = q_out + (r0 + row[j]) * a.q_out_stride + (int64_t)head[j] * D;
                Four<T>::store(to + e.off0, x[j]);
                Four<T>::store(to + e.off1, x[j] + 4);
            }
            continue;
        }
        const uint32_t top = top_of_row<kLanes>(tops, sub);       // of head row sub % 4
        const bool good = top < 0x7f800000u;
        const float amax = fmaxf(__uint_as_float(top), 0x1p-100f);
        const float mul_of = good ? __fdiv_rn(kTop, amax) : 0.f;
        if (sub < 4) {
            int my_row = row[0], my_head = head[0];
#pragma unroll
            for (int j = 1; j < 4; ++j)
                if (sub == j) my_row = row[j], my_head = head[j];
            if (my_row >= 0 && place[my_row] >= 0) {
                nonfinite |= !good;
                (is_v ? c.v_scale : c.k_scale)[place[my_row] + (int64_t)my_head * c.page_size] =
                    good ? __fdiv_rn(amax, kTop) : __int_as_float(0x7fffffff);
            }
        }
        unsigned char *codes = static_cast<unsigned char *>(is_v ? c.v : c.k);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float mul = __shfl_sync(0xffffffffu, mul_of, j, kLanes);
            if (row[j] < 0 || !in_row || place[row[j]] < 0) continue;
            uint2 w;
            w.x = encode4<kFormat>(x[j][0] * mul, x[j][1] * mul, x[j][2] * mul, x[j][3] * mul);
            w.y = encode4<kFormat>(x[j][4] * mul, x[j][5] * mul, x[j][6] * mul, x[j][7] * mul);
            if (mul == 0.f) w = make_uint2(0u, 0u);               // 0 * inf is NaN
            unsigned char *to = codes + (place[row[j]] + (int64_t)head[j] * c.page_size) * D;
            *reinterpret_cast<uint32_t *>(to + e.off0) = w.x;
            *reinterpret_cast<uint32_t *>(to + e.off1) = w.y;
        }
    }
    if (nonfinite) atomicOr(c.flags, kFlagNonfinite);
}

template <typename T, int kFormat, int kLanes>
void append_pairs(const AppendRotary &a, const T *q, const T *k, const T *v, T *q_out, cudaStream_t s) {
    const int blocks = (a.p.n_rows + a.rows - 1) / a.rows;
    if (a.z.adjacent)
        kv_append_rotary_kernel<T, kFormat, kLanes, true><<<blocks, kAppendThreads, 0, s>>>(a, q, k, v, q_out);
    else
        kv_append_rotary_kernel<T, kFormat, kLanes, false><<<blocks, kAppendThreads, 0, s>>>(a, q, k, v, q_out);
}

template <typename T>
void append_t(const AppendRotary &a, const void *q, const void *k, const void *v, void *q_out, cudaStream_t s) {
    const T *qt = static_cast<const T *>(q), *kt = static_cast<const T *>(k), *vt = static_cast<const T *>(v);
    T *ot = static_cast<T *>(q_out);
    const bool e4m3 = a.c.format == DSPARK_KV_E4M3, narrow = a.c.head_dim <= 64;
    if (e4m3 && narrow) append_pairs<T, DSPARK_KV_E4M3, 8>(a, qt, kt, vt, ot, s);
    else if (e4m3) append_pairs<T, DSPARK_KV_E4M3, 16>(a, qt, kt, vt, ot, s);
    else if (narrow) append_pairs<T, DSPARK_KV_INT8, 8>(a, qt, kt, vt, ot, s);
    else append_pairs<T, DSPARK_KV_INT8, 16>(a, qt, kt, vt, ot, s);
}

template <typename T>
void rows_t(const TurnRows &a, const void *x, void *out, int blocks, size_t smem, cudaStream_t s) {
    if (a.z.adjacent)
        rotary_rows_kernel<T, true><<<blocks, kRowThreads, smem, s>>>(a, static_cast<const T *>(x), static_cast<T *>(out));
    else
        rotary_rows_kernel<T, false><<<blocks, kRowThreads, smem, s>>>(a, static_cast<const T *>(x), static_cast<T *>(out));
}

}  // namespace

cudaError_t launch_rotary_rows(const RotaryRowsArgs &g, cudaStream_t s) {
    // rows a block: two rounds of its threads' items, fewer where that would leave SMs without a block
    const int per_row = g.n_heads * (g.head_dim / 8);
    int rows = 2 * kRowThreads * kRowUnroll / per_row;
    const int even = (g.n_rows + 2 * kNumSMs - 1) / (2 * kNumSMs), fit = (32 << 10) / (g.z.n_pairs * 8);
    rows = rows < even ? rows : even;
    rows = rows < fit ? rows : fit;
    if (rows < 1) rows = 1;
    const TurnRows a{g.z, g.row_stride, g.head_stride, g.out_row_stride, g.out_head_stride, g.positions,
                     g.n_rows, g.n_heads, g.head_dim, rows, g.inverse, g.row_stride < g.head_stride};
    const int blocks = (g.n_rows + rows - 1) / rows;
    const size_t smem = (size_t)rows * g.z.n_pairs * 2 * sizeof(float);
    if (g.dt == DSPARK_BF16) rows_t<__nv_bfloat16>(a, g.x, g.out, blocks, smem, s);
    else if (g.dt == DSPARK_F16) rows_t<__half>(a, g.x, g.out, blocks, smem, s);
    else rows_t<float>(a, g.x, g.out, blocks, smem, s);
    return cudaGetLastError();
}

cudaError_t launch_kv_append_rotary(const AppendRotaryArgs &g, cudaStream_t s) {
    const int rows = g.rows.n_rows >= 4 * kAppendRows * kNumSMs ? kAppendRows : 1;
    const AppendRotary a{g.cache, g.rows, g.z, g.q_stride, g.k_stride, g.v_stride, g.q_out_stride, g.offset,
                         g.positions, g.q ? g.n_q_heads : 0, rows};
    if (g.dt == DSPARK_BF16) append_t<__nv_bfloat16>(a, g.q, g.k, g.v, g.q_out, s);
    else if (g.dt == DSPARK_F16) append_t<__half>(a, g.q, g.k, g.v, g.q_out, s);
    else append_t<float>(a, g.q, g.k, g.v, g.q_out, s);
    return cudaGetLastError();
}

}  // namespace dspark
