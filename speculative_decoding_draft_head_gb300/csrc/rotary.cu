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
// nearest quarter turn, in [-1/8, 1/8] of a turn, goes through short series in fp32: sine
// and cosine are off by less than 2^-23, the turned values by that times their pair's
// size, in fp32; keys are rounded once, to their codes, other rows once, to
// their type.
//
// What bounds it: memory, when large (see the figures at the launches), as long as
// an element costs few instructions; the launch and the chain row -> request ->
// page and position -> angle -> store when small.  A lane takes four pairs, so
// that both halves of a pair are in its registers: two groups of four elements,
// which lie half the turned width apart (halves) or side by side (adjacent).  It
// keeps its row and pairs and goes through the heads, so that their sines and
// cosines are made once and stay in registers.
#include "paged_rows.cuh"

namespace dspark {
namespace {

// Cosine and sine of a 64-bit fraction of a turn.  To the nearest quarter turn r is left, |r| <= 1/8, which is one
// rounding off (2^-24 of it); then the Taylor series of sin(2 pi r) and cos(2 pi r) up to r^9 and r^10, whose rest is
// below 2^-28.  The sine's first factor is in two parts, so that only r's rounding and the last sum's count: off by
// less than 2^-23.6; the cosine's sum of terms, at most 0.3, is some four roundings off: less than 2^-23.2.
__device__ __forceinline__ void turn(uint64_t phase, float &c, float &s) {
    constexpr double t = 6.283185307179586476925286766559, t2 = t * t;
    constexpr float s1 = (float)t, s1_rest = (float)(t - (double)s1);
    constexpr float s3 = (float)(-t * t2 / 6), s5 = (float)(t * t2 * t2 / 120), s7 = (float)(-t * t2 * t2 * t2 / 5040),
                    s9 = (float)(t * t2 * t2 * t2 * t2 / 362880);
    constexpr float c2 = (float)(-t2 / 2), c4 = (float)(t2 * t2 / 24), c6 = (float)(-t2 * t2 * t2 / 720),
                    c8 = (float)(t2 * t2 * t2 * t2 / 40320), c10 = (float)(-t2 * t2 * t2 * t2 * t2 / 3628800);
    const uint32_t hi = (uint32_t)(phase >> 32), quarter = hi + 0x20000000u & 0xc0000000u;
    const float r = (float)(int)(hi - quarter) * 0x1p-32f, r2 = r * r;
    const float sum = fmaf(r2, fmaf(r2, fmaf(r2, fmaf(r2, s9, s7), s5), s3), s1_rest);
    const float s0 = fmaf(r, s1, r * sum);
    const float c0 = fmaf(r2, fmaf(r2, fmaf(r2, fmaf(r2, fmaf(r2, c10, c8), c6), c4), c2), 1.f);
    // a quarter turn on: (c, s) -> (-s, c)
    const bool odd = quarter & 0x40000000u;
    c = __uint_as_float(__float_as_uint(odd ? s0 : c0) ^ (quarter + 0x40000000u & 0x80000000u));
    s = __uint_as_float(__float_as_uint(odd ? c0 : s0) ^ (quarter & 0x80000000u));
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
__device__ __forceinline__ void turn8(float (&x)[8], const float (&c)[4], const float (&s)[4]) {
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

// the angles of a lane's four pairs at a row's positions (or at `at`, where there are none)
__device__ __forceinline__ void angles(const dspark_rotary &z, int pair, const int32_t *positions, int64_t n_rows, int64_t row,
                                       int64_t at, float (&c)[4], float (&s)[4]) {
    const ulonglong2 lo = __ldg(reinterpret_cast<const ulonglong2 *>(z.step + pair));
    const ulonglong2 hi = __ldg(reinterpret_cast<const ulonglong2 *>(z.step + pair) + 1);
    const uint64_t steps[4] = {lo.x, lo.y, hi.x, hi.y};
    if (positions && !z.axis) at = positions[row];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (positions && z.axis) at = positions[axis_of(z, pair + i) * n_rows + row];
        turn((uint64_t)at * steps[i], c[i], s[i]);
    }
}

// ---------------------------------------------------------------- rows alone --
// A block takes `rows` consecutive rows, a thread eight elements of kRowsEach of them,
// `rows` / kRowsEach apart, for every `phases`-th head: four heads at a time, or four rows
// where there are few heads, so that enough loads are under way.  Measured: 60,001 rows of
// 16 heads of 80 bf16 elements, heads first, 51 us (6.0 TB/s, 89% of a copy's rate); 9,000
// rows of 32 heads of 128 fp32 elements 50 us (5.9 TB/s); 200,000 rows of one head of
// 128 bf16 elements 41 us (2.5 TB/s): there the sines and cosines, one for two elements,
// are what bounds it.
constexpr int kRowThreads = 256;
constexpr int kRowUnroll = 4;

struct TurnRows {
    dspark_rotary z;
    int64_t row_stride, head_stride, out_row_stride, out_head_stride;
    const int32_t *positions;
    int n_rows, n_heads, eighths, rows, phases;
    bool inverse;
};

template <typename T, bool kAdjacent, int kRowsEach>
__global__ void __launch_bounds__(kRowThreads)
rotary_rows_kernel(const __grid_constant__ TurnRows a, const T *x, T *out) {     // (may be the same rows)
    constexpr int kHeadsEach = kRowUnroll / kRowsEach;
    const int at = (int)threadIdx.x / a.eighths, eighth = (int)threadIdx.x - at * a.eighths;
    const int every = a.rows / kRowsEach, phase = at / every, row = blockIdx.x * a.rows + at - phase * every;
    if (phase >= a.phases || row >= a.n_rows) return;
    const Eighth e(eighth, a.z.n_pairs, kAdjacent);
    const int64_t begin = row * a.row_stride + phase * a.head_stride + e.off0;
    const T *from = x + begin;
    T *to = out + row * a.out_row_stride + phase * a.out_head_stride + e.off0;
    const int apart = e.off1 - e.off0;
    // item j of a step: row j, or head j
    const int64_t item = kRowsEach > 1 ? every * a.row_stride : a.phases * a.head_stride;
    const int64_t out_item = kRowsEach > 1 ? every * a.out_row_stride : a.phases * a.out_head_stride;
    const int64_t step = kHeadsEach * a.phases * a.head_stride, out_step = kHeadsEach * a.phases * a.out_head_stride;
    auto there = [&](int h, int j) { return kRowsEach > 1 ? row + j * every < a.n_rows : h + j * a.phases < a.n_heads; };
    Four<T> in[kRowUnroll][2];
    auto load = [&](int h) {
#pragma unroll
        for (int j = 0; j < kRowUnroll; ++j)
            if (there(h, j)) in[j][0].load(from + j * item), in[j][1].load(from + j * item + apart);
        from += step;
    };
    load(phase);
    float c[kRowsEach][4], s[kRowsEach][4];
    if (e.pair >= 0) {
#pragma unroll
        for (int j = 0; j < kRowsEach; ++j) {
            if (j > 0 && !there(0, j)) break;
            angles(a.z, e.pair, a.positions, a.n_rows, row + j * every, 0, c[j], s[j]);
            if (a.inverse) {
#pragma unroll
                for (int i = 0; i < 4; ++i) s[j][i] = -s[j][i];
            }
        }
    }
    for (int h = phase; h < a.n_heads; h += kHeadsEach * a.phases) {
        if (h > phase) load(h);
#pragma unroll
        for (int j = 0; j < kRowUnroll; ++j) {
            if (!there(h, j)) break;
            float y[8];
            in[j][0].get(y);
            in[j][1].get(y + 4);
            if (e.pair >= 0) turn8<kAdjacent>(y, c[kRowsEach > 1 ? j : 0], s[kRowsEach > 1 ? j : 0]);
            Four<T>::store(to + j * out_item, y);
            Four<T>::store(to + j * out_item + apart, y + 4);
        }
        to += out_step;
    }
}

// ------------------------------------------------------------ into the cache --
// A group of kLanes lanes (8 for D <= 64, 16 for D <= 128) takes a row and of its
// heads four at a time: of the queries, turned and written; of the keys, turned
// and quantised; of the values, quantised.  Each warp has rows of its own, or
// (`phases` > 1) several warps, of a block and of several, share the steps of the
// same rows.  The one-off work of a quantised head row, its maximum's exchange and two
// divisions, is done for four at once, by a lane each; a step's rows are loaded during
// the one before.
//
// Measured (one GB300, cold caches): 55,000 tokens of 13 prompts, 32 query and 8 kv heads of
// 128 bf16 elements, 201 us (6.3 TB/s, 93% of a copy's rate); with sines and cosines in
// shared memory and made for four rows a block 258 us.  Blocks an SM (by registers): four
// 209 us, five 201, six 209 (spills); of fp32 rows four 352, five 360.  One token of 32
// requests: 6.2 us, of a Python call's 15.
constexpr int kAppendThreads = 128;

struct AppendRotary {
    dspark_kv_cache c;
    PagedRows p;
    dspark_rotary z;
    int64_t q_stride, k_stride, v_stride, q_out_stride, offset;
    const int32_t *positions;
    int n_q_heads, phases;
};

template <typename T, int kFormat, int kLanes, bool kAdjacent>
__global__ void __launch_bounds__(kAppendThreads, sizeof(T) == 4 ? 4 : 5)
kv_append_rotary_kernel(const __grid_constant__ AppendRotary a, const T *q, const T *__restrict__ k,
                        const T *__restrict__ v, T *q_out) {
    constexpr float kTop = kFormat == DSPARK_KV_E4M3 ? 448.f : 127.f;
    constexpr int kGroups = 32 / kLanes;
    const dspark_kv_cache &c = a.c;
    const int lane = threadIdx.x & 31, warp = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    const int sub = lane % kLanes, group = lane / kLanes;
    const int phase = warp % a.phases, first = warp / a.phases * kGroups, r = first + group;
    const int D = c.head_dim, H = c.n_kv_heads, Hq = a.n_q_heads;
    const bool in_row = sub * 8 < D && r < a.p.n_rows;
    const Eighth e(sub, a.z.n_pairs, kAdjacent);
    const int steps_q = (Hq + 3) / 4, steps_kv = (H + 3) / 4, steps = steps_q + 2 * steps_kv;
    if (first >= a.p.n_rows || phase >= steps) return;

    Four<T> in[4][2];
    auto load = [&](int step) {
        const bool is_q = step < steps_q, is_v = step >= steps_q + steps_kv;
        const int heads = is_q ? Hq : H, h0 = 4 * (step - (is_q ? 0 : is_v ? steps_q + steps_kv : steps_q));
        const T *from = is_q ? q + r * a.q_stride : is_v ? v + r * a.v_stride : k + r * a.k_stride;
        from += (int64_t)h0 * D;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (in_row && h0 + j < heads) in[j][0].load(from + j * D + e.off0), in[j][1].load(from + j * D + e.off1);
    };
    load(phase);

    // the row's request, place and position
    int b = -1;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        const int found = first + i < a.p.n_rows ? find_request(a.p.row0, a.p.B, first + i, lane) : -1;
        if (group == i) b = found;
    }
    int64_t place = -1, pos = 0;
    if (b >= 0) {
        const int start = a.p.start[b];
        pos = (int64_t)start + (r - a.p.row0[b]);
        place = start < 0 ? -1 - (int64_t)kFlagBadLength : find_place(a.p, b, pos, c.n_pages, H, c.page_size);
        if (place < 0 && sub == 0 && phase == 0) atomicOr(c.flags, (uint32_t)(-1 - place));
    }
    float cos[4], sin[4];
    if (e.pair >= 0 && b >= 0 && phase < steps_q + steps_kv)
        angles(a.z, e.pair, a.positions, a.p.n_rows, r, pos + a.offset, cos, sin);

    bool nonfinite = false;
    for (int step = phase; step < steps; step += a.phases) {
        const bool is_q = step < steps_q, is_v = step >= steps_q + steps_kv;
        const int heads = is_q ? Hq : H, h0 = 4 * (step - (is_q ? 0 : is_v ? steps_q + steps_kv : steps_q));
        float x[4][8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[j][i] = 0.f;
            if (!in_row || h0 + j >= heads) continue;
            in[j][0].get(x[j]);
            in[j][1].get(x[j] + 4);
        }
        if (step + a.phases < steps) load(step + a.phases);
        if (!is_v && e.pair >= 0 && b >= 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) turn8<kAdjacent>(x[j], cos, sin);
        }
        if (is_q) {
            if (b < 0 || !in_row) continue;
            T *to = q_out + r * a.q_out_stride + (int64_t)h0 * D;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (h0 + j >= heads) break;
                Four<T>::store(to + j * D + e.off0, x[j]);
                Four<T>::store(to + j * D + e.off1, x[j] + 4);
            }
            continue;
        }
        uint32_t tops[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            tops[j] = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) tops[j] = max(tops[j], __float_as_uint(x[j][i]) & 0x7fffffffu);
        }
        __syncwarp();
        const uint32_t top = top_of_row<kLanes>(tops, sub);       // of head h0 + sub % 4
        const bool good = top < 0x7f800000u;
        const float amax = fmaxf(__uint_as_float(top), 0x1p-100f);
        const float mul_of = good ? __fdiv_rn(kTop, amax) : 0.f;
        const int64_t to = place + (int64_t)h0 * c.page_size;     // head row of head h0
        if (sub < 4 && place >= 0 && h0 + sub < heads) {
            nonfinite |= !good;
            (is_v ? c.v_scale : c.k_scale)[to + (int64_t)sub * c.page_size] =
                good ? __fdiv_rn(amax, kTop) : __int_as_float(0x7fffffff);
        }
        unsigned char *codes = static_cast<unsigned char *>(is_v ? c.v : c.k) + to * D;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float mul = __shfl_sync(0xffffffffu, mul_of, j, kLanes);
            if (!in_row || place < 0 || h0 + j >= heads) continue;
            uint2 w;
            w.x = encode4<kFormat>(x[j][0] * mul, x[j][1] * mul, x[j][2] * mul, x[j][3] * mul);
            w.y = encode4<kFormat>(x[j][4] * mul, x[j][5] * mul, x[j][6] * mul, x[j][7] * mul);
            if (mul == 0.f) w = make_uint2(0u, 0u);               // 0 * inf is NaN
            unsigned char *at = codes + (int64_t)j * c.page_size * D;
            *reinterpret_cast<uint32_t *>(at + e.off0) = w.x;
            *reinterpret_cast<uint32_t *>(at + e.off1) = w.y;
        }
    }
    if (nonfinite) atomicOr(c.flags, kFlagNonfinite);
}

template <typename T, int kFormat, int kLanes>
void append_pairs(AppendRotary a, const T *q, const T *k, const T *v, T *q_out, cudaStream_t s) {
    constexpr int kGroups = 32 / kLanes, kBlockWarps = kAppendThreads / 32;
    const int64_t warps = ((int64_t)a.p.n_rows + kGroups - 1) / kGroups;
    // several warps a row while the SMs have room for them, as many as there are steps at most
    const int steps = (a.n_q_heads + 3) / 4 + 2 * ((a.c.n_kv_heads + 3) / 4);
    a.phases = 1;
    while (a.phases < steps && warps * a.phases < 8 * kNumSMs) a.phases *= 2;
    const int blocks = (int)((warps * a.phases + kBlockWarps - 1) / kBlockWarps);
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

template <typename T, int kRowsEach>
void rows_t(const TurnRows &a, const void *x, void *out, cudaStream_t s) {
    const int blocks = (a.n_rows + a.rows - 1) / a.rows;
    const T *from = static_cast<const T *>(x);
    T *to = static_cast<T *>(out);
    if (a.z.adjacent) rotary_rows_kernel<T, true, kRowsEach><<<blocks, kRowThreads, 0, s>>>(a, from, to);
    else rotary_rows_kernel<T, false, kRowsEach><<<blocks, kRowThreads, 0, s>>>(a, from, to);
}

template <typename T>
void rows_each(TurnRows a, const void *x, void *out, cudaStream_t s) {
    // Heads of a row that a block takes side by side: a stretch of 1 KB, where they lie so (the turns of a row are made
    // once for each; fp32 rows of 32 heads of 128 took 60 us without, 50 with four).
    const int bytes = a.eighths * 8 * (int)sizeof(T);
    int side = a.head_stride < a.row_stride ? (1024 + bytes - 1) / bytes : 1;
    side = side < a.n_heads ? side : a.n_heads;
    int most = kRowThreads / (a.eighths * side);
    most = most > 1 ? most : 1;
    // four rows a thread where there are fewer heads, and rows enough for every SM
    const bool rows4 = a.n_heads <= 2 * side && (int64_t)a.n_rows >= (int64_t)most * kRowUnroll * 2 * kNumSMs;
    const int even = (a.n_rows + 2 * kNumSMs - 1) / (2 * kNumSMs);
    const int every = most < even ? most : even;
    a.rows = rows4 ? kRowUnroll * every : every;
    a.phases = kRowThreads / (every * a.eighths);
    a.phases = a.phases < a.n_heads ? a.phases : a.n_heads;
    if (rows4) rows_t<T, kRowUnroll>(a, x, out, s);
    else rows_t<T, 1>(a, x, out, s);
}

}  // namespace

cudaError_t launch_rotary_rows(const RotaryRowsArgs &g, cudaStream_t s) {
    const TurnRows a{g.z, g.row_stride, g.head_stride, g.out_row_stride, g.out_head_stride, g.positions,
                     g.n_rows, g.n_heads, g.head_dim / 8, 1, 1, g.inverse};
    if (g.dt == DSPARK_BF16) rows_each<__nv_bfloat16>(a, g.x, g.out, s);
    else if (g.dt == DSPARK_F16) rows_each<__half>(a, g.x, g.out, s);
    else rows_each<float>(a, g.x, g.out, s);
    return cudaGetLastError();
}

cudaError_t launch_kv_append_rotary(const AppendRotaryArgs &g, cudaStream_t s) {
    const AppendRotary a{g.cache, g.rows, g.z, g.q_stride, g.k_stride, g.v_stride, g.q_out_stride, g.offset,
                         g.positions, g.q ? g.n_q_heads : 0, 1};
    if (g.dt == DSPARK_BF16) append_t<__nv_bfloat16>(a, g.q, g.k, g.v, g.q_out, s);
    else if (g.dt == DSPARK_F16) append_t<__half>(a, g.q, g.k, g.v, g.q_out, s);
    else append_t<float>(a, g.q, g.k, g.v, g.q_out, s);
    return cudaGetLastError();
}

}  // namespace dspark
