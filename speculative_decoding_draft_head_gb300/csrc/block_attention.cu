// Attention of each request's block rows over a shared prefix and the
// request's own tokens, both in the quantised cache.
//
// Mathematics.  Row m (a block row of a query head) against tokens j, with 8-bit
// codes k~, v~ and scales ks, vs: x_j = ks_j (q . k~_j), s_j = c x_j in log2
// units, and with any reference r
//   O = sum_j [2^(s_j - r) vs_j] v~_j,   l = sum_j 2^(s_j - r),   out = O / l,
//   lse = ln 2 (r + log2 l).
// The bracket is the fp16 operand P of the second product, so r follows
// max_j s_j + log2 vs_j (an integer, moved only when P would pass 2^15 of
// fp16's 2^16, then starting again at 2^7; O is scaled by an exact power of
// two).  Codes are exact in fp16 and so is q after a power-of-two scaling per
// row (exact to 2^-32 of the row's largest element), hence both products run
// on fp16 tensor cores with fp32 sums, and the only rounding of the inner
// terms is P's, 2^-11.  Neither scale is folded into codes: that would round
// every key and value.
//
// One CTA per SM walks its part of the plan's line of tiles (attention_plan.h),
// 128 tokens a tile.  Roles (16 warps):
//   0-7   two softmax groups of 128 threads, a thread per row (TMEM lane)
//   8-11  converters: raw codes -> fp16 operands in the swizzled layout
//   12    producer: plans pieces, loads codes and scales (cp.async.bulk)
//   13    issues the tensor-core products;  14, 15  load and scale q
// A piece of more than 128 rows gives each softmax group 128 rows of the same
// tokens; one of fewer rows gives the groups alternate tiles of the same rows,
// joined at the end, so that one group's softmax always runs under the other's
// products.  Every wait is bounded.
#include "attention_plan.h"
#include "paged_rows.cuh"
#include "tc_primitives.cuh"

namespace dspark {
namespace {

using namespace tc;

constexpr int kThreads = 512;
constexpr int kCtas = kNumSMs;
constexpr int kPieces = 4;        // piece descriptors in flight
constexpr int kScaleSlots = 4;    // tiles whose scales are held
constexpr long long kSpinLimit = 4000000000LL;  // ~2 s of clock cycles
constexpr long long kDrainLimit = 200000000LL;  // ~0.1 s: copies and products in flight after a timeout

constexpr uint32_t kColS = 0, kColO = 256;  // TMEM columns: scores (and P) of the groups, then their outputs

constexpr float kScaleFloor = 0x1p-100f;   // value scales below it lose precision, not range
constexpr float kPeak = 7.f;               // log2 of P's largest bound when the reference moves
constexpr float kSlack = 15.f;             // ... and the bound at which it has to

enum { kDirect = 0, kFirst = 1, kContinued = 2 };

// Shared memory: operands first (1024-byte aligned for the swizzle)
template <int DP>
struct Layout {
    static constexpr int kOps = DP == 128 ? 3 : 4;    // fp16 operand ring (K and V tiles)
    static constexpr int kRaw = DP == 128 ? 3 : 6;    // ring of tiles as loaded
    static constexpr uint32_t kTileBytes = 128 * DP * 2;
    static constexpr uint32_t kRawBytes = 128 * DP + 1024;  // codes; with the keys both scales
    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kOp = kQ + 2 * kTileBytes;
    static constexpr uint32_t kRawAt = kOp + kOps * kTileBytes;
    static constexpr uint32_t kScale = kRawAt + kRaw * kRawBytes;        // [slots][ks 128, vs 128]
    static constexpr uint32_t kQScale = kScale + kScaleSlots * 1024;     // [pieces][256]
    static constexpr uint32_t kStats = kQScale + kPieces * 1024;         // [2][128] (r, l)
    static constexpr uint32_t kBytes = kStats + 2048 + 1024;             // + alignment slack
};

struct Piece {
    int tiles;          // tiles of this piece, 0: no more pieces
    int first;          // its first tile of the item
    int rows, m0;       // rows of the row tile, and their first
    int row_base;       // packed row of the item's row 0
    int head;           // kv head
    int len;            // tokens of the list
    int ctx;            // tokens every row sees
    int n;              // block rows (own tokens)
    int request;        // -1: the prefix
    int out;            // kDirect, kFirst, kContinued
    int pad;
};

// Device workspace: where partial results go
struct Partials {
    int64_t *unit0;     // [B] first own unit of each request
    float2 *stats;      // (r, l): [R Hq] prefix, [R Hq] own, [kCtas][256] continued
    float *o;           // the same rows of D unnormalised outputs
};

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

__device__ __forceinline__ int prefix_rows(const AttentionArgs &a) {
    const int64_t r = a.rows.row0[a.rows.B];
    return r < 0 ? 0 : r > a.rows.n_rows ? a.rows.n_rows : (int)r;
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
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
__device__ __forceinline__ float fast_exp2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t half_pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}

// Bounded wait of a whole warp on one barrier.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort) {
    const bool ok = mbar_wait(bar, parity, abort, kSpinLimit);
    return __all_sync(0xffffffffu, ok);
}

// Steps of a piece in the order its operands are loaded, converted and used:
// step s is tile s' of K or V.  Row halves (pair): K0 V0 K1 V1 ..; alternate
// tiles: K0 K1 V0 K2 V1 .., one key tile ahead, as the products need them.
__device__ __forceinline__ void step_of(int s, int tiles, bool pair, bool &is_v, int &j) {
    if (pair) {
        is_v = s & 1;
        j = s >> 1;
    } else if (s == 0) {
        is_v = false;
        j = 0;
    } else if (s == 2 * tiles - 1) {
        is_v = true;
        j = tiles - 1;
    } else {
        is_v = !(s & 1);
        j = is_v ? s / 2 - 1 : (s + 1) / 2;
    }
}

// ------------------------------------------------------------------ the plan --
// Walks a CTA's pieces (one warp, all lanes alike).
struct Walk {
    const AttentionArgs &a;
    int lane, group, prefix_m, prefix_tiles;
    int64_t prefix_head, prefix_total, u, hi;
    // the item at the cursor
    int b, head, rt, m, tiles;
    int64_t start;
    // 32 requests' sizes, a lane each, from request wb on
    int wb, w_n, w_len;
    int64_t w_first;

    __device__ __forceinline__ void window(int from) {
        wb = from;
        w_n = 0;
        if (from + lane < a.rows.B) {
            const Request q = load_request(a, from + lane);
            w_n = q.len_ok ? q.n : 0;
            w_len = q.len;
            w_first = q.first;
        }
    }
    // the next request with rows, from b on; false when there is none
    __device__ __forceinline__ bool seek() {
        while (b < a.rows.B) {
            if (b >= wb + 32) window(b);
            const unsigned with = __ballot_sync(0xffffffffu, w_n > 0) & (0xffffffffu << (b - wb));
            if (with) {
                b = wb + __ffs(with) - 1;
                m = __shfl_sync(0xffffffffu, w_n, b - wb) * group;
                tiles = plan::token_tiles(__shfl_sync(0xffffffffu, w_len, b - wb));
                return true;
            }
            b = wb + 32;
        }
        return false;
    }
    __device__ __forceinline__ void begin(int64_t lo, int64_t to, int b0, int64_t own0) {
        u = lo;
        hi = to;
        wb = -32;
        w_n = w_len = 0;
        w_first = 0;
        if (u < prefix_total) {
            b = -1;
            head = (int)(u / prefix_head);
            const int64_t rest = u - head * prefix_head;
            m = prefix_m;
            tiles = prefix_tiles;
            rt = plan::row_tile_of(rest, m, tiles);
            start = head * prefix_head + plan::row_tile_start(rt, tiles);
        } else {
            b = b0;
            window(b0);
            if (!seek()) {
                u = hi;
                return;
            }
            const int64_t per = plan::head_units(m, tiles), at = prefix_total + own0;
            head = (int)((u - at) / per);
            const int64_t rest = u - at - head * per;
            rt = plan::row_tile_of(rest, m, tiles);
            start = at + head * per + plan::row_tile_start(rt, tiles);
        }
    }
    __device__ __forceinline__ bool next(Piece &p) {
        while (u < hi) {
            const int rows = plan::tile_rows(m, rt), w = plan::weight(rows);
            const int t0 = plan::first_tile(u, start, w, tiles), t1 = plan::first_tile(hi, start, w, tiles);
            p.tiles = t1 - t0;
            p.first = t0;
            p.rows = rows;
            p.m0 = rt * plan::kTileRows;
            p.head = head;
            p.request = b;
            if (b < 0) {
                p.row_base = 0;
                p.len = p.ctx = a.prefix_len;
                p.n = 0;
            } else {
                p.row_base = (int)__shfl_sync(0xffffffffu, w_first, b - wb);
                p.len = __shfl_sync(0xffffffffu, w_len, b - wb);
                p.n = __shfl_sync(0xffffffffu, w_n, b - wb);
                p.ctx = p.len - p.n;
            }
            p.out = t0 > 0 ? kContinued : (b >= 0 && prefix_total == 0 && t1 == tiles) ? kDirect : kFirst;
            p.pad = 0;
            // the cursor moves to the next item
            start += (int64_t)tiles * w;
            u = start;
            if (++rt == plan::row_tiles(m)) {
                rt = 0;
                if (++head == a.cache.n_kv_heads) {
                    head = 0;
                    ++b;
                    if (!seek()) u = hi;
                }
            }
            if (p.tiles > 0) return true;
        }
        p.tiles = 0;
        return false;
    }
};

// ------------------------------------------------------------------------- q --
// Up to 128 rows of a row tile, from its row t0 on, to fp16 in the swizzled
// layout, each scaled by the power of two that takes its largest element into
// [2^7, 2^8); qscale[row of the tile] is what its scores still lack (the power,
// the caller's scale and log2 e).  Warp `part` of `parts` takes every parts-th
// group of rows.
template <typename T, int DP>
__device__ __forceinline__ void load_q(const AttentionArgs &a, const Piece &p, int t0, int part, int parts, int group,
                                       uint32_t dst, float *qscale, int lane) {
    constexpr int kLanes = DP / 8, kPer = 32 / kLanes;  // lanes of a row (8 elements each), rows a warp takes at once
    constexpr int kBatch = 4;
    const int D = a.cache.head_dim, sub = lane % kLanes, d = sub * 8;
    const int here = min(p.rows - t0, plan::kHalfRows);
    const float inv_group = 1.f / (float)group;
    const int blk0 = (p.m0 + t0) / group, g0 = p.m0 + t0 - blk0 * group;
    const T *q0 = static_cast<const T *>(a.q) + ((int64_t)p.row_base + blk0) * a.q_stride + (int64_t)p.head * group * D + d;
#pragma unroll 1
    for (int r00 = part * kPer; r00 < here; r00 += parts * kPer * kBatch) {
        const int r0 = r00 + lane / kLanes;
        uint4 in[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = r0 + i * parts * kPer;
            in[i] = make_uint4(0, 0, 0, 0);
            if (r < here && d < D) {
                // (g0 + r) / group: below 2^21, where this product is exact enough
                const int g = g0 + r, row = (int)(((float)g + 0.5f) * inv_group);
                in[i] = __ldg(reinterpret_cast<const uint4 *>(q0 + row * a.q_stride + (int64_t)(g - row * group) * D));
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = r0 + i * parts * kPer;
            const uint32_t w[4] = {in[i].x, in[i].y, in[i].z, in[i].w};
            float2 x[4];
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] = pair_to_float<T>(w[e]);
                top = max(top, max(__float_as_uint(x[e].x) & 0x7fffffffu, __float_as_uint(x[e].y) & 0x7fffffffu));
            }
#pragma unroll
            for (int k = kLanes / 2; k > 0; k >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, k));
            if (r < here) {
                const int e2 = top == 0 ? 7 : max((int)(top >> 23) - 127, -110);
                const float mul = top >= 0x7f800000u ? __int_as_float(0x7fffffff) : __uint_as_float((uint32_t)(127 + 7 - e2) << 23);
                if (sub == 0)
                    qscale[t0 + r] = fmaxf(__uint_as_float((uint32_t)(127 - 7 + min(e2, 127)) << 23) * (a.scale * kLog2e), 1e-37f);
                if (d < D)
                    st_shared_v4(dst + (uint32_t)(d >> 6) * (128u * 128u) + (uint32_t)r * 128u +
                                     ((((uint32_t)d >> 3 & 7u) ^ ((uint32_t)r & 7u)) << 4),
                                 make_uint4(half_pair(x[0].x * mul, x[0].y * mul), half_pair(x[1].x * mul, x[1].y * mul),
                                            half_pair(x[2].x * mul, x[2].y * mul), half_pair(x[3].x * mul, x[3].y * mul)));
            }
            __syncwarp();
        }
    }
}

// ----------------------------------------------------------------- the kernel --
template <typename T, int kFormat, int DP>
__global__ void __launch_bounds__(kThreads, 1)
attention_kernel(const __grid_constant__ AttentionArgs a, const Partials parts) {
    using L = Layout<DP>;
    constexpr int kOps = L::kOps, kRaw = L::kRaw;
    extern __shared__ unsigned char dyn[];
    __shared__ __align__(8) uint64_t bars[2 * kRaw + 2 * kOps + 2 * kPieces + 16];
    __shared__ Piece pieces[kPieces];
    __shared__ __align__(16) float vmax[kScaleSlots][4];
    __shared__ int raw_bad[kRaw];
    __shared__ int64_t scan[kThreads / 32 + 1];
    __shared__ int64_t found_units;
    __shared__ int found_request;
    __shared__ int misc[3];       // abort, a word that stays 0, TMEM address

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const dspark_kv_cache &c = a.cache;
    const int D = c.head_dim, group = a.n_q_heads / c.n_kv_heads;
    const uint32_t base = (smem_u32(dyn) + 1023u) & ~1023u;
    unsigned char *gen = dyn + (base - smem_u32(dyn));
    volatile int *abort = misc, *never = misc + 1;

    // barriers
    const uint32_t bar0 = smem_u32(bars);
    auto raw_full = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    auto raw_empty = [&](int i) { return bar0 + 8u * (uint32_t)(kRaw + i); };
    auto op_full = [&](int i) { return bar0 + 8u * (uint32_t)(2 * kRaw + i); };
    auto op_empty = [&](int i) { return bar0 + 8u * (uint32_t)(2 * kRaw + kOps + i); };
    auto piece_full = [&](int i) { return bar0 + 8u * (uint32_t)(2 * kRaw + 2 * kOps + i); };
    auto piece_empty = [&](int i) { return bar0 + 8u * (uint32_t)(2 * kRaw + 2 * kOps + kPieces + i); };
    const uint32_t bar1 = bar0 + 8u * (uint32_t)(2 * kRaw + 2 * kOps + 2 * kPieces);
    auto q_full = [&](int i) { return bar1 + 8u * (uint32_t)i; };
    auto q_empty = [&](int i) { return bar1 + 8u * (uint32_t)(2 + i); };
    auto s_full = [&](int i) { return bar1 + 8u * (uint32_t)(4 + i); };
    auto p_ready = [&](int i) { return bar1 + 8u * (uint32_t)(6 + i); };
    auto o_full = [&](int i) { return bar1 + 8u * (uint32_t)(8 + i); };
    auto stat_full = [&](int i) { return bar1 + 8u * (uint32_t)(10 + i); };
    const uint32_t o_free = bar1 + 8u * 12u, drain = bar1 + 8u * 13u;

    if (tid == 0) {
        for (int i = 0; i < kRaw; ++i) mbar_init(raw_full(i), 33), mbar_init(raw_empty(i), 4);
        for (int i = 0; i < kOps; ++i) mbar_init(op_full(i), 4), mbar_init(op_empty(i), 1);
        for (int i = 0; i < kPieces; ++i) mbar_init(piece_full(i), 1), mbar_init(piece_empty(i), 15);
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full(i), 4), mbar_init(q_empty(i), 1);
            mbar_init(s_full(i), 1), mbar_init(p_ready(i), 4);
            mbar_init(o_full(i), 1), mbar_init(stat_full(i), 4);
        }
        mbar_init(o_free, 8), mbar_init(drain, 1);
        fence_mbar_init();
        misc[0] = misc[1] = 0;
        found_request = a.rows.B;
        found_units = 0;
    }
    if (warp == 13) {
        tmem_alloc(smem_u32(misc + 2), 512);
        tmem_relinquish();
    }

    // ---- the line of units: total, and the request this CTA's own part starts in
    const int R = prefix_rows(a);
    const int prefix_tiles = plan::token_tiles(a.prefix_len), prefix_m = R * group;
    const int64_t prefix_head = plan::head_units(prefix_m, prefix_tiles);
    const int64_t prefix_total = prefix_head * c.n_kv_heads;
    auto request_units = [&](int b) -> int64_t {
        if (b >= a.rows.B) return 0;
        const Request q = load_request(a, b);
        if (blockIdx.x == 0 && (!q.rows_ok || (q.n > 0 && !q.len_ok)))
            atomicOr(c.flags, kFlagBadLength);
        if (!q.len_ok || q.n == 0) return 0;
        return plan::head_units(q.n * group, plan::token_tiles(q.len)) * c.n_kv_heads;
    };
    const int64_t mine = request_units(tid);   // the first 512 requests' units stay in registers
    int64_t sum = mine;
    for (int b = tid + kThreads; b < a.rows.B; b += kThreads) sum += request_units(b);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) scan[warp] = sum;
    __syncthreads();
    int64_t own_total = 0;
    for (int w = 0; w < kThreads / 32; ++w) own_total += scan[w];
    const int64_t total = prefix_total + own_total;
    const int64_t lo = plan::cta_begin(blockIdx.x, total, kCtas), hi = plan::cta_begin(blockIdx.x + 1, total, kCtas);
    {
        int64_t before = 0;
        const int64_t want = lo > prefix_total ? lo - prefix_total : 0;  // own unit to start at
        for (int b0 = 0; b0 < a.rows.B; b0 += kThreads) {
            const int b = b0 + tid;
            const int64_t x = b0 == 0 ? mine : request_units(b);
            int64_t v = x;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, v, d);
                if (lane >= d) v += y;
            }
            __syncthreads();
            if (lane == 31) scan[warp] = v;
            __syncthreads();
            int64_t at = before + v - x;
            for (int w = 0; w < kThreads / 32; ++w) {
                if (w < warp) at += scan[w];
                before += scan[w];
            }
            if (b < a.rows.B) {
                if (blockIdx.x == 0) parts.unit0[b] = at;
                if (x > 0 && at <= want && want < at + x) {
                    found_request = b;
                    found_units = at;
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)misc[2];

    if (warp >= 8) {
        if (warp == 12) {
            // ------------------------------------------------------ producer --
            Walk walk{a, lane, group, prefix_m, prefix_tiles, prefix_head, prefix_total};
            walk.begin(lo, hi, found_request, found_units);
            Piece cur, nxt;
            bool have = walk.next(cur), ok = true;
            uint32_t raw = 0, count = 0;   // tiles issued, pieces published
            // Pages of 32 chunks of 16 tokens (4 tiles) from tile t of a piece on, one a lane; the
            // chunk's number in the cache (in units of 16 head rows) is made from it when the page is
            // first needed, 128 tokens x 4 later than its load.  A chunk lies inside one page.
            const int chunks_per_page = c.page_size / 16;
            const uint32_t page_chunks = (uint32_t)c.n_kv_heads * (uint32_t)chunks_per_page;
            constexpr uint32_t kNone = 0xffffffffu, kBad = 0xfffffffeu;
            auto load_pages = [&](const Piece &p, int t, int &off) -> int {
                const int chunk = (p.first + t) * 8 + lane;
                if (t >= p.tiles || (int64_t)chunk * 16 >= p.len) {
                    off = -1;
                    return 0;
                }
                const int slot = chunk / chunks_per_page;
                off = p.head * chunks_per_page + (chunk - slot * chunks_per_page);
                return p.request < 0 ? a.prefix_pages[slot] : a.rows.block_table[(int64_t)p.request * a.rows.max_pages + slot];
            };
            auto number = [&](int page, int off) -> uint32_t {
                return off < 0 ? kNone : (page < 0 || page >= c.n_pages) ? kBad : (uint32_t)page * page_chunks + (uint32_t)off;
            };
            const unsigned char *k_lane = static_cast<const unsigned char *>(c.k) + lane * 16;
            const unsigned char *v_lane = static_cast<const unsigned char *>(c.v) + lane * 16;
            // scales: lane's 16 bytes are tokens 4 (lane & 3) .. of chunk lane / 4
            const float *ks_lane = c.k_scale + (lane & 3) * 4, *vs_lane = c.v_scale + (lane & 3) * 4;
            int off_next = -1;
            int page_next = have ? load_pages(cur, 0, off_next) : 0;
            while (ok) {
                int page = page_next, off = off_next;            // the next window to be needed
                uint32_t chunk_id[2] = {kNone, kNone};            // this lane's chunk in even and odd windows
                const bool more = have && walk.next(nxt);
                page_next = more ? load_pages(nxt, 0, off_next) : 0;
                const int ps = (int)(count % kPieces);
                if (!warp_wait(piece_empty(ps), ((count / kPieces) & 1) ^ 1, abort)) { ok = false; break; }
                if (!have) cur.tiles = 0;
                if (lane == 0) {
                    pieces[ps] = cur;
                    mbar_arrive(piece_full(ps));
                }
                ++count;
                if (!have) break;
                const bool pair = cur.rows > plan::kHalfRows;
                bool flagged = false;
                const int steps = 2 * cur.tiles;
                for (int s = 0; s < steps; ++s, ++raw) {
                    bool is_v;
                    int j;
                    step_of(s, cur.tiles, pair, is_v, j);
                    const bool odd = (j >> 2) & 1;
                    if (!is_v && (j & 3) == 0) {
                        // a new window; the one before it is still needed for values
                        const uint32_t id = number(page, off);
                        if (odd) chunk_id[1] = id; else chunk_id[0] = id;
                        page = load_pages(cur, j + 4, off);
                    }
                    const uint32_t mine = odd ? chunk_id[1] : chunk_id[0];
                    const int from = (j & 3) << 3;
                    const int slot = (int)(raw % kRaw);
                    if (!warp_wait(raw_empty(slot), ((raw / kRaw) & 1) ^ 1, abort)) { ok = false; break; }
                    const uint32_t at = base + L::kRawAt + (uint32_t)slot * L::kRawBytes + (uint32_t)lane * 16u;
                    const unsigned char *codes = is_v ? v_lane : k_lane;
                    const unsigned bad = (__ballot_sync(0xffffffffu, mine == kBad) >> from) & 0xffu;
#pragma unroll
                    for (int ch = 0; ch < 8; ++ch) {
                        const uint32_t id = __shfl_sync(0xffffffffu, mine, from + ch);
                        if (id >= kBad) continue;
                        const unsigned char *src = codes + (uint64_t)id * (uint32_t)(16 * D);
                        const uint32_t dst = at + (uint32_t)(ch * 16 * D);
                        if (D == 128) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) cp_async_16(dst + 512u * i, src + 512 * i, 16);
                        } else {
                            for (int i = lane; i < D; i += 32) cp_async_16(dst + 16u * (uint32_t)(i - lane), src + 16 * (i - lane), 16);
                        }
                    }
                    if (!is_v) {
                        const uint32_t id = __shfl_sync(0xffffffffu, mine, from + (lane >> 2));
                        if (id < kBad) {
                            cp_async_16(at + 128u * DP, ks_lane + (uint64_t)id * 16u, 16);
                            cp_async_16(at + 128u * DP + 512u, vs_lane + (uint64_t)id * 16u, 16);
                        }
                    }
                    cp_async_arrive(raw_full(slot));
                    if (lane == 0) {
                        raw_bad[slot] = (int)bad;
                        mbar_arrive(raw_full(slot));
                    }
                    flagged |= bad != 0;
                }
                if (flagged && lane == 0) atomicOr(c.flags, kFlagBadPage);
                cur = nxt;
                have = more;
            }
            if (!ok && lane == 0) *abort = 1;
            cp_async_wait_all();   // nothing may be in flight when the block's memory goes
        } else if (warp == 13) {
            // ------------------------------------------- tensor-core products --
            {
                const bool leader = elect_one();
                const uint32_t hi_desc = (uint32_t)(sw128_kmajor_desc(0) >> 32);
                const uint32_t id_qk = idesc_f16_f32(128, 128, false), id_pv = idesc_f16_f32(128, D, true);
                constexpr uint32_t kAtom = 128 * 128;  // bytes of a 64-column atom of a 128-row tile
                uint32_t op = 0, qc = 0, count = 0, pc[2] = {0, 0};
                bool ok = true;
                const int k_steps = D / 16;
                auto wait = [&](uint32_t bar, uint32_t parity) {
                    if (!ok) return false;
                    ok = warp_wait(bar, parity, abort);
                    tc_fence_after();
                    return ok;
                };
                // the whole warp walks the loop, so that addresses stay warp-uniform; one lane issues
                auto commit = [&](uint32_t bar) {
                    if (leader) umma_commit(bar);
                };
                auto qk = [&](int w, uint32_t qbuf, uint32_t slot) {
                    const uint32_t qa = (base + L::kQ + qbuf * L::kTileBytes) >> 4 | 1u << 16;
                    const uint32_t ka = (base + L::kOp + slot * L::kTileBytes) >> 4 | 1u << 16;
                    const uint32_t d = tmem + kColS + 128u * (uint32_t)w;
                    if (leader) {
#pragma unroll
                        for (int k = 0; k < DP / 16; ++k) {
                            const uint32_t off = ((uint32_t)(k >> 2) * kAtom + (uint32_t)(k & 3) * 32u) >> 4;
                            if (k < k_steps) umma_bf16_w(d, qa + off, ka + off, hi_desc, id_qk, k > 0);
                        }
                        umma_commit(s_full(w));
                    }
                };
                auto pv = [&](int w, uint32_t slot, bool accumulate) {
                    const uint32_t va = (base + L::kOp + slot * L::kTileBytes) >> 4 | (kAtom >> 4) << 16;
                    const uint32_t d = tmem + kColO + 128u * (uint32_t)w, pa = tmem + kColS + 128u * (uint32_t)w;
                    if (leader) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            umma_bf16_ts(d, pa + 8u * (uint32_t)k, va + (uint32_t)k * (2048u >> 4), hi_desc, id_pv,
                                         k > 0 ? 1u : (uint32_t)accumulate);
                    }
                };
                while (true) {
                    const int ps = (int)(count % kPieces);
                    if (!wait(piece_full(ps), (count / kPieces) & 1)) break;
                    const int n = pieces[ps].tiles;
                    const bool pair = pieces[ps].rows > plan::kHalfRows;
                    if (lane == 0) mbar_arrive(piece_empty(ps));
                    if (n == 0) break;
                    // this piece's q tiles: one, or one per group
                    uint32_t qb[2] = {qc & 1, qc & 1}, qp[2] = {(qc >> 1) & 1, (qc >> 1) & 1};
                    if (pair) qb[1] = (qc + 1) & 1, qp[1] = ((qc + 1) >> 1) & 1;
                    qc += pair ? 2 : 1;
                    auto op_ready = [&](uint32_t i) { return wait(op_full((int)(i % kOps)), (i / kOps) & 1); };
                    if (!wait(q_full((int)qb[0]), qp[0])) break;
                    if (pair) {
                        if (!wait(q_full((int)qb[1]), qp[1])) break;
                        if (!op_ready(op)) break;
                        for (int w = 0; w < 2; ++w) {
                            qk(w, qb[w], op % kOps);
                            if (n == 1) commit(q_empty((int)qb[w]));
                        }
                        commit(op_empty((int)(op % kOps)));
                        if (count > 0 && !wait(o_free, (count - 1) & 1)) break;
                        for (int j = 0; j < n && ok; ++j) {
                            const uint32_t vi = op + 2 * j + 1, ki = op + 2 * j + 2;
                            if (!op_ready(vi)) break;
                            for (int w = 0; w < 2; ++w) {
                                if (!wait(p_ready(w), pc[w] & 1)) break;
                                ++pc[w];
                                pv(w, vi % kOps, j > 0);
                                if (w == 1) commit(op_empty((int)(vi % kOps)));
                                if (j + 1 < n) {
                                    if (w == 0 && !op_ready(ki)) break;
                                    qk(w, qb[w], ki % kOps);
                                    if (j + 2 == n) commit(q_empty((int)qb[w]));
                                    if (w == 1) commit(op_empty((int)(ki % kOps)));
                                } else {
                                    commit(o_full(w));
                                }
                            }
                        }
                    } else {
                        // step indices: K0 = 0, K(j) = 2j - 1, V(j) = 2j + 2, the last V = 2n - 1
                        auto k_at = [&](int j) { return op + (uint32_t)(j == 0 ? 0 : 2 * j - 1); };
                        auto v_at = [&](int j) { return op + (uint32_t)(j == n - 1 ? 2 * n - 1 : 2 * j + 2); };
                        for (int j = 0; j < 2 && j < n; ++j) {
                            if (!op_ready(k_at(j))) break;
                            qk(j, qb[0], k_at(j) % kOps);
                            commit(op_empty((int)(k_at(j) % kOps)));
                            if (j == n - 1) commit(q_empty((int)qb[0]));
                        }
                        if (!ok) break;
                        if (count > 0 && !wait(o_free, (count - 1) & 1)) break;
                        for (int j = 0; j < n && ok; ++j) {
                            const int w = j & 1;
                            if (!op_ready(v_at(j)) || !wait(p_ready(w), pc[w] & 1)) break;
                            ++pc[w];
                            pv(w, v_at(j) % kOps, j >= 2);
                            commit(op_empty((int)(v_at(j) % kOps)));
                            if (j + 2 < n) {
                                if (!op_ready(k_at(j + 2))) break;
                                qk(w, qb[0], k_at(j + 2) % kOps);
                                commit(op_empty((int)(k_at(j + 2) % kOps)));
                                if (j + 3 == n) commit(q_empty((int)qb[0]));
                            } else {
                                commit(o_full(w));
                            }
                        }
                    }
                    if (!ok) break;
                    op += 2 * n;
                    ++count;
                }
                if (!ok) {
                    if (lane == 0) *abort = 1;
                    commit(drain);
                    mbar_wait(drain, 0, never, kDrainLimit);
                }
            }
        } else if (warp >= 14) {
            // ------------------------------------------------------------ q --
            // (pieces of at most 128 rows, ahead of their use)
            uint32_t qc = 0, count = 0;
            bool ok = true;
            while (ok) {
                const int ps = (int)(count % kPieces);
                if (!warp_wait(piece_full(ps), (count / kPieces) & 1, abort)) { ok = false; break; }
                const int n = pieces[ps].tiles, rows = pieces[ps].rows;
                if (n > 0 && rows > plan::kHalfRows) qc += 2;
                else if (n > 0) {
                    const int buf = (int)(qc & 1);
                    if (!warp_wait(q_empty(buf), ((qc >> 1) & 1) ^ 1, abort)) { ok = false; break; }
                    load_q<T, DP>(a, pieces[ps], 0, warp - 14, 2, group, base + L::kQ + (uint32_t)buf * L::kTileBytes,
                                  reinterpret_cast<float *>(gen + L::kQScale) + ps * 256, lane);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane < 2) mbar_arrive(q_full(buf));
                    ++qc;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(piece_empty(ps));
                ++count;
                if (n == 0) break;
            }
            if (!ok && lane == 0) *abort = 1;
        } else {
            // ---------------------------------------------------- converters --
            const int t = tid - 256;
            const int cpr = D / 16;                      // 16-code chunks of a token
            uint32_t op = 0, count = 0, tile0 = 0;
            bool ok = true;
            while (ok) {
                const int ps = (int)(count % kPieces);
                if (!warp_wait(piece_full(ps), (count / kPieces) & 1, abort)) { ok = false; break; }
                const int n = pieces[ps].tiles, first = pieces[ps].first, len = pieces[ps].len;
                const bool pair = pieces[ps].rows > plan::kHalfRows;
                for (int s = 0; s < 2 * n && ok; ++s, ++op) {
                    bool is_v;
                    int j;
                    step_of(s, n, pair, is_v, j);
                    const uint32_t dst = base + L::kOp + (op % kOps) * L::kTileBytes;
                    if (!warp_wait(op_empty((int)(op % kOps)), ((op / kOps) & 1) ^ 1, abort)) { ok = false; break; }
                    const int slot = (int)(op % kRaw);
                    if (!warp_wait(raw_full(slot), (op / kRaw) & 1, abort)) { ok = false; break; }
                    const uint32_t src = base + L::kRawAt + (uint32_t)slot * L::kRawBytes;
                    const int bad = raw_bad[slot];
                    const int valid = len - (first + j) * plan::kTile;   // tokens of this tile that exist (128 or more: all)
                    const bool whole = valid >= plan::kTile && bad == 0;
                    auto decode_store = [&](uint4 in, int row, int ch) {
                        __half2 h[8];
                        decode4<kFormat>(in.x, h[0], h[1]);
                        decode4<kFormat>(in.y, h[2], h[3]);
                        decode4<kFormat>(in.z, h[4], h[5]);
                        decode4<kFormat>(in.w, h[6], h[7]);
                        const uint32_t *u = reinterpret_cast<const uint32_t *>(h);
                        const uint4 lo4 = make_uint4(u[0], u[1], u[2], u[3]), hi4 = make_uint4(u[4], u[5], u[6], u[7]);
                        const uint32_t r = (uint32_t)row, c8 = (uint32_t)(ch & 3) * 2u;
                        const uint32_t line = dst + (uint32_t)(ch >> 2) * (128u * 128u) + r * 128u;
                        // lanes of the upper 64 columns write their second half first: no two of a
                        // row's lanes then meet in a bank
                        const uint32_t o = (uint32_t)(ch >> 2) & 1u;
                        st_shared_v4(line + (((c8 + o) ^ (r & 7u)) << 4), o ? hi4 : lo4);
                        st_shared_v4(line + (((c8 + 1u - o) ^ (r & 7u)) << 4), o ? lo4 : hi4);
                    };
                    auto keep = [&](uint4 in, int row) {   // nothing of a token that is not there
                        return row < valid && !(bad >> (row >> 4) & 1) ? in : make_uint4(0, 0, 0, 0);
                    };
                    float ks = 0.f, vs = 0.f;
                    if (!is_v && t < valid) {
                        // a token whose value scale (or page) is no number carries its NaN in the key's
                        // scale alone: where it is masked, P is 0 times the value's
                        const float *rs = reinterpret_cast<const float *>(gen + L::kRawAt + (uint32_t)slot * L::kRawBytes + 128 * DP);
                        ks = rs[t];
                        vs = rs[128 + t];
                        if ((bad >> (t >> 4) & 1) || !(vs <= 3.4028235e38f)) ks = __int_as_float(0x7fffffff), vs = 0.f;
                    }
                    if (D == DP) {
                        // all loads first: the slot goes back before the decoding
                        constexpr int kCpr = DP / 16, kEach = kCpr;
                        uint4 in[kEach];
#pragma unroll
                        for (int i = 0; i < kEach; ++i) in[i] = ld_shared_v4(src + (uint32_t)(t + 128 * i) * 16u);
                        if (!whole) {
#pragma unroll
                            for (int i = 0; i < kEach; ++i) in[i] = keep(in[i], (t + 128 * i) / kCpr);
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(raw_empty(slot));
#pragma unroll
                        for (int i = 0; i < kEach; ++i) decode_store(in[i], (t + 128 * i) / kCpr, (t + 128 * i) % kCpr);
                    } else {
                        for (int i = t; i < 128 * cpr; i += 128) {
                            const int row = i / cpr;
                            decode_store(keep(ld_shared_v4(src + (uint32_t)i * 16u), row), row, i - row * cpr);
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(raw_empty(slot));
                    }
                    if (!is_v) {
                        // the tile's scales, for the softmax groups
                        const int ss = (int)((tile0 + j) % kScaleSlots);
                        float *sc = reinterpret_cast<float *>(gen + L::kScale) + ss * 256;
                        sc[t] = ks;
                        sc[128 + t] = vs;
                        const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(vs, 0.f)));
                        if (lane == 0) vmax[ss][t >> 5] = __uint_as_float(top);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(op_full((int)(op % kOps)));
                }
                tile0 += (uint32_t)n;
                __syncwarp();
                if (lane == 0) mbar_arrive(piece_empty(ps));
                ++count;
                if (n == 0) break;
            }
            if (!ok && lane == 0) *abort = 1;
        }
    } else {
        // -------------------------------------------------------------- softmax --
        const int w = warp >> 2, row = tid & 127;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);   // this warp's 32 TMEM lanes
        const uint32_t my_s = lanes + kColS + 128u * w, my_o = lanes + kColO + 128u * w;
        float2 *stats = reinterpret_cast<float2 *>(gen + L::kStats);
        uint32_t sc_count = 0, oc = 0, xc = 0, count = 0, tile0 = 0, qc = 0;
        bool ok = true;
        while (ok) {
            const int ps = (int)(count % kPieces);
            if (!warp_wait(piece_full(ps), (count / kPieces) & 1, abort)) { ok = false; break; }
            const Piece p = pieces[ps];
            if (p.tiles == 0) {
                if (lane == 0) mbar_arrive(piece_empty(ps));
                break;
            }
            const bool pair = p.rows > plan::kHalfRows;
            if (pair) {
                const uint32_t q = qc + (uint32_t)w;
                const int buf = (int)(q & 1);
                if (!warp_wait(q_empty(buf), ((q >> 1) & 1) ^ 1, abort)) { ok = false; break; }
                load_q<T, DP>(a, p, w * 128, warp & 3, 4, group, base + L::kQ + (uint32_t)buf * L::kTileBytes,
                              reinterpret_cast<float *>(gen + L::kQScale) + ps * 256, lane);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full(buf));
            }
            qc += pair ? 2 : 1;
            const int step = pair ? 1 : 2, t_first = pair ? 0 : w;
            const int rows = pair ? min(max(p.rows - w * 128, 0), 128) : p.rows;
            const int mt = pair ? w * 128 + row : row;       // row of the row tile
            const bool live = row < rows, warp_live = (warp & 3) * 32 < rows;
            const int m = p.m0 + mt, blk = m / group;
            // what this row sees of the list: tokens below `sees`, and with a mask word those of its bits
            int sees = p.ctx;
            uint64_t word = 0;
            if (p.request >= 0) {
                if (a.row_mask) {
                    if (live) word = a.row_mask[p.row_base + blk];
                    if (p.n < 64) word &= (1ull << p.n) - 1;
                } else {
                    sees = a.mask == DSPARK_MASK_CAUSAL ? p.ctx + min(blk, p.n - 1) + 1 : p.len;
                }
            }
            float r = -INFINITY, l = 0.f, cm = 0.f;
            for (int j = t_first; j < p.tiles && ok; j += step, ++sc_count) {
                if (!warp_wait(s_full(w), sc_count & 1, abort)) { ok = false; break; }
                tc_fence_after();
                if (warp_live) {
                    if (j == t_first) cm = live ? (reinterpret_cast<const float *>(gen + L::kQScale))[ps * 256 + mt] : 0.f;
                    const int ss = (int)((tile0 + j) % kScaleSlots);
                    const float *ks = reinterpret_cast<const float *>(gen + L::kScale) + ss * 256, *vs = ks + 128;
                    const float4 vm = *reinterpret_cast<const float4 *>(vmax[ss]);
                    const int t0 = (p.first + j) * plan::kTile;
                    const bool masked = t0 > p.ctx - plan::kTile;   // some row does not see some token of this tile
                    __syncwarp();
                    // x = ks * (q . k~) of 32 columns, those the row does not see -inf
                    auto scores = [&](uint32_t (&x)[32], int q) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 k4 = *reinterpret_cast<const float4 *>(ks + 32 * q + e);
                            float y0, y1, y2, y3;
                            unpack2(mul2(pack2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), pack2(k4.x, k4.y)), y0, y1);
                            unpack2(mul2(pack2(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])), pack2(k4.z, k4.w)), y2, y3);
                            x[e] = __float_as_uint(y0), x[e + 1] = __float_as_uint(y1);
                            x[e + 2] = __float_as_uint(y2), x[e + 3] = __float_as_uint(y3);
                        }
                        if (masked) {
                            const int from = t0 + 32 * q, full = min(max(sees - from, 0), 32);
                            uint32_t bits = full == 32 ? 0xffffffffu : (1u << full) - 1u;
                            const int sh = from - p.ctx;   // block token of the first column
                            if (sh > -32 && sh < 64) bits |= (uint32_t)(sh >= 0 ? word >> sh : word << -sh);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(bits >> e & 1u)) x[e] = 0xff800000u;
                        }
                    };
                    float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    auto maxima = [&](uint32_t (&x)[32], int q) {
                        scores(x, q);
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                tops[k] = max3(tops[k], __uint_as_float(x[e + 2 * k]), __uint_as_float(x[e + 2 * k + 1]));
                    };
                    // the scores are read twice from tensor memory, 32 columns at a time and one load
                    // ahead: holding a row's 128 scores instead spills
                    uint32_t xa[32], xb[32];
                    tmem_ld32(my_s, xa);
#pragma unroll 1
                    for (int q = 0; q < 4; q += 2) {
                        tmem_ld_wait32(xa);
                        tmem_ld32(my_s + 32u * (q + 1), xb);
                        maxima(xa, q);
                        tmem_ld_wait32(xb);
                        tmem_ld32(my_s + 32u * ((q + 2) & 3), xa);
                        maxima(xb, q + 1);
                    }
                    tmem_ld_wait32(xa);
                    const float top = fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]);
                    // P <= 2^(bound - r): the row's largest score with the tile's largest value scale
                    const float vt = fmaxf(fmaxf(fmaxf(vm.x, vm.y), fmaxf(vm.z, vm.w)), kScaleFloor);
                    const float bound = top * cm + (float)((int)(__float_as_uint(vt) >> 23) - 126);
                    const bool moves = live && bound - r > kSlack;   // (also when r is still -inf)
                    if (__any_sync(0xffffffffu, moves)) {
                        const float r_new = moves ? ceilf(bound) - kPeak : r;
                        const float f = moves ? fast_exp2(r - r_new) : 1.f;
                        r = r_new;
                        l *= f;
                        if (j != t_first) {
                            // the group's previous product has ended (the scores came after it)
#pragma unroll 1
                            for (int q = 0; q < DP / 32; ++q) {
                                tmem_ld32(my_o + 32u * q, xb);
                                tmem_ld_wait32(xb);
#pragma unroll
                                for (int e = 0; e < 32; ++e) xb[e] = __float_as_uint(__uint_as_float(xb[e]) * f);
                                tmem_st32(my_o + 32u * q, xb);
                            }
                        }
                    }
                    const float ref = r == -INFINITY ? 0.f : r;
                    const uint64_t c2 = pack2(cm, cm), r2 = pack2(-ref, -ref);
                    uint64_t sum[2] = {0, 0};
                    auto terms = [&](uint32_t (&x)[32], int q) {
                        scores(x, q);
                        uint32_t pr[16];
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 v4 = *reinterpret_cast<const float4 *>(vs + 32 * q + e);
                            float y0, y1, y2, y3;
                            unpack2(fma2(pack2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), c2, r2), y0, y1);
                            unpack2(fma2(pack2(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])), c2, r2), y2, y3);
                            const uint64_t e0 = pack2(fast_exp2(y0), fast_exp2(y1)), e1 = pack2(fast_exp2(y2), fast_exp2(y3));
                            sum[0] = add2(sum[0], e0);
                            sum[1] = add2(sum[1], e1);
                            unpack2(mul2(e0, pack2(v4.x, v4.y)), y0, y1);
                            unpack2(mul2(e1, pack2(v4.z, v4.w)), y2, y3);
                            pr[e >> 1] = half_pair(y0, y1);
                            pr[(e >> 1) + 1] = half_pair(y2, y3);
                        }
                        // P's 16 columns lie below the scores still to be read
                        tmem_st16(my_s + 16u * q, pr);
                    };
#pragma unroll 1
                    for (int q = 0; q < 4; q += 2) {
                        tmem_ld32(my_s + 32u * (q + 1), xb);
                        terms(xa, q);
                        tmem_ld_wait32(xb);
                        if (q == 0) tmem_ld32(my_s + 64u, xa);
                        terms(xb, q + 1);
                        if (q == 0) tmem_ld_wait32(xa);
                    }
                    float s0, s1;
                    unpack2(add2(sum[0], sum[1]), s0, s1);
                    l += s0 + s1;
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_ready(w));
            }
            if (!ok) break;
            // ---- the piece's result
            const bool takes_part = pair || p.tiles > w;
            if (takes_part) {
                if (!warp_wait(o_full(w), oc & 1, abort)) { ok = false; break; }
                ++oc;
            } else if (count > 0 && !warp_wait(o_free, (count - 1) & 1, abort)) {
                // nothing held this group back: the other one may still read the last piece's sums
                ok = false;
                break;
            }
            float f_own = 1.f, f_other = 0.f;
            if (!pair) {
                // both groups' sums of these rows: exchanged, and each group writes half the columns
                stats[w * 128 + row] = make_float2(r, l);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(stat_full(w));
                if (!warp_wait(stat_full(w ^ 1), xc & 1, abort)) { ok = false; break; }
                ++xc;
                const float2 other = stats[(w ^ 1) * 128 + row];
                const float top = fmaxf(r, other.x);
                f_own = (r == -INFINITY && l == 0.f) ? 0.f : fast_exp2(r - top);
                f_other = (other.x == -INFINITY && other.y == 0.f) ? 0.f : fast_exp2(other.x - top);
                l = l * f_own + other.y * f_other;
                r = top;
                // a group without a tile has nothing in its columns
                if (!takes_part) f_own = 0.f;
                if (p.tiles < 2 && w == 0) f_other = 0.f;
            }
            tc_fence_after();
            __syncwarp();
            if (warp_live) {
                const int64_t packed = (int64_t)p.row_base + blk;
                const int head = p.head * group + (m - blk * group);
                const int64_t place = packed * a.n_q_heads + head, all = (int64_t)a.rows.n_rows * a.n_q_heads;
                const int64_t part = p.out == kContinued ? 2 * all + (int64_t)blockIdx.x * plan::kTileRows + mt
                                                         : (p.request < 0 ? place : all + place);
                float inv = 1.f;
                if (p.out == kDirect) inv = l == 0.f ? 0.f : 1.f / l;
                const int q0 = pair ? 0 : w * (DP / 64), q1 = pair ? DP / 32 : q0 + DP / 64;
                for (int q = q0; q < q1; ++q) {
                    if (q * 32 >= D) break;
                    uint32_t o[32];
                    tmem_ld32(my_o + 32u * q, o);
                    tmem_ld_wait32(o);
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = f_own == 0.f ? 0u : __float_as_uint(__uint_as_float(o[e]) * f_own);
                    if (!pair) {
                        uint32_t o2[32];
                        tmem_ld32(lanes + kColO + 128u * (w ^ 1) + 32u * q, o2);
                        tmem_ld_wait32(o2);
                        if (f_other != 0.f) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                o[e] = __float_as_uint(fmaf(__uint_as_float(o2[e]), f_other, __uint_as_float(o[e])));
                        }
                    }
                    if (live && p.out == kDirect) {
                        T *dst = static_cast<T *>(a.out) + place * D + 32 * q;
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            if (32 * q + e >= D) break;
                            uint32_t v[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                v[k] = float_to_pair<T>(__uint_as_float(o[e + 2 * k]) * inv, __uint_as_float(o[e + 2 * k + 1]) * inv);
                            *reinterpret_cast<uint4 *>(dst + e) = make_uint4(v[0], v[1], v[2], v[3]);
                        }
                    } else if (live) {
                        float *dst = parts.o + part * D + 32 * q;
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            if (32 * q + e >= D) break;
                            *reinterpret_cast<uint4 *>(dst + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                        }
                    }
                    __syncwarp();
                }
                if (live && (pair || w == 0)) {
                    if (p.out != kDirect) parts.stats[part] = make_float2(r, l);
                    else if (a.lse) a.lse[place] = l == 0.f ? -INFINITY : kLn2 * (r + log2f(l));
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(o_free);
                mbar_arrive(piece_empty(ps));
            }
            tile0 += (uint32_t)p.tiles;
            ++count;
        }
        if (!ok && lane == 0) *abort = 1;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 13) tmem_dealloc(tmem, 512);
    if (tid == 0 && *abort) atomicOr(c.flags, kFlagTimeout);
}

// ---------------------------------------------------------------- the joining --
// One warp per (packed row, query head) adds up the parts of its row: the
// prefix's and its request's own item's, each cut where a CTA's part of the
// line ends.  Rows that one CTA finished alone are already written.
constexpr int kJoinWarps = 8;

template <typename T>
__global__ void __launch_bounds__(kJoinWarps * 32)
attention_join_kernel(const __grid_constant__ AttentionArgs a, const Partials parts) {
    griddep_wait();
    const int lane = threadIdx.x & 31, b = blockIdx.x;
    const dspark_kv_cache &c = a.cache;
    const int D = c.head_dim, group = a.n_q_heads / c.n_kv_heads, Hq = a.n_q_heads;
    const Request q = load_request(a, b);
    if (q.n == 0) return;
    const int R = prefix_rows(a), prefix_m = R * group, prefix_tiles = plan::token_tiles(a.prefix_len);
    const int64_t prefix_head = plan::head_units(prefix_m, prefix_tiles), prefix_total = prefix_head * c.n_kv_heads;
    // the total of all units: the last request's end
    int64_t total;
    {
        const int last = a.rows.B - 1;
        const Request z = load_request(a, last);
        total = prefix_total + parts.unit0[last] +
                (z.len_ok && z.n > 0 ? plan::head_units(z.n * group, plan::token_tiles(z.len)) * c.n_kv_heads : 0);
    }
    const int64_t all = (int64_t)a.rows.n_rows * Hq;
    const int m_own = q.n * group, own_tiles = plan::token_tiles(q.len);
    const int64_t own_head = plan::head_units(m_own, own_tiles);
    for (int i = blockIdx.y * kJoinWarps + (threadIdx.x >> 5); i < q.n * Hq; i += gridDim.y * kJoinWarps) {
        const int blk = i / Hq, head = i - blk * Hq, h = head / group, g = head - h * group;
        const int64_t place = (q.first + blk) * Hq + head;
        T *out = static_cast<T *>(a.out) + place * D;
        if (!q.len_ok) {
            if (lane * 4 < D) *reinterpret_cast<uint2 *>(out + lane * 4) = make_uint2(0x7fff7fffu, 0x7fff7fffu);
            if (lane == 0 && a.lse) a.lse[place] = __int_as_float(0x7fffffff);
            continue;
        }
        float top = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
        auto add = [&](int64_t part) {
            const float2 st = parts.stats[part];
            if (st.x == -INFINITY && st.y == 0.f) return;   // saw nothing
            const float t = fmaxf(top, st.x);
            const float f0 = top == -INFINITY && l == 0.f ? 0.f : fast_exp2(top - t), f1 = fast_exp2(st.x - t);
            l = l * f0 + st.y * f1;
            top = t;
            if (lane * 4 < D) {
                const float4 o = *reinterpret_cast<const float4 *>(parts.o + part * D + lane * 4);
                acc[0] = acc[0] * f0 + o.x * f1, acc[1] = acc[1] * f0 + o.y * f1;
                acc[2] = acc[2] * f0 + o.z * f1, acc[3] = acc[3] * f0 + o.w * f1;
            }
        };
        // parts of one item: its first CTA's, then those of the CTAs that go on with it
        auto add_item = [&](int64_t start, int tiles, int w, int mt, int64_t first_part, bool alone_is_done) {
            const int64_t end = start + (int64_t)tiles * w;
            const int c0 = plan::cta_of(start, total, kCtas);
            if (alone_is_done && plan::first_tile(plan::cta_begin(c0 + 1, total, kCtas), start, w, tiles) == tiles) return false;
            add(first_part);
            for (int k = c0 + 1; k < kCtas; ++k) {
                const int64_t from = plan::cta_begin(k, total, kCtas);
                if (from >= end) break;
                if (plan::first_tile(from, start, w, tiles) <
                    plan::first_tile(plan::cta_begin(k + 1, total, kCtas), start, w, tiles))
                    add(2 * all + (int64_t)k * plan::kTileRows + mt);
            }
            return true;
        };
        if (prefix_total > 0) {
            const int m = (int)(q.first + blk) * group + g, rt = m / plan::kTileRows;
            add_item(h * prefix_head + plan::row_tile_start(rt, prefix_tiles), prefix_tiles,
                     plan::weight(plan::tile_rows(prefix_m, rt)), m - rt * plan::kTileRows, place, false);
        }
        const int m = blk * group + g, rt = m / plan::kTileRows;
        if (!add_item(prefix_total + parts.unit0[b] + h * own_head + plan::row_tile_start(rt, own_tiles), own_tiles,
                      plan::weight(plan::tile_rows(m_own, rt)), m - rt * plan::kTileRows, all + place, prefix_total == 0))
            continue;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        if (lane * 4 < D) {
            uint2 v;
            v.x = float_to_pair<T>(acc[0] * inv, acc[1] * inv);
            v.y = float_to_pair<T>(acc[2] * inv, acc[3] * inv);
            *reinterpret_cast<uint2 *>(out + lane * 4) = v;
        }
        if (lane == 0 && a.lse) a.lse[place] = l == 0.f ? -INFINITY : kLn2 * (top + log2f(l));
    }
}

struct Regions {
    size_t stats, o, bytes;
};
Regions regions(int B, int n_rows, int n_q_heads, int D) {
    const size_t parts = 2 * (size_t)n_rows * n_q_heads + (size_t)kCtas * plan::kTileRows;
    Regions g;
    g.stats = align_up((size_t)B * sizeof(int64_t), 256);
    g.o = align_up(g.stats + parts * sizeof(float2), 256);
    g.bytes = align_up(g.o + parts * D * sizeof(float), 256);
    return g;
}

template <typename T, int kFormat, int DP>
cudaError_t launch_t(const AttentionArgs &a, const Partials &p, cudaStream_t s) {
    static PerDeviceOnce once;
    auto *kernel = attention_kernel<T, kFormat, DP>;
    cudaError_t e = once.run([&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<DP>::kBytes);
    });
    if (e != cudaSuccess) return e;
    kernel<<<kCtas, kThreads, Layout<DP>::kBytes, s>>>(a, p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    // enough blocks per request for the rows of an average one
    const int64_t per = ((int64_t)a.rows.n_rows * a.n_q_heads + a.rows.B - 1) / a.rows.B;
    const int y = (int)((per + kJoinWarps - 1) / kJoinWarps);
    return launch_dependent(attention_join_kernel<T>, dim3(a.rows.B, y < 1024 ? y : 1024), dim3(kJoinWarps * 32), 0, s, a, p);
}

template <typename T>
cudaError_t launch_format(const AttentionArgs &a, const Partials &p, cudaStream_t s) {
    const bool e4m3 = a.cache.format == DSPARK_KV_E4M3;
    if (a.cache.head_dim <= 64)
        return e4m3 ? launch_t<T, DSPARK_KV_E4M3, 64>(a, p, s) : launch_t<T, DSPARK_KV_INT8, 64>(a, p, s);
    return e4m3 ? launch_t<T, DSPARK_KV_E4M3, 128>(a, p, s) : launch_t<T, DSPARK_KV_INT8, 128>(a, p, s);
}

}  // namespace

size_t attention_ws_bytes(int B, int n_rows, int n_q_heads, int, int head_dim) {
    return regions(B, n_rows, n_q_heads, head_dim).bytes;
}

cudaError_t launch_block_attention(const AttentionArgs &a, cudaStream_t s) {
    const Regions g = regions(a.rows.B, a.rows.n_rows, a.n_q_heads, a.cache.head_dim);
    const Partials p{reinterpret_cast<int64_t *>(a.ws), reinterpret_cast<float2 *>(a.ws + g.stats),
                     reinterpret_cast<float *>(a.ws + g.o)};
    return a.dt == DSPARK_BF16 ? launch_format<__nv_bfloat16>(a, p, s) : launch_format<__half>(a, p, s);
}

}  // namespace dspark
