// Attention of each request's block rows over a shared prefix and the
// request's own tokens, both in the quantised cache.
//
// Mathematics.  Row m (a block row of a query head) against tokens j, with 8-bit
// codes k~, v~ and scales ks, vs: scores s_j = c ks_j (q . k~_j) in log2 units,
// and with any reference r
//   O = sum_j 2^(s_j - r) v_j,   l = sum_j 2^(s_j - r),   out = O / l,
//   lse = ln 2 (r + log2 l).
// Both products run on the fp16 tensor cores with fp32 sums:
//   q . k~   codes are exact in fp16, and so is q after a power-of-two scaling (to
//            2^-25 of its row's largest element); ks_j stays in fp32 and multiplies
//            the sums, since rounding keys would err by 2^-11 of every score.
//   P . V    codes are exact again; P = 2^(s_j - r) (2^12 vs_j) rounded to fp16, from
//            fp32 factors.  r is an integer, the row's own: it follows the largest
//            s_j + log2 vs_j of the tokens that the row sees, whatever values
//            others hold, and moves only when a P passes fp16's range, then
//            starting again at 2^7, and O is scaled by an exact power of two.
// So the inner terms take one rounding of 2^-11, everything else is fp32.
// (The 2^12 sets where a term of l lies in fp32's range: the largest is 2^-105 for value
// scales of 2^100 and 2^95 for those of 2^-100.  The reference also moves when 32 terms pass
// 2^105, which those of values near 0 could without P showing it.)
//
// One CTA per SM walks its part of the plan's line of tiles (attention_plan.h),
// 128 tokens a tile.  Roles (20 warps):
//   0      issues the tensor-core products
//   1      plans: rounds of up to four tiles for each group
//   2      loads codes, 3 scales (bulk copies)
//   4-11   two softmax groups of 128 threads, a thread per row (TMEM lane)
//   12-15  keys to fp16 operands in the swizzled layout, 16-19 values; queries by both
// A pair tile's keys and values serve both groups; single tiles alternate
// between the groups' own items.  Operands are loaded, converted and used in
// one order: of pairs K0 V0 K1 V1 .., so that a tile's values are converted
// under the products of the tile before; of singles K0 K1 V0 K2 V1 .., keys one
// tile ahead, so that a group's scores are ready while the other group's softmax
// runs.  Every ring is filled in this order or freed in it, both loaders arrive on
// every place of theirs (so that neither can be a lap ahead of the other), and the
// converter teams wait for their operand's place before they look for its codes: so
// no wait is more than one lap of a ring away from the phase that it tests, whose
// parity would deceive it.  Every wait is bounded.
//
// What bounds it (SM clocks): a pair tile takes 5,100 to 5,600 where its products
// take 2,048, its exponentials 1,024 and all its instructions 2,900 of every
// scheduler; a single tile 2,700 to 3,000 where its products take 1,024: the
// chain of issuer, product, softmax and issuer, as P takes its scores' columns.  An
// item adds some 6,700 to a CTA with two groups at work (queries, first reference,
// result), which is why the plan counts it.  Measured: 153 rows of 32 query
// heads over 131,000 shared tokens in 408 us (805 TFLOP/s of the rows' products),
// 64 single tokens of 64 heads over 300,000 own tokens in 240 us (2.7 TB/s).
// The roles' loops together nearly fill the instruction cache, so less code
// was faster again and again: 64 scores at a time instead of 32 cost 1 to 10%, two
// issuing warps 7%, 24 warps with the issuer apart from the converters 15%.
#include <type_traits>

#include "attention_plan.h"
#include "paged_rows.cuh"
#include "tc_primitives.cuh"

namespace dspark {
namespace {

using namespace tc;

constexpr int kThreads = 640;
// warps of the roles
constexpr int kIssuer = 0, kPlanner = 1, kCodes = 2, kSoftmaxAt = 4, kConvertAt = 12, kTeamWarps = 4;
// registers a thread: of the launch, and as the roles share them out (a role that asks for more than
// there is would wait for ever: checked before the launch)
constexpr int kLaunchRegs = 96, kSoftmaxRegs = 128, kConvertRegs = 64;
static_assert(256 * kSoftmaxRegs + 2 * kTeamWarps * 32 * kConvertRegs + 128 * kLaunchRegs <= kThreads * kLaunchRegs, "");
constexpr int kCtas = kNumSMs;
constexpr int kRing = 8;          // pieces of a group told ahead
constexpr int kRounds = 4;        // rounds planned ahead
constexpr int kScaleSlots = 3;    // tiles of a group whose scales are held: the keys of tile t wait for a place that the
                                  // values of tile t - 3 (or later ones) have left, so for the end of its softmax
constexpr uint32_t kSpinLimit = 2000000000u;    // ~1 s of clock cycles (below the 32-bit clock's lap)
constexpr long long kDrainLimit = 200000000LL;  // ~0.1 s: products in flight after a timeout

constexpr uint32_t kColS = 0, kColO = 256;  // TMEM columns: scores (and P) of the groups, then their outputs

constexpr float kVUp = 0x1p12f, kVDown = 0x1p-12f;   // what value scales are multiplied by, and its inverse
constexpr float kVLeast = -88.f;           // log2 of the least of these that the reference counts: value scales
                                           // below 2^-100 lose precision, not range
constexpr float kPeak = 7.f;               // log2 of P's largest bound when the reference moves ...
constexpr uint32_t kPast = 0x7c00u;        // ... which it does when a P reaches these bits, fp16's infinity,
constexpr float kSumMost = 0x1p105f;       // or when 32 terms of l sum to more than this
constexpr float kQUp = 16.f;               // what q is multiplied by before it becomes fp16 ...
constexpr int kQLow = -4, kQHigh = 11;     // ... when its row's largest element lies in [2^-4, 2^11)

enum { kDirect = 0, kFirst = 1, kContinued = 2 };
// tile flags: bits 0, 1 the groups that take part
enum { kTileFirst = 4, kTileLast = 8, kTileEnd = 16 };

// Shared memory: operands first (1024-byte aligned for the swizzle)
template <int DP>
struct Layout {
    static constexpr int kOps = 3;                    // fp16 operand ring (K and V tiles)
    static constexpr int kRaw = DP == 128 ? 3 : 6;    // ring of tiles as loaded
    static constexpr uint32_t kTileBytes = 128 * DP * 2;
    static constexpr uint32_t kRawBytes = 128 * DP + 1024;  // codes; with the keys both scales
    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kOp = kQ + 2 * kTileBytes;
    static constexpr uint32_t kRawAt = kOp + kOps * kTileBytes;
    static constexpr uint32_t kScale = kRawAt + kRaw * kRawBytes;         // [groups][slots][2][128] scales: keys', values'
    static constexpr uint32_t kQScale = kScale + 2 * kScaleSlots * 1024;  // [groups][2 pieces][128]
    static constexpr uint32_t kBytes = kQScale + 2048 + 1024;            // + alignment slack
};

// Consecutive tiles of one item
struct Piece {
    int tiles, first;   // how many, and the first one's number in the item
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
// Up to four tiles of each group, taken in turns: 0 of the first, 0 of the
// second, 1 of the first ..; pairs as tiles of the first.
struct Round {
    int flags;                    // kRoundPair, kRoundEnd; bits 2 s, 2 s + 1: the first / last tile of stream s's piece is here
    int n[2], token[2], piece[2]; // of the streams: tiles, first token, place of the piece
    uint32_t chunks[2][32];       // where the tokens are, 16 a chunk, 8 chunks a tile
};
enum { kRoundPair = 16, kRoundEnd = 32 };

// The order of operands: places of the keys of tile after tile, and of the values
// that go with them (of the same pair, or of the single before).
struct Order {
    uint32_t tile, k, v;
    bool has_v, single;           // values at `v`; the last tile was a single
    __device__ __forceinline__ void step(int flags) {
        const bool end = flags & kTileEnd, pair = (flags & 3) == 3;
        k = 2 * tile - (!pair && single ? 1 : 0);
        v = pair ? 2 * tile + 1 : end ? 2 * tile - 1 : 2 * tile;
        has_v = pair || single;
        single = !pair;
        ++tile;
    }
};

// Device workspace: where partial results go
struct Partials {
    int64_t *unit0[2];  // [B] first own unit of each request in the class's part of the line, after the prefix's
    float2 *stats;      // (r, l): [R Hq] prefix, [R Hq] own, [kCtas][256] continued pairs, [2 kCtas][128] continued singles
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
__device__ __forceinline__ float fast_exp2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float fast_log2(float x) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
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

// Bounded wait of a whole warp on one barrier: false when it took longer than
// about a second or another warp gave up.  (Kept small: it stands in the code
// some thirty times, and the roles' loops have to stay in the instruction cache
// together.)
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort) {
    const uint32_t t0 = (uint32_t)clock();
    bool ok;
#pragma unroll 1
    while (!(ok = mbar_try_wait_sleep(bar, parity, 20000u)))
        if (*abort || (uint32_t)clock() - t0 > kSpinLimit) break;
    return __all_sync(0xffffffffu, ok);
}

// A value that all lanes hold, in the form the compiler knows to be so.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

template <int kRegs>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// ---------------------------------------------------------------- the result --
// eight floats times f, a whole 32-byte sector at once
__device__ __forceinline__ void store8(float *to, const uint32_t *x, float f) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __uint_as_float(x[i]) * f;
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "f"(y[0]), "f"(y[1]), "f"(y[2]),
                 "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7])
                 : "memory");
}

// ------------------------------------------------------------------ the plan --
// The line as a CTA sees it.
struct Line {
    int group, prefix_m, prefix_tiles;
    int64_t prefix[2], pairs, total;   // units of the prefix's items by class, of all pairs, of all
};

// Walks one worker's pieces of a class.  Lives in shared memory and is stepped
// out of line by the planner's warp, all lanes alike: it runs once a piece, and
// its registers and code would burden the loop over tiles.
struct Walk {
    int64_t u, hi, start;             // cursor, end, first unit of the item at the cursor
    int cls, b, head, k, m, tiles;    // that item: request (-1: the prefix), head, row tile of the class, rows, tiles
    int wb;                           // 32 requests' sizes from request wb on:
    int w_n[32], w_len[32], w_first[32];

    __device__ __forceinline__ void window(const AttentionArgs &a, int group, int from, int lane) {
        __syncwarp();
        int n = 0, len = 0, first = 0;
        if (from + lane < a.rows.B) {
            const Request q = load_request(a, from + lane);
            n = q.len_ok && plan::class_tiles(cls, q.n * group) > 0 ? q.n : 0;
            len = q.len;
            first = (int)q.first;
        }
        w_n[lane] = n;
        w_len[lane] = len;
        w_first[lane] = first;
        wb = from;
        __syncwarp();
    }
    // the next request with items of the class, from b on; false when there is none
    __device__ __forceinline__ bool seek(const AttentionArgs &a, int group, int lane) {
        int at = b;
        while (at < a.rows.B) {
            if (at >= wb + 32) window(a, group, at, lane);
            const unsigned with = __ballot_sync(0xffffffffu, w_n[lane] > 0) & (0xffffffffu << (at - wb));
            if (with) {
                at = wb + __ffs(with) - 1;
                __syncwarp();
                b = at;
                m = w_n[at - wb] * group;
                tiles = plan::token_tiles(w_len[at - wb]);
                __syncwarp();
                return true;
            }
            at = wb + 32;
        }
        __syncwarp();
        b = at;
        __syncwarp();
        return false;
    }
};
// (All lanes store the same values to a walk's fields.)

// from unit `lo` to `to` of the line; own items begin in request b0 at unit own0 of the class's
__device__ __noinline__ void walk_begin(const AttentionArgs &a, const Line &z, Walk &k, int cls, int64_t lo, int64_t to,
                                        int b0, int64_t own0, int lane) {
    __syncwarp();
    k.cls = cls;
    k.u = lo;
    k.hi = to;
    k.wb = -32;
    k.b = -1;
    __syncwarp();
    if (lo >= to) return;
    int64_t at = cls == plan::kPair ? 0 : z.pairs;
    if (lo - at < z.prefix[cls]) {
        k.m = z.prefix_m;
        k.tiles = z.prefix_tiles;
    } else {
        k.b = b0;
        k.window(a, z.group, b0, lane);
        if (!k.seek(a, z.group, lane)) {
            k.u = to;
            __syncwarp();
            return;
        }
        at += z.prefix[cls] + own0;
    }
    __syncwarp();
    const int64_t per = plan::head_units(cls, k.m, k.tiles), item = plan::item_total(cls, k.tiles);
    const int64_t head = (lo - at) / per, t = (lo - at - head * per) / item;
    k.head = (int)head;
    k.k = (int)t;
    k.start = at + head * per + t * item;
    __syncwarp();
}
// the next piece, to `slot`; its tiles, 0 when there is none
__device__ __noinline__ int walk_next(const AttentionArgs &a, const Line &z, Walk &k, Piece &slot, int lane) {
    __syncwarp();
    while (k.u < k.hi) {
        const int cls = k.cls, b = k.b, m = k.m, tiles = k.tiles, head = k.head, kk = k.k;
        const int64_t start = k.start;
        const int t0 = plan::first_tile(cls, k.u, start, tiles), t1 = plan::first_tile(cls, k.hi, start, tiles);
        const int rt = plan::class_row_tile(cls, m, kk);
        Piece p;
        p.tiles = t1 - t0;
        p.first = t0;
        p.rows = plan::tile_rows(m, rt);
        p.m0 = rt * plan::kTileRows;
        p.head = head;
        p.request = b;
        p.row_base = b < 0 ? 0 : k.w_first[b - k.wb];
        p.len = b < 0 ? a.prefix_len : k.w_len[b - k.wb];
        p.n = b < 0 ? 0 : k.w_n[b - k.wb];
        p.ctx = p.len - p.n;
        p.out = t0 > 0 ? kContinued : (b >= 0 && z.prefix_tiles == 0 && t1 == tiles) ? kDirect : kFirst;
        p.pad = 0;
        __syncwarp();
        // the cursor moves to the next item
        k.start = k.u = start + plan::item_total(cls, tiles);
        if (kk + 1 < plan::class_tiles(cls, m)) {
            k.k = kk + 1;
        } else {
            k.k = 0;
            if (head + 1 < a.cache.n_kv_heads) {
                k.head = head + 1;
            } else {
                k.head = 0;
                k.b = b + 1;
                __syncwarp();
                if (!k.seek(a, z.group, lane)) k.u = k.hi;
            }
        }
        if (p.tiles > 0) {
            if (lane == 0) slot = p;
            __syncwarp();
            return p.tiles;
        }
        __syncwarp();
    }
    return 0;
}

// A worker's tiles in order, with the cache places of their tokens.  Places are
// kept by chunk of 16 tokens (a chunk lies inside one page), as the chunk's
// number in the cache, in units of 16 head rows: 32 chunks (4 tiles) at a time,
// one a lane, their pages loaded four tiles before they are needed.
constexpr uint32_t kNoChunk = 0xffffffffu, kBadChunk = 0xfffffffeu;
// Pieces a stream's tiles refer to: a slot is written again only after every
// tile of its piece has left the rings (the next piece is planned while the last
// one's tiles are taken, hence more than kRing slots).
constexpr int kPieces = 2 * kRing;
// (In shared memory, as there are two and the loop over tiles should be one.)
struct Stream {
    int j, tiles;                      // next tile of the piece, its tiles (0: no more pieces)
    uint32_t count;                    // pieces begun
    int page[32], off[32];             // of the next four tiles' chunks, a lane each
    Walk walk;
    Piece slots[kPieces];

    __device__ __forceinline__ void load_pages(const AttentionArgs &a, const Piece &p, int t, int lane) {
        const int per_page = a.cache.page_size / 16, chunk = (p.first + t) * 8 + lane;
        int place = -1, pg = 0;
        if ((int64_t)chunk * 16 < p.len) {
            const int slot = chunk / per_page;
            place = p.head * per_page + (chunk - slot * per_page);
            pg = p.request < 0 ? a.prefix_pages[slot] : a.rows.block_table[(int64_t)p.request * a.rows.max_pages + slot];
        }
        page[lane] = pg;
        off[lane] = place;
    }
};

__device__ __noinline__ void stream_begin(const AttentionArgs &a, const Line &z, Stream &s, int cls, int64_t lo, int64_t to,
                                          int b0, int64_t own0, int lane) {
    walk_begin(a, z, s.walk, cls, lo, to, b0, own0, lane);
    Piece &p = s.slots[s.count % kPieces];
    const int tiles = walk_next(a, z, s.walk, p, lane);
    s.tiles = tiles;
    s.j = 0;
    if (tiles) s.load_pages(a, p, 0, lane);
    __syncwarp();
}

// up to four tiles of the stream (s.tiles > 0) to stream `id` of a round; the round's bits of it
__device__ __noinline__ int stream_round(const AttentionArgs &a, const Line &z, Stream &s, Round &r, int id, int lane) {
    const int j = s.j, tiles = s.tiles, n = min(tiles - j, 4);
    const uint32_t count = s.count;
    const int off = s.off[lane], page = s.page[lane];
    r.chunks[id][lane] = off < 0 ? kNoChunk
                         : (page < 0 || page >= a.cache.n_pages)
                             ? kBadChunk
                             : (uint32_t)page * (uint32_t)(a.cache.n_kv_heads * (a.cache.page_size / 16)) + (uint32_t)off;
    const bool last = j + n == tiles;
    const Piece *p = s.slots + count % kPieces;
    if (lane == 0) {
        r.n[id] = n;
        r.token[id] = (p->first + j) * plan::kTile;
        r.piece[id] = id * kPieces + (int)(count % kPieces);
    }
    __syncwarp();
    int next = tiles;
    if (last) {
        p = s.slots + (count + 1) % kPieces;
        next = walk_next(a, z, s.walk, s.slots[(count + 1) % kPieces], lane);
    }
    s.j = last ? 0 : j + n;
    s.tiles = next;
    s.count = count + (last ? 1 : 0);
    if (next) s.load_pages(a, *p, last ? 0 : j + n, lane);
    __syncwarp();
    return (j == 0 ? 1 << (2 * id) : 0) | (last ? 2 << (2 * id) : 0);
}

// ------------------------------------------------------------------------- q --
// Up to 128 rows of a row tile, from its row t0 on, to fp16 in the swizzled
// layout, all multiplied by kQUp; a row whose largest element is far from 1 is
// instead taken into [2^7, 2^8) by a power of two of its own, and qscale[row] is
// the factor its scores then lack (1 for the others).  Warp `part` of `parts`
// takes every parts-th group of rows.
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
                const int e2 = max((int)(top >> 23) - 127, -110);
                float mul = kQUp, lack = 1.f;
                if (top >= 0x7f800000u) {
                    mul = __int_as_float(0x7fffffff);
                } else if (top != 0 && (e2 < kQLow || e2 >= kQHigh)) {
                    mul = __uint_as_float((uint32_t)(127 + 7 - e2) << 23);
                    lack = __uint_as_float((uint32_t)(127 - 7 + e2) << 23) * kQUp;
                }
                if (sub == 0) qscale[r] = lack;
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
    __shared__ __align__(8) uint64_t bars[2 * kRaw + 2 * kOps + 4 * kRing + 2 * kRounds + 16];
    __shared__ int group_pieces[2][kRing];          // pieces of the softmax groups: slot, flags
    __shared__ Stream streams[2];
    __shared__ Round rounds[kRounds];
    __shared__ int raw_bad[kRaw];
    __shared__ int64_t scan[2][kThreads / 32];
    __shared__ Line line;
    __shared__ int64_t found_units[3], from_s[3], to_s[3];   // of the workers: pairs, and each group's singles
    __shared__ int found_request[3];
    __shared__ int misc[3];       // abort, a word that stays 0, TMEM address

    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    const dspark_kv_cache &c = a.cache;
    const int D = c.head_dim, group = a.n_q_heads / c.n_kv_heads;
    const uint32_t base = (smem_u32(dyn) + 1023u) & ~1023u;
    unsigned char *gen = dyn + (base - smem_u32(dyn));
    volatile int *abort = misc, *never = misc + 1;
    auto piece_at = [&](int i) -> const Piece & { return streams[i / kPieces].slots[i % kPieces]; };

    // barriers
    const uint32_t bar0 = smem_u32(bars);
    auto raw_full = [&](uint32_t i) { return bar0 + 8u * i; };
    auto raw_empty = [&](uint32_t i) { return bar0 + 8u * (kRaw + i); };
    auto op_full = [&](uint32_t i) { return bar0 + 8u * (2 * kRaw + i); };
    auto op_empty = [&](uint32_t i) { return bar0 + 8u * (2 * kRaw + kOps + i); };
    auto piece_full = [&](int w, uint32_t i) { return bar0 + 8u * (2 * kRaw + 2 * kOps + (uint32_t)w * kRing + i); };
    auto piece_empty = [&](int w, uint32_t i) { return bar0 + 8u * (2 * kRaw + 2 * kOps + (uint32_t)(w + 2) * kRing + i); };
    auto round_full = [&](uint32_t i) { return bar0 + 8u * (2 * kRaw + 2 * kOps + 4 * kRing + i); };
    auto round_empty = [&](uint32_t i) { return bar0 + 8u * (2 * kRaw + 2 * kOps + 4 * kRing + kRounds + i); };
    const uint32_t bar1 = bar0 + 8u * (uint32_t)(2 * kRaw + 2 * kOps + 4 * kRing + 2 * kRounds);
    auto q_full = [&](int i) { return bar1 + 8u * (uint32_t)i; };
    auto q_empty = [&](int i) { return bar1 + 8u * (uint32_t)(2 + i); };
    auto s_full = [&](int i) { return bar1 + 8u * (uint32_t)(4 + i); };
    auto p_ready = [&](int i) { return bar1 + 8u * (uint32_t)(6 + i); };
    auto o_full = [&](int i) { return bar1 + 8u * (uint32_t)(8 + i); };
    auto o_free = [&](int i) { return bar1 + 8u * (uint32_t)(10 + i); };
    const uint32_t drain = bar1 + 8u * 12u;

    if (tid == 0) {
        for (int i = 0; i < kRaw; ++i) mbar_init(raw_full(i), 2), mbar_init(raw_empty(i), kTeamWarps);
        for (int i = 0; i < kOps; ++i) mbar_init(op_full(i), kTeamWarps), mbar_init(op_empty(i), 1);
        for (int i = 0; i < kRounds; ++i) mbar_init(round_full(i), 1), mbar_init(round_empty(i), 3 + 2 * kTeamWarps);
        for (int i = 0; i < kRing; ++i)
            for (int w = 0; w < 2; ++w) mbar_init(piece_full(w, i), 1), mbar_init(piece_empty(w, i), 4);
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full(i), 2 * kTeamWarps), mbar_init(q_empty(i), 1);
            mbar_init(s_full(i), 1), mbar_init(p_ready(i), 4);
            mbar_init(o_full(i), 1), mbar_init(o_free(i), 4);
        }
        mbar_init(drain, 1);
        fence_mbar_init();
        misc[0] = misc[1] = 0;
        for (int i = 0; i < 3; ++i) found_request[i] = a.rows.B, found_units[i] = 0;
    }
    if (warp == kIssuer) {
        tmem_alloc(smem_u32(misc + 2), 512);
        tmem_relinquish();
    }

    // ---- the line of units, and the requests this CTA's workers start in
    const int prefix_m = prefix_rows(a) * group, prefix_tiles = plan::token_tiles(a.prefix_len);
    int64_t prefix[2];
    for (int k = 0; k < 2; ++k) prefix[k] = plan::head_units(k, prefix_m, prefix_tiles) * c.n_kv_heads;
    auto request_units = [&](int b, int64_t (&x)[2]) {
        x[0] = x[1] = 0;
        if (b >= a.rows.B) return;
        const Request q = load_request(a, b);
        if (blockIdx.x == 0 && (!q.rows_ok || (q.n > 0 && !q.len_ok))) atomicOr(c.flags, kFlagBadLength);
        if (!q.len_ok || q.n == 0) return;
        const int tiles = plan::token_tiles(q.len);
        for (int k = 0; k < 2; ++k) x[k] = plan::head_units(k, q.n * group, tiles) * c.n_kv_heads;
    };
    int64_t mine[2];
    request_units(tid, mine);   // the first kThreads requests' units stay in registers
    {
        int64_t sum[2] = {mine[0], mine[1]};
        for (int b = tid + kThreads; b < a.rows.B; b += kThreads) {
            int64_t x[2];
            request_units(b, x);
            sum[0] += x[0], sum[1] += x[1];
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], d);
            sum[1] += __shfl_xor_sync(0xffffffffu, sum[1], d);
        }
        if (lane == 0) scan[0][warp] = sum[0], scan[1][warp] = sum[1];
    }
    __syncthreads();
    int64_t pairs = prefix[0], total = prefix[1];
    for (int w = 0; w < kThreads / 32; ++w) pairs += scan[0][w], total += scan[1][w];
    total += pairs;
    int64_t from[3];
    from[0] = plan::cta_begin(blockIdx.x, total, kCtas);
    for (int w = 0; w < 2; ++w) from[1 + w] = plan::single_begin(2 * blockIdx.x + w, pairs, total, kCtas);
    if (tid == 0) {
        line.group = group;
        line.prefix_m = prefix_m;
        line.prefix_tiles = prefix_tiles;
        line.prefix[0] = prefix[0];
        line.prefix[1] = prefix[1];
        line.pairs = pairs;
        line.total = total;
        for (int i = 0; i < 3; ++i) from_s[i] = from[i];
        const int64_t end = plan::cta_begin(blockIdx.x + 1, total, kCtas);
        to_s[0] = end < pairs ? end : pairs;
        to_s[1] = from[2];
        to_s[2] = plan::single_begin(2 * blockIdx.x + 2, pairs, total, kCtas);
    }
    {
        int64_t before[2] = {0, 0};
        for (int b0 = 0; b0 < a.rows.B; b0 += kThreads) {
            const int b = b0 + tid;
            int64_t x[2] = {mine[0], mine[1]};
            if (b0 > 0) request_units(b, x);
            int64_t v[2] = {x[0], x[1]};
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t y0 = __shfl_up_sync(0xffffffffu, v[0], d), y1 = __shfl_up_sync(0xffffffffu, v[1], d);
                if (lane >= d) v[0] += y0, v[1] += y1;
            }
            __syncthreads();
            if (lane == 31) scan[0][warp] = v[0], scan[1][warp] = v[1];
            __syncthreads();
            for (int k = 0; k < 2; ++k) {
                int64_t at = before[k] + v[k] - x[k];
                for (int w = 0; w < kThreads / 32; ++w) {
                    if (w < warp) at += scan[k][w];
                    before[k] += scan[k][w];
                }
                if (b >= a.rows.B) continue;
                if (blockIdx.x == 0) parts.unit0[k][b] = at;
                for (int i = k == 0 ? 0 : 1; i < (k == 0 ? 1 : 3); ++i) {
                    // the own unit to start at
                    const int64_t want = max(from[i] - (k == 0 ? 0 : pairs) - prefix[k], (int64_t)0);
                    if (x[k] > 0 && at <= want && want < at + x[k]) {
                        found_request[i] = b;
                        found_units[i] = at;
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform(misc[2]);

    // Walks the planned tiles: body(flags, stream, number in the round, round) for each, and for the end;
    // false when it or a wait gives up.
    auto for_tiles = [&](auto body) {
#pragma unroll 1
        for (uint32_t k = 0;; ++k) {
            const uint32_t e = k % kRounds;
            if (!warp_wait(round_full(e), (k / kRounds) & 1, abort)) return false;
            const Round &r = rounds[e];
            const int bits = uniform(r.flags);
            const int n0 = uniform(r.n[0]), n1 = uniform(r.n[1]);
            const int turns = (bits & kRoundEnd) ? 1 : 2 * max(n0, n1);
#pragma unroll 1
            for (int x = 0; x < turns; x += (bits & kRoundPair) ? 2 : 1) {
                const int id = x & 1, i = x >> 1, n = id ? n1 : n0;
                int flags = kTileEnd;
                if (!(bits & kRoundEnd)) {
                    if (i >= n) continue;
                    flags = ((bits & kRoundPair) ? 3 : 1 << id) | (i == 0 && (bits >> (2 * id) & 1) ? kTileFirst : 0) |
                            (i + 1 == n && (bits >> (2 * id + 1) & 1) ? kTileLast : 0);
                }
                if (!body(flags, id, i, r)) return false;
            }
            if (bits & kRoundEnd) return true;
            __syncwarp();
            if (lane == 0) mbar_arrive(round_empty(e));
        }
    };

    // Loads the keys or values of a tile, chunk `mine` in lanes 0 .. 7 (and again in 8 .. 15 and so
    // on), to place `position` of the order of operands, in runs of tokens that share a page: their
    // codes or (another warp) with the keys the scales of both.  (Copies by the warp's own cp.async,
    // 512 bytes at a time, held it up: 2300 clocks a tile.)
    const int run = min(c.page_size & -c.page_size, plan::kTile), runs = plan::kTile / run;
    auto load = [&](uint32_t mine, bool is_v, uint32_t position, bool codes) {
        const int i = lane & 7;
        const uint32_t id = __shfl_sync(0xffffffffu, mine, (i * (run / 16)) & 7);
        const bool good = i < runs && id < kBadChunk;
        const unsigned bad = __ballot_sync(0xffffffffu, mine == kBadChunk) & 0xffu;
        const uint32_t n = (uint32_t)__popc(__ballot_sync(0xffffffffu, good) & 0xffu);
        const uint32_t slot = position % kRaw;
        if (!warp_wait(raw_empty(slot), ((position / kRaw) & 1) ^ 1, abort)) return false;
        const uint32_t at = base + L::kRawAt + slot * L::kRawBytes;
        if (lane == 0) {
            if (codes) raw_bad[slot] = (int)bad;
            mbar_arrive_expect_tx(raw_full(slot), n * (uint32_t)(run * (codes ? D : is_v ? 0 : 8)));
        }
        __syncwarp();
        const bool leader = elect_one();
#pragma unroll 1
        for (int r = 0; r < runs; ++r) {
            const uint32_t from = (uint32_t)uniform((int)__shfl_sync(0xffffffffu, mine, r * (run / 16)));
            if (from >= kBadChunk || !leader) continue;
            const uint64_t first = (uint64_t)from * 16u;      // head row of the run's first token
            if (codes) {
                bulk_load(at + (uint32_t)(r * run * D),
                          static_cast<const unsigned char *>(is_v ? c.v : c.k) + first * (uint32_t)D, (uint32_t)(run * D),
                          raw_full(slot));
            } else if (!is_v) {
                const uint32_t to = at + 128u * DP + (uint32_t)(r * run * 4), bytes = (uint32_t)(run * 4);
                bulk_load(to + 512u, c.v_scale + first, bytes, raw_full(slot));
                bulk_load(to, c.k_scale + first, bytes, raw_full(slot));
            }
        }
        __syncwarp();
        if (codes && bad && lane == 0) atomicOr(c.flags, kFlagBadPage);
        return true;
    };
    // One team of converters: the keys or the values of all tiles, and half of the queries.  The lanes of a quarter
    // warp take four chunks each of the lower and the upper 64 columns of an even and an odd row:
    // neither their loads nor their stores (the swizzle takes even chunks of an odd row to odd places)
    // meet in a bank.
    auto convert_all = [&](const bool is_v) {
        const int t = (tid - kConvertAt * 32) & (kTeamWarps * 32 - 1);
        const float up = a.scale * kLog2e / kQUp;    // scores in log2 units: folded into the keys' scales
        uint32_t scale_slots = 0;                    // where the groups' next scales go, 8 bits each
        uint32_t group_pieces_seen = 0;              // parity of the groups' pieces
        int valid = 0;                               // tokens of the tile that exist (128 or more: all)
        Order order = {0, 0, 0, false, false};
        return for_tiles([&](int flags, int id, int i, const Round &r) {
            const bool end = flags & kTileEnd, pair = (flags & 3) == 3;
            const int valid_before = valid;
            order.step(flags);
            if (!end) {
                const Piece &p = piece_at(uniform(r.piece[id]));
                valid = uniform(p.len) - uniform(r.token[id]) - i * plan::kTile;
                if (flags & kTileFirst) {
                    // the piece's queries, by both teams
#pragma unroll 1
                    for (int w = 0; w < 2; ++w) {
                        if (!(flags >> w & 1)) continue;
                        const uint32_t seen = group_pieces_seen >> w & 1;
                        if (!warp_wait(q_empty(w), seen ^ 1, abort)) return false;
                        load_q<T, DP>(a, p, pair ? w * 128 : 0, warp - kConvertAt, 2 * kTeamWarps, group,
                                      base + L::kQ + (uint32_t)w * L::kTileBytes,
                                      reinterpret_cast<float *>(gen + L::kQScale) + w * 256 + (int)seen * 128, lane);
                        group_pieces_seen ^= 1u << w;
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(q_full(w));
                    }
                }
            }
            if (is_v ? !order.has_v : end) return true;
            // the operand: the tile's keys, or the values whose turn it is
            const int there_are = is_v && !pair ? valid_before : valid;
            const uint32_t position = is_v ? order.v : order.k;
            const uint32_t slot = position % kRaw, op = position % kOps;
            if (!warp_wait(op_empty(op), ((position / kOps) & 1) ^ 1, abort)) return false;
            if (!warp_wait(raw_full(slot), (position / kRaw) & 1, abort)) return false;
            const uint32_t src = base + L::kRawAt + slot * L::kRawBytes, dst = base + L::kOp + op * L::kTileBytes;
            const uint32_t raw_scale = src + 128u * DP;   // with the keys: key scales, then value scales
            const int bad = uniform(raw_bad[slot]);
            const bool whole = there_are >= plan::kTile && bad == 0;
            auto there = [&](int row) { return whole || (row < there_are && !(bad >> (row >> 4) & 1)); };
            auto decode_store = [&](uint4 in, uint32_t row, uint32_t ch) {
                __half2 h[8];
                decode4<kFormat>(in.x, h[0], h[1]);
                decode4<kFormat>(in.y, h[2], h[3]);
                decode4<kFormat>(in.z, h[4], h[5]);
                decode4<kFormat>(in.w, h[6], h[7]);
                const uint32_t *u = reinterpret_cast<const uint32_t *>(h);
                const uint32_t at = dst + (ch >> 2) * (128u * 128u) + row * 128u, c8 = (ch & 3u) * 2u;
                st_shared_v4(at + ((c8 ^ (row & 7u)) << 4), make_uint4(u[0], u[1], u[2], u[3]));
                st_shared_v4(at + (((c8 + 1u) ^ (row & 7u)) << 4), make_uint4(u[4], u[5], u[6], u[7]));
            };
            // nothing of a token that is not there
            auto read = [&](int row, int ch, int width) {
                const uint4 in = ld_shared_v4(src + (uint32_t)(row * width + ch) * 16u);
                return there(row) ? in : make_uint4(0, 0, 0, 0);
            };
            if (!is_v) {
                // the tile's scales for the softmax groups: keys' (of scores in log2 units) and values'; a token
                // whose value scale (or page) is no number carries its NaN in the key's alone: where it is
                // masked, its zero weight must not become 0 times NaN
                float ks = 0.f, vs = 0.f;
                if (t < there_are) {
                    const float v = ld_shared_f32(raw_scale + 512u + 4u * (uint32_t)t);
                    const bool good = there(t) && v <= 3.4028235e38f;
                    ks = good ? ld_shared_f32(raw_scale + 4u * (uint32_t)t) * up : __int_as_float(0x7fffffff);
                    vs = good ? fminf(v * kVUp, 3.4028235e38f) : 0.f;
                }
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    if (!(flags >> w & 1)) continue;
                    const uint32_t i = scale_slots >> (8 * w) & 3u;
                    const uint32_t to = base + L::kScale + ((uint32_t)(w * kScaleSlots) + i) * 1024u + 4u * (uint32_t)t;
                    st_shared_f32(to, ks);
                    st_shared_f32(to + 512u, vs);
                    scale_slots += i + 1 == kScaleSlots ? 0u - (i << (8 * w)) : 1u << (8 * w);
                }
            }
            if (D == DP) {
                constexpr int kSteps = DP / 32;     // two chunks each: of one row (D = 128), of two rows
                const int odd = t >> 2 & 1;
#pragma unroll 1
                for (int step = 0; step < kSteps; ++step) {
                    uint4 in[2];
                    auto row_of = [&](int i) {
                        return DP == 128 ? 2 * ((t >> 3) + 16 * step) + odd : (t >> 2) + 32 * (2 * step + i);
                    };
                    auto chunk_of = [&](int i) { return (t & 3) + (DP == 128 ? 4 * (odd ^ i) : 0); };
#pragma unroll
                    for (int i = 0; i < 2; ++i) in[i] = read(row_of(i), chunk_of(i), DP / 16);
                    if (step + 1 == kSteps) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(raw_empty(slot));
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) decode_store(in[i], (uint32_t)row_of(i), (uint32_t)chunk_of(i));
                }
            } else {
                const int width = D / 16;
#pragma unroll 1
                for (int i = t; i < 128 * width; i += 32 * kTeamWarps) {
                    const int row = i / width;
                    decode_store(read(row, i - row * width, width), (uint32_t)row, (uint32_t)(i - row * width));
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(raw_empty(slot));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(op_full(op));
            return true;
        });
    };

    if (warp < kSoftmaxAt || warp >= kConvertAt) {
        if (warp == kPlanner) {
            // -------------------------------------------------------- planner --
            // pairs, then the first group's singles, are stream 0's tiles, the second group's singles stream 1's
            if (lane < 2) streams[lane].count = 0;
            __syncwarp();
            bool ok = true, pairing = true;
#pragma unroll 1
            for (int i = 2; i >= 0; i -= 2)
                stream_begin(a, line, streams[i >> 1], i == 0 ? plan::kPair : plan::kSingle, from_s[i], to_s[i], found_request[i],
                             found_units[i], lane);
            uint32_t taken = 0;                  // pieces given to the groups, modulo 2^16 (a multiple of the ring's laps)
#pragma unroll 1
            for (uint32_t k = 0; ok; ++k) {
                if (pairing && streams[0].tiles == 0) {
                    pairing = false;
                    stream_begin(a, line, streams[0], plan::kSingle, from_s[1], to_s[1], found_request[1], found_units[1], lane);
                }
                const uint32_t e = k % kRounds;
                if (!warp_wait(round_empty(e), ((k / kRounds) & 1) ^ 1, abort)) { ok = false; break; }
                Round &r = rounds[e];
                int bits = pairing ? kRoundPair : 0;
                if (lane < 2) r.n[lane] = 0;
                __syncwarp();
#pragma unroll 1
                for (int id = 0; id < (pairing ? 1 : 2); ++id)
                    if (streams[id].tiles) bits |= stream_round(a, line, streams[id], r, id, lane);
                __syncwarp();
                const bool end = r.n[0] + r.n[1] == 0;
                // a new piece (or the end) is told to the groups it is for
#pragma unroll 1
                for (int w = 0; w < 2 && ok; ++w) {
                    const int id = pairing ? 0 : w;
                    if (!end && !(bits >> (2 * id) & 1)) continue;
                    const uint32_t n = w ? taken >> 16 : taken & 0xffffu, i = n % kRing;
                    ok = warp_wait(piece_empty(w, i), ((n / kRing) & 1) ^ 1, abort);
                    if (ok && lane == 0) {
                        group_pieces[w][i] = end ? kTileEnd << 16 : r.piece[id] | (pairing ? 3 : 1 << w) << 16;
                        mbar_arrive(piece_full(w, i));
                    }
                    taken = w ? taken + 0x10000u : (taken & 0xffff0000u) | ((taken + 1) & 0xffffu);
                }
                if (!ok) break;
                if (lane == 0) {
                    r.flags = end ? kRoundEnd : bits;
                    mbar_arrive(round_full(e));
                }
                if (end) break;
            }
            if (!ok && lane == 0) *abort = 1;
        } else if (warp >= kCodes && warp < kSoftmaxAt) {
            // -------------------------------------------------------- loaders --
            uint32_t ids = kNoChunk;
            Order order = {0, 0, 0, false, false};
            plan::Filled filled = {0};
            const bool ok = for_tiles([&](int flags, int id, int i, const Round &r) {
                const bool end = flags & kTileEnd, pair = (flags & 3) == 3;
                const uint32_t before = ids;
                order.step(flags);
                if (!end) ids = r.chunks[id][i * 8 + (lane & 7)];
#pragma unroll 1
                for (int v = end ? 1 : 0; v < (order.has_v ? 2 : 1); ++v) {
                    const uint32_t position = v ? order.v : order.k;
                    if (!load(v && !pair ? before : ids, v, position, warp == kCodes)) return false;
                    filled.add(position);
                }
                return true;
            });
            if (!ok) {
                // whatever failed, the copies under way must land before the block's memory goes (the place that
                // the other loader has not filled too takes the whole limit)
                if (lane == 0) *abort = 1;
                for (uint32_t i = 0; i < filled.held(kRaw); ++i)
                    mbar_wait(raw_full(filled.place(i) % kRaw), (filled.place(i) / kRaw) & 1, never, kDrainLimit);
            }
        } else if (warp == kIssuer) {
            // ------------------------------------------- tensor-core products --
            // the whole warp walks the loop, so that addresses stay warp-uniform; one lane issues
            const bool leader = elect_one();
            const uint32_t hi_desc = (uint32_t)(sw128_kmajor_desc(0) >> 32);
            const uint32_t id_qk = idesc_f16_f32(128, 128, false), id_pv = idesc_f16_f32(128, D, true);
            constexpr uint32_t kAtom = 128 * 128;  // bytes of a 64-column atom of a 128-row tile
            Order order = {0, 0, 0, false, false};
            uint32_t laps = 0;      // bits: parity of the next q, P and result of the groups; 6, 7: a group has had a result
            bool ok = true;
            auto wait = [&](uint32_t bar, uint32_t parity) {
                if (ok) ok = warp_wait(bar, parity, abort);
                tc_fence_after();
                return ok;
            };
            auto commit = [&](uint32_t bar) {
                if (leader) umma_commit(bar);
            };
            // scores of group w for a tile: waits for the item's q with its first tile, gives it back with its last
            auto qk = [&](int w, uint32_t k, int flags) {
                if (flags & kTileFirst) {
                    if (!wait(q_full(w), laps >> w & 1)) return;
                    laps ^= 1u << w;
                }
                if (!wait(op_full(k % kOps), (k / kOps) & 1)) return;
                const uint32_t qa = (base + L::kQ + (uint32_t)w * L::kTileBytes) >> 4 | 1u << 16;
                const uint32_t ka = (base + L::kOp + (k % kOps) * L::kTileBytes) >> 4 | 1u << 16;
                const uint32_t d = tmem + kColS + 128u * (uint32_t)w;
                if (leader) {
                    auto step = [&](int i) {
                        const uint32_t off = ((uint32_t)(i >> 2) * kAtom + (uint32_t)(i & 3) * 32u) >> 4;
                        umma_bf16_w(d, qa + off, ka + off, hi_desc, id_qk, i > 0);
                    };
                    if (D == DP) {
#pragma unroll
                        for (int i = 0; i < DP / 16; ++i) step(i);
                    } else {
#pragma unroll 1
                        for (int i = 0; i < D / 16; ++i) step(i);
                    }
                    umma_commit(s_full(w));
                    if (flags & kTileLast) umma_commit(q_empty(w));
                }
            };
            auto pv = [&](int w, uint32_t v, int flags) {
                if (flags & kTileFirst) {
                    if ((laps >> (6 + w) & 1) && !wait(o_free(w), (laps >> (4 + w) & 1) ^ 1)) return;
                    laps = (laps ^ 1u << (4 + w)) | 1u << (6 + w);
                }
                if (!wait(p_ready(w), laps >> (2 + w) & 1)) return;
                laps ^= 1u << (2 + w);
                const uint32_t va = (base + L::kOp + (v % kOps) * L::kTileBytes) >> 4 | (kAtom >> 4) << 16;
                const uint32_t pa = tmem + kColS + 128u * (uint32_t)w, d = pa + kColO - kColS;
                if (leader) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        umma_bf16_ts(d, pa + 8u * (uint32_t)i, va + (uint32_t)i * (2048u >> 4), hi_desc, id_pv,
                                     i > 0 ? 1u : (flags & kTileFirst) ? 0u : 1u);
                    if (flags & kTileLast) umma_commit(o_full(w));
                }
            };
            // Step g: the scores of tile g as soon as a group is free for them (those of the groups that
            // tile g - 1 does not use before tile g - 1's P is waited for), and tile g - 1's output.
            int now = 0;
            uint32_t pair_v = 0;    // place of the last pair's values
            const bool walked = for_tiles([&](int nxt, int, int, const Round &) {
                const int next_mask = nxt & 3, mask = now & 3;
                order.step(nxt);
                const uint32_t ki = order.k, vi = mask == 3 ? pair_v : order.v;
                if (next_mask == 3) pair_v = order.v;
                // passes: 0 and 1 the early scores of the groups, 2 and 3 their outputs and later scores
                uint32_t work = (uint32_t)(next_mask & ~mask) | (uint32_t)mask << 2;
#pragma unroll 1
                while (work && ok) {
                    const int i = __ffs((int)work) - 1, w = i & 1;
                    work &= work - 1;
                    if (i >= 2) {
                        if ((i == 2 || mask == 2) && !wait(op_full(vi % kOps), (vi / kOps) & 1)) break;
                        pv(w, vi, now);
                    }
                    if (ok && next_mask >> w & 1) qk(w, ki, nxt);
                }
                if (!ok) return false;
                // (in the order of their places)
                if (mask == 3) commit(op_empty(vi % kOps));
                if (next_mask) commit(op_empty(ki % kOps));
                if (mask == 1 || mask == 2) commit(op_empty(vi % kOps));
                now = nxt;
                return true;
            });
            ok = ok && walked;
            if (!ok) {
                if (lane == 0) *abort = 1;
                commit(drain);
                mbar_wait(drain, 0, never, kDrainLimit);
            }
        } else {
            // ---------------------------------------------------- converters --
            regs_dec<kConvertRegs>();
            const bool ok = convert_all(warp >= kConvertAt + kTeamWarps);
            if (!ok && lane == 0) *abort = 1;
        }
    } else {
        // -------------------------------------------------------------- softmax --
        regs_inc<kSoftmaxRegs>();
        const int w = (warp - kSoftmaxAt) >> 2, row = tid & 127;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);   // this warp's 32 TMEM lanes
        const uint32_t my_s = lanes + kColS + 128u * (uint32_t)w, my_o = lanes + kColO + 128u * (uint32_t)w;
        bool ok = true;
        uint32_t n = 0;       // tiles of the group so far
        for (uint32_t k = 0; ok; ++k) {
            if (!warp_wait(piece_full(w, k % kRing), (k / kRing) & 1, abort)) { ok = false; break; }
            const int told = uniform(group_pieces[w][k % kRing]), flags = told >> 16;
            if (flags & kTileEnd) break;
            const Piece &p = piece_at(told & 0xffff);
            const bool pair = (flags & 3) == 3;
            const float *qscale = reinterpret_cast<float *>(gen + L::kQScale) + w * 256 + (int)(k & 1) * 128;
            const int rows = uniform(pair ? min(p.rows - w * 128, 128) : p.rows);
            const int mt = pair ? w * 128 + row : row;       // row of the row tile
            const bool live = row < rows, warp_live = (warp & 3) * 32 < rows;
            const int m = p.m0 + mt, blk = m / group;
            // what this row sees of the list: tokens below `sees`, and with a mask word those of its bits
            const int ctx = uniform(p.ctx), tiles = uniform(p.tiles);
            int sees = ctx, token = uniform(p.first) * plan::kTile;
            uint64_t word = 0;
            if (p.request >= 0) {
                if (a.row_mask) {
                    if (live) word = a.row_mask[p.row_base + blk];
                    if (p.n < 64) word &= (1ull << p.n) - 1;
                } else {
                    sees = a.mask == DSPARK_MASK_CAUSAL ? ctx + min(blk, p.n - 1) + 1 : p.len;
                }
            }
            float r = -INFINITY, l = 0.f, lack = 1.f;
            bool rescale_q = false;
#pragma unroll 1
            for (int j = 0; j < tiles; ++j, ++n, token += plan::kTile) {
                const bool first = j == 0;
                if (!warp_wait(s_full(w), n & 1, abort)) { ok = false; break; }
                tc_fence_after();
                if (first) {
                    lack = live ? qscale[row] : 1.f;
                    rescale_q = __any_sync(0xffffffffu, lack != 1.f);
                }
                if (warp_live) {
                    const uint32_t ss = n % kScaleSlots;
                    const float *ks = reinterpret_cast<const float *>(gen + L::kScale) + (w * kScaleSlots + ss) * 256, *vs = ks + 128;
                    const bool masked = token > ctx - plan::kTile;   // some row does not see some token of this tile
                    float ref = r == -INFINITY ? 0.f : r;
                    __syncwarp();
                    // the row's scores 32 columns at a time: more would spill, and with this much shared
                    // memory a spilled register comes back from L2
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        uint32_t pr[16], bits = ~0u;
                        bool some_hidden = false;
                        if (masked) {
                            const int from_t = token + 32 * q, full = min(max(sees - from_t, 0), 32);
                            bits = full == 32 ? ~0u : (1u << full) - 1;
                            const int sh = from_t - ctx;   // block token of the first column
                            if (sh > -32 && sh < 64) bits |= (uint32_t)(sh >= 0 ? word >> sh : word << -sh);
                            some_hidden = __any_sync(0xffffffffu, bits != ~0u);
                            if (!__any_sync(0xffffffffu, live && bits != 0)) {
#pragma unroll
                                for (int i = 0; i < 16; ++i) pr[i] = 0;
                                tmem_st16(my_s + 16u * (uint32_t)q, pr);
                                continue;
                            }
                        }
                        // the columns' sums, with the row's own factor
                        auto load_x = [&](uint32_t (&x)[32]) {
                            tmem_ld32(my_s + 32u * (uint32_t)q, x);
                            tmem_ld_wait32(x);
                            if (rescale_q) {
#pragma unroll
                                for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * lack);
                            }
                        };
                        // scores in log2 units less `ref2` of four columns; those the row does not see -inf
                        auto four = [&](const uint32_t (&x)[32], int i, uint64_t ref2, float (&y)[4], auto hidden) {
                            const float4 k4 = *reinterpret_cast<const float4 *>(ks + 32 * q + i);
                            unpack2(fma2(pack2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), pack2(k4.x, k4.y), ref2), y[0], y[1]);
                            unpack2(fma2(pack2(__uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])), pack2(k4.z, k4.w), ref2), y[2], y[3]);
                            if constexpr (decltype(hidden)::value) {
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    if (!(bits >> (i + k) & 1u)) y[k] = -INFINITY;
                            }
                        };
                        // the softmax terms' sum; to `pr` what they weigh the values' codes with
                        auto terms = [&](const uint32_t (&x)[32], auto hidden) {
                            const uint64_t ref2 = pack2(-ref, -ref);
                            uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
                            for (int i = 0; i < 32; i += 4) {
                                float y[4];
                                four(x, i, ref2, y, hidden);
#pragma unroll
                                for (int k = 0; k < 4; ++k) y[k] = fast_exp2(y[k]);
                                const uint64_t y01 = pack2(y[0], y[1]), y23 = pack2(y[2], y[3]);
                                sum[i >> 1 & 2] = add2(sum[i >> 1 & 2], y01);
                                sum[(i >> 1 & 2) + 1] = add2(sum[(i >> 1 & 2) + 1], y23);
                                const float4 v4 = *reinterpret_cast<const float4 *>(vs + 32 * q + i);
                                unpack2(mul2(y01, pack2(v4.x, v4.y)), y[0], y[1]);
                                unpack2(mul2(y23, pack2(v4.z, v4.w)), y[2], y[3]);
                                pr[i >> 1] = half_pair(y[0], y[1]);
                                pr[(i >> 1) + 1] = half_pair(y[2], y[3]);
                            }
                            float s0, s1;
                            unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), s0, s1);
                            return s0 + s1;
                        };
                        float s;
#pragma unroll 1
                        for (int again = 0;; ++again) {
                            uint32_t x[32];
                            load_x(x);
                            s = some_hidden ? terms(x, std::true_type{}) : terms(x, std::false_type{});
                            // the reference has to move when a P or the sum has passed its bound, or when there
                            // is none yet (never for a row that is NaN already)
                            uint32_t most = 0;
#pragma unroll
                            for (int i = 0; i < 16; i += 2) most = __vimax3_u16x2(most, pr[i], pr[i + 1]);
                            const bool past = max(most & 0xffffu, most >> 16) >= kPast || s > kSumMost;
                            const bool moves = live && l == l && (past || (r == -INFINITY && bits != 0));
                            if (again || !__any_sync(0xffffffffu, moves)) break;
                            float top = -INFINITY;
                            load_x(x);
#pragma unroll
                            for (int i = 0; i < 32; i += 4) {
                                float y[4];
                                four(x, i, 0, y, std::true_type{});
#pragma unroll
                                for (int k = 0; k < 4; ++k) y[k] += fmaxf(fast_log2(vs[32 * q + i + k]), kVLeast);
                                top = max3(max3(top, y[0], y[1]), y[2], y[3]);
                            }
                            float f = 1.f;
                            if (moves && top != -INFINITY) {     // (-inf: there is no number)
                                const float r_new = ceilf(top) - kPeak;   // P <= 2^7
                                f = scale_down(1.f, r - r_new);
                                l = scale_down(l, r - r_new);
                                r = r_new;
                            }
                            ref = r == -INFINITY ? 0.f : r;
                            // what is summed so far: the output of earlier tiles (their product has ended, these
                            // scores came after it) and this tile's P
                            if (!first) {
#pragma unroll 1
                                for (int i = 0; i < DP / 16; ++i) {
                                    uint32_t o[16];
                                    tmem_ld16(my_o + 16u * (uint32_t)i, o);
                                    tmem_ld_wait16(o);
#pragma unroll
                                    for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                                    tmem_st16(my_o + 16u * (uint32_t)i, o);
                                }
                            }
                            const __half2 f2 = __float2half2_rn(f);
                            tmem_st_wait();
#pragma unroll 1
                            for (int i = 0; i < q; ++i) {
                                uint32_t o[16];
                                tmem_ld16(my_s + 16u * (uint32_t)i, o);
                                tmem_ld_wait16(o);
#pragma unroll
                                for (int k = 0; k < 16; ++k) {
                                    const __half2 h = __hmul2(*reinterpret_cast<__half2 *>(&o[k]), f2);
                                    o[k] = *reinterpret_cast<const uint32_t *>(&h);
                                }
                                tmem_st16(my_s + 16u * (uint32_t)i, o);
                            }
                        }
                        l += s;
                        // P's 16 columns lie below the scores still to be read
                        tmem_st16(my_s + 16u * (uint32_t)q, pr);
                    }
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_ready(w));
            }
            if (!ok) break;
            {
                // ---- the piece's result
                if (!warp_wait(o_full(w), k & 1, abort)) { ok = false; break; }
                tc_fence_after();
                __syncwarp();
                if (warp_live) {
                    const int64_t packed = (int64_t)p.row_base + blk;
                    const int head = p.head * group + (m - blk * group), out_kind = p.out;
                    const int64_t place = packed * a.n_q_heads + head, all = (int64_t)a.rows.n_rows * a.n_q_heads;
                    const int64_t part =
                        out_kind != kContinued ? (p.request < 0 ? place : all + place)
                        : pair ? 2 * all + (int64_t)blockIdx.x * plan::kTileRows + mt
                               : 2 * all + (int64_t)kCtas * plan::kTileRows + ((int64_t)blockIdx.x * 2 + w) * plan::kHalfRows + mt;
                    const float inv = out_kind == kDirect ? (l == 0.f ? 0.f : kVDown / l) : kVDown;
#pragma unroll 1
                    for (int q = 0; q * 16 < D; ++q) {
                        uint32_t o[16];
                        tmem_ld16(my_o + 16u * (uint32_t)q, o);
                        tmem_ld_wait16(o);
                        if (live && out_kind == kDirect) {
                            T *dst = static_cast<T *>(a.out) + place * D + 16 * q;
#pragma unroll
                            for (int i = 0; i < 16; i += 8) {
                                uint32_t v[4];
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    v[k] = float_to_pair<T>(__uint_as_float(o[i + 2 * k]) * inv, __uint_as_float(o[i + 2 * k + 1]) * inv);
                                *reinterpret_cast<uint4 *>(dst + i) = make_uint4(v[0], v[1], v[2], v[3]);
                            }
                        } else if (live) {
                            float *dst = parts.o + part * D + 16 * q;
                            store8(dst, &o[0], inv);
                            store8(dst + 8, &o[8], inv);
                        }
                        __syncwarp();
                    }
                    if (live) {
                        if (out_kind != kDirect) parts.stats[part] = make_float2(r, l);
                        else if (a.lse) a.lse[place] = l == 0.f ? -INFINITY : kLn2 * (r + log2f(l));
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(o_free(w));
                    mbar_arrive(piece_empty(w, k % kRing));
                }
            }
        }
        if (!ok && lane == 0) *abort = 1;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kIssuer) tmem_dealloc(tmem, 512);
    if (tid == 0 && *abort) atomicOr(c.flags, kFlagTimeout);
}

// ---------------------------------------------------------------- the joining --
// Adds up the parts of each (packed row, query head): the prefix's and its
// request's own item's, each cut where a worker's part of the line ends.  Rows
// that one worker finished alone are already written.
//
// A warp takes `per` rows of one kv head and request, one after another: they
// nearly always belong to the same two items, so that where their parts are is
// found once, a half of the warp looking at an item and each lane at one of its
// workers (an item of more than 16 workers is looked at in turns).  What then
// bounds it is reading the parts.
constexpr int kJoinWarps = 8, kJoinRows = 4;

template <typename T>
__global__ void __launch_bounds__(kJoinWarps * 32)
attention_join_kernel(const __grid_constant__ AttentionArgs a, const Partials parts, const int per) {
    griddep_wait();
    const int lane = threadIdx.x & 31, b = blockIdx.x;
    const dspark_kv_cache &c = a.cache;
    const int D = c.head_dim, group = a.n_q_heads / c.n_kv_heads, Hq = a.n_q_heads;
    const Request q = load_request(a, b);
    if (q.n == 0) return;
    // the line: units of the prefix by class, of all pairs, of all (the last request's end)
    const int prefix_m = prefix_rows(a) * group, prefix_tiles = plan::token_tiles(a.prefix_len);
    int64_t prefix[2], pairs, total;
    {
        const int last = a.rows.B - 1;
        const Request z = load_request(a, last);
        int64_t end[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            prefix[k] = plan::head_units(k, prefix_m, prefix_tiles) * c.n_kv_heads;
            end[k] = prefix[k] + parts.unit0[k][last] +
                     (z.len_ok && z.n > 0 ? plan::head_units(k, z.n * group, plan::token_tiles(z.len)) * c.n_kv_heads : 0);
        }
        pairs = end[0];
        total = end[0] + end[1];
    }
    const int64_t own0 = parts.unit0[0][b] + prefix[0], own1 = parts.unit0[1][b] + prefix[1];
    const int64_t all = (int64_t)a.rows.n_rows * Hq;
    const int own_m = q.n * group, chunks = (own_m + per - 1) / per;
    // this lane's item (0 the prefix's, 1 the request's own) and its place among the item's workers
    const int side = lane >> 4, at = lane & 15;
    const int m_of = side ? 0 : (int)q.first * group, rows = side ? own_m : prefix_m;
    const int tiles = side ? plan::token_tiles(q.len) : prefix_tiles;
    for (int i = blockIdx.y * kJoinWarps + (threadIdx.x >> 5); i < c.n_kv_heads * chunks; i += gridDim.y * kJoinWarps) {
        const int h = i / chunks, m0 = (i - h * chunks) * per, m1 = min(m0 + per, own_m);
        int item = -1;             // the row tile that is looked at
        bool has = false, first = false, more = false, done = false;
        int64_t part0 = 0;
        // the lane's part of the item, when its worker (the `turn`-th 16 of them) has one
        auto look = [&](int turn) {
            const int cls = plan::class_of(plan::tile_rows(rows, item));
            const int64_t start = (!side ? 0 : cls == plan::kPair ? own0 : own1) + (cls == plan::kPair ? 0 : pairs) +
                                  h * plan::head_units(cls, rows, tiles) +
                                  (cls == plan::kPair ? item * plan::item_total(cls, tiles) : 0);
            const int64_t end = start + plan::item_total(cls, tiles);
            const int v0 = plan::worker_of(cls, start + plan::item_units(cls), pairs, total, kCtas), v = v0 + turn * 16 + at;
            const int workers = cls == plan::kPair ? kCtas : 2 * kCtas;
            has = first = false;
            bool go_on = false, alone = false;
            if (tiles > 0 && v < workers) {
                const int64_t from = plan::worker_begin(cls, v, pairs, total, kCtas);
                const int64_t to = plan::worker_begin(cls, v + 1, pairs, total, kCtas);
                const int t = plan::first_tile(cls, to, start, tiles);
                first = v == v0;
                has = first || (from < end && plan::first_tile(cls, from, start, tiles) < t);
                go_on = at == 15 && to < end && v + 1 < workers;
                alone = first && t == tiles;
            }
            part0 = first ? (side ? all : 0)
                          : 2 * all + (cls == plan::kPair ? 0 : (int64_t)kCtas * plan::kTileRows) +
                                (int64_t)v * (cls == plan::kPair ? plan::kTileRows : plan::kHalfRows);
            more = __any_sync(0xffffffffu, go_on);
            if (turn == 0) done = __any_sync(0xffffffffu, side && alone && prefix_tiles == 0);
        };
        for (int m = m0; m < m1; ++m) {
            const int blk = m / group;
            const int64_t place = (q.first + blk) * Hq + h * group + (m - blk * group);
            T *out = static_cast<T *>(a.out) + place * D;
            if (!q.len_ok) {
                if (lane * 4 < D) *reinterpret_cast<uint2 *>(out + lane * 4) = make_uint2(0x7fff7fffu, 0x7fff7fffu);
                if (lane == 0 && a.lse) a.lse[place] = __int_as_float(0x7fffffff);
                continue;
            }
            const int mt = m_of + m, now = mt / plan::kTileRows;
            const bool other = __any_sync(0xffffffffu, now != item);
            item = now;
            if (other) look(0);
            if (done) continue;
            float top = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
            int turn = 0;
            while (true) {
                const int64_t part = part0 + (first ? place : mt - now * plan::kTileRows);
                float2 st = make_float2(-INFINITY, 0.f);
                if (has && mt < rows) st = parts.stats[part];
                const bool saw = !(st.x == -INFINITY && st.y == 0.f);
                float t = fmaxf(top, st.x);
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, d));
                const float keep = top == -INFINITY && l == 0.f ? 0.f : scale_down(1.f, top - t);
                const float f = saw ? scale_down(1.f, st.x - t) : 0.f;
                float s = saw ? scale_down(st.y, st.x - t) : 0.f;
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
                l = (top == -INFINITY && l == 0.f ? 0.f : scale_down(l, top - t)) + s;
                top = t;
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[k] *= keep;
                unsigned left = __ballot_sync(0xffffffffu, saw);
                while (left) {
                    // two parts at a time
                    const int x = __ffs(left) - 1;
                    left &= left - 1;
                    const int y = left ? __ffs(left) - 1 : x;
                    const float fx = __shfl_sync(0xffffffffu, f, x), fy = left ? __shfl_sync(0xffffffffu, f, y) : 0.f;
                    const int64_t px = __shfl_sync(0xffffffffu, part, x), py = __shfl_sync(0xffffffffu, part, y);
                    if (lane * 4 < D) {
                        const float4 ox = *reinterpret_cast<const float4 *>(parts.o + px * D + lane * 4);
                        const float4 oy = left ? *reinterpret_cast<const float4 *>(parts.o + py * D + lane * 4)
                                               : make_float4(0.f, 0.f, 0.f, 0.f);
                        acc[0] += ox.x * fx + oy.x * fy, acc[1] += ox.y * fx + oy.y * fy;
                        acc[2] += ox.z * fx + oy.z * fy, acc[3] += ox.w * fx + oy.w * fy;
                    }
                    left &= left - 1;   // (none left: stays 0)
                }
                if (!more) break;
                look(++turn);
            }
            if (turn > 0) item = -1;
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
}

struct Regions {
    size_t unit1, stats, o, bytes;
};
Regions regions(int B, int n_rows, int n_q_heads, int D) {
    const size_t parts = 2 * (size_t)n_rows * n_q_heads + 2 * (size_t)kCtas * plan::kTileRows;
    Regions g;
    g.unit1 = align_up((size_t)B * sizeof(int64_t), 256);
    g.stats = 2 * g.unit1;
    g.o = align_up(g.stats + parts * sizeof(float2), 256);
    g.bytes = align_up(g.o + parts * D * sizeof(float), 256);
    return g;
}

template <typename T, int kFormat, int DP>
cudaError_t launch_t(const AttentionArgs &a, const Partials &p, cudaStream_t s) {
    static PerDeviceOnce once;
    auto *kernel = attention_kernel<T, kFormat, DP>;
    cudaError_t e = once.run([&] {
        cudaFuncAttributes attr{};
        const cudaError_t got = cudaFuncGetAttributes(&attr, kernel);
        if (got != cudaSuccess) return got;
        if (attr.numRegs < kLaunchRegs) return cudaErrorInvalidConfiguration;
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<DP>::kBytes);
    });
    if (e != cudaSuccess) return e;
    kernel<<<kCtas, kThreads, Layout<DP>::kBytes, s>>>(a, p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    // rows a warp: several, or one where that would leave SMs without warps (the whole call with one / several:
    // 1,280 rows of heads 36.9 / 43.0 us, 5,120 rows 55.3 / 55.3, 9,600 rows 75.8 / 69.6, 76,800 rows 397 / 344);
    // and enough blocks per request for the rows of an average one
    const int64_t rows = (int64_t)a.rows.n_rows * a.n_q_heads;
    const int per = rows >= kJoinRows * 8 * kNumSMs ? kJoinRows : 1;
    const int64_t warps = (rows + (int64_t)a.rows.B * per - 1) / ((int64_t)a.rows.B * per);
    const int y = (int)((warps + kJoinWarps - 1) / kJoinWarps);
    return launch_dependent(attention_join_kernel<T>, dim3(a.rows.B, y < 1024 ? y : 1024), dim3(kJoinWarps * 32), 0, s, a, p,
                            per);
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
    const Partials p{{reinterpret_cast<int64_t *>(a.ws), reinterpret_cast<int64_t *>(a.ws + g.unit1)},
                     reinterpret_cast<float2 *>(a.ws + g.stats), reinterpret_cast<float *>(a.ws + g.o)};
    return a.dt == DSPARK_BF16 ? launch_format<__nv_bfloat16>(a, p, s) : launch_format<__half>(a, p, s);
}

}  // namespace dspark
