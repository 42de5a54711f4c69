// How the block attention's work is cut: items, units and the pieces a worker
// takes.  Plain integer arithmetic, the same on the device and on the host.
//
// An item is one kv head's row tile (up to 256 rows = block rows x query heads
// of the kv head) against one token list: the shared prefix (rows of the whole
// batch) or one request's own tokens.  Its work in units is a cost per
// 128-token tile plus one for the item itself (its queries in, its result
// out).  Two classes:
//   pairs    129 .. 256 rows: both softmax groups of a CTA take 128 rows each of
//            the same tokens;
//   singles  1 .. 128 rows: each group takes items of its own, so that one's
//            softmax and result run under the other's products.
// The pairs in order (prefix: head, row tile; then request, head, row tile) and
// after them the singles in the same order make one line of units, cut into
// equal parts, one per CTA; a CTA's part of the singles is cut again in half,
// one half per group.  A tile belongs to the worker whose part holds its first
// unit.  So a worker's pieces are consecutive, at most its first one begins
// inside an item, and which workers share an item follows from a division, with
// no list in memory.
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define DSPARK_HD __host__ __device__ __forceinline__
#else
#define DSPARK_HD inline
#endif

namespace dspark {
namespace plan {

constexpr int kTile = 128;        // tokens
constexpr int kHalfRows = 128;    // rows of one accumulator
constexpr int kTileRows = 256;    // rows of a row tile

enum Class { kPair = 0, kSingle = 1 };
DSPARK_HD int tile_units(int cls) { return cls == kPair ? 8 : 5; }
DSPARK_HD int item_units(int cls) { return cls == kPair ? 18 : 16; }

DSPARK_HD int row_tiles(int rows) { return (int)(((int64_t)rows + kTileRows - 1) / kTileRows); }
DSPARK_HD int token_tiles(int tokens) { return (int)(((int64_t)tokens + kTile - 1) / kTile); }
DSPARK_HD int tile_rows(int rows, int rt) {
    const int left = rows - rt * kTileRows;
    return left < kTileRows ? left : kTileRows;
}
DSPARK_HD int class_of(int rows_in_tile) { return rows_in_tile > kHalfRows ? kPair : kSingle; }
// row tiles of a class among `rows` rows; the single one, if any, is the last
DSPARK_HD int class_tiles(int cls, int rows) {
    if (rows <= 0) return 0;
    const int n = row_tiles(rows);
    const bool last_single = class_of(tile_rows(rows, n - 1)) == kSingle;
    return cls == kPair ? n - (last_single ? 1 : 0) : (last_single ? 1 : 0);
}
// the class's k-th row tile
DSPARK_HD int class_row_tile(int cls, int rows, int k) { return cls == kPair ? k : row_tiles(rows) - 1; }

// units of one item, and of all of a head's items of a class
DSPARK_HD int64_t item_total(int cls, int tiles) { return (int64_t)tiles * tile_units(cls) + item_units(cls); }
DSPARK_HD int64_t head_units(int cls, int rows, int tiles) {
    return tiles <= 0 ? 0 : class_tiles(cls, rows) * item_total(cls, tiles);
}

// CTA c of n takes units [cta_begin(c), cta_begin(c + 1)) of `total`
DSPARK_HD int64_t cta_begin(int64_t c, int64_t total, int n) { return total * c / n; }
// (a guess, off by one at most, and a look: a 64-bit division costs some hundred instructions)
DSPARK_HD int cta_of(int64_t u, int64_t total, int n) {
    int c = (int)((float)u * (float)n / (float)total);
    if (c > n - 1) c = n - 1;
    while (c > 0 && cta_begin(c, total, n) > u) --c;
    while (c + 1 < n && cta_begin(c + 1, total, n) <= u) ++c;
    return c;
}

// worker v = 2 c + group of the singles takes units [single_begin(v), single_begin(v + 1)), all of
// them from `pairs`, the units of all pairs, on
DSPARK_HD int64_t single_begin(int v, int64_t pairs, int64_t total, int n) {
    int64_t lo = cta_begin(v >> 1, total, n);
    if (lo < pairs) lo = pairs;
    if (!(v & 1)) return lo;
    int64_t hi = cta_begin((v >> 1) + 1, total, n);
    if (hi < pairs) hi = pairs;
    return lo + (hi - lo) / 2;
}
DSPARK_HD int single_of(int64_t u, int64_t pairs, int64_t total, int n) {
    const int v = 2 * cta_of(u, total, n);
    return u >= single_begin(v + 1, pairs, total, n) ? v + 1 : v;
}
// the same for either class, worker v (a CTA for pairs)
DSPARK_HD int64_t worker_begin(int cls, int v, int64_t pairs, int64_t total, int n) {
    return cls == kPair ? cta_begin(v, total, n) : single_begin(v, pairs, total, n);
}
DSPARK_HD int worker_of(int cls, int64_t u, int64_t pairs, int64_t total, int n) {
    return cls == kPair ? cta_of(u, total, n) : single_of(u, pairs, total, n);
}

// first tile of an item (its first unit `start`) whose first unit is `u` or
// later, at most `tiles`; the item's own units come before its tiles'
DSPARK_HD int first_tile(int cls, int64_t u, int64_t start, int tiles) {
    const int64_t at = start + item_units(cls);
    if (u <= at) return 0;
    const int64_t t = (u - at + tile_units(cls) - 1) / tile_units(cls);
    return (int)(t < tiles ? t : tiles);
}

// Places of a ring that a loader has filled, 0, 1, 2 .. in order: those whose
// copies may still be under way are the last `held` ones.
struct Filled {
    uint32_t n;
    DSPARK_HD void add(uint32_t position) { n = position + 1; }
    DSPARK_HD uint32_t held(uint32_t ring) const { return n < ring ? n : ring; }
    DSPARK_HD uint32_t place(uint32_t i) const { return n - 1 - i; }   // the i-th last
};

}  // namespace plan
}  // namespace dspark
