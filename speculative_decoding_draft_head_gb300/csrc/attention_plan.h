// How the block attention's work is cut: items, units and the pieces a CTA
// takes.  Plain integer arithmetic, the same on the device and on the host.
//
// An item is one kv head's row tile (up to 256 rows = block rows x query heads
// of the kv head) against one token list: the shared prefix (rows of the whole
// batch) or one request's own tokens.  Its work is its number of 128-token
// tiles times a weight: a tile against more than 128 rows keeps the tensor
// cores busy (two 128-row halves), a tile against at most 128 rows is bound by
// reading it.  The items in order (prefix: head, row tile; then request, head,
// row tile) make one line of units, cut into equal parts, one per CTA; a tile
// belongs to the CTA whose part holds its first unit.  So a CTA's pieces are
// consecutive, at most its first one begins inside an item, and which CTAs
// share an item follows from two divisions, with no list in memory.
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
constexpr int kWeightPair = 3;    // units of a tile against 129 .. 256 rows
constexpr int kWeightSingle = 2;  // units of a tile against 1 .. 128 rows

DSPARK_HD int row_tiles(int rows) { return (int)(((int64_t)rows + kTileRows - 1) / kTileRows); }
DSPARK_HD int token_tiles(int tokens) { return (int)(((int64_t)tokens + kTile - 1) / kTile); }
DSPARK_HD int tile_rows(int rows, int rt) {
    const int left = rows - rt * kTileRows;
    return left < kTileRows ? left : kTileRows;
}
DSPARK_HD int weight(int rows_in_tile) { return rows_in_tile > kHalfRows ? kWeightPair : kWeightSingle; }

// units of all row tiles of one head
DSPARK_HD int64_t head_units(int rows, int tiles) {
    if (rows <= 0 || tiles <= 0) return 0;
    const int n = row_tiles(rows);
    return (int64_t)tiles * ((int64_t)(n - 1) * kWeightPair + weight(tile_rows(rows, n - 1)));
}
// first unit of row tile rt, counted from the head's first
DSPARK_HD int64_t row_tile_start(int rt, int tiles) { return (int64_t)rt * tiles * kWeightPair; }
// the row tile that holds unit u of a head
DSPARK_HD int row_tile_of(int64_t u, int rows, int tiles) {
    const int64_t rt = u / ((int64_t)tiles * kWeightPair), last = row_tiles(rows) - 1;
    return (int)(rt < last ? rt : last);
}

// CTA c of n takes units [cta_begin(c), cta_begin(c + 1)) of `total`
DSPARK_HD int64_t cta_begin(int64_t c, int64_t total, int n) { return total * c / n; }
DSPARK_HD int cta_of(int64_t u, int64_t total, int n) { return (int)(((u + 1) * n - 1) / total); }

// first tile of an item (first unit `start`, `w` units a tile) whose first unit
// is `u` or later, at most `tiles`
DSPARK_HD int first_tile(int64_t u, int64_t start, int w, int tiles) {
    if (u <= start) return 0;
    const int64_t t = (u - start + w - 1) / w;
    return (int)(t < tiles ? t : tiles);
}

}  // namespace plan
}  // namespace dspark
