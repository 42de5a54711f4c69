// dspark_window_attention of blocks with many rows: the kernels of block_attention.cu,
// compiled for rows that see through a window, and a joining of their own.
//
// What bounds it: a pair tile's chain of softmax and products, as there (5,500 clocks), and
// what an item of few tiles adds (its queries, first reference, masked ends and result: as
// long as four to five tiles).  Four prompts of up to 4,096 rows of 32 heads over 1,028
// tokens take 385 us (470 TFLOP/s of what is seen), of it 25 for the joining; a gap in
// whole tiles of 128 tokens 506 us, in chunks of 16, which makes nine tiles an item of
// eleven, 467; joining only what workers left unfinished 397; telling by the rows' ranges
// which columns all of a warp's rows see, or none, 385.  Queries fetched ahead, runs of
// chunks loaded as one copy and references from a whole first tile made no difference.
#define DSPARK_WINDOW_BLOCKS
#include "block_attention.cu"
