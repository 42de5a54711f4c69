// dspark_window_attention of blocks with many rows: the kernels of block_attention.cu,
// compiled for rows that see through a window.
#define DSPARK_WINDOW_BLOCKS
#include "block_attention.cu"
