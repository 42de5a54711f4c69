// The fp16 kernels of window_attention.cu, in a translation unit of their own.
#define DSPARK_WINDOW_F16
#include "window_attention.cu"
