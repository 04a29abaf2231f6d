// k_attend_mma_fp32.cu -- the kernels of k_attend_mma.cu for fp32 queries, compiled beside those for 16-bit ones.
#define DIT_ATTEND_FP32
#include "k_attend_mma.cu"
