// residual_norm_bf16.hip -- the norm of whole tokens with bfloat16 storage.
#include "residual_norm_kernels.h"

HY_NORM_INSTANTIATE(uint16_t)
