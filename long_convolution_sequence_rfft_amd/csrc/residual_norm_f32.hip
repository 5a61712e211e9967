// residual_norm_f32.hip -- the norm of whole tokens with float32 storage.
#include "residual_norm_kernels.h"

HY_NORM_INSTANTIATE(float)
