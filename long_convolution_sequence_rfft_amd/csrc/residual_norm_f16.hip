// residual_norm_f16.hip -- the norm of whole tokens with binary16 storage.
#include "residual_norm_kernels.h"

HY_NORM_INSTANTIATE(_Float16)
