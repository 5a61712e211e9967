// token_loss_f32.hip -- the loss over a vocabulary with float32 storage.
#include "token_loss_kernels.h"

HY_LOSS_INSTANTIATE(float)
