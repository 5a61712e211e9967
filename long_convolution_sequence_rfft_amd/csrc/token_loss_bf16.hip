// token_loss_bf16.hip -- the loss over a vocabulary with bfloat16 storage.
#include "token_loss_kernels.h"

HY_LOSS_INSTANTIATE(uint16_t)
