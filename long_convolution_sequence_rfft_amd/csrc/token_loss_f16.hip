// token_loss_f16.hip -- the loss over a vocabulary with binary16 storage.
#include "token_loss_kernels.h"

HY_LOSS_INSTANTIATE(_Float16)
