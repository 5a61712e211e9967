// recurrence_bf16.hip -- the gated linear recurrence with bfloat16 storage.
#include "recurrence_launch.h"

HY_REC_INSTANTIATE(uint16_t)
