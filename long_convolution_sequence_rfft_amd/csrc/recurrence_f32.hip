// recurrence_f32.hip -- the gated linear recurrence with float32 storage.
#include "recurrence_launch.h"

HY_REC_INSTANTIATE(float)
