// recurrence_f16.hip -- the gated linear recurrence with binary16 storage.
#include "recurrence_launch.h"

HY_REC_INSTANTIATE(_Float16)
