// residual_norm.h -- arguments of the kernels of the norm of whole tokens.
#pragma once

#include "rows.h"

namespace hy {

struct NormArgs {
    Rows x, res;         // res: the residual; backward: the sum's own gradient
    Rows dy;
    const float* w;
    void* sum;
    void* y;             // backward: dx
    float* scales;
    float* dw_part;      // [workgroups][d]
    int64_t rows;
    uint32_t N;          // row_at
    int32_t d;
    int32_t lanes;       // of a team that is part of a wave
    int32_t weight_vectors;  // weight is 16-byte aligned
    int32_t int8;
    int32_t group_lanes; // 0: a scale for each row
    int32_t groups;      // of a row
    float largest, inverse;
    float eps;
};

// Units of a lane where a workgroup holds a row: 16 channels, which with three tensors and
// the sums for the weights' gradient fill the registers of 1024 threads.
template <typename T> constexpr int kWideUnits = 16 / kUnit<T>;

struct NormLaunch {
    bool units;          // rows are made of whole aligned units
    bool workgroup;
    int per;             // units of a lane
    int threads;
    int64_t groups;      // workgroups
};

// kind 0: y in the io dtype, 1: y in 8 bits, 2: backward.
template <typename T> hyena_status norm_launch(const NormArgs& a, const NormLaunch& l, int kind, hipStream_t s);
extern template hyena_status norm_launch<float>(const NormArgs&, const NormLaunch&, int, hipStream_t);
extern template hyena_status norm_launch<uint16_t>(const NormArgs&, const NormLaunch&, int, hipStream_t);
extern template hyena_status norm_launch<_Float16>(const NormArgs&, const NormLaunch&, int, hipStream_t);

}  // namespace hy
