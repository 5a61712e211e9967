// recurrence.h -- arguments of the gated linear recurrence's kernels
// (recurrence_kernels.h, recurrence.hip).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "hyena.h"
#include "plan.h"
#include "recurrence_device.h"
#include "recurrence_plan.h"

namespace hy {

// Tokens that one pass of a kernel's loop handles (a chunk): 64, or 32 in
// float32, whose operands take twice the LDS.
template <typename T> constexpr int kRecChunk = sizeof(T) == 4 ? 32 : 64;

// Arguments of the kernels that walk a row's chunks.  a, b of width da and c
// of width dc are the tensors by role: out_i = f_i scale a_i . S + scale
// sum_j w_ij (a_i . b_j) c_j with S <- decay S + sum_j f'_j b_j c_j^T.
struct RecArgs {
    RView a, b, c, r;      // r: width dc, for sum(r . out) per token
    RView g;
    const int32_t* lengths;
    void* out;             // dense [B][N][heads][dc]
    const float* state;    // before each segment [bh][state_n][dk dv], or NULL
    float* last;           // final state [bh][dk dv], or NULL (one segment)
    float* rq;             // [bh][N]
    int64_t N, heads;
    int32_t da, dc;
    int32_t nseg, state_n;
    float scale;
};

// Local states: role 0 sums tail_j k_j v_j^T over each segment going forward,
// role 1 head_i scale q_i do_i^T going back.
struct RecStateArgs {
    RView x[2], y[2];
    RView g;
    const int32_t* lengths;
    float* local[2];       // [bh][nseg + 1][dk dv]; role 0 writes entries 1.., role 1 0..nseg-1
    float* decay;          // [bh][nseg]
    int64_t N, heads;
    int32_t dk, dv;
    int32_t nseg;
    float scale;           // role 1
};

struct RecScanArgs {
    float* local[2];
    const float* first[2]; // initial state, gradient of the final state (or NULL)
    float* last[2];        // final state, gradient of the initial state (or NULL)
    const float* decay;
    int64_t per;           // dk * dv
    int64_t total;         // B heads dk dv
    int32_t nseg;
};

struct RecGradArgs {
    RView q, k, v, o;      // o: gradient of the output
    RView g;
    const int32_t* lengths;
    void* dk_out;
    void* dv_out;
    float* dg;
    const float* rq;       // [bh][N]: q . (state's part of dq)
    const float* start;    // [bh][nseg every + 1][dk dv] or NULL (no gradient comes from the end)
    const float* end;      // the same, or NULL with start
    int64_t N, heads;
    int32_t dk, dv;
    int32_t nseg, every;   // its segments are `every` of those that have states
    float scale;
};

struct RecStepArgs {
    RView q, k, v, g;      // token stride unused
    const int32_t* slots;
    float* states;
    void* o;
    int64_t n_slots, heads;
    int32_t dk, dv;
    float scale;
};

// One translation unit per storage type instantiates these.
template <typename T> hyena_status rec_launch_states(const RecStateArgs& a, int64_t bh, int roles, hipStream_t s);
template <typename T> hyena_status rec_launch_out(const RecArgs& a, int64_t bh, bool transposed, hipStream_t s);
template <typename T> hyena_status rec_launch_grad(const RecGradArgs& a, int64_t bh, hipStream_t s);
template <typename T> hyena_status rec_launch_step(const RecStepArgs& a, int64_t B, hipStream_t s);

}  // namespace hy
