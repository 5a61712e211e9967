// recurrence_plan.h -- the gated linear recurrence's plan, and checks of strided
// views (pure host code, no HIP).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "hyena.h"

namespace hy {

// Workgroups that the cut into segments aims at: one round of those that are
// resident together.  More segments mean more states to write, scan and read,
// fewer leave compute units empty.  Measured, all kernels of a call repeated on
// the same inputs:
// forward, 64K tokens, 12 heads of 64, bfloat16: 220, 183, 156, 141, 161 us at
// 256, 384, 512, 768, 1024; 2 x 8K tokens, 6 heads of 128: 89, 84, 74, 77, 87
// at 192, 256, 384, 512, 768;
// backward, 2 x 8K tokens, 12 heads of 64, its dk and dv in 256 and its states
// and dq in 256, 512, 768: 148, 137, 140; all in 384 and 512: 157, 150.
// 4 x 2K tokens in float32: 155, 150, 155; 165, 164.  3 x 4100 tokens, 5 heads
// of 40 and 72, float16: 92, 92, 92; 90, 92.
constexpr int64_t kRecForwardGroups = 768;
constexpr int64_t kRecWideGroups = 384;  // forward, dk or dv above 64
constexpr int64_t kRecBackwardGroups = 256;
constexpr int64_t kRecStateGroups = 512;

struct RecPlan {
    int64_t B = 0, N = 0, heads = 0;
    int32_t dk = 0, dv = 0;
    int32_t io_dtype = HYENA_F32;
    // The sequence is cut into nseg segments that run in parallel; the backward
    // pass's dk and dv into nseg_b, its states and dq into nseg_b * every.
    int32_t nseg = 0;
    int32_t nseg_b = 0, every = 1;
    size_t forward_bytes = 0, backward_bytes = 0;
};

// Workspace, all float32.  start: [B heads][nseg + 1][dk dv] states before each
// segment (the last entry: the final state); decay [B heads][nseg].  Backward
// also end: gradients of the states after each segment (entry 0: of the initial
// state), and rq [B heads][N].
struct RecSpace {
    float* start = nullptr;
    float* end = nullptr;
    float* decay = nullptr;
    float* rq = nullptr;
};

hyena_status rec_plan_build(RecPlan& p, int64_t B, int64_t N, int64_t heads, int64_t dk, int64_t dv,
                            int32_t io_dtype);
RecSpace rec_space(const RecPlan& p, bool backward, void* workspace);

inline size_t element_bytes(int32_t io_dtype) { return io_dtype == HYENA_F32 ? 4 : 2; }

struct Span {
    const void* p;
    size_t bytes;
};
hyena_status check_view(const hyena_view& v, const char* name, size_t element);
// The recurrence's kernels address the tokens of a chunk by 32-bit byte offsets.
hyena_status check_token_stride(const hyena_view& v, const char* name, int64_t N);
Span view_span(const hyena_view& v, int64_t B, int64_t N, int64_t heads, int64_t width, size_t element);
bool spans_overlap(const Span& a, const Span& b);

}  // namespace hy
