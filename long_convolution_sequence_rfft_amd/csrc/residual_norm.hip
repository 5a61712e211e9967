// residual_norm.hip -- entry points of the norm of whole tokens (include/hyena.h):
// checks, and the launches of a call.
#include "residual_norm.h"

namespace hy {

// dw[c] = sum over the workgroups' rows, in float64, 16 channels by 64 rows at a time.
__global__ __launch_bounds__(1024) void hyena_residual_weight_grad(const float* part, float* out, int groups, int d)
{
    __shared__ double sums[1024];
    const int c = blockIdx.x * 16 + (threadIdx.x & 15), r = threadIdx.x >> 4;
    double s = 0.0;
    if (c < d) {
#pragma unroll 8
        for (int g = r; g < groups; g += 64) s += (double)part[(int64_t)g * d + c];
    }
    sums[threadIdx.x] = s;
    __syncthreads();
    if (r == 0 && c < d) {
        double x = 0.0;
        for (int i = 0; i < 64; ++i) x += sums[i * 16 + threadIdx.x];
        out[c] = (float)x;
    }
}

namespace {

constexpr const char* kWho = "residual norm";

// Workgroups of 256 threads that run through the rows, forward and backward, where each adds a
// row of sums for the weights (gradients of 16384 rows of 768: 256 workgroups 30.7, 512 26.5, 768 33.0,
// 1024 31.4, 2048 41.2 us).
constexpr int64_t kNormGroups = 2048;
constexpr int64_t kNormGradGroups = 512;

hyena_status refuse(const char* what) { return fail(HYENA_ERR_INVALID_ARGUMENT, std::string(kWho) + ": " + what); }

hyena_status norm_sizes(const hyena_residual_norm* op)
{
    if (op == nullptr) return refuse("the description is NULL");
    if (op->B < 1 || op->N < 1 || op->d < 1) return refuse("B, N and d must be at least 1");
    if (op->d > 16384) return fail(HYENA_ERR_UNSUPPORTED, "residual norm: d must be in 1..16384");
    if (op->B > 0x7fffffff || op->N > 0x7fffffff || op->B * op->N > 0x7fffffff)
        return fail(HYENA_ERR_UNSUPPORTED, "residual norm: at most 2^31 - 1 tokens");
    if (!(op->eps >= 0.0f)) return refuse("eps must be at least 0");
    return check_io(kWho, op->io_dtype);
}

// Teams: as many lanes of a wave, a power of two, as leave the fewest idle with at
// most 4 units each; wider rows take a workgroup (gradients of rows of 5120 by one wave
// spilled registers: 116 us, 30 so).  least: lanes of a group of scales.
NormLaunch shape(const NormArgs& a, size_t element, bool whole, bool grad, int least, int32_t* lanes)
{
    NormLaunch l{};
    l.units = whole;
    const int units = (int)((a.d * element + 15) / 16);
    l.workgroup = units > 256;
    if (l.workgroup) {
        l.per = (int)element;  // kWideUnits
        l.threads = ((units + l.per - 1) / l.per + 63) / 64 * 64;
        *lanes = l.threads;
    } else {
        int best = 64;
        for (int n = 64; n >= least && n >= 1; n /= 2) {
            const int per = (units + n - 1) / n;
            if (per > 4) break;
            if (per * n < ((units + best - 1) / best) * best) best = n;
        }
        l.threads = 256;
        l.per = (units + best - 1) / best;
        *lanes = best;
    }
    const int64_t teams = l.workgroup ? 1 : 256 / *lanes, need = (a.rows + teams - 1) / teams;
    const int64_t most = (grad ? kNormGradGroups : kNormGroups) * 256 / l.threads;
    l.groups = need < most ? need : most;
    return l;
}

}  // namespace
}  // namespace hy

using namespace hy;

extern "C" {

hyena_status hyena_residual_norm_forward(const hyena_residual_norm* op, void* sum, void* y, float* scales, void* stream)
{
    hyena_status st = norm_sizes(op);
    if (st != HYENA_OK) return st;
    const bool eight = op->format != HYENA_NORM_IO;
    if (eight && op->format != HYENA_NORM_E4M3 && op->format != HYENA_NORM_INT8)
        return fail(HYENA_ERR_UNSUPPORTED, "residual norm: unknown format");
    if (op->group != 0 && (!eight || (op->group != 32 && op->group != 64 && op->group != 128)))
        return refuse("group must be 0, or 32, 64 or 128 with a format of 8 bits");
    if (op->group != 0 && op->d % op->group != 0) return refuse("d must be a multiple of group");
    const size_t e = element_bytes(op->io_dtype);
    if ((st = check_rows(kWho, op->x, "x", e)) != HYENA_OK) return st;
    const bool added = op->residual.data != nullptr;
    if (added && (st = check_rows(kWho, op->residual, "residual", e)) != HYENA_OK) return st;
    if (added != (sum != nullptr)) return refuse("sum must be given with a residual, and only then");
    if (y == nullptr) return refuse("y is NULL");
    if (eight != (scales != nullptr)) return refuse("scales must be given with a format of 8 bits, and only then");
    if ((uintptr_t)op->weight % 4 != 0 || (uintptr_t)scales % 4 != 0 || (uintptr_t)sum % e != 0 ||
        (!eight && (uintptr_t)y % e != 0))
        return refuse("weight or an output is not aligned to its element");

    hyena_rows x = plain_rows(op->x, op->B, op->N), res = plain_rows(op->residual, op->B, op->N);
    const int64_t rows = op->B * op->N, groups = op->group ? op->d / op->group : 1;
    const size_t all = (size_t)rows * (size_t)op->d;
    // the sum may lie on x or on the residual, row on row
    auto on = [&](const hyena_rows& v) {
        return sum == v.data && (op->N == 1 || v.token == op->d) && (op->B == 1 || v.batch == op->N * op->d);
    };
    const Span ins[3] = {rows_span(x, op->B, op->N, op->d, e),
                         added ? rows_span(res, op->B, op->N, op->d, e) : Span{nullptr, 0},
                         Span{op->weight, (size_t)op->d * 4}};
    const Named outs[3] = {{Span{y, all * (eight ? 1 : e)}, "y"},
                           {Span{scales, (size_t)(rows * groups) * 4}, "scales"},
                           {Span{sum, all * e}, "sum"}};
    if ((st = check_apart(kWho, ins, 3, outs, 2)) != HYENA_OK) return st;
    for (int j = 0; j < 2; ++j)
        if (spans_overlap(outs[2].span, outs[j].span)) return refuse("sum overlaps another output");
    for (int j = 0; j < 3; ++j)
        if (spans_overlap(outs[2].span, ins[j]) && !(j == 0 && on(x)) && !(j == 1 && on(res)))
            return refuse("sum overlaps an input");

    NormArgs a{};
    RowShape made(op->d, e);
    made.add(x);
    if (added) made.add(res), made.dense(sum);
    if (!eight) made.dense(y);
    // (8-bit rows of whole units are written by 4 bytes)
    const bool units = made.units() && (!eight || (uintptr_t)y % 4 == 0);
    int64_t N = op->N;
    hyena_rows* all_rows[2] = {&x, &res};
    flatten_rows(all_rows, added ? 2 : 1, op->B, &N);
    a.x = Rows{x.data, x.batch, x.token};
    a.res = Rows{res.data, res.batch, res.token};
    a.w = op->weight;
    a.weight_vectors = (uintptr_t)op->weight % 16 == 0;
    a.sum = sum;
    a.y = y;
    a.scales = scales;
    a.rows = rows;
    a.N = (uint32_t)N;
    a.d = (int32_t)op->d;
    a.int8 = op->format == HYENA_NORM_INT8;
    a.group_lanes = (int32_t)(op->group * (int64_t)e / 16);
    a.groups = (int32_t)groups;
    a.largest = a.int8 ? 127.0f : 448.0f;
    a.inverse = 1.0f / a.largest;
    a.eps = op->eps;
    const NormLaunch l = shape(a, e, units, false, a.group_lanes, &a.lanes);
    return by_io(op->io_dtype, [&](auto* t) {
        return norm_launch<std::remove_pointer_t<decltype(t)>>(a, l, eight ? 1 : 0, (hipStream_t)stream);
    });
}

hyena_status hyena_residual_norm_scratch_bytes(const hyena_residual_norm* op, size_t* bytes)
{
    const hyena_status st = norm_sizes(op);
    if (st != HYENA_OK) return st;
    if (bytes == nullptr) return refuse("bytes is NULL");
    NormArgs a{};
    a.rows = op->B * op->N;
    a.d = (int32_t)op->d;
    *bytes = (size_t)shape(a, element_bytes(op->io_dtype), false, true, 1, &a.lanes).groups * (size_t)op->d * 4;
    return HYENA_OK;
}

hyena_status hyena_residual_norm_backward(const hyena_residual_norm* op, const hyena_rows* d_y, const hyena_rows* d_sum,
                                          void* d_x, float* d_weight, void* scratch, void* stream)
{
    hyena_status st = norm_sizes(op);
    if (st != HYENA_OK) return st;
    const size_t e = element_bytes(op->io_dtype);
    if (d_y == nullptr) return refuse("d_y is NULL");
    const bool more = d_sum != nullptr;
    if ((st = check_rows(kWho, op->x, "x", e)) != HYENA_OK || (st = check_rows(kWho, *d_y, "d_y", e)) != HYENA_OK ||
        (more && (st = check_rows(kWho, *d_sum, "d_sum", e)) != HYENA_OK))
        return st;
    if (d_x == nullptr) return refuse("d_x is NULL");
    if ((uintptr_t)d_x % e != 0 || (uintptr_t)d_weight % 4 != 0 || (uintptr_t)op->weight % 4 != 0)
        return refuse("weight or an output is not aligned to its element");
    if (d_weight != nullptr && (scratch == nullptr || (uintptr_t)scratch % 16 != 0))
        return refuse("scratch is NULL or not 16-byte aligned");

    hyena_rows x = plain_rows(op->x, op->B, op->N), dy = plain_rows(*d_y, op->B, op->N),
               ds = more ? plain_rows(*d_sum, op->B, op->N) : hyena_rows{nullptr, 0, 0};
    NormArgs a{};
    a.rows = op->B * op->N;
    a.d = (int32_t)op->d;
    RowShape made(op->d, e);
    made.add(x);
    made.add(dy);
    if (more) made.add(ds);
    made.dense(d_x);
    const NormLaunch l = shape(a, e, made.units(), true, 1, &a.lanes);

    const bool on = more && d_x == ds.data && (op->N == 1 || ds.token == op->d) && (op->B == 1 || ds.batch == op->N * op->d);
    const Span ins[4] = {rows_span(x, op->B, op->N, op->d, e), rows_span(dy, op->B, op->N, op->d, e),
                         Span{op->weight, (size_t)op->d * 4},
                         more ? rows_span(ds, op->B, op->N, op->d, e) : Span{nullptr, 0}};
    const Named outs[3] = {{Span{d_x, (size_t)a.rows * (size_t)op->d * e}, "d_x"},
                           {Span{d_weight, (size_t)op->d * 4}, "d_weight"},
                           {Span{d_weight ? scratch : nullptr, (size_t)l.groups * (size_t)op->d * 4}, "scratch"}};
    if ((st = check_apart(kWho, ins, 3, outs, 3)) != HYENA_OK) return st;
    for (int i = 0; i < 3; ++i)
        if (spans_overlap(outs[i].span, ins[3]) && !(i == 0 && on)) return refuse("an output overlaps d_sum");

    int64_t N = op->N;
    hyena_rows* all_rows[3] = {&x, &dy, &ds};
    flatten_rows(all_rows, more ? 3 : 2, op->B, &N);
    a.x = Rows{x.data, x.batch, x.token};
    a.dy = Rows{dy.data, dy.batch, dy.token};
    a.res = Rows{ds.data, ds.batch, ds.token};
    a.w = op->weight;
    a.weight_vectors = (uintptr_t)op->weight % 16 == 0;
    a.y = d_x;
    a.dw_part = d_weight ? (float*)scratch : nullptr;
    a.N = (uint32_t)N;
    a.eps = op->eps;
    const hipStream_t s = (hipStream_t)stream;
    st = by_io(op->io_dtype, [&](auto* t) { return norm_launch<std::remove_pointer_t<decltype(t)>>(a, l, 2, s); });
    if (st != HYENA_OK || d_weight == nullptr) return st;
    HY_LAUNCH(kernel_label("hyena_residual_weight_grad"), hyena_residual_weight_grad, dim3((unsigned)((a.d + 15) / 16)),
              dim3(1024), 0, s, a.dw_part, d_weight, (int)l.groups, a.d);
    return launched();
}

}  // extern "C"
