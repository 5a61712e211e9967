// recurrence_plan.cpp -- argument validation, segments and workspace sizes of
// the gated linear recurrence.  Pure host code.
#include <string>

#include "plan.h"
#include "recurrence_plan.h"

namespace hy {

namespace {
// Segments per (row, head): as many as give `want` workgroups in all and no
// more (one round of the chip), of at least about 128 tokens each.
int32_t cut(int64_t N, int64_t bh, int64_t want)
{
    int64_t n = want / bh;
    const int64_t most = (N + 127) / 128;
    if (n > most) n = most;
    return (int32_t)(n < 1 ? 1 : n);
}
size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
}  // namespace

hyena_status rec_plan_build(RecPlan& p, int64_t B, int64_t N, int64_t heads, int64_t dk, int64_t dv,
                            int32_t io_dtype)
{
    if (B < 1 || N < 1 || heads < 1 || dk < 1 || dv < 1)
        return fail(HYENA_ERR_INVALID_ARGUMENT, "recurrence: B, N, heads, dk and dv must be at least 1");
    if (dk > 128 || dv > 128) return fail(HYENA_ERR_UNSUPPORTED, "recurrence: dk and dv must be in 1..128");
    if (N >= ((int64_t)1 << 31) - 64) return fail(HYENA_ERR_UNSUPPORTED, "recurrence: N must be below 2^31 - 64");
    if (heads > 65536) return fail(HYENA_ERR_UNSUPPORTED, "recurrence: at most 65536 heads");
    // (a launch holds less than 2^32 threads: a workgroup per row and head has up to 512)
    if (B > ((int64_t)1 << 22) || B * heads > ((int64_t)1 << 22))
        return fail(HYENA_ERR_UNSUPPORTED, "recurrence: B * heads must be at most 2^22");
    if (io_dtype != HYENA_F32 && io_dtype != HYENA_BF16 && io_dtype != HYENA_F16)
        return fail(HYENA_ERR_UNSUPPORTED, "recurrence: unknown io dtype");
    p.B = B;
    p.N = N;
    p.heads = heads;
    p.dk = (int32_t)dk;
    p.dv = (int32_t)dv;
    p.io_dtype = io_dtype;
    const int64_t bh = B * heads;
    p.nseg = cut(N, bh, dk <= 64 && dv <= 64 ? kRecForwardGroups : kRecWideGroups);
    p.nseg_b = cut(N, bh, kRecBackwardGroups);
    p.every = cut(N, bh, kRecStateGroups) / p.nseg_b;
    if (p.every < 1) p.every = 1;
    const size_t state = (size_t)bh * (size_t)(dk * dv) * sizeof(float);
    p.forward_bytes = p.nseg == 1 ? 0 : align256(state * (p.nseg + 1)) + align256((size_t)bh * p.nseg * 4);
    const size_t n = (size_t)p.nseg_b * p.every;
    p.backward_bytes = 2 * align256(state * (n + 1)) + align256((size_t)bh * n * 4) +
                       align256((size_t)bh * (size_t)N * 4);
    log_msg("recurrence plan: B %lld N %lld heads %lld dk %lld dv %lld dtype %d, segments %d (backward %d, %d), "
            "workspace %zu (backward %zu)",
            (long long)B, (long long)N, (long long)heads, (long long)dk, (long long)dv, (int)io_dtype, p.nseg,
            p.nseg_b, p.nseg_b * p.every, p.forward_bytes, p.backward_bytes);
    return HYENA_OK;
}

RecSpace rec_space(const RecPlan& p, bool backward, void* workspace)
{
    RecSpace w;
    if (workspace == nullptr) return w;
    const size_t bh = (size_t)(p.B * p.heads);
    const size_t n = backward ? (size_t)p.nseg_b * p.every : (size_t)p.nseg;
    const size_t states = align256(bh * (size_t)p.dk * (size_t)p.dv * sizeof(float) * (n + 1));
    char* at = (char*)workspace;
    w.start = (float*)at;
    at += states;
    if (backward) {
        w.end = (float*)at;
        at += states;
    }
    w.decay = (float*)at;
    at += align256(bh * n * 4);
    if (backward) w.rq = (float*)at;
    return w;
}

hyena_status check_view(const hyena_view& v, const char* name, size_t element)
{
    if (v.data == nullptr) return fail(HYENA_ERR_INVALID_ARGUMENT, std::string(name) + " is NULL");
    if ((uintptr_t)v.data % element != 0)
        return fail(HYENA_ERR_INVALID_ARGUMENT, std::string(name) + " is not aligned to its element");
    if (v.batch < 0 || v.token < 0 || v.head < 0)
        return fail(HYENA_ERR_INVALID_ARGUMENT, std::string(name) + " has a negative stride");
    return HYENA_OK;
}

hyena_status check_token_stride(const hyena_view& v, const char* name, int64_t N)
{
    if (N > 1 && v.token >= ((int64_t)1 << 23))
        return fail(HYENA_ERR_UNSUPPORTED, std::string(name) + " has a token stride of 2^23 elements or more");
    return HYENA_OK;
}

Span view_span(const hyena_view& v, int64_t B, int64_t N, int64_t heads, int64_t width, size_t element)
{
    return Span{v.data, ((size_t)(B - 1) * (size_t)v.batch + (size_t)(N - 1) * (size_t)v.token +
                         (size_t)(heads - 1) * (size_t)v.head + (size_t)width) * element};
}

bool spans_overlap(const Span& a, const Span& b)
{
    if (a.p == nullptr || b.p == nullptr || a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

}  // namespace hy
