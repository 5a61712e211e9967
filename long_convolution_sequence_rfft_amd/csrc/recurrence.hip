// recurrence.hip -- entry points of the gated linear recurrence (include/hyena.h):
// checks, and the launches of a call.
#include <hip/hip_runtime.h>

#include <new>

#include "recurrence.h"
#include "timing.h"

struct hyena_recurrence_s {
    hy::RecPlan p;
};

namespace hy {

// The states before the segments (role 0: S <- decay S + local, first to last)
// and the gradients after them (role 1: the same backwards), in place of the
// local sums; one thread per element.  Local sums are read kScanBatch segments
// at a time, ahead of the stores that a compiler cannot tell apart from them.
// Bound by memory and by the latency of its few rounds: 64 segments of 12 heads
// of 64 x 64 (25 MB) in 11 us, 32 of 128 x 128 (50 MB) in 13; with batches of 32
// 10.6 and 15.1, of 64 12.4 and 14.5.
constexpr int kScanBatch = 16;

__global__ __launch_bounds__(256) void hyena_rec_scan(RecScanArgs p)
{
    const int role = blockIdx.y;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < p.total; i += (int64_t)gridDim.x * 256) {
        const int64_t bh = i / p.per, e = i % p.per;
        // entry n of role 0 goes to n + 1; role 1 counts entries and segments from the last
        const int64_t step = role ? -p.per : p.per;
        float* x = p.local[role] + bh * (p.nseg + 1) * p.per + e + (role ? p.nseg * p.per : 0);
        const float* d = p.decay + bh * p.nseg + (role ? p.nseg - 1 : 0);
        const int dstep = role ? -1 : 1;
        float s = p.first[role] ? p.first[role][i] : 0.0f;
        *x = s;
        for (int n0 = 0; n0 < p.nseg; n0 += kScanBatch) {
            float local[kScanBatch], decay[kScanBatch];
#pragma unroll
            for (int n = 0; n < kScanBatch; ++n)
                if (n0 + n < p.nseg) {
                    local[n] = x[(n0 + n + 1) * step];
                    decay[n] = d[(n0 + n) * dstep];
                }
#pragma unroll
            for (int n = 0; n < kScanBatch; ++n)
                if (n0 + n < p.nseg) {
                    s = decay[n] != 0.0f ? fmaf(decay[n], s, local[n]) : local[n];  // (s may be infinite)
                    x[(n0 + n + 1) * step] = s;
                }
        }
        if (p.last[role]) p.last[role][i] = s;
    }
}

namespace {

bool aligned(const void* p, size_t n) { return (uintptr_t)p % n == 0; }

// A view as the kernels take it.
RView rview(const hyena_view& v, int64_t width, size_t element)
{
    auto made_of = [&](int64_t n) {
        return width % n == 0 && aligned(v.data, (size_t)n * element) && v.batch % n == 0 && v.token % n == 0 && v.head % n == 0;
    };
    const int32_t vec = made_of(16 / (int64_t)element) ? kRowVectors : made_of(2) ? kRowPairs : kRowElements;
    return RView{v.data, v.batch, v.token, v.head, vec};
}

hyena_status refuse(const char* what) { return fail(HYENA_ERR_INVALID_ARGUMENT, std::string("recurrence: ") + what); }

// Checks shared by the three calls; n: tokens of the views; spans: the inputs.
hyena_status check_inputs(const RecPlan& p, const hyena_recurrence_inputs* in, int64_t n, Span* spans)
{
    if (in == nullptr) return refuse("inputs are NULL");
    const size_t e = element_bytes(p.io_dtype);
    hyena_status st;
    if ((st = check_view(in->q, "q", e)) != HYENA_OK || (st = check_view(in->k, "k", e)) != HYENA_OK ||
        (st = check_view(in->v, "v", e)) != HYENA_OK || (st = check_view(in->g, "g", 4)) != HYENA_OK)
        return st;
    if ((st = check_token_stride(in->q, "q", n)) != HYENA_OK || (st = check_token_stride(in->k, "k", n)) != HYENA_OK ||
        (st = check_token_stride(in->v, "v", n)) != HYENA_OK || (st = check_token_stride(in->g, "g", n)) != HYENA_OK)
        return st;
    spans[0] = view_span(in->q, p.B, n, p.heads, p.dk, e);
    spans[1] = view_span(in->k, p.B, n, p.heads, p.dk, e);
    spans[2] = view_span(in->v, p.B, n, p.heads, p.dv, e);
    spans[3] = view_span(in->g, p.B, n, p.heads, 1, 4);
    return HYENA_OK;
}

// Outputs may not overlap each other, an input or the workspace.  The first `vectors`
// of them are stored by vectors, the others, all float32, by elements.
hyena_status check_outputs(const Span* in, int nin, const Span* out, const char* const* names, int nout, int vectors)
{
    for (int i = 0; i < nout; ++i) {
        if (out[i].p == nullptr) continue;
        if (i < vectors && !aligned(out[i].p, 16))
            return fail(HYENA_ERR_INVALID_ARGUMENT, std::string(names[i]) + " must be 16-byte aligned");
        if (!aligned(out[i].p, 4))
            return fail(HYENA_ERR_INVALID_ARGUMENT, std::string(names[i]) + " is not aligned to its element");
        for (int j = 0; j < nin; ++j)
            if (spans_overlap(out[i], in[j]))
                return fail(HYENA_ERR_INVALID_ARGUMENT, std::string(names[i]) + " overlaps an input or the workspace");
        for (int j = 0; j < i; ++j)
            if (spans_overlap(out[i], out[j]))
                return fail(HYENA_ERR_INVALID_ARGUMENT, std::string(names[i]) + " overlaps " + names[j]);
    }
    return HYENA_OK;
}

hyena_status launch_scan(const RecScanArgs& a, int roles, hipStream_t s)
{
    const int64_t groups = (a.total + 255) / 256, most = (int64_t)1 << 22;  // the rest is looped over
    HY_LAUNCH(kernel_label("hyena_rec_scan"), hyena_rec_scan, dim3((unsigned)(groups < most ? groups : most), (unsigned)roles),
              dim3(256), 0, s, a);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? HYENA_OK : fail(HYENA_ERR_DEVICE, hipGetErrorString(e));
}

// States before the segments (and, roles = 2, gradients after them).
template <typename T>
hyena_status rec_states(const RecPlan& p, const hyena_recurrence_inputs& in, const hyena_view* d_o, const float* d_final,
                        float* last, float* d_state, const RecSpace& w, int nseg, hipStream_t s)
{
    const size_t e = sizeof(T);
    const int roles = d_o ? 2 : 1;
    RecStateArgs a{};
    a.x[0] = rview(in.k, p.dk, e);
    a.y[0] = rview(in.v, p.dv, e);
    if (d_o) {
        a.x[1] = rview(in.q, p.dk, e);
        a.y[1] = rview(*d_o, p.dv, e);
    }
    a.g = rview(in.g, 1, 4);
    a.lengths = in.lengths;
    a.local[0] = w.start;
    a.local[1] = w.end;
    a.decay = w.decay;
    a.N = p.N;
    a.heads = p.heads;
    a.dk = p.dk;
    a.dv = p.dv;
    a.nseg = nseg;
    a.scale = in.scale;
    hyena_status st = rec_launch_states<T>(a, p.B * p.heads, roles, s);
    if (st != HYENA_OK) return st;
    RecScanArgs c{};
    c.local[0] = w.start;
    c.local[1] = w.end;
    c.first[0] = in.state;
    c.first[1] = d_final;
    c.last[0] = last;
    c.last[1] = d_state;
    c.decay = w.decay;
    c.per = (int64_t)p.dk * p.dv;
    c.total = p.B * p.heads * c.per;
    c.nseg = nseg;
    return launch_scan(c, roles, s);
}

template <typename T>
hyena_status run_forward(const RecPlan& p, const hyena_recurrence_inputs& in, void* o, float* last, void* workspace,
                         hipStream_t s)
{
    const RecSpace w = p.nseg > 1 ? rec_space(p, false, workspace) : RecSpace{};
    if (p.nseg > 1) {
        const hyena_status st = rec_states<T>(p, in, nullptr, nullptr, last, nullptr, w, p.nseg, s);
        if (st != HYENA_OK) return st;
    }
    const size_t e = sizeof(T);
    RecArgs a{};
    a.a = rview(in.q, p.dk, e);
    a.b = rview(in.k, p.dk, e);
    a.c = rview(in.v, p.dv, e);
    a.g = rview(in.g, 1, 4);
    a.lengths = in.lengths;
    a.out = o;
    a.state = p.nseg > 1 ? w.start : in.state;
    a.state_n = p.nseg > 1 ? p.nseg + 1 : 1;
    a.last = p.nseg > 1 ? nullptr : last;
    a.N = p.N;
    a.heads = p.heads;
    a.da = p.dk;
    a.dc = p.dv;
    a.nseg = p.nseg;
    a.scale = in.scale;
    return rec_launch_out<T>(a, p.B * p.heads, false, s);
}

template <typename T>
hyena_status run_backward(const RecPlan& p, const hyena_recurrence_inputs& in, const hyena_view& d_o,
                          const float* d_final, const hyena_recurrence_grads& out, void* workspace, hipStream_t s)
{
    const RecSpace w = rec_space(p, true, workspace);
    const int64_t bh = p.B * p.heads;
    const size_t e = sizeof(T);
    // one segment, dq's (nseg_b * every) included, and nothing coming from the end
    // or asked for at the start: no state is needed before the main passes
    const bool states = p.nseg_b * p.every > 1 || d_final != nullptr || out.d_state != nullptr;
    if (states) {
        const hyena_status st =
            rec_states<T>(p, in, &d_o, d_final, nullptr, out.d_state, w, p.nseg_b * p.every, s);
        if (st != HYENA_OK) return st;
    }
    RecArgs a{};
    a.a = rview(d_o, p.dv, e);
    a.b = rview(in.v, p.dv, e);
    a.c = rview(in.k, p.dk, e);
    a.r = rview(in.q, p.dk, e);
    a.g = rview(in.g, 1, 4);
    a.lengths = in.lengths;
    a.out = out.dq;
    a.state = states ? w.start : in.state;
    a.state_n = states ? p.nseg_b * p.every + 1 : 1;
    a.rq = w.rq;
    a.N = p.N;
    a.heads = p.heads;
    a.da = p.dv;
    a.dc = p.dk;
    a.nseg = p.nseg_b * p.every;
    a.scale = in.scale;
    hyena_status st = rec_launch_out<T>(a, bh, true, s);
    if (st != HYENA_OK) return st;
    RecGradArgs g{};
    g.q = rview(in.q, p.dk, e);
    g.k = rview(in.k, p.dk, e);
    g.v = rview(in.v, p.dv, e);
    g.o = rview(d_o, p.dv, e);
    g.g = a.g;
    g.lengths = in.lengths;
    g.dk_out = out.dk;
    g.dv_out = out.dv;
    g.dg = out.dg;
    g.rq = w.rq;
    g.start = states ? w.start : nullptr;
    g.end = states ? w.end : nullptr;
    g.N = p.N;
    g.heads = p.heads;
    g.dk = p.dk;
    g.dv = p.dv;
    g.every = p.every;
    g.nseg = p.nseg_b;
    g.scale = in.scale;
    return rec_launch_grad<T>(g, bh, s);
}

template <typename T>
hyena_status run_step(const RecPlan& p, const hyena_recurrence_inputs& in, const int32_t* slots, int64_t n_slots,
                      float* states, void* o, hipStream_t s)
{
    RecStepArgs a{};
    a.q = rview(in.q, p.dk, sizeof(T));
    a.k = rview(in.k, p.dk, sizeof(T));
    a.v = rview(in.v, p.dv, sizeof(T));
    a.g = rview(in.g, 1, 4);
    a.slots = slots;
    a.states = states;
    a.o = o;
    a.n_slots = n_slots;
    a.heads = p.heads;
    a.dk = p.dk;
    a.dv = p.dv;
    a.scale = in.scale;
    return rec_launch_step<T>(a, p.B, s);
}

template <typename F> hyena_status by_type(int32_t io_dtype, F f)
{
    if (io_dtype == HYENA_F32) return f(float{});
    if (io_dtype == HYENA_BF16) return f(uint16_t{});
    return f(_Float16{});
}

}  // namespace
}  // namespace hy

using namespace hy;

extern "C" {

hyena_status hyena_recurrence_create(hyena_recurrence_t* plan, int64_t B, int64_t N, int64_t heads, int64_t dk,
                                     int64_t dv, int32_t io_dtype)
{
    if (plan == nullptr) return refuse("plan output pointer is NULL");
    hyena_recurrence_s* s = new (std::nothrow) hyena_recurrence_s;
    if (s == nullptr) return refuse("out of host memory");
    const hyena_status st = rec_plan_build(s->p, B, N, heads, dk, dv, io_dtype);
    if (st != HYENA_OK) {
        delete s;
        return st;
    }
    *plan = s;
    return HYENA_OK;
}

hyena_status hyena_recurrence_query(hyena_recurrence_t plan, size_t* forward_bytes, size_t* backward_bytes)
{
    if (plan == nullptr) return refuse("plan is NULL");
    if (forward_bytes) *forward_bytes = plan->p.forward_bytes;
    if (backward_bytes) *backward_bytes = plan->p.backward_bytes;
    return HYENA_OK;
}

hyena_status hyena_recurrence_forward(hyena_recurrence_t plan, const hyena_recurrence_inputs* in, void* o,
                                      float* final_state, void* workspace, void* stream)
{
    if (plan == nullptr) return refuse("plan is NULL");
    const RecPlan& p = plan->p;
    Span spans[7];
    hyena_status st = check_inputs(p, in, p.N, spans);
    if (st != HYENA_OK) return st;
    if (o == nullptr) return refuse("o is NULL");
    if (p.forward_bytes > 0 && workspace == nullptr) return refuse("workspace is NULL");
    if (!aligned(workspace, 16)) return refuse("workspace is not 16-byte aligned");
    if (!aligned(in->state, 4) || !aligned(in->lengths, 4)) return refuse("state or lengths is not aligned to its element");
    const size_t state = (size_t)(p.B * p.heads) * (size_t)p.dk * (size_t)p.dv * 4;
    spans[4] = Span{in->state, state};
    spans[5] = Span{in->lengths, (size_t)p.B * 4};
    spans[6] = Span{workspace, p.forward_bytes};
    const Span out[2] = {{o, (size_t)(p.B * p.heads) * (size_t)p.N * (size_t)p.dv * element_bytes(p.io_dtype)},
                         {final_state, state}};
    const char* const names[2] = {"o", "final_state"};
    if ((st = check_outputs(spans, 7, out, names, 2, 1)) != HYENA_OK) return st;
    return by_type(p.io_dtype, [&](auto t) {
        return run_forward<decltype(t)>(p, *in, o, final_state, workspace, (hipStream_t)stream);
    });
}

hyena_status hyena_recurrence_backward(hyena_recurrence_t plan, const hyena_recurrence_inputs* in,
                                       const hyena_view* d_o, const float* d_final, const hyena_recurrence_grads* out,
                                       void* workspace, void* stream)
{
    if (plan == nullptr) return refuse("plan is NULL");
    const RecPlan& p = plan->p;
    Span spans[9];
    hyena_status st = check_inputs(p, in, p.N, spans);
    if (st != HYENA_OK) return st;
    if (d_o == nullptr) return refuse("d_o is NULL");
    const size_t e = element_bytes(p.io_dtype);
    if ((st = check_view(*d_o, "d_o", e)) != HYENA_OK || (st = check_token_stride(*d_o, "d_o", p.N)) != HYENA_OK) return st;
    if (out == nullptr || out->dq == nullptr || out->dk == nullptr || out->dv == nullptr || out->dg == nullptr)
        return refuse("an output pointer is NULL");
    if (workspace == nullptr) return refuse("workspace is NULL");
    if (!aligned(workspace, 16)) return refuse("workspace is not 16-byte aligned");
    if (!aligned(in->state, 4) || !aligned(in->lengths, 4) || !aligned(d_final, 4))
        return refuse("state, d_final or lengths is not aligned to its element");
    const size_t n = (size_t)(p.B * p.heads) * (size_t)p.N;
    const size_t state = (size_t)(p.B * p.heads) * (size_t)p.dk * (size_t)p.dv * 4;
    spans[4] = Span{in->state, state};
    spans[5] = Span{in->lengths, (size_t)p.B * 4};
    spans[6] = Span{workspace, p.backward_bytes};
    spans[7] = view_span(*d_o, p.B, p.N, p.heads, p.dv, e);
    spans[8] = Span{d_final, state};
    const Span outs[5] = {{out->dq, n * p.dk * e}, {out->dk, n * p.dk * e}, {out->dv, n * p.dv * e},
                          {out->dg, n * 4}, {out->d_state, state}};
    const char* const names[5] = {"dq", "dk", "dv", "dg", "d_state"};
    if ((st = check_outputs(spans, 9, outs, names, 5, 3)) != HYENA_OK) return st;
    return by_type(p.io_dtype, [&](auto t) {
        return run_backward<decltype(t)>(p, *in, *d_o, d_final, *out, workspace, (hipStream_t)stream);
    });
}

hyena_status hyena_recurrence_step(hyena_recurrence_t plan, const hyena_recurrence_inputs* in, const int32_t* slots,
                                   int64_t n_slots, float* states, void* o, void* stream)
{
    if (plan == nullptr) return refuse("plan is NULL");
    const RecPlan& p = plan->p;
    Span spans[5];
    hyena_status st = check_inputs(p, in, 1, spans);
    if (st != HYENA_OK) return st;
    if (states == nullptr || o == nullptr) return refuse("states or o is NULL");
    if (n_slots < 1 || (slots == nullptr && n_slots < p.B)) return refuse("n_slots is below the rows that use the states");
    if (n_slots > ((int64_t)1 << 31) - 1) return refuse("n_slots must be below 2^31");
    if (!aligned(slots, 4)) return refuse("slots is not aligned to its element");
    spans[4] = Span{slots, (size_t)p.B * 4};
    const Span outs[2] = {{o, (size_t)(p.B * p.heads) * (size_t)p.dv * element_bytes(p.io_dtype)},
                          {states, (size_t)n_slots * (size_t)p.heads * (size_t)p.dk * (size_t)p.dv * 4}};
    const char* const names[2] = {"o", "states"};
    if ((st = check_outputs(spans, 5, outs, names, 2, 1)) != HYENA_OK) return st;
    return by_type(p.io_dtype, [&](auto t) {
        return run_step<decltype(t)>(p, *in, slots, n_slots, states, o, (hipStream_t)stream);
    });
}

hyena_status hyena_recurrence_destroy(hyena_recurrence_t plan)
{
    delete plan;
    return HYENA_OK;
}

}  // extern "C"
