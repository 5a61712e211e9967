// recurrence_launch.h -- instantiates the recurrence's kernels for one storage
// type: head widths are padded to 64 or 128 channels.
#pragma once

#include "recurrence_kernels.h"

namespace hy {

inline hyena_status rec_done()
{
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? HYENA_OK : fail(HYENA_ERR_DEVICE, hipGetErrorString(e));
}

// Rows that are all made of 16-byte vectors have kernels of their own (VEC): the
// others choose by tensor what they load.
template <typename... V> bool by_vectors(const V&... v) { return ((v.vec == kRowVectors) && ...); }

template <typename T, int DK, int DV>
hyena_status rec_states_one(const RecStateArgs& a, int64_t bh, int roles, hipStream_t s)
{
    const bool vec = by_vectors(a.x[0], a.y[0]) && (roles == 1 || by_vectors(a.x[1], a.y[1]));
    const dim3 grid((unsigned)(bh * a.nseg), (unsigned)roles);
    if (vec)
        HY_LAUNCH(kernel_label("hyena_rec_states", type_label<T>(), DK, DV, true), (hyena_rec_states<T, DK, DV, true>), grid,
                  dim3(256), 0, s, a);
    else
        HY_LAUNCH(kernel_label("hyena_rec_states", type_label<T>(), DK, DV, false), (hyena_rec_states<T, DK, DV, false>), grid,
                  dim3(256), 0, s, a);
    return rec_done();
}

template <typename T> hyena_status rec_launch_states(const RecStateArgs& a, int64_t bh, int roles, hipStream_t s)
{
    if (a.dk <= 64) return a.dv <= 64 ? rec_states_one<T, 64, 64>(a, bh, roles, s) : rec_states_one<T, 64, 128>(a, bh, roles, s);
    return a.dv <= 64 ? rec_states_one<T, 128, 64>(a, bh, roles, s) : rec_states_one<T, 128, 128>(a, bh, roles, s);
}

template <typename T, int DA, int DC, bool TRANS, bool VEC>
hyena_status rec_out_as(const RecArgs& a, int64_t bh, hipStream_t s)
{
    HY_LAUNCH(kernel_label("hyena_rec_out", type_label<T>(), DA, DC, TRANS, VEC),
              (hyena_rec_out<T, DA, DC, TRANS, VEC>), dim3((unsigned)(bh * a.nseg)), dim3(256), 0, s, a);
    return rec_done();
}

template <typename T, int DA, int DC, bool TRANS>
hyena_status rec_out_one(const RecArgs& a, int64_t bh, hipStream_t s)
{
    const bool vec = by_vectors(a.a, a.b, a.c) && (!TRANS || by_vectors(a.r));
    return vec ? rec_out_as<T, DA, DC, TRANS, true>(a, bh, s) : rec_out_as<T, DA, DC, TRANS, false>(a, bh, s);
}

template <typename T, bool TRANS> hyena_status rec_out_pick(const RecArgs& a, int64_t bh, hipStream_t s)
{
    if (a.da <= 64)
        return a.dc <= 64 ? rec_out_one<T, 64, 64, TRANS>(a, bh, s) : rec_out_one<T, 64, 128, TRANS>(a, bh, s);
    return a.dc <= 64 ? rec_out_one<T, 128, 64, TRANS>(a, bh, s) : rec_out_one<T, 128, 128, TRANS>(a, bh, s);
}

template <typename T> hyena_status rec_launch_out(const RecArgs& a, int64_t bh, bool transposed, hipStream_t s)
{
    return transposed ? rec_out_pick<T, true>(a, bh, s) : rec_out_pick<T, false>(a, bh, s);
}

template <typename T, int DK, int DV, bool VEC>
hyena_status rec_grad_as(const RecGradArgs& a, int64_t bh, hipStream_t s)
{
    HY_LAUNCH(kernel_label("hyena_rec_grad", type_label<T>(), DK, DV, VEC), (hyena_rec_grad<T, DK, DV, VEC>),
              dim3((unsigned)(bh * a.nseg)), dim3(512), 0, s, a);
    return rec_done();
}

template <typename T, int DK, int DV> hyena_status rec_grad_one(const RecGradArgs& a, int64_t bh, hipStream_t s)
{
    return by_vectors(a.q, a.k, a.v, a.o) ? rec_grad_as<T, DK, DV, true>(a, bh, s) : rec_grad_as<T, DK, DV, false>(a, bh, s);
}

template <typename T> hyena_status rec_launch_grad(const RecGradArgs& a, int64_t bh, hipStream_t s)
{
    if (a.dk <= 64) return a.dv <= 64 ? rec_grad_one<T, 64, 64>(a, bh, s) : rec_grad_one<T, 64, 128>(a, bh, s);
    return a.dv <= 64 ? rec_grad_one<T, 128, 64>(a, bh, s) : rec_grad_one<T, 128, 128>(a, bh, s);
}

template <typename T> hyena_status rec_launch_step(const RecStepArgs& a, int64_t B, hipStream_t s)
{
    const bool vec = a.dv % 4 == 0 && ((uintptr_t)a.states & 15) == 0;
    if (vec) {
        HY_LAUNCH(kernel_label("hyena_rec_step", type_label<T>(), 4), (hyena_rec_step<T, 4>),
                  dim3((unsigned)(B * a.heads)), dim3(256), 0, s, a);
    } else {
        HY_LAUNCH(kernel_label("hyena_rec_step", type_label<T>(), 1), (hyena_rec_step<T, 1>),
                  dim3((unsigned)(B * a.heads)), dim3(256), 0, s, a);
    }
    return rec_done();
}

}  // namespace hy

#define HY_REC_INSTANTIATE(T)                                                                        \
    namespace hy {                                                                                   \
    template hyena_status rec_launch_states<T>(const RecStateArgs&, int64_t, int, hipStream_t);      \
    template hyena_status rec_launch_out<T>(const RecArgs&, int64_t, bool, hipStream_t);             \
    template hyena_status rec_launch_grad<T>(const RecGradArgs&, int64_t, hipStream_t);              \
    template hyena_status rec_launch_step<T>(const RecStepArgs&, int64_t, hipStream_t);              \
    }
