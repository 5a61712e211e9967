// rows.h -- rows of channels for the operators on whole tokens: strided rows,
// 16-byte units of a row, and the teams of lanes that hold one.
//
// A row is cut into units of 16 bytes of the storage type.  A team of lanes holds
// it, lane l the units l, l + lanes, ...: part of a wave (lanes a power of two) or
// a whole workgroup.  Where every row of a call is made of whole aligned units
// they are moved by 16-byte accesses (VEC); else by pairs of elements or by
// elements, whichever the call's rows allow, with the same units per lane.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <string>

#include "hyena.h"
#include "plan.h"
#include "recurrence_device.h"
#include "recurrence_plan.h"
#include "timing.h"

namespace hy {

template <typename T> constexpr int kUnit = 16 / (int)sizeof(T);

// Strided rows (strides in elements); row r of N to a batch row.
struct Rows {
    const void* p;
    int64_t b, t;
};

template <typename T> __device__ __forceinline__ const T* row_at(const Rows& x, int64_t r, uint32_t N)
{
    // N = 0: rows at one distance (b * N = t * N or one batch row)
    if (N == 0) return (const T*)x.p + r * x.t;
    const uint32_t b = (uint32_t)r / N, n = (uint32_t)r - b * N;
    return (const T*)x.p + (int64_t)b * x.b + (int64_t)n * x.t;
}

// The unit at channel c of a row of d.  Channels at d and after it are 0.
template <typename T, bool VEC>
__device__ __forceinline__ void load_unit(const T* row, int c, int d, bool pairs, float (&x)[kUnit<T>])
{
    typedef T pair __attribute__((ext_vector_type(2)));
    if constexpr (VEC) {
        const uint4 v = *(const uint4*)(row + c);
        const T* e = (const T*)&v;
#pragma unroll
        for (int i = 0; i < kUnit<T>; ++i) x[i] = load_one<T>(e + i);
    } else if (pairs) {
#pragma unroll
        for (int i = 0; i < kUnit<T>; i += 2) {
            pair v = {};
            if (c + i < d) v = *(const pair*)(row + c + i);
            const T a = v[0], b = v[1];
            x[i] = load_one<T>(&a);
            x[i + 1] = load_one<T>(&b);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kUnit<T>; ++i) x[i] = c + i < d ? load_one<T>(row + c + i) : 0.0f;
    }
}

// A unit as loaded, for loads that are to be under way together: 16-byte accesses
// keep its 16 bytes and widen them later.
template <typename T, bool VEC> struct RawUnit {
    float x[kUnit<T>];
    __device__ __forceinline__ void load(const T* row, int c, int d, bool pairs) { load_unit<T, false>(row, c, d, pairs, x); }
    __device__ __forceinline__ void widen(float (&y)[kUnit<T>]) const
    {
#pragma unroll
        for (int i = 0; i < kUnit<T>; ++i) y[i] = x[i];
    }
};
template <typename T> struct RawUnit<T, true> {
    uint4 v;
    __device__ __forceinline__ void load(const T* row, int c, int, bool) { v = *(const uint4*)(row + c); }
    __device__ __forceinline__ void widen(float (&y)[kUnit<T>]) const
    {
        const T* e = (const T*)&v;
#pragma unroll
        for (int i = 0; i < kUnit<T>; ++i) y[i] = load_one<T>(e + i);
    }
};

template <typename T, bool VEC>
__device__ __forceinline__ void store_unit(T* row, int c, int d, bool pairs, const float (&x)[kUnit<T>])
{
    typedef T pair __attribute__((ext_vector_type(2)));
    if constexpr (VEC) {
        uint4 v;
        T* e = (T*)&v;
#pragma unroll
        for (int i = 0; i < kUnit<T>; ++i) store_one<T>(e + i, x[i]);
        *(uint4*)(row + c) = v;
    } else if (pairs) {
#pragma unroll
        for (int i = 0; i < kUnit<T>; i += 2)
            if (c + i < d) {
                T a, b;
                store_one<T>(&a, x[i]);
                store_one<T>(&b, x[i + 1]);
                *(pair*)(row + c + i) = pair{a, b};
            }
    } else {
#pragma unroll
        for (int i = 0; i < kUnit<T>; ++i)
            if (c + i < d) store_one<T>(row + c + i, x[i]);
    }
}

// ---------------------------------------------------------------- host side

// What all of a call's rows are made of: whole aligned units, pairs or elements.
enum : int32_t { kMadeOfElements = 0, kMadeOfPairs = 1, kMadeOfUnits = 2 };

class RowShape {
public:
    RowShape(int64_t d, size_t element) : d_(d), e_(element) {}
    void add(const hyena_rows& v) { add(v.data, v.batch, v.token); }
    void dense(const void* p) { add(p, 0, 0); }
    int32_t made_of() const { return fits_[1] ? kMadeOfUnits : fits_[0] ? kMadeOfPairs : kMadeOfElements; }

private:
    void add(const void* p, int64_t b, int64_t t)
    {
        const int64_t n[2] = {2, 16 / (int64_t)e_};
        for (int i = 0; i < 2; ++i)
            if (d_ % n[i] != 0 || (uintptr_t)p % (n[i] * e_) != 0 || b % n[i] != 0 || t % n[i] != 0) fits_[i] = false;
    }
    int64_t d_;
    size_t e_;
    bool fits_[2] = {true, true};
};

// Strides that B = 1 or N = 1 leaves open are 0.
inline hyena_rows plain_rows(const hyena_rows& v, int64_t B, int64_t N)
{
    return hyena_rows{v.data, B > 1 ? v.batch : 0, N > 1 ? v.token : 0};
}

// The rows of a call as one axis where all of its tensors allow it: *N becomes 0
// and the token stride the distance of any two neighbouring rows.
inline void flatten_rows(hyena_rows* const* v, int n, int64_t B, int64_t* N)
{
    bool flat = true;
    for (int i = 0; i < n; ++i) flat = flat && (B == 1 || *N == 1 || v[i]->batch == *N * v[i]->token);
    if (!flat) return;
    for (int i = 0; i < n; ++i)
        if (*N == 1) v[i]->token = v[i]->batch;
    *N = 0;
}

inline hyena_status check_rows(const char* who, const hyena_rows& v, const char* name, size_t element)
{
    const std::string at = std::string(who) + ": " + name;
    if (v.data == nullptr) return fail(HYENA_ERR_INVALID_ARGUMENT, at + " is NULL");
    if ((uintptr_t)v.data % element != 0) return fail(HYENA_ERR_INVALID_ARGUMENT, at + " is not aligned to its element");
    if (v.batch < 0 || v.token < 0) return fail(HYENA_ERR_INVALID_ARGUMENT, at + " has a negative stride");
    if (v.batch > ((int64_t)1 << 40) || v.token > ((int64_t)1 << 40))
        return fail(HYENA_ERR_UNSUPPORTED, at + " has a stride above 2^40 elements");
    return HYENA_OK;
}

inline hyena_status check_io(const char* who, int32_t io_dtype)
{
    if (io_dtype != HYENA_F32 && io_dtype != HYENA_BF16 && io_dtype != HYENA_F16)
        return fail(HYENA_ERR_UNSUPPORTED, std::string(who) + ": unknown io dtype");
    return HYENA_OK;
}

inline Span rows_span(const hyena_rows& v, int64_t B, int64_t N, int64_t width, size_t element)
{
    const unsigned __int128 n = ((unsigned __int128)(B - 1) * (uint64_t)v.batch +
                                 (unsigned __int128)(N - 1) * (uint64_t)v.token + (uint64_t)width) * element;
    const unsigned __int128 most = (unsigned __int128)1 << 62;
    return Span{v.data, (size_t)(n < most ? n : most)};
}

struct Named {
    Span span;
    const char* name;
};

// No output may overlap an input or another output.
inline hyena_status check_apart(const char* who, const Span* in, int nin, const Named* out, int nout)
{
    for (int i = 0; i < nout; ++i) {
        for (int j = 0; j < nin; ++j)
            if (spans_overlap(out[i].span, in[j]))
                return fail(HYENA_ERR_INVALID_ARGUMENT, std::string(who) + ": " + out[i].name + " overlaps an input");
        for (int j = 0; j < i; ++j)
            if (spans_overlap(out[i].span, out[j].span))
                return fail(HYENA_ERR_INVALID_ARGUMENT,
                            std::string(who) + ": " + out[i].name + " overlaps " + out[j].name);
    }
    return HYENA_OK;
}

inline hyena_status launched()
{
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? HYENA_OK : fail(HYENA_ERR_DEVICE, hipGetErrorString(e));
}

// f(type_tag) for an io dtype.
template <typename F> hyena_status by_io(int32_t io_dtype, F&& f)
{
    if (io_dtype == HYENA_F32) return f((float*)nullptr);
    if (io_dtype == HYENA_BF16) return f((uint16_t*)nullptr);
    return f((_Float16*)nullptr);
}

}  // namespace hy
