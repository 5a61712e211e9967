// rows.h -- rows of channels for the operators on whole tokens: strided rows,
// 16-byte units of a row, and the teams of lanes that hold one.
//
// A row is cut into units of 16 bytes of the storage type.  A team of lanes holds it,
// lane l the units l, l + lanes, ...: part of a wave (lanes a power of two) or a whole
// workgroup.  Rows that are not made of whole aligned units are moved by 16-byte accesses
// all the same, at their elements' alignment, which the machine takes; only what is left
// at a row's end goes by elements (norm of 16320 rows of 771 channels in bf16: 29 us so,
// 62 by elements; of 16384 rows of 768: 17).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <string>
#include <type_traits>

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

// 16 bytes at an element's alignment.
template <typename T> struct __attribute__((packed, aligned(sizeof(T)))) Loose {
    uint32_t w[4];
};

// A unit as loaded (channels at d and after it are 0), and widened.  UNITS: the rows are made
// of whole aligned units.
template <typename T, bool UNITS> struct Unit {
    static constexpr int K = kUnit<T>;
    uint4 v;
    __device__ __forceinline__ void load(const T* row, int c, int d)
    {
        if constexpr (UNITS) {
            // no branch, so that loads stay together (gradient of 65536 tokens 38 us with one, 28 without)
            const uint4 x = *(const uint4*)(row + (c < d ? c : 0));
            v = make_uint4(c < d ? x.x : 0, c < d ? x.y : 0, c < d ? x.z : 0, c < d ? x.w : 0);
            return;
        }
        v = make_uint4(0, 0, 0, 0);
        if (c + K <= d) {
            const Loose<T> x = *(const Loose<T>*)(row + c);
            v = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
        } else if (c < d) {
            T* e = (T*)&v;
#pragma unroll
            for (int i = 0; i < K; ++i)
                if (c + i < d) e[i] = row[c + i];
        }
    }
    __device__ __forceinline__ void widen(float (&x)[K]) const
    {
        const T* e = (const T*)&v;
#pragma unroll
        for (int i = 0; i < K; ++i) x[i] = load_one<T>(e + i);
    }
    __device__ __forceinline__ void set(const float (&x)[K])
    {
        T* e = (T*)&v;
#pragma unroll
        for (int i = 0; i < K; ++i) store_one<T>(e + i, x[i]);
    }
    __device__ __forceinline__ void store(T* row, int c, int d) const
    {
        if constexpr (UNITS) {
            if (c < d) *(uint4*)(row + c) = v;
        } else if (c + K <= d) {
            Loose<T> x;
            x.w[0] = v.x, x.w[1] = v.y, x.w[2] = v.z, x.w[3] = v.w;
            *(Loose<T>*)(row + c) = x;
        } else if (c < d) {
            const T* e = (const T*)&v;
#pragma unroll
            for (int i = 0; i < K; ++i)
                if (c + i < d) row[c + i] = e[i];
        }
    }
};

template <typename T, bool UNITS>
__device__ __forceinline__ void load_unit(const T* row, int c, int d, float (&x)[kUnit<T>])
{
    Unit<T, UNITS> y;
    y.load(row, c, d);
    y.widen(x);
}
template <typename T, bool UNITS>
__device__ __forceinline__ void store_unit(T* row, int c, int d, const float (&x)[kUnit<T>])
{
    Unit<T, UNITS> y;
    y.set(x);
    y.store(row, c, d);
}

// ---------------------------------------------------------------- host side

// Whether all of a call's rows are made of whole aligned units.
class RowShape {
public:
    RowShape(int64_t d, size_t element) : n_(16 / (int64_t)element), units_(d % n_ == 0) {}
    void add(const hyena_rows& v)
    {
        if ((uintptr_t)v.data % 16 != 0 || v.batch % n_ != 0 || v.token % n_ != 0) units_ = false;
    }
    void dense(const void* p) { add(hyena_rows{p, 0, 0}); }
    bool units() const { return units_; }

private:
    int64_t n_;
    bool units_;
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
    auto at = [&](const char* what) { return std::string(who) + ": " + name + what; };
    if (v.data == nullptr) return fail(HYENA_ERR_INVALID_ARGUMENT, at(" is NULL"));
    if ((uintptr_t)v.data % element != 0) return fail(HYENA_ERR_INVALID_ARGUMENT, at(" is not aligned to its element"));
    if (v.batch < 0 || v.token < 0) return fail(HYENA_ERR_INVALID_ARGUMENT, at(" has a negative stride"));
    if (v.batch > ((int64_t)1 << 40) || v.token > ((int64_t)1 << 40))
        return fail(HYENA_ERR_UNSUPPORTED, at(" has a stride above 2^40 elements"));
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

// f(std::bool_constant) for whether rows are made of units.
template <typename F> hyena_status by_units(bool units, F&& f)
{
    return units ? f(std::true_type{}) : f(std::false_type{});
}

// f(a null pointer to the type) for an io dtype.
template <typename F> hyena_status by_io(int32_t io_dtype, F&& f)
{
    if (io_dtype == HYENA_F32) return f((float*)nullptr);
    if (io_dtype == HYENA_BF16) return f((uint16_t*)nullptr);
    return f((_Float16*)nullptr);
}

}  // namespace hy
