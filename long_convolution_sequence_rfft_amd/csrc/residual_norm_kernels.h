// residual_norm_kernels.h -- RMS norm of whole tokens with the residual's
// addition, and its backward pass (include/hyena.h).
//
// Forward, for a row of d channels with s = x + residual:
//   r = 1 / sqrt(mean(s^2) + eps),  y = w r s,
// or y in 8 bits, value = round(y / a), a = max|y| of a group / the largest value.
// Backward, with n = r s and dn = w dy:
//   dx = ds + r (dn - n mean(dn n)),  dw = sum over rows of dy n.
//
// Bound by memory: each tensor is read or written once.  A row stays in the
// registers of the team of lanes that holds it; teams go through the rows in
// steps, so that the weights, and backward the sums for their gradient, are
// loaded (stored) once for each team and not for each row.
//
// 16384 rows of 768 in bf16 with a residual: 16.9 us for 101 MB, to e4m3 20.6 us (by groups of 128
// 21.3) for 88 MB, their gradients 23.2 us for as much as the first and 4.0 us for the weights' sums; 8192 rows
// of 1000 in binary16, gradients 14.7 us for 49 MB.  The next row's loads ahead of this one's work
// made none of them faster, and loads past the caches only rows that came from memory (21 us
// instead of 23.5, and 14 instead of 13 of rows that did not).  32 rows in 8 bits: 5.0 us.
#pragma once

#include "residual_norm.h"

namespace hy {

// Sum over a team's lanes (WG: a workgroup).
template <bool WG> __device__ __forceinline__ void team_sum(float& a, float& b, bool two, int lanes, float* lds)
{
    const int within = WG ? 64 : lanes;
    for (int m = 1; m < within; m *= 2) {
        a += __shfl_xor(a, m);
        if (two) b += __shfl_xor(b, m);
    }
    if constexpr (WG) {
        const int wave = threadIdx.x >> 6, waves = lanes >> 6;
        __syncthreads();  // the last row's sums have been read
        if ((threadIdx.x & 63) == 0) {
            lds[wave] = a;
            if (two) lds[16 + wave] = b;
        }
        __syncthreads();
        a = 0.0f;
        for (int w = 0; w < waves; ++w) a += lds[w];
        if (two) {
            b = 0.0f;
            for (int w = 0; w < waves; ++w) b += lds[16 + w];
        }
    }
}

// Largest of the bits of absolute values: a NaN is above everything.
template <bool WG> __device__ __forceinline__ uint32_t team_max(uint32_t a, int lanes, float* lds)
{
    const int within = WG ? 64 : lanes;
    for (int m = 1; m < within; m *= 2) a = max(a, (uint32_t)__shfl_xor((int)a, m));
    if constexpr (WG) {
        const int wave = threadIdx.x >> 6, waves = lanes >> 6;
        __syncthreads();  // the sums have been read
        if ((threadIdx.x & 63) == 0) lds[wave] = __uint_as_float(a);
        __syncthreads();
        a = 0;
        for (int w = 0; w < waves; ++w) a = max(a, __float_as_uint(lds[w]));
        __syncthreads();
    }
    return a;
}

__device__ __forceinline__ float rms(float squares, int d, float eps) { return 1.0f / sqrtf(squares / (float)d + eps); }

// The weights of a unit (ones without).
template <bool UNITS, int K> __device__ __forceinline__ void load_weights(const NormArgs& p, int c, float (&w)[K])
{
#pragma unroll
    for (int i = 0; i < K; ++i) w[i] = 1.0f;
    if (p.w == nullptr || c >= p.d) return;
    if (UNITS && p.weight_vectors) {
#pragma unroll
        for (int i = 0; i < K; i += 4) {
            const f32x4 v = *(const f32x4*)(p.w + c + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) w[i + j] = v[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < K; ++i)
            if (c + i < p.d) w[i] = p.w[c + i];
    }
}

// K units of 8-bit values, K = 4 or 8.
template <int K> __device__ __forceinline__ void pack8(const float (&y)[K], bool int8, uint32_t (&w)[K / 4])
{
#pragma unroll
    for (int i = 0; i < K; i += 4) {
        if (int8) {
            uint32_t v = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) v |= ((uint32_t)(int)rintf(fminf(fmaxf(y[i + j], -127.0f), 127.0f)) & 255u) << (8 * j);
            w[i / 4] = v;
        } else {
            int v = __builtin_amdgcn_cvt_pk_fp8_f32(y[i], y[i + 1], 0, false);
            w[i / 4] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[i + 2], y[i + 3], v, true);
        }
    }
}

template <typename T, bool UNITS, bool WG, int U, bool EIGHT>
__global__ __launch_bounds__(WG ? 1024 : 256) void hyena_residual_norm(NormArgs p)
{
    constexpr int K = kUnit<T>;
    __shared__ float lds[32];
    const int lanes = WG ? (int)blockDim.x : p.lanes;
    const int teams = WG ? 1 : 256 / lanes, team = WG ? 0 : (int)threadIdx.x / lanes, tl = WG ? (int)threadIdx.x : (int)threadIdx.x % lanes;
    float w[U][K];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        load_weights<UNITS>(p, (tl + u * lanes) * K, w[u]);
    }
    for (int64_t r = (int64_t)blockIdx.x * teams + team; r < p.rows; r += (int64_t)gridDim.x * teams) {
        const T* x = row_at<T>(p.x, r, p.N);
        const T* res = p.res.p != nullptr ? row_at<T>(p.res, r, p.N) : nullptr;
        float s[U][K];
#pragma unroll
        for (int u = 0; u < U; ++u) load_unit<T, UNITS>(x, (tl + u * lanes) * K, p.d, s[u]);
        if (res != nullptr) {
            float y[U][K];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                load_unit<T, UNITS>(res, (tl + u * lanes) * K, p.d, y[u]);
#pragma unroll
                for (int i = 0; i < K; ++i) s[u][i] += y[u][i];
            }
            T* sum = (T*)p.sum + r * p.d;
#pragma unroll
            for (int u = 0; u < U; ++u) store_unit<T, UNITS>(sum, (tl + u * lanes) * K, p.d, s[u]);
        }
        float squares = 0.0f, none = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < K; ++i) squares = fmaf(s[u][i], s[u][i], squares);
        team_sum<WG>(squares, none, false, lanes, lds);
        const float rstd = rms(squares, p.d, p.eps);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < K; ++i) s[u][i] = s[u][i] * rstd * w[u][i];
        if constexpr (!EIGHT) {
            T* y = (T*)p.y + r * p.d;
#pragma unroll
            for (int u = 0; u < U; ++u) store_unit<T, UNITS>(y, (tl + u * lanes) * K, p.d, s[u]);
        } else {
            uint32_t top[U], row = 0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = (tl + u * lanes) * K;
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < K; ++i)
                    if (c + i < p.d) m = max(m, __float_as_uint(s[u][i]) & 0x7fffffffu);
                // a group is group_lanes lanes side by side
                for (int k = 1; k < p.group_lanes; k *= 2) m = max(m, (uint32_t)__shfl_xor((int)m, k));
                top[u] = m;
                row = max(row, m);
            }
            if (p.group_lanes == 0) {
                row = team_max<WG>(row, lanes, lds);
#pragma unroll
                for (int u = 0; u < U; ++u) top[u] = row;
            }
            uint8_t* y = (uint8_t*)p.y + r * p.d;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int unit = tl + u * lanes, c = unit * K;
                const float most = __uint_as_float(top[u]);
                // (a largest value under 2^-100 has no reciprocal worth having)
                const bool some = !(most < 0x1p-100f);
                const float scale = some ? most * p.inverse : 0.0f, down = some ? p.largest / most : 0.0f;
                if (c < p.d) {
                    float v[K];
#pragma unroll
                    for (int i = 0; i < K; ++i) v[i] = some ? s[u][i] * down : 0.0f;
                    uint32_t q[K / 4];
                    pack8<K>(v, p.int8, q);
                    if (UNITS) {
#pragma unroll
                        for (int i = 0; i < K / 4; ++i) *(uint32_t*)(y + c + 4 * i) = q[i];
                    } else {
#pragma unroll
                        for (int i = 0; i < K; ++i)
                            if (c + i < p.d) y[c + i] = (uint8_t)(q[i / 4] >> (8 * (i % 4)));
                    }
                    if (p.group_lanes != 0 && unit % p.group_lanes == 0) p.scales[r * p.groups + unit / p.group_lanes] = scale;
                }
                if (p.group_lanes == 0 && u == 0 && tl == 0) p.scales[r] = scale;
            }
        }
    }
}

// Rows of a team whose part of the weights' gradient is summed in float32; such sums go to
// float64 ones in LDS, so that what is lost does not grow with the rows (256 equal rows of a team in
// one float32 sum are up to 63 2^-24 off, 16 of them 4.5 2^-24; gradients of 16384 rows of 768 in bf16
// 18.6 us with one sum, 19.2 so, of 2^20 rows of 256 366 and 385).
constexpr int kWeightRows = 16;

template <typename T, bool UNITS, bool WG, int U>
__global__ __launch_bounds__(WG ? 1024 : 256) void hyena_residual_norm_grad(NormArgs p)
{
    constexpr int K = kUnit<T>;
    __shared__ float lds[32];
    extern __shared__ double sums[];  // [teams][whole units of a row], an element one lane's
    const int lanes = WG ? (int)blockDim.x : p.lanes;
    const int teams = WG ? 1 : 256 / lanes, team = WG ? 0 : (int)threadIdx.x / lanes, tl = WG ? (int)threadIdx.x : (int)threadIdx.x % lanes;
    float w[U][K], dw[U][K];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        load_weights<UNITS>(p, (tl + u * lanes) * K, w[u]);
#pragma unroll
        for (int i = 0; i < K; ++i) dw[u][i] = 0.0f;
    }
    const int width = (p.d + K - 1) / K * K;
    int rows = 0;        // in dw
    bool more = false;   // there are sums in LDS
    // dw to LDS.  (Its addresses are not to be held in registers over the rows.)
    auto put_sums = [&]() {
        int at = (team * width + tl * K) * (int)sizeof(double);
        asm volatile("" : "+v"(at));
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if ((tl + u * lanes) * K >= p.d) break;
            double* own = (double*)((char*)sums + at + u * lanes * K * (int)sizeof(double));
#pragma unroll
            for (int i = 0; i < K; ++i) {
                own[i] = (more ? own[i] : 0.0) + (double)dw[u][i];
                dw[u][i] = 0.0f;
            }
        }
        rows = 0;
        more = true;
    };
    for (int64_t r = (int64_t)blockIdx.x * teams + team; r < p.rows; r += (int64_t)gridDim.x * teams) {
        const T* x = row_at<T>(p.x, r, p.N);
        const T* dyr = row_at<T>(p.dy, r, p.N);
        float s[U][K], dy[U][K], ds[U][K];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            load_unit<T, UNITS>(x, (tl + u * lanes) * K, p.d, s[u]);
            load_unit<T, UNITS>(dyr, (tl + u * lanes) * K, p.d, dy[u]);
#pragma unroll
            for (int i = 0; i < K; ++i) ds[u][i] = 0.0f;
        }
        if (p.res.p != nullptr) {
            const T* dsr = row_at<T>(p.res, r, p.N);
#pragma unroll
            for (int u = 0; u < U; ++u) load_unit<T, UNITS>(dsr, (tl + u * lanes) * K, p.d, ds[u]);
        }
        float squares = 0.0f, along = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < K; ++i) {
                squares = fmaf(s[u][i], s[u][i], squares);
                along = fmaf(s[u][i], dy[u][i] * w[u][i], along);
            }
        team_sum<WG>(squares, along, true, lanes, lds);
        const float rstd = rms(squares, p.d, p.eps), mean = along * rstd / (float)p.d;
        T* dx = (T*)p.y + r * p.d;
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < K; ++i) {
                const float n = s[u][i] * rstd;
                s[u][i] = fmaf(rstd, fmaf(-n, mean, dy[u][i] * w[u][i]), ds[u][i]);
                dw[u][i] = fmaf(dy[u][i], n, dw[u][i]);
            }
            store_unit<T, UNITS>(dx, (tl + u * lanes) * K, p.d, s[u]);
        }
        if (++rows == kWeightRows && p.dw_part != nullptr) put_sums();
    }
    if (p.dw_part == nullptr) return;
    float* part = p.dw_part + (int64_t)blockIdx.x * p.d;
    put_sums();
    // the upper half of many teams onto the lower one, the last four together
    int left = teams;
    for (; left > 4; left /= 2) {
        __syncthreads();
        for (int k = threadIdx.x; k < left / 2 * width; k += (int)blockDim.x) sums[k] += sums[k + left / 2 * width];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.d; c += (int)blockDim.x) {
        double x = sums[c];
#pragma unroll
        for (int k = 1; k < 4; ++k)
            if (k < left) x += sums[k * width + c];
        part[c] = (float)x;
    }
}

template <typename T, bool UNITS, bool WG, int U, int KIND> hyena_status norm_as(const NormArgs& a, const NormLaunch& l, hipStream_t s)
{
    if constexpr (KIND == 2)
        HY_LAUNCH(kernel_label("hyena_residual_norm_grad", type_label<T>(), UNITS, WG, U), (hyena_residual_norm_grad<T, UNITS, WG, U>),
                  dim3((unsigned)l.groups), dim3((unsigned)l.threads), a.dw_part ? (size_t)(WG ? 1 : 256 / a.lanes) * ((a.d + kUnit<T> - 1) / kUnit<T> * kUnit<T>) * sizeof(double) : 0, s, a);
    else
        HY_LAUNCH(kernel_label("hyena_residual_norm", type_label<T>(), UNITS, WG, U, KIND == 1), (hyena_residual_norm<T, UNITS, WG, U, KIND == 1>),
                  dim3((unsigned)l.groups), dim3((unsigned)l.threads), 0, s, a);
    return launched();
}

template <typename T, bool UNITS, int KIND> hyena_status norm_sized(const NormArgs& a, const NormLaunch& l, hipStream_t s)
{
    if (l.workgroup) return norm_as<T, UNITS, true, kWideUnits<T>, KIND>(a, l, s);
    if (l.per == 1) return norm_as<T, UNITS, false, 1, KIND>(a, l, s);
    if (l.per == 2) return norm_as<T, UNITS, false, 2, KIND>(a, l, s);
    if (l.per == 3) return norm_as<T, UNITS, false, 3, KIND>(a, l, s);
    return norm_as<T, UNITS, false, 4, KIND>(a, l, s);
}

template <typename T> hyena_status norm_launch(const NormArgs& a, const NormLaunch& l, int kind, hipStream_t s)
{
    return by_units(l.units, [&](auto u) {
        constexpr bool UNITS = decltype(u)::value;
        if (kind == 0) return norm_sized<T, UNITS, 0>(a, l, s);
        return kind == 1 ? norm_sized<T, UNITS, 1>(a, l, s) : norm_sized<T, UNITS, 2>(a, l, s);
    });
}

}  // namespace hy

#define HY_NORM_INSTANTIATE(T)                                                                                       \
    namespace hy {                                                                                                  \
    template hyena_status norm_launch<T>(const NormArgs&, const NormLaunch&, int, hipStream_t);                      \
    }
