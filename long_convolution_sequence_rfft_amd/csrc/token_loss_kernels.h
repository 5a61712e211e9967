// token_loss_kernels.h -- softmax cross entropy over a vocabulary and its
// gradients (include/hyena.h).
//
//   hyena_loss_gather   the tokens that take part, their rows of x side by side
//   hyena_loss_pack     the table as a matrix operand, where it is not one as given
//   hyena_loss_logits   a tile of logits; forward: each token's largest and the sum
//                       of the exponentials over the tile's values; backward: G
//   hyena_loss_join     the tiles' sums joined: loss, lse
//   hyena_loss_products d_table of a piece of the vocabulary, and its share of d_x
//   hyena_loss_finish   d_x from its sums
// Bound by the matrix instructions: 2 tokens V d operations forward, 6 backward.
#pragma once

#include "matmul_device.h"
#include "token_loss.h"

namespace hy {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Storage types' matrix operands: float32 as three planes of bfloat16.
template <typename T> struct LossType {
    using E = T;
    static constexpr int P = 1;
};
template <> struct LossType<float> {
    using E = uint16_t;
    static constexpr int P = 3;
};

// Eight float32 values as P planes of E, by cutting (bfloat16, P = 3) or rounding.
template <typename E, int P> __device__ __forceinline__ void store_planes8(char* to, int64_t plane, f32x8 x)
{
    Split<E, P> s;
    s.set(x);
#pragma unroll
    for (int n = 0; n < P; ++n) *(typename Mx<E>::frag*)(to + n * plane) = s.f[n];
}

__device__ __forceinline__ int workgroup_sum16(int x, int* lds)
{
    for (int m = 1; m < 64; m *= 2) x += __shfl_xor(x, m);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    x = 0;
    for (int w = 0; w < 16; ++w) x += lds[w];
    __syncthreads();
    return x;
}

// Each workgroup counts the tokens that take part before its own, lists its own
// after them and gathers their rows of x.
template <typename T, bool VEC, bool GRAD> __global__ __launch_bounds__(1024) void hyena_loss_gather(LossArgs p)
{
    using E = typename LossType<T>::E;
    constexpr int P = LossType<T>::P;
    __shared__ int lds[16];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t first = (int64_t)blockIdx.x * p.each, last = first + p.each < p.total ? first + p.each : p.total;
    auto takes_part = [&](int64_t t) { return (uint32_t)*row_at<int32_t>(p.targets, t, p.targets_N) < (uint32_t)p.V; };
    int n = 0;
#pragma unroll 4
    for (int64_t t = threadIdx.x; t < first; t += 1024) n += takes_part(t);
    int64_t before = workgroup_sum16(n, lds);
    const int64_t begin = before;
    for (int64_t t0 = first; t0 < last; t0 += 1024) {
        const int64_t t = t0 + threadIdx.x;
        const int target = t < last ? *row_at<int32_t>(p.targets, t, p.targets_N) : -1;
        const bool in = (uint32_t)target < (uint32_t)p.V;
        const uint64_t all = __ballot(in);
        if (lane == 0) lds[wave] = __popcll(all);
        __syncthreads();
        int at = __popcll(all & (((uint64_t)1 << lane) - 1)), total = 0;
        for (int w = 0; w < 16; ++w) {
            if (w < wave) at += lds[w];
            total += lds[w];
        }
        __syncthreads();
        if (in) {
            p.index[before + at] = (int32_t)t;
            p.target[before + at] = target;
            if constexpr (GRAD) {
                p.weight[before + at] = *row_at<float>(p.d_loss, t, p.d_loss_N);
                p.lse2[before + at] = p.lse_in[t] * kLog2e;
            }
        }
        if (t < last) {
            if constexpr (GRAD) {
                p.place[t] = in ? (int32_t)(before + at) : -1;
            } else if (!in) {
                p.loss[t] = 0.0f;
                p.lse[t] = 0.0f;
            }
        }
        before += total;
    }
    __syncthreads();  // index is read back below
    // rows, a wave each, and after the last one zeros up to a whole step of 32
    int64_t end = before;
    if (blockIdx.x + 1 == gridDim.x) {
        if (threadIdx.x == 0) *p.count = before;
        end = (before + 31) / 32 * 32;
    }
    for (int64_t a = begin + wave; a < end; a += 16) {
        const T* x = a < before ? row_at<T>(p.x, p.index[a], p.x_N) : nullptr;
        char* to = p.rows + a * p.kd * 2;
        for (int c = lane * 8; c < p.kd; c += 512) {
            f32x8 v = {};
            if (x != nullptr && c < p.d) {
                float e[8];
                if constexpr (kUnit<T> == 8) {
                    load_unit<T, VEC>(x, c, p.d, p.pairs, e);
                } else {
                    float lo[kUnit<T>], hi[kUnit<T>];
                    load_unit<T, VEC>(x, c, p.d, p.pairs, lo);
#pragma unroll
                    for (int i = 0; i < 4; ++i) hi[i] = 0.0f;
                    if (c + 4 < p.d) load_unit<T, VEC>(x, c + 4, p.d, p.pairs, hi);
#pragma unroll
                    for (int i = 0; i < 4; ++i) e[i] = lo[i], e[4 + i] = hi[i];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = e[i];
            }
            store_planes8<E, P>(to + c * 2, p.rows_plane, v);
        }
    }
    if constexpr (GRAD) {
        // binary16 holds G over the power of two above the largest |d_loss|, times 2^15
        if (blockIdx.x == 0) {
            float up = 1.0f, down = 1.0f;
            if constexpr (Mx<E>::kTerms == 2) {
                uint32_t m = 0;
#pragma unroll 4
                for (int64_t t = threadIdx.x; t < p.total; t += 1024)
                    if (takes_part(t)) m = max(m, __float_as_uint(*row_at<float>(p.d_loss, t, p.d_loss_N)) & 0x7fffffffu);
                for (int k = 1; k < 64; k *= 2) m = max(m, (uint32_t)__shfl_xor((int)m, k));
                __syncthreads();
                if (lane == 0) lds[wave] = (int)m;
                __syncthreads();
                for (int w = 0; w < 16; ++w) m = max(m, (uint32_t)lds[w]);
                uint32_t e = m >> 23;  // the largest is below 2^(e - 126)
                e = e < 20 ? 20 : e > 250 ? 250 : e;
                up = __uint_as_float((268 - e) << 23);    // 2^(141 - e)
                down = __uint_as_float((e - 14) << 23);   // 2^(e - 141)
            }
            if (threadIdx.x == 0) {
                p.norm[0] = up;
                p.norm[1] = down * p.scale;
            }
        }
    }
}

// The table in rows of kd, as P planes.
template <typename T, bool VEC> __global__ __launch_bounds__(256) void hyena_loss_pack(LossArgs p)
{
    using E = typename LossType<T>::E;
    constexpr int P = LossType<T>::P;
    const int lane = threadIdx.x & 63;
    for (int64_t v = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); v < p.V; v += (int64_t)gridDim.x * 4) {
        const T* row = (const T*)p.table + v * p.d;
        char* to = const_cast<char*>(p.values) + v * p.values_row;
        for (int c = lane * 8; c < p.kd; c += 512) {
            f32x8 x = {};
#pragma unroll
            for (int h = 0; h < 8; h += kUnit<T>) {
                float e[kUnit<T>];
#pragma unroll
                for (int i = 0; i < kUnit<T>; ++i) e[i] = 0.0f;
                if (c + h < p.d) load_unit<T, VEC>(row, c + h, p.d, p.pairs, e);
#pragma unroll
                for (int i = 0; i < kUnit<T>; ++i) x[h + i] = e[i];
            }
            store_planes8<E, P>(to + c * 2, p.values_plane, x);
        }
    }
}

// Logits of kLossValues values (rows of the tile) and kLossTokens tokens (columns).
template <typename T, bool GRAD> __global__ __launch_bounds__(256, 2) void hyena_loss_logits(LossArgs p)
{
    using E = typename LossType<T>::E;
    constexpr int P = LossType<T>::P;
    using Tile = MatTile<E, kLossValues, kLossTokens, 2, 2, true, true, P>;
    __shared__ __attribute__((aligned(16))) char lds[Tile::kLds];
    const int64_t count = *p.count;
    const int64_t t0 = (int64_t)blockIdx.y * kLossTokens;
    if (t0 >= count) return;
    const int32_t v0 = p.first + (int32_t)blockIdx.x * kLossValues;
    Tile tile;
    const Operand values{p.values + (int64_t)v0 * p.values_row, p.values + (int64_t)p.V * p.values_row, p.values_row};
    const Operand rows{p.rows + t0 * p.kd * 2, p.rows + p.tokens * p.kd * 2, (int64_t)p.kd * 2};
    tile.run(lds, values, p.values_plane, rows, p.rows_plane, p.kd / 32);

    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4;
    const int wm = wave / 2, wn = wave % 2;
    const float scale2 = p.scale * kLog2e;
    const bool whole = v0 + kLossValues <= p.V;
    if constexpr (!GRAD) {
        __shared__ float2 halves[2][kLossTokens];
#pragma unroll
        for (int j = 0; j < Tile::NI; ++j) {
            const int n = wn * (kLossTokens / 2) + 16 * j + (lane & 15);
            const int64_t t = t0 + n;
            const int target = t < count ? p.target[t] - v0 : -1;
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < Tile::MI; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int v = wm * (kLossValues / 2) + 16 * i + 4 * g + r;
                    float l = tile.c[i][j][r] * scale2;
                    if (!whole && v0 + v >= p.V) l = -INFINITY;
                    if (v == target) p.hit[t] = l;
                    tile.c[i][j][r] = l;
                    m = fmaxf(m, l);
                }
            m = fmaxf(m, __shfl_xor(m, 16));
            m = fmaxf(m, __shfl_xor(m, 32));
            const float base = m == -INFINITY ? 0.0f : m;  // (no value of the tile's half is in the vocabulary)
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < Tile::MI; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) s += __builtin_amdgcn_exp2f(tile.c[i][j][r] - base);
            s += __shfl_xor(s, 16);
            s += __shfl_xor(s, 32);
            if (g == 0) halves[wm][n] = make_float2(m, s);
        }
        __syncthreads();
        if (threadIdx.x < kLossTokens) {
            const float2 a = halves[0][threadIdx.x], b = halves[1][threadIdx.x];
            const float m = fmaxf(a.x, b.x);
            // (the first half always has a value)
            const float s = a.y * __builtin_amdgcn_exp2f(a.x - m) + b.y * __builtin_amdgcn_exp2f(b.x - m);
            p.part[(int64_t)blockIdx.x * p.tokens + t0 + threadIdx.x] = make_float2(m, s);
        }
    } else {
        const float up = p.norm[0];
#pragma unroll
        for (int j = 0; j < Tile::NI; ++j) {
            const int n = wn * (kLossTokens / 2) + 16 * j + (lane & 15);
            const int64_t t = t0 + n;
            const bool in = t < count;
            const int target = in ? p.target[t] - v0 : -1;
            const float lse2 = in ? p.lse2[t] : 0.0f, weight = in ? p.weight[t] * up : 0.0f;
            char* to = p.g + t * p.g_row + ((int64_t)blockIdx.x * kLossValues) * 2;
#pragma unroll
            for (int i = 0; i < Tile::MI; ++i) {
                const int v = wm * (kLossValues / 2) + 16 * i + 4 * g;
                f32x4 x;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float q = __builtin_amdgcn_exp2f(fmaf(tile.c[i][j][r], scale2, -lse2));
                    if (v + r == target) q -= 1.0f;
                    q *= weight;
                    if (!in || (!whole && v0 + v + r >= p.V)) q = 0.0f;
                    x[r] = q;
                }
                if constexpr (P == 1) {
                    *(typename Mx<E>::vec4*)(to + v * 2) = Mx<E>::narrow(x);
                } else {
#pragma unroll
                    for (int k = 0; k < P; ++k) {
                        const typename Mx<E>::vec4 y = Mx<E>::narrow(x);
                        *(typename Mx<E>::vec4*)(to + v * 2 + k * p.g_plane) = y;
                        x -= Mx<E>::widen(y);
                    }
                }
            }
        }
    }
}

// Loss and lse of 16 tokens: 16 threads each go through the tiles' sums.
template <int kUnused> __global__ __launch_bounds__(256) void hyena_loss_join(LossArgs p, int tiles)
{
    __shared__ float2 lds[16][17];
    const int64_t count = *p.count, a = (int64_t)blockIdx.x * 16 + (threadIdx.x & 15);
    const int k = threadIdx.x >> 4;
    if ((int64_t)blockIdx.x * 16 >= count) return;
    float m = -INFINITY, s = 0.0f;
#pragma unroll 4
    for (int i = k; i < tiles; i += 16) {
        const float2 x = p.part[(int64_t)i * p.tokens + a];
        const float top = fmaxf(m, x.x);
        s = s * __builtin_amdgcn_exp2f(m - top) + x.y * __builtin_amdgcn_exp2f(x.x - top);
        m = top;
    }
    lds[k][threadIdx.x & 15] = make_float2(m, s);
    __syncthreads();
    if (k == 0 && a < count) {
        for (int i = 1; i < 16; ++i) {
            const float2 x = lds[i][threadIdx.x];
            if (x.x == -INFINITY) continue;  // fewer tiles than threads
            const float top = fmaxf(m, x.x);
            s = s * __builtin_amdgcn_exp2f(m - top) + x.y * __builtin_amdgcn_exp2f(x.x - top);
            m = top;
        }
        const float log2s = __builtin_amdgcn_logf(s);
        const int32_t t = p.index[a];
        p.lse[t] = (m + log2s) * kLn2;
        p.loss[t] = ((m - p.hit[a]) + log2s) * kLn2;
    }
}

// The first `tiles` workgroups: d_table of kGradRows values of this piece and
// kGradChannels channels.  The others: a share of d_x of kGradRows tokens, the sum
// over one of p.splits parts of the piece's values.
template <typename T> __global__ __launch_bounds__(256, 2) void hyena_loss_products(LossArgs p, int table_tiles, int channel_tiles)
{
    using E = typename LossType<T>::E;
    constexpr int P = LossType<T>::P;
    using Table = MatTile<E, kGradChannels, kGradRows, 2, 2, false, false, P>;
    using Dx = MatTile<E, kGradChannels, kGradRows, 2, 2, false, true, P>;
    __shared__ __attribute__((aligned(16))) char lds[Table::kLds];
    const int64_t count = *p.count;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4;
    const int wm = wave / 2, wn = wave % 2;
    const int32_t values = p.V - p.first < p.chunk ? p.V - p.first : p.chunk;  // of this piece
    if ((int)blockIdx.x < table_tiles) {
        const int c0 = (int)blockIdx.x % channel_tiles * kGradChannels;
        const int32_t v0 = (int)blockIdx.x / channel_tiles * kGradRows;
        Table tile;
        const Operand x{p.rows + c0 * 2, p.rows + p.tokens * p.kd * 2, (int64_t)p.kd * 2};
        const Operand y{p.g + (int64_t)v0 * 2, p.g + p.tokens * p.g_row, p.g_row};
        if (count > 0) {
            tile.run(lds, x, p.rows_plane, y, p.g_plane, (int)((count + 31) / 32));
        } else {
#pragma unroll
            for (int i = 0; i < Table::MI; ++i)
#pragma unroll
                for (int j = 0; j < Table::NI; ++j) tile.c[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        const float down = p.norm[1];
#pragma unroll
        for (int j = 0; j < Table::NI; ++j) {
            const int32_t v = v0 + wn * (kGradRows / 2) + 16 * j + (lane & 15);
            if (v >= values) continue;
            T* to = (T*)p.d_table + (int64_t)(p.first + v) * p.d;
#pragma unroll
            for (int i = 0; i < Table::MI; ++i) {
                const int c = c0 + wm * (kGradChannels / 2) + 16 * i + 4 * g;
                const f32x4 r = tile.c[i][j] * down;
                if (p.d % 4 == 0) {
                    if (c < p.d) *(typename Mx<T>::vec4*)(to + c) = Mx<T>::narrow(r);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (c + e < p.d) store_one<T>(to + c + e, r[e]);
                }
            }
        }
        return;
    }
    int64_t b = (int64_t)blockIdx.x - table_tiles;
    const int c0 = (int)(b % channel_tiles) * kGradChannels;
    b /= channel_tiles;
    const int split = (int)(b % p.splits);
    const int64_t t0 = b / p.splits * kGradRows;
    if (t0 >= count) return;
    // this part's values, whole steps of 32
    const int steps = (values + 31) / 32, per = (steps + p.splits - 1) / p.splits;
    const int k0 = split * per, k1 = k0 + per < steps ? k0 + per : steps;
    if (k0 >= k1 && p.first != 0) return;
    Dx tile;
    if (k0 < k1) {
        const Operand x{p.values + (int64_t)(p.first + 32 * k0) * p.values_row + c0 * 2, p.values + (int64_t)p.V * p.values_row, p.values_row};
        const Operand y{p.g + t0 * p.g_row + k0 * 64, p.g + p.tokens * p.g_row, p.g_row};
        tile.run(lds, x, p.values_plane, y, p.g_plane, k1 - k0);
    } else {
#pragma unroll
        for (int i = 0; i < Dx::MI; ++i)
#pragma unroll
            for (int j = 0; j < Dx::NI; ++j) tile.c[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll
    for (int j = 0; j < Dx::NI; ++j) {
        const int64_t t = t0 + wn * (kGradRows / 2) + 16 * j + (lane & 15);
        float* to = p.acc + ((int64_t)split * p.tokens + t) * p.acc_row;
#pragma unroll
        for (int i = 0; i < Dx::MI; ++i) {
            const int c = c0 + wm * (kGradChannels / 2) + 16 * i + 4 * g;
            if (c >= p.acc_row) continue;
            f32x4 r = tile.c[i][j];
            if (p.first != 0) r += *(const f32x4*)(to + c);
            *(f32x4*)(to + c) = r;
        }
    }
}

template <typename T, bool VEC> __global__ __launch_bounds__(256) void hyena_loss_finish(LossArgs p)
{
    constexpr int K = kUnit<T>;
    const int lane = threadIdx.x & 63;
    const float down = p.norm[1];
    for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < p.total; t += (int64_t)gridDim.x * 4) {
        const int32_t a = p.place[t];
        T* to = (T*)p.d_x + t * p.d;
        for (int c = lane * K; c < p.d; c += 64 * K) {
            float x[K];
#pragma unroll
            for (int i = 0; i < K; ++i) x[i] = 0.0f;
            if (a >= 0) {
                for (int s = 0; s < p.splits; ++s) {
                    const float* from = p.acc + ((int64_t)s * p.tokens + a) * p.acc_row + c;
#pragma unroll
                    for (int i = 0; i < K; i += 4) {
                        if (c + i >= p.acc_row) break;
                        const f32x4 y = *(const f32x4*)(from + i);
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[i + e] += y[e];
                    }
                }
#pragma unroll
                for (int i = 0; i < K; ++i) x[i] *= down;
            }
            store_unit<T, VEC>(to, c, p.d, p.d % 2 == 0, x);
        }
    }
}

template <typename T, bool GRAD> hyena_status loss_begin(const LossArgs& a, bool pack, bool units, hipStream_t s)
{
    hyena_status st;
    const dim3 grid((unsigned)((a.total + a.each - 1) / a.each));
    if (units)
        HY_LAUNCH(kernel_label("hyena_loss_gather", type_label<T>(), true, GRAD), (hyena_loss_gather<T, true, GRAD>), grid, dim3(1024), 0, s, a);
    else
        HY_LAUNCH(kernel_label("hyena_loss_gather", type_label<T>(), false, GRAD), (hyena_loss_gather<T, false, GRAD>), grid, dim3(1024), 0, s, a);
    if ((st = launched()) != HYENA_OK || !pack) return st;
    LossArgs b = a;
    b.pairs = a.d % 2 == 0;
    const int64_t need = ((int64_t)a.V + 3) / 4;
    const dim3 pgrid((unsigned)(need < 4096 ? need : 4096));
    if (a.d % kUnit<T> == 0)
        HY_LAUNCH(kernel_label("hyena_loss_pack", type_label<T>(), true), (hyena_loss_pack<T, true>), pgrid, dim3(256), 0, s, b);
    else
        HY_LAUNCH(kernel_label("hyena_loss_pack", type_label<T>(), false), (hyena_loss_pack<T, false>), pgrid, dim3(256), 0, s, b);
    return launched();
}

template <typename T> hyena_status loss_forward(const LossArgs& a, bool pack, bool units, hipStream_t s)
{
    hyena_status st = loss_begin<T, false>(a, pack, units, s);
    if (st != HYENA_OK) return st;
    const int tiles = (a.V + kLossValues - 1) / kLossValues;
    HY_LAUNCH(kernel_label("hyena_loss_logits", type_label<T>(), false), (hyena_loss_logits<T, false>),
              dim3((unsigned)tiles, (unsigned)(a.tokens / kLossTokens)), dim3(256), 0, s, a);
    if ((st = launched()) != HYENA_OK) return st;
    HY_LAUNCH(kernel_label("hyena_loss_join", 0), hyena_loss_join<0>, dim3((unsigned)((a.total + 15) / 16)), dim3(256), 0, s, a, tiles);
    return launched();
}

template <typename T> hyena_status loss_backward(const LossArgs& a, bool pack, bool units, hipStream_t s)
{
    hyena_status st = loss_begin<T, true>(a, pack, units, s);
    if (st != HYENA_OK) return st;
    LossArgs b = a;
    const int channel_tiles = (a.d + kGradChannels - 1) / kGradChannels;
    for (int64_t first = 0; first < a.V; first += a.chunk) {
        b.first = (int32_t)first;
        const int values = a.V - first < a.chunk ? (int)(a.V - first) : a.chunk;
        const dim3 grid((unsigned)((values + kLossValues - 1) / kLossValues), (unsigned)(a.tokens / kLossTokens));
        HY_LAUNCH(kernel_label("hyena_loss_logits", type_label<T>(), true), (hyena_loss_logits<T, true>), grid, dim3(256), 0, s, b);
        if ((st = launched()) != HYENA_OK) return st;
        const int table_tiles = a.d_table ? channel_tiles * ((values + kGradRows - 1) / kGradRows) : 0;
        const int64_t dx_tiles = a.d_x ? (int64_t)channel_tiles * a.splits * (a.tokens / kGradRows) : 0;
        HY_LAUNCH(kernel_label("hyena_loss_products", type_label<T>()), hyena_loss_products<T>, dim3((unsigned)(table_tiles + dx_tiles)),
                  dim3(256), 0, s, b, table_tiles, channel_tiles);
        if ((st = launched()) != HYENA_OK) return st;
    }
    if (a.d_x == nullptr) return HYENA_OK;
    const int64_t need = (a.total + 3) / 4;
    const dim3 grid((unsigned)(need < 4096 ? need : 4096));
    if (a.d % kUnit<T> == 0)
        HY_LAUNCH(kernel_label("hyena_loss_finish", type_label<T>(), true), (hyena_loss_finish<T, true>), grid, dim3(256), 0, s, a);
    else
        HY_LAUNCH(kernel_label("hyena_loss_finish", type_label<T>(), false), (hyena_loss_finish<T, false>), grid, dim3(256), 0, s, a);
    return launched();
}

}  // namespace hy

#define HY_LOSS_INSTANTIATE(T)                                                                  \
    namespace hy {                                                                             \
    template hyena_status loss_forward<T>(const LossArgs&, bool, bool, hipStream_t);            \
    template hyena_status loss_backward<T>(const LossArgs&, bool, bool, hipStream_t);           \
    }
