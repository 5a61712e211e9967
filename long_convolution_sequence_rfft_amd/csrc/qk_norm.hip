// qk_norm.hip -- norms of queries and keys per head with the position rotation
// in the same pass, and their backward pass (include/hyena.h).
//
// With r = 1 / sqrt(mean(x^2) + eps) (L2: the sum) a head's x becomes
//   y = turn(w r x),
// and its gradient, with d = w turn^T(dy) and z = r x,
//   dx = r (d - z mean(d z)),   dw = sum over tokens and heads of turn^T(dy) z.
//
// Bound by memory: each channel is read and written once (the backward pass
// reads two tensors).  What is shared by all heads of a token, the sines and
// cosines and the token's place, is computed once per tile and kept in LDS;
// everything else of a head stays in the registers of the few lanes that hold
// it.  A workgroup serves one of the two tensors: with both, the kernel held
// two sets of weights and of their sums, 165 instead of 131 registers, and the
// two heads' worth of a decoding token came one after the other (8.0 us
// instead of 6.5).
//
// A head is cut into units of 2 W channels, two vectors of W: W pairs of the
// rotation (in the half layout the vectors are rotary_dim / 2 apart, else side
// by side) or 2 W channels that are not rotated.  A lane holds U units, a power
// of two of lanes one head, so a pair is always within a lane and the norm's
// sum is a few steps across lanes.  W is as wide as the widths and strides allow
// (2 x 8192 tokens, 12 + 12 heads of 100 in bf16: 93 us forward with W = 1, 56
// with 2, where heads of 128 take 38 with 8).
//
// Tiles of 48 KB: the backward pass at 16384 tokens of 12 + 4 heads of 64 in
// bf16 takes 26.7 us (100 MB, 4.4 TB/s less 4 us of launch), with 32 KB 31,
// with 64 KB 30 (fewer workgroups than the card holds); at 8192 tokens of
// 12 + 12 heads in float32 35.6 us (151 MB) against 39.6 and 40.0.  Forward at
// 16384 tokens of 12 + 12 heads, bf16: 24.6 us (101 MB).
#include <hip/hip_runtime.h>

#include <string>
#include <type_traits>

#include "recurrence_device.h"
#include "recurrence_plan.h"
#include "plan.h"
#include "timing.h"

namespace hy {

namespace {

constexpr int kQkThreads = 256;
constexpr int kQkTokens = 64;      // most tokens of a workgroup's tile
constexpr int kQkTile = 48 << 10;  // bytes of a tensor that a tile is meant to hold
constexpr int kQkAngles = 2048;    // most (token, frequency) pairs of a tile: 16 KB of LDS
constexpr int kQkTiles = 256;      // fewest tiles of a tensor, if it has that many tokens
constexpr int kQkGroups = 1 << 16; // most workgroups of a tensor, forward: the rest of the tiles is looped over
constexpr int kQkGradGroups = 1024;    // backward: what runs at once, the most rows of the partial sums
constexpr int kQkGradGroupsWide = 768; // the same where a lane holds 16 channels (W = 8)

struct QkTensor {
    RView x, dy;
    void* out;
    const float* w;
    float* dw_part;     // [groups][D]
    int32_t heads;
    uint32_t magic;     // ceil(2^32 / heads), heads > 1: item / heads = item * magic >> 32, item < 2^16
    int32_t tokens;     // per tile
    int32_t groups;     // workgroups
    int64_t tiles;
};

struct QkArgs {
    QkTensor t[2];
    const double* freqs;
    const int32_t* positions;
    int64_t offset;
    int64_t N, rows;    // rows: B * N
    int32_t D, rotary;
    int32_t half, norm;
    int32_t lanes;      // per head, a power of two
    float mean;         // 1 / m
    float eps, rscale;
};

// W channels as loaded, and widened.
template <typename T, int W> struct QkRaw {
    typename Mx<T>::vec4 v[W / 4];
    __device__ __forceinline__ void load(const T* p)
    {
        if constexpr (W == 8) *(uint4*)v = *(const uint4*)p;
        else v[0] = *(const typename Mx<T>::vec4*)p;
    }
    __device__ __forceinline__ void widen(float (&x)[W]) const
    {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            const f32x4 f = Mx<T>::widen(v[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[4 * i + j] = f[j];
        }
    }
};
template <typename T> struct QkRaw<T, 2> {
    typedef T pair __attribute__((ext_vector_type(2)));
    pair v;
    __device__ __forceinline__ void load(const T* p) { v = *(const pair*)p; }
    __device__ __forceinline__ void widen(float (&x)[2]) const
    {
        const T a = v[0], b = v[1];
        x[0] = load_one<T>(&a);
        x[1] = load_one<T>(&b);
    }
};
template <typename T> struct QkRaw<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T* p) { v = *p; }
    __device__ __forceinline__ void widen(float (&x)[1]) const { x[0] = load_one<T>(&v); }
};

template <typename T, int W>
__device__ __forceinline__ void qk_store(T* p, const float (&x)[W])
{
    if constexpr (W == 1) {
        store_one<T>(p, x[0]);
    } else if constexpr (W == 2) {
        T a, b;
        store_one<T>(&a, x[0]);
        store_one<T>(&b, x[1]);
        *(typename QkRaw<T, 2>::pair*)p = typename QkRaw<T, 2>::pair{a, b};
    } else {
        typename Mx<T>::vec4 v[W / 4];
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            f32x4 f;
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = x[4 * i + j];
            v[i] = Mx<T>::narrow(f);
        }
        if constexpr (W == 8) *(uint4*)p = *(const uint4*)v;
        else *(typename Mx<T>::vec4*)p = v[0];
    }
}

// Sine and cosine of position * frequency.  The angle in float64 is reduced by
// pi / 2 in two parts (error below 2^-52 of the angle plus 2e-16 at 2^31 turns),
// so far positions keep float32 accuracy.  What is left is within pi / 4, where
// Taylor's series end: the terms left out are below 2e-9 of the sum.
__device__ __forceinline__ float2 qk_turn(int64_t pos, double freq, float scale)
{
    const double a = (double)pos * freq;
    const double n = rint(a * 0.63661977236758134308);
    double r = fma(-n, 1.5707963267948965580, a);
    r = fma(-n, 6.123233995736766036e-17, r);
    const float x = (float)r, z = x * x;
    float s = fmaf(z, 1.0f / 362880, -1.0f / 5040), c = fmaf(z, -1.0f / 3628800, 1.0f / 40320);
    s = fmaf(z, s, 1.0f / 120);
    c = fmaf(z, c, -1.0f / 720);
    s = fmaf(z, s, -1.0f / 6);
    c = fmaf(z, c, 1.0f / 24);
    s = fmaf(z * x, s, x);
    c = fmaf(z, c, -0.5f);
    c = fmaf(z, c, 1.0f);
    const int turn = (int)(int64_t)n & 3;  // quarter turns
    const float u = turn & 1 ? s : c, v = turn & 1 ? c : s;
    const float co = turn == 1 || turn == 2 ? -u : u, si = turn & 2 ? -v : v;
    return make_float2(co * scale, si * scale);
}

// y = turn(x) for GRAD = false, its transpose for GRAD = true; a pair's members
// are (x0[e], x1[e]) in the half layout, neighbours otherwise.
template <int W, bool GRAD>
__device__ __forceinline__ void qk_rotate(float (&x0)[W], float (&x1)[W], const float2* turn, bool half)
{
    auto one = [](float& a, float& b, float2 t) {
        const float s = GRAD ? -t.y : t.y;
        const float u = a * t.x - b * s;
        b = a * s + b * t.x;
        a = u;
    };
    if (half || W == 1) {
#pragma unroll
        for (int e = 0; e < W; ++e) one(x0[e], x1[e], turn[e]);
    } else {
#pragma unroll
        for (int e = 0; e < W / 2; ++e) {
            one(x0[2 * e], x0[2 * e + 1], turn[e]);
            one(x1[2 * e], x1[2 * e + 1], turn[W / 2 + e]);
        }
    }
}

// Sum over a group of `lanes` (a power of two) lanes, in each of them.
__device__ __forceinline__ float sum_lanes(float x, int lanes)
{
    if (lanes > 1) x += dpp_f32<0xb1>(x);   // the steps of sum16
    if (lanes > 2) x += dpp_f32<0x4e>(x);
    if (lanes > 4) x += dpp_f32<0x141>(x);
    if (lanes > 8) x += dpp_f32<0x140>(x);
    if (lanes > 16) x += __shfl_xor(x, 16);
    if (lanes > 32) x += __shfl_xor(x, 32);
    return x;
}

template <typename T, int W, int U, bool GRAD>
__global__ __launch_bounds__(kQkThreads, U == 1 ? 3 : 2) void hyena_qk_norm_pass(QkArgs p)
{
    __shared__ float2 turns[kQkAngles];
    __shared__ int64_t at[GRAD ? 2 : 1][kQkTokens];  // elements to each token of the tile, in x and dy
    __shared__ float sums[GRAD ? kQkThreads * 2 * W : 1];
    const bool second = (int)blockIdx.x >= p.t[0].groups;
    const QkTensor q = second ? p.t[1] : p.t[0];
    const int mine = (int)blockIdx.x - (second ? p.t[0].groups : 0);
    const int tid = threadIdx.x;
    const int lane = tid & (p.lanes - 1), group = tid / p.lanes, groups = kQkThreads / p.lanes;
    const int units = (p.D + 2 * W - 1) / (2 * W), turned = p.rotary / (2 * W), nf = p.rotary / 2;

    // the lane's units: places of their two vectors
    int c0[U], c1[U];
    bool in0[U], in1[U], rot[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int n = lane + u * p.lanes;
        rot[u] = n < turned;
        const bool apart = rot[u] && p.half;
        c0[u] = apart ? n * W : 2 * n * W;
        c1[u] = apart ? nf + n * W : 2 * n * W + W;
        in0[u] = n < units;
        in1[u] = n < units && c1[u] < p.D;
    }
    float w[U][2][W], dw[GRAD ? U : 1][2][W];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < W; ++e) {
            w[u][0][e] = q.w && in0[u] ? q.w[c0[u] + e] : 1.0f;
            w[u][1][e] = q.w && in1[u] ? q.w[c1[u] + e] : 1.0f;
            if constexpr (GRAD) dw[u][0][e] = dw[u][1][e] = 0.0f;
        }

    for (int64_t tile = mine; tile < q.tiles; tile += q.groups) {
        const int64_t row0 = tile * q.tokens;
        const int ntok = p.rows - row0 < q.tokens ? (int)(p.rows - row0) : q.tokens;
        if (tile != mine) __syncthreads();
        if (tid < ntok) {
            const uint64_t row = (uint64_t)(row0 + tid);
            const int64_t b = (int64_t)(row / (uint64_t)p.N), t = (int64_t)(row - (uint64_t)b * (uint64_t)p.N);
            at[0][tid] = b * q.x.b + t * q.x.t;
            if constexpr (GRAD) at[1][tid] = b * q.dy.b + t * q.dy.t;
        }
        for (int i = tid; i < ntok * nf; i += kQkThreads) {
            const uint64_t row = (uint64_t)(row0 + i / nf);
            const int64_t pos = p.positions ? (int64_t)p.positions[row] : p.offset + (int64_t)(row % (uint64_t)p.N);
            turns[i] = qk_turn(pos, p.freqs[i % nf], p.rscale);
        }
        __syncthreads();
        const int items = ntok * q.heads;
        for (int item = group; item < items; item += groups) {
            QkRaw<T, W> rx[U][2], rd[GRAD ? U : 1][2];
            const int tok = q.heads == 1 ? item : (int)__umulhi((uint32_t)item, q.magic), head = item - tok * q.heads;
            const T* xp = (const T*)q.x.p + at[0][tok] + head * q.x.h;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (in0[u]) rx[u][0].load(xp + c0[u]);
                if (in1[u]) rx[u][1].load(xp + c1[u]);
            }
            if constexpr (GRAD) {
                const T* dp = (const T*)q.dy.p + at[1][tok] + head * q.dy.h;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (in0[u]) rd[u][0].load(dp + c0[u]);
                    if (in1[u]) rd[u][1].load(dp + c1[u]);
                }
            }
            T* op = (T*)q.out + (row0 * q.heads + item) * p.D;
            float x[U][2][W], d[U][2][W];
            float ss = 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int e = 0; e < W; ++e) x[u][0][e] = x[u][1][e] = d[u][0][e] = d[u][1][e] = 0.0f;
                if (in0[u]) rx[u][0].widen(x[u][0]);
                if (in1[u]) rx[u][1].widen(x[u][1]);
                if constexpr (GRAD) {
                    if (in0[u]) rd[u][0].widen(d[u][0]);
                    if (in1[u]) rd[u][1].widen(d[u][1]);
                }
            }
            float r = 1.0f;
            if (p.norm) {
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int e = 0; e < W; ++e) ss += x[u][0][e] * x[u][0][e] + x[u][1][e] * x[u][1][e];
                ss = sum_lanes(ss, p.lanes);
                r = 1.0f / sqrtf(ss * p.mean + p.eps);
            }
            const float2* turn = turns + tok * nf;
            if constexpr (!GRAD) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (p.norm) {
#pragma unroll
                        for (int e = 0; e < W; ++e) {
                            x[u][0][e] *= r * w[u][0][e];
                            x[u][1][e] *= r * w[u][1][e];
                        }
                    }
                    if (rot[u]) qk_rotate<W, false>(x[u][0], x[u][1], turn + (lane + u * p.lanes) * W, p.half);
                    if (in0[u]) qk_store<T, W>(op + c0[u], x[u][0]);
                    if (in1[u]) qk_store<T, W>(op + c1[u], x[u][1]);
                }
            } else {
                float along = 0.0f;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (rot[u]) qk_rotate<W, true>(d[u][0], d[u][1], turn + (lane + u * p.lanes) * W, p.half);
                    if (p.norm) {
#pragma unroll
                        for (int v = 0; v < 2; ++v)
#pragma unroll
                            for (int e = 0; e < W; ++e) {
                                x[u][v][e] *= r;
                                dw[u][v][e] += d[u][v][e] * x[u][v][e];
                                d[u][v][e] *= w[u][v][e];
                                along += d[u][v][e] * x[u][v][e];
                            }
                    }
                }
                if (p.norm) along = sum_lanes(along, p.lanes) * p.mean;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (p.norm) {
#pragma unroll
                        for (int v = 0; v < 2; ++v)
#pragma unroll
                            for (int e = 0; e < W; ++e) d[u][v][e] = (d[u][v][e] - x[u][v][e] * along) * r;
                    }
                    if (in0[u]) qk_store<T, W>(op + c0[u], d[u][0]);
                    if (in1[u]) qk_store<T, W>(op + c1[u], d[u][1]);
                }
            }
        }
    }
    if constexpr (GRAD) {
        // the workgroup's sums for the weights, over its groups in order
        if (q.dw_part == nullptr) return;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < W; ++e) {
                sums[(e * 2) * kQkThreads + tid] = dw[u][0][e];
                sums[(e * 2 + 1) * kQkThreads + tid] = dw[u][1][e];
            }
            __syncthreads();
            for (int i = tid; i < p.lanes * 2 * W; i += kQkThreads) {
                const int l = i / (2 * W), ev = i % (2 * W), e = ev / 2, v = ev % 2;
                const int n = l + u * p.lanes;
                const bool apart = n < turned && p.half;
                const int c = (v ? (apart ? nf + n * W : 2 * n * W + W) : (apart ? n * W : 2 * n * W)) + e;
                if (n < units && c < p.D) {
                    float s = 0.0f;
                    for (int g = 0; g < groups; ++g) s += sums[ev * kQkThreads + g * p.lanes + l];
                    q.dw_part[(int64_t)mine * p.D + c] = s;
                }
            }
        }
    }
}

// dw[c] = sum over the workgroups' rows, 16 channels by 64 rows at a time: what
// takes time here is one load after the other.
__global__ __launch_bounds__(1024) void hyena_qk_weight_grad(const float* part0, const float* part1, float* out0,
                                                            float* out1, int groups0, int groups1, int D)
{
    __shared__ double sums[1024];
    const float* part = blockIdx.y ? part1 : part0;
    float* out = blockIdx.y ? out1 : out0;
    const int groups = blockIdx.y ? groups1 : groups0;
    if (out == nullptr) return;
    const int c = blockIdx.x * 16 + (threadIdx.x & 15), r = threadIdx.x >> 4;
    double s = 0.0;
    if (c < D) {
#pragma unroll 8
        for (int g = r; g < groups; g += 64) s += (double)part[(int64_t)g * D + c];
    }
    sums[threadIdx.x] = s;
    __syncthreads();
    if (r == 0 && c < D) {
        double x = 0.0;
        for (int i = 0; i < 64; ++i) x += sums[i * 16 + threadIdx.x];
        out[c] = (float)x;
    }
}

bool all_zero_mod(const RView& v, size_t element, int w)
{
    return (uintptr_t)v.p % (element * w) == 0 && v.b % w == 0 && v.t % w == 0 && v.h % w == 0;
}

// Largest W whose vectors stay whole and aligned: the width in groups of W
// channels, the rotated part in units of 2 W.
int vector_width(const QkArgs& a, size_t element, bool grad)
{
    for (int w = element == 2 ? 8 : 4; w >= 2; w /= 2) {
        bool ok = a.D % w == 0 && a.rotary % (2 * w) == 0;
        for (int k = 0; k < 2 && ok; ++k)
            ok = all_zero_mod(a.t[k].x, element, w) && (!grad || all_zero_mod(a.t[k].dy, element, w)) &&
                 (uintptr_t)a.t[k].out % (element * w) == 0;
        if (ok) return w;
    }
    return 1;
}

// The tensors' tiles and workgroups.  Tiles of kQkTile bytes, or less so that
// there are kQkTiles of them, and a workgroup for each.  Backward, where a
// workgroup keeps sums for the weights, no more workgroups than run at once: if
// there are more tiles, they are shared out by heads, and the tiles made smaller
// so that each workgroup of a tensor has as many (2 x 8192 tokens, 12 + 12 heads
// of 64, 128 and 256 in bf16, a workgroup per tile up to 1024 of them: 41, 106
// and 171 us, so: 40, 92 and 141).
void shape_tiles(QkArgs& a, size_t element, bool grad)
{
    const int64_t nf = a.rotary / 2 > 0 ? a.rotary / 2 : 1, heads = a.t[0].heads + a.t[1].heads;
    const bool wide = element == 2 && a.D % 8 == 0 && a.rotary % 16 == 0;
    const int64_t resident = wide ? kQkGradGroupsWide : kQkGradGroups;
    int64_t most[2], total = 0;
    for (int k = 0; k < 2; ++k) {
        int64_t t = kQkTile / ((int64_t)a.t[k].heads * a.D * (int64_t)element);
        if (t > kQkTokens) t = kQkTokens;
        if (t > kQkAngles / nf) t = kQkAngles / nf;
        if (t > a.rows / kQkTiles) t = a.rows / kQkTiles;
        most[k] = t < 1 ? 1 : t;
        total += (a.rows + most[k] - 1) / most[k];
    }
    for (int k = 0; k < 2; ++k) {
        QkTensor& q = a.t[k];
        int64_t t = most[k], groups = kQkGroups;
        if (grad && total > resident) {
            groups = resident * (int64_t)q.heads / heads;
            if (groups < 1) groups = 1;
            const int64_t each = (a.rows + groups * t - 1) / (groups * t);
            t = (a.rows + groups * each - 1) / (groups * each);
        }
        q.tokens = (int32_t)t;
        q.tiles = (a.rows + t - 1) / t;
        q.groups = (int32_t)(q.tiles < groups ? q.tiles : groups);
    }
}

template <typename T, int W, int U, bool GRAD>
hyena_status qk_launch_one(const QkArgs& a, hipStream_t s)
{
    HY_LAUNCH(kernel_label("hyena_qk_norm_pass", type_label<T>(), W, U, GRAD), (hyena_qk_norm_pass<T, W, U, GRAD>),
              dim3((unsigned)(a.t[0].groups + a.t[1].groups)), dim3(kQkThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? HYENA_OK : fail(HYENA_ERR_DEVICE, hipGetErrorString(e));
}

template <typename T, int W, bool GRAD> hyena_status qk_launch_w(QkArgs& a, hipStream_t s)
{
    // lanes per head: a power of two, at most a wave; more units go to a lane
    const int units = (a.D + 2 * W - 1) / (2 * W);
    int lanes = 1;
    while (lanes < units && lanes < 64) lanes *= 2;
    a.lanes = lanes;
    const int per = (units + lanes - 1) / lanes;
    constexpr int most = 1024 / (2 * W * 64);  // of the widest heads: 1, 2, 4, 8
    if (per <= 1) return qk_launch_one<T, W, 1, GRAD>(a, s);
    if constexpr (most > 2)
        if (per <= 2) return qk_launch_one<T, W, 2, GRAD>(a, s);
    return qk_launch_one<T, W, most, GRAD>(a, s);
}

template <typename T, bool GRAD> hyena_status qk_launch(QkArgs& a, hipStream_t s)
{
    const int w = vector_width(a, sizeof(T), GRAD);
    if constexpr (sizeof(T) == 2)
        if (w == 8) return qk_launch_w<T, 8, GRAD>(a, s);
    if (w == 4) return qk_launch_w<T, 4, GRAD>(a, s);
    if (w == 2) return qk_launch_w<T, 2, GRAD>(a, s);
    return qk_launch_w<T, 1, GRAD>(a, s);
}

hyena_status qk_refuse(const char* what) { return fail(HYENA_ERR_INVALID_ARGUMENT, std::string("qk norm: ") + what); }

RView plain_view(const hyena_view& v) { return RView{v.data, v.batch, v.token, v.head, 0}; }

hyena_status qk_sizes(const hyena_qk_norm* op)
{
    if (op == nullptr) return qk_refuse("the description is NULL");
    if (op->B < 1 || op->N < 1 || op->q_heads < 1 || op->k_heads < 1 || op->D < 1)
        return qk_refuse("B, N, q_heads, k_heads and D must be at least 1");
    if (op->D > 1024) return fail(HYENA_ERR_UNSUPPORTED, "qk norm: D must be in 1..1024");
    if (op->q_heads > 4096 || op->k_heads > 4096)
        return fail(HYENA_ERR_UNSUPPORTED, "qk norm: at most 4096 heads");
    if (op->B > ((int64_t)1 << 31) || op->N > ((int64_t)1 << 31) || op->B * op->N > ((int64_t)1 << 31))
        return fail(HYENA_ERR_UNSUPPORTED, "qk norm: at most 2^31 tokens");
    if (op->io_dtype != HYENA_F32 && op->io_dtype != HYENA_BF16 && op->io_dtype != HYENA_F16)
        return fail(HYENA_ERR_UNSUPPORTED, "qk norm: unknown io dtype");
    if (op->norm != HYENA_NORM_NONE && op->norm != HYENA_NORM_RMS && op->norm != HYENA_NORM_L2)
        return fail(HYENA_ERR_UNSUPPORTED, "qk norm: unknown norm");
    if (op->layout != HYENA_ROTARY_HALF && op->layout != HYENA_ROTARY_INTERLEAVED)
        return fail(HYENA_ERR_UNSUPPORTED, "qk norm: unknown layout");
    if (op->rotary_dim < 0 || op->rotary_dim > op->D || op->rotary_dim % 2 != 0)
        return qk_refuse("rotary_dim must be even and in 0..D");
    if (op->rotary_dim > 0 && op->freqs == nullptr) return qk_refuse("freqs is NULL");
    if (!(op->eps >= 0.0f)) return qk_refuse("eps must be at least 0");
    return HYENA_OK;
}

// Checks and kernel arguments shared by both directions; ins: 7 spans.
hyena_status qk_args(const hyena_qk_norm* op, void* q_out, void* k_out, QkArgs& a, Span* ins, Span* outs)
{
    hyena_status st = qk_sizes(op);
    if (st != HYENA_OK) return st;
    const size_t e = element_bytes(op->io_dtype);
    if ((st = check_view(op->q, "q", e)) != HYENA_OK || (st = check_view(op->k, "k", e)) != HYENA_OK) return st;
    if (q_out == nullptr || k_out == nullptr) return qk_refuse("an output pointer is NULL");
    if ((uintptr_t)q_out % 16 != 0 || (uintptr_t)k_out % 16 != 0) return qk_refuse("outputs must be 16-byte aligned");
    if ((uintptr_t)op->freqs % 8 != 0 || (uintptr_t)op->q_weight % 4 != 0 || (uintptr_t)op->k_weight % 4 != 0 ||
        (uintptr_t)op->positions % 4 != 0)
        return qk_refuse("freqs, a weight or positions is not aligned to its element");
    const size_t rows = (size_t)(op->B * op->N);
    ins[0] = view_span(op->q, op->B, op->N, op->q_heads, op->D, e);
    ins[1] = view_span(op->k, op->B, op->N, op->k_heads, op->D, e);
    ins[2] = Span{op->freqs, (size_t)op->rotary_dim / 2 * 8};
    ins[3] = Span{op->q_weight, (size_t)op->D * 4};
    ins[4] = Span{op->k_weight, (size_t)op->D * 4};
    ins[5] = Span{op->positions, rows * 4};
    outs[0] = Span{q_out, rows * (size_t)(op->q_heads * op->D) * e};
    outs[1] = Span{k_out, rows * (size_t)(op->k_heads * op->D) * e};

    a = QkArgs{};
    a.t[0].x = plain_view(op->q);
    a.t[1].x = plain_view(op->k);
    a.t[0].out = q_out;
    a.t[1].out = k_out;
    a.t[0].w = op->norm == HYENA_NORM_NONE ? nullptr : op->q_weight;
    a.t[1].w = op->norm == HYENA_NORM_NONE ? nullptr : op->k_weight;
    a.t[0].heads = (int32_t)op->q_heads;
    a.t[1].heads = (int32_t)op->k_heads;
    for (int k = 0; k < 2; ++k)
        a.t[k].magic = (uint32_t)((((uint64_t)1 << 32) + (uint64_t)a.t[k].heads - 1) / (uint64_t)a.t[k].heads);
    a.freqs = op->freqs;
    a.positions = op->positions;
    a.offset = op->position_offset;
    a.N = op->N;
    a.rows = op->B * op->N;
    a.D = (int32_t)op->D;
    a.rotary = (int32_t)op->rotary_dim;
    a.half = op->layout == HYENA_ROTARY_HALF;
    a.norm = op->norm;
    a.mean = op->norm == HYENA_NORM_RMS ? 1.0f / (float)op->D : 1.0f;
    a.eps = op->eps;
    a.rscale = op->rotary_scale;
    return HYENA_OK;
}

hyena_status qk_overlaps(const Span* ins, int nin, const Span* outs, int nout)
{
    for (int i = 0; i < nout; ++i) {
        for (int j = 0; j < nin; ++j)
            if (spans_overlap(outs[i], ins[j])) return qk_refuse("an output overlaps an input");
        for (int j = 0; j < i; ++j)
            if (spans_overlap(outs[i], outs[j])) return qk_refuse("two outputs overlap");
    }
    return HYENA_OK;
}

size_t part_bytes(int64_t groups, int64_t D) { return ((size_t)groups * (size_t)D * 4 + 255) & ~(size_t)255; }

template <bool GRAD> hyena_status qk_by_type(int32_t io_dtype, QkArgs& a, hipStream_t s)
{
    if (io_dtype == HYENA_F32) return qk_launch<float, GRAD>(a, s);
    if (io_dtype == HYENA_BF16) return qk_launch<uint16_t, GRAD>(a, s);
    return qk_launch<_Float16, GRAD>(a, s);
}

}  // namespace
}  // namespace hy

using namespace hy;

extern "C" {

hyena_status hyena_qk_norm_forward(const hyena_qk_norm* op, void* q_out, void* k_out, void* stream)
{
    QkArgs a;
    Span ins[6], outs[2];
    hyena_status st = qk_args(op, q_out, k_out, a, ins, outs);
    if (st != HYENA_OK) return st;
    if ((st = qk_overlaps(ins, 6, outs, 2)) != HYENA_OK) return st;
    shape_tiles(a, element_bytes(op->io_dtype), false);
    return qk_by_type<false>(op->io_dtype, a, (hipStream_t)stream);
}

hyena_status hyena_qk_norm_scratch_bytes(const hyena_qk_norm* op, size_t* bytes)
{
    const hyena_status st = qk_sizes(op);
    if (st != HYENA_OK) return st;
    if (bytes == nullptr) return qk_refuse("bytes is NULL");
    QkArgs a{};
    a.rows = op->B * op->N;
    a.D = (int32_t)op->D;
    a.rotary = (int32_t)op->rotary_dim;
    a.t[0].heads = (int32_t)op->q_heads;
    a.t[1].heads = (int32_t)op->k_heads;
    shape_tiles(a, element_bytes(op->io_dtype), true);
    *bytes = part_bytes(a.t[0].groups, op->D) + part_bytes(a.t[1].groups, op->D);
    return HYENA_OK;
}

hyena_status hyena_qk_norm_backward(const hyena_qk_norm* op, const hyena_view* dq_out, const hyena_view* dk_out,
                                    void* dq, void* dk, float* dq_weight, float* dk_weight, void* scratch,
                                    void* stream)
{
    QkArgs a;
    Span ins[8], outs[5];
    hyena_status st = qk_args(op, dq, dk, a, ins, outs);
    if (st != HYENA_OK) return st;
    if (dq_out == nullptr || dk_out == nullptr) return qk_refuse("a gradient view is NULL");
    const size_t e = element_bytes(op->io_dtype);
    if ((st = check_view(*dq_out, "dq_out", e)) != HYENA_OK || (st = check_view(*dk_out, "dk_out", e)) != HYENA_OK)
        return st;
    ins[6] = view_span(*dq_out, op->B, op->N, op->q_heads, op->D, e);
    ins[7] = view_span(*dk_out, op->B, op->N, op->k_heads, op->D, e);
    if ((uintptr_t)dq_weight % 4 != 0 || (uintptr_t)dk_weight % 4 != 0)
        return qk_refuse("a weight's gradient is not aligned to its element");
    const bool weights = op->norm != HYENA_NORM_NONE && (dq_weight || dk_weight);
    if (op->norm == HYENA_NORM_NONE && (dq_weight || dk_weight)) return qk_refuse("no norm, so no weights' gradients");
    if (weights && (scratch == nullptr || (uintptr_t)scratch % 16 != 0))
        return qk_refuse("scratch is NULL or not 16-byte aligned");
    shape_tiles(a, e, true);
    const size_t part = part_bytes(a.t[0].groups, op->D), parts = part + part_bytes(a.t[1].groups, op->D);
    outs[2] = Span{dq_weight, (size_t)op->D * 4};
    outs[3] = Span{dk_weight, (size_t)op->D * 4};
    outs[4] = Span{weights ? scratch : nullptr, parts};
    if ((st = qk_overlaps(ins, 8, outs, 5)) != HYENA_OK) return st;
    a.t[0].dy = plain_view(*dq_out);
    a.t[1].dy = plain_view(*dk_out);
    a.t[0].dw_part = dq_weight ? (float*)scratch : nullptr;
    a.t[1].dw_part = dk_weight ? (float*)((char*)scratch + part) : nullptr;
    const hipStream_t s = (hipStream_t)stream;
    if ((st = qk_by_type<true>(op->io_dtype, a, s)) != HYENA_OK) return st;
    if (!weights) return HYENA_OK;
    HY_LAUNCH(kernel_label("hyena_qk_weight_grad"), hyena_qk_weight_grad, dim3((unsigned)((a.D + 15) / 16), 2), dim3(1024),
              0, s, a.t[0].dw_part, a.t[1].dw_part, dq_weight, dk_weight, a.t[0].groups, a.t[1].groups, a.D);
    const hipError_t err = hipGetLastError();
    return err == hipSuccess ? HYENA_OK : fail(HYENA_ERR_DEVICE, hipGetErrorString(err));
}

}  // extern "C"
