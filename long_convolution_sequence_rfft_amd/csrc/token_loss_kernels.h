// token_loss_kernels.h -- softmax cross entropy over a vocabulary and its
// gradients (include/hyena.h).
//
//   hyena_loss_gather   the tokens that take part, their rows of x side by side
//   hyena_loss_pack     the table as a matrix operand, where it is not one as given
//   hyena_loss_logits   a tile of logits; forward: each token's largest and the sum
//                       of the exponentials over the tile's values; backward: G
//   hyena_loss_few      the same for few tokens, hyena_loss_few_grads their gradients
//   hyena_loss_join     the tiles' sums joined: loss, lse
//   hyena_loss_products d_table of a piece of the vocabulary, and its share of d_x
//   hyena_loss_table    d_table of a piece from its sums, where the tokens are cut
//   hyena_loss_finish   d_x from its sums (hyena_loss_finish_few where they are many)
//   hyena_loss_zeros    zeros for the other tokens, where the products write d_x themselves
//
// Bound by the matrix instructions, 2 tokens V d operations forward, 10 backward with 16-bit storage
// (6, and G's products by two terms each), and these by the power the card may take.  16384 tokens, 50257
// values, width 768 in bf16: logits 1090 to 1120 us, 1130 to 1160 TFLOP/s (the matrix units are
// busy for 66% of the cycles, of 1.64 to 1.68 GHz; a large product of the library's reaches 1279,
// this one 953).  12288 of them backward: logits 1360 us, of which the 2.5 GB of G's two terms take a third; products 3150 us
// (1205 TFLOP/s; of one term two products of the library's 944 and 822; the matrix units are busy for
// 72% of the cycles, of 1.60 GHz).  2048 tokens, 31999 values in float32, whose six products are
// counted: 515 us (1172) and 988 us (1222).
#pragma once

#include "matmul_device.h"
#include "token_loss.h"

namespace hy {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Storage types' matrix operands, float32 as three planes of bfloat16, and the waves of a
// tile of a product, WM x WN.  With three planes a step's operands take 72 KB of LDS and a
// compute unit holds one workgroup, of 8 waves (gradients of 2000 tokens, 50257 values and
// 768 channels in float32: 1492 us, with 4 waves 1568, with one plane after the other and
// two workgroups of 4 waves 1676).
template <typename T> struct LossType {
    using E = T;
    static constexpr int P = 1, WM = 2, WN = 2, kThreads = WM * WN * 64;
};
template <> struct LossType<float> {
    using E = uint16_t;
    static constexpr int P = 3, WM = 4, WN = 2, kThreads = WM * WN * 64;
};

// Eight float32 values as P planes of E, by cutting (bfloat16, P = 3) or rounding (P = 1).
template <typename E, int P> __device__ __forceinline__ void store_planes(char* to, int64_t plane, f32x8 x)
{
    Split<E, P> s;
    s.set(x);
#pragma unroll
    for (int n = 0; n < P; ++n) *(typename Mx<E>::frag*)(to + n * plane) = s.f[n];
}

// Planes of G.  It is float32, and with 16-bit storage two terms of that type (rounded, what is
// left rounded): off by 2^-16 of itself in bfloat16, 2^-22 in binary16, so that the gradients'
// rounding is their results' only.  One term leaves as much again in every row of d_table that is
// nobody's target, and more in sums that cancel (d_x: G of a token sums to 0); its products take
// half the matrix instructions (16384 tokens, a quarter masked, 50257 values, width 768 in bf16: logits
// 890 us with one, 1370 with two, products 1890 and 3150).
template <typename T> constexpr int kGradPlanes = LossType<T>::P == 1 ? 2 : LossType<T>::P;
template <typename T> __device__ __forceinline__ void store_grads(char* to, int64_t plane, f32x8 x)
{
    using E = typename LossType<T>::E;
    if constexpr (LossType<T>::P == 1) {
        const typename Mx<E>::frag first = Mx<E>::narrow8(x);
        *(typename Mx<E>::frag*)to = first;
        *(typename Mx<E>::frag*)(to + plane) = Mx<E>::narrow8(x - Mx<E>::widen8(first));
    } else {
        store_planes<E, kGradPlanes<T>>(to, plane, x);
    }
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
template <typename T, bool UNITS, bool GRAD> __global__ __launch_bounds__(1024) void hyena_loss_gather(LossArgs p)
{
    using E = typename LossType<T>::E;
    constexpr int P = LossType<T>::P;
    __shared__ int lds[16];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t first = (int64_t)blockIdx.x * p.each, last = first + p.each < p.total ? first + p.each : p.total;
    auto takes_part = [&](int64_t t) { return (uint32_t)*row_at<int32_t>(p.targets, t, p.targets_N) < (uint32_t)p.V; };
    int n = 0;
#pragma unroll 16
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
    // rows: teams of lanes with a unit of 8 channels each, kRows rows of a team under way
    constexpr int kRows = 4, kUnits = 8 / kUnit<T>;
    int lanes = 64;
    while (lanes * 4 >= p.kd) lanes /= 2;
    const int teams = 1024 / lanes, team = threadIdx.x / lanes, tl = threadIdx.x % lanes;
    for (int64_t a0 = begin + team; a0 < before; a0 += kRows * teams) {
        const T* x[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int64_t a = a0 + k * teams < before ? a0 + k * teams : before - 1;
            x[k] = row_at<T>(p.x, p.index[a], p.x_N);
        }
        for (int c = tl * 8; c < p.kd; c += lanes * 8) {
            Unit<T, UNITS> u[kRows][kUnits];
#pragma unroll
            for (int k = 0; k < kRows; ++k)
#pragma unroll
                for (int h = 0; h < kUnits; ++h) u[k][h].load(x[k], c + h * kUnit<T>, p.d);
            char* to = p.rows + (c >> 5) * p.block + (c & 31) * 2;
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                if (a0 + k * teams >= before) break;
                f32x8 v;
#pragma unroll
                for (int h = 0; h < kUnits; ++h) {
                    float e[kUnit<T>];
                    u[k][h].widen(e);
#pragma unroll
                    for (int i = 0; i < kUnit<T>; ++i) v[h * kUnit<T> + i] = e[i];
                }
                store_planes<E, P>(to + (a0 + k * teams) * 64, p.rows_plane, v);
            }
        }
    }
    if (blockIdx.x + 1 == gridDim.x) {
        if (threadIdx.x == 0) *p.count = before;
        // after the last one zeros up to a whole step of 32
        const f32x8 none = {};
        for (int64_t a = before + team; a < (before + 31) / 32 * 32; a += teams)
            for (int c = tl * 8; c < p.kd; c += lanes * 8)
                store_planes<E, P>(p.rows + a * 64 + (c >> 5) * p.block + (c & 31) * 2, p.rows_plane, none);
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

// The table in blocks of 32 channels, [kd / 32][V][32], as P planes.
template <typename T, bool UNITS> __global__ __launch_bounds__(256) void hyena_loss_pack(LossArgs p)
{
    using E = typename LossType<T>::E;
    constexpr int P = LossType<T>::P;
    const int lane = threadIdx.x & 63;
    for (int64_t v = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); v < p.V; v += (int64_t)gridDim.x * 4) {
        const T* row = (const T*)p.table + v * p.d;
        char* to = const_cast<char*>(p.values) + v * 64;
        for (int c = lane * 8; c < p.kd; c += 512) {
            f32x8 x = {};
#pragma unroll
            for (int h = 0; h < 8; h += kUnit<T>) {
                float e[kUnit<T>];
                load_unit<T, UNITS>(row, c + h, p.d, e);
#pragma unroll
                for (int i = 0; i < kUnit<T>; ++i) x[h + i] = e[i];
            }
            store_planes<E, P>(to + (c >> 5) * p.values_block + (c & 31) * 2, p.values_plane, x);
        }
    }
}

// The workgroups of one XCD (every eighth) take tiles of the same rows or columns
// side by side, so that what they share comes from its L2: `inner` tiles of one axis,
// `outer` of the other; the outer axis is dealt out to the XCDs.
__device__ __forceinline__ bool deal(int64_t id, int inner, int outer, int& i, int& o)
{
    const int64_t local = id >> 3;
    i = (int)(local % inner);
    const int64_t k = local / inner * 8 + (id & 7);
    o = (int)k;
    return k < outer;
}
inline int64_t dealt(int64_t inner, int64_t outer) { return inner * ((outer + 7) / 8 * 8); }

// Tiles of values of one XCD whose part of the table stays in its L2 while the tokens'
// tiles go by (16384 tokens, 50257 values: 2 1076, 6 1066, 12 1079, 25 1284 us).
constexpr int kLossGroup = 6;
// Fewer tiles of values than this, and fewer than tiles of tokens: the tokens' tiles are dealt
// out to the XCDs.
constexpr int kDealValues = 64;
inline __host__ __device__ bool deal_tokens(int value_tiles, int token_tiles) { return value_tiles < kDealValues && value_tiles < token_tiles; }

// Two sums of exponentials, each with what was taken from its exponents.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2)
{
    const float top = fmaxf(m, m2);
    const float base = top == -INFINITY ? 0.0f : top;  // both are empty
    s = s * __builtin_amdgcn_exp2f(m - base) + s2 * __builtin_amdgcn_exp2f(m2 - base);
    m = top;
}

// Logits of TM values (rows of the tile) and TN tokens (columns).  Small tiles have more of
// their short steps under way.
template <typename T, bool SMALL> struct LogitsTile {
    static constexpr int TM = SMALL ? kSmallTile : kLossValues, TN = SMALL ? kSmallTile : kLossTokens;
    static constexpr int P = LossType<T>::P, WM = SMALL ? 2 : LossType<T>::WM, WN = SMALL ? 2 : LossType<T>::WN;
    static constexpr int kThreads = WM * WN * 64, kStages = SMALL ? (P == 1 ? 4 : 3) : 2;
    static constexpr int kWaves = P == 1 && !SMALL ? 3 : 2;  // of a SIMD
};
template <typename T, bool GRAD, bool SMALL>
__global__ __launch_bounds__((LogitsTile<T, SMALL>::kThreads), (LogitsTile<T, SMALL>::kWaves)) void hyena_loss_logits(LossArgs p, int value_tiles)
{
    using L = LogitsTile<T, SMALL>;
    using E = typename LossType<T>::E;
    constexpr int P = L::P, WM = L::WM, WN = L::WN, TM = L::TM, TN = L::TN;
    using Tile = MatTile<E, TM, TN, WM, WN, kInColumnsPaired, kInColumns, P, P, L::kStages>;
    __shared__ __attribute__((aligned(16))) char lds[Tile::kLds];
    const int64_t count = *p.count;
    const int token_tiles = (int)(p.tokens / TN);
    int value_tile, token_tile;
    if (deal_tokens(value_tiles, token_tiles)) {
        deal(blockIdx.x, value_tiles, token_tiles, value_tile, token_tile);
    } else {
        // XCD x has the tiles of values x, x + 8, ..., kLossGroup of them at a time
        const int64_t local = blockIdx.x >> 3, each = (int64_t)kLossGroup * token_tiles;
        const int mine = (value_tiles + 7) / 8, group = (int)(local / each), in_group = mine - group * kLossGroup;
        const int width = in_group < kLossGroup ? in_group : kLossGroup;
        const int64_t rest = local - group * each;
        value_tile = (group * kLossGroup + (int)(rest % width)) * 8 + (int)(blockIdx.x & 7);
        token_tile = (int)(rest / width);
    }
    const int64_t t0 = (int64_t)token_tile * TN;
    if (t0 >= count || value_tile >= value_tiles) return;
    const int32_t v0 = p.first + value_tile * TM;
    Tile tile;
    const Operand values{p.values + (int64_t)v0 * p.values_row, p.values + p.values_bytes, p.values_row, p.values_block};
    const Operand rows{p.rows + t0 * 64, p.rows + p.rows_plane, 64, p.block};
    tile.run(lds, values, p.values_plane, rows, p.rows_plane, p.kd / 32);

    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4;
    const int wm = wave / WN, wn = wave % WN;
    const float scale2 = p.scale * kLog2e;
    const int first = wm * (TM / WM) + 8 * g;  // this lane's values: first + at(i) + r
    auto at = [](int i) { return 32 * (i >> 1) + 4 * (i & 1); };
    const int left = p.V - v0;                         // values of the tile that there are
    if constexpr (!GRAD) {
        float2* shares = (float2*)lds;  // [WM][TN]
#pragma unroll
        for (int j = 0; j < Tile::NI; ++j) {
            const int n = wn * (TN / WN) + 16 * j + (lane & 15);
            const int64_t t = t0 + n;
#pragma unroll
            for (int i = 0; i < Tile::MI; ++i) tile.c[i][j] *= scale2;
            if (left < TM) {
#pragma unroll
                for (int i = 0; i < Tile::MI; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (first + at(i) + r >= left) tile.c[i][j][r] = -INFINITY;
            }
            const int target = t < count ? p.target[t] - v0 - first : -1;
            if (__any((uint32_t)target < (uint32_t)(TM / WM))) {
                float hit = 0.0f;
#pragma unroll
                for (int i = 0; i < Tile::MI; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) hit = target == at(i) + r ? tile.c[i][j][r] : hit;
                if ((uint32_t)target < (uint32_t)(TM / WM) && (target & 31) < 8) p.hit[t] = hit;
            }
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < Tile::MI; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) m = fmaxf(m, tile.c[i][j][r]);
            m = fmaxf(m, __shfl_xor(m, 16));
            m = fmaxf(m, __shfl_xor(m, 32));
            const float base = m == -INFINITY ? 0.0f : m;  // (no value of this share is in the vocabulary)
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < Tile::MI; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) s += __builtin_amdgcn_exp2f(tile.c[i][j][r] - base);
            s += __shfl_xor(s, 16);
            s += __shfl_xor(s, 32);
            if (g == 0) shares[wm * TN + n] = make_float2(m, s);
        }
        __syncthreads();
        if (threadIdx.x < TN) {
            float2 a = shares[threadIdx.x];
#pragma unroll
            for (int w = 1; w < WM; ++w) join(a.x, a.y, shares[w * TN + threadIdx.x].x, shares[w * TN + threadIdx.x].y);
            p.part[(int64_t)value_tile * p.tokens + t0 + threadIdx.x] = a;
        }
    } else {
        const float up = p.norm[0];
        const bool rim = left < TM || t0 + TN > count;
#pragma unroll
        for (int j = 0; j < Tile::NI; ++j) {
            const int n = wn * (TN / WN) + 16 * j + (lane & 15);
            const int64_t t = t0 + n;
            const bool in = t < count;
            const int target = in ? p.target[t] - v0 - first : -1;
            const float lse2 = in ? p.lse2[t] : 0.0f, weight = in ? p.weight[t] * up : 0.0f;
#pragma unroll
            for (int i = 0; i < Tile::MI; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    tile.c[i][j][r] = weight * __builtin_amdgcn_exp2f(fmaf(tile.c[i][j][r], scale2, -lse2));
            if (rim) {  // zeros where no token or no value is
#pragma unroll
                for (int i = 0; i < Tile::MI; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (!in || first + at(i) + r >= left) tile.c[i][j][r] = 0.0f;
            }
            if (__any((uint32_t)target < (uint32_t)(TM / WM))) {
#pragma unroll
                for (int i = 0; i < Tile::MI; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (target == at(i) + r) tile.c[i][j][r] -= weight;
            }
            char* to = p.g + (int64_t)((value_tile * TM + wm * (TM / WM)) >> 5) * p.block + t * 64 + g * 16;
#pragma unroll
            for (int i = 0; i < Tile::MI; i += 2)
                store_grads<T>(to + (int64_t)(i >> 1) * p.block, p.g_plane, join8(tile.c[i][j], tile.c[i + 1][j]));
        }
    }
}

// Logits of few tokens, 16 N of them: bound by reading the table once (8 tokens of width 768 in bf16,
// 50257 values: 17.0 us for 77 MB).  Workgroups take
// tiles of 16 values in turn, so that all of them together read one piece of the table after
// the other (a part of the table for each workgroup was a third slower); within a tile each
// wave has a quarter of the channels.  The operands go from memory to the registers, the
// next piece ahead of the products; the waves' sums are joined in LDS.  A table in float32
// is read as given and becomes three terms in the registers.  Forward a workgroup keeps each
// token's largest and sum; backward G stays float32, [values rounded up][16].
//
// OWN: there is no gather before it.  The call has at most 16 N tokens, in rows of whole
// units, and each workgroup finds by itself which take part, while its first piece of the
// table is under way, and reads their rows as given (8 tokens in bf16: 21 us so, 28
// with a gather).
template <typename T, int N, bool GRAD, bool OWN> __global__ __launch_bounds__(256) void hyena_loss_few(LossArgs p)
{
    using E = typename LossType<T>::E;
    using frag = typename Mx<E>::frag;
    using Raw = std::conditional_t<LossType<T>::P == 3, f32x8, frag>;  // as loaded
    constexpr int P = LossType<T>::P, kPiece = P == 3 && N > 1 ? 3 : 6;        // steps of a piece
    static_assert(!GRAD || (N == 1 && !OWN), "");
    static_assert(N <= 4, "");
    __shared__ f32x4 lds[2][4][N][64];
    __shared__ int own_index[16 * N], own_target[16 * N];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, g = lane >> 4, i = lane & 15;
    const int64_t t0 = (int64_t)blockIdx.y * (16 * N);
    int64_t count = 0;
    if constexpr (!OWN) {
        count = *p.count;
        if (t0 >= count) return;
    }
    const int tiles = (p.V + 15) / 16, steps = p.kd / 32, each = (steps + 3) / 4, pieces = (each + kPiece - 1) / kPiece;
    const int k0 = wave * each, k1 = k0 + each < steps ? k0 + each : steps;  // this wave's steps (none: k0 >= k1)
    const int64_t rows_block = p.block, step_bytes = P == 3 ? 128 : p.values_block;
    const uint32_t aoff = (uint32_t)i * (uint32_t)p.values_row + g * (P == 3 ? 32 : 16), boff = i * 64 + g * 16;
    const char* end = p.values + p.values_bytes;
    auto load_a = [&](int tile, int s, Raw (&a)[kPiece]) {
        const __amdgpu_buffer_rsrc_t r = operand_rsrc(p.values + (int64_t)tile * 16 * p.values_row + s * step_bytes, end);
#pragma unroll
        for (int k = 0; k < kPiece; ++k) {
            const uint32_t off = aoff + (uint32_t)k * (uint32_t)step_bytes;
            if constexpr (P == 3) {
                const f32x4 lo = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
                const f32x4 hi = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off + 16, 0, 0));
                a[k] = join8(lo, hi);
            } else {
                a[k] = __builtin_bit_cast(frag, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
            }
        }
    };
    frag b[kPiece][P][N];
    const T* own_row[N];
    auto load_b = [&](int s) {
        if constexpr (OWN) {
#pragma unroll
            for (int k = 0; k < kPiece; ++k)
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const int c = (s + k) * 32 + g * 8;
                    if constexpr (P == 1) {
                        Unit<T, true> u;
                        u.load(own_row[j], c, p.d);
                        b[k][0][j] = __builtin_bit_cast(frag, u.v);
                    } else {
                        Unit<T, true> lo, hi;
                        lo.load(own_row[j], c, p.d);
                        hi.load(own_row[j], c + 4, p.d);
                        Split<E, P> x;
                        x.set(join8(__builtin_bit_cast(f32x4, lo.v), __builtin_bit_cast(f32x4, hi.v)));
#pragma unroll
                        for (int n = 0; n < P; ++n) b[k][n][j] = x.f[n];
                    }
                }
            return;
        }
#pragma unroll
        for (int n = 0; n < P; ++n) {
            const char* plane = p.rows + n * p.rows_plane;
            const __amdgpu_buffer_rsrc_t r = operand_rsrc(plane + t0 * 64 + s * rows_block, plane + p.rows_plane);
#pragma unroll
            for (int k = 0; k < kPiece; ++k)
#pragma unroll
                for (int j = 0; j < N; ++j)
                    b[k][n][j] = __builtin_bit_cast(frag, __builtin_amdgcn_raw_buffer_load_b128(r, (int)(boff + j * 1024 + (uint32_t)k * (uint32_t)rows_block), 0, 0));
        }
    };
    const float scale2 = p.scale * kLog2e;
    // the waves take turns at the 16s of tokens
    constexpr int kOwn = (N + 3) / 4;
    float top[kOwn], sum[kOwn];
#pragma unroll
    for (int o = 0; o < kOwn; ++o) top[o] = -INFINITY, sum[o] = 0.0f;
    f32x4 c[N];
    // tile and piece of it that are loaded next
    int next_tile = blockIdx.x, next_piece = 0;
    auto ahead = [&](Raw (&a)[kPiece]) {
        if (next_tile < tiles) load_a(next_tile, k0 + next_piece * kPiece, a);
        if (++next_piece == pieces) next_piece = 0, next_tile += gridDim.x;
    };
    int tile = blockIdx.x, piece = 0, half = 0;
    auto work = [&](const Raw (&a)[kPiece]) {
        if (piece == 0) {
#pragma unroll
            for (int j = 0; j < N; ++j) c[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        const int s = k0 + piece * kPiece;
        if (pieces > 1) load_b(s);
#pragma unroll
        for (int k = 0; k < kPiece; ++k) {
            if (s + k >= k1) break;
            if constexpr (P == 3) {
                Split<E, 3> x;
                x.set(a[k]);
#pragma unroll
                for (int q = 0; q < Planes<3>::kPairs; ++q)
#pragma unroll
                    for (int j = 0; j < N; ++j) c[j] = Mx<E>::mma(x.f[Planes<3>::a(q)], b[k][Planes<3>::b(q)][j], c[j]);
            } else {
#pragma unroll
                for (int j = 0; j < N; ++j) c[j] = Mx<E>::mma(a[k], b[k][0][j], c[j]);
            }
        }
        if (++piece < pieces) return;
        piece = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) lds[half][wave][j][lane] = c[j];
        __syncthreads();  // (the other half is written before the next one, and read after it)
        const int left = p.V - tile * 16;
#pragma unroll
        for (int o = 0; o < kOwn; ++o) {
            const int j = o * 4 + wave;
            if (j >= N) break;
            f32x4 l = lds[half][0][j][lane];
#pragma unroll
            for (int w = 1; w < 4; ++w) l += lds[half][w][j][lane];
            const int64_t t = t0 + 16 * j + i;
            int target = -1;
            if (t < count) target = (OWN ? own_target[t] : p.target[t]) - tile * 16 - 4 * g;
            if constexpr (!GRAD) {
                float m = -INFINITY, e = 0.0f;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    l[r] = 4 * g + r < left ? l[r] * scale2 : -INFINITY;
                    if (target == r) p.hit[t] = l[r];
                    m = fmaxf(m, l[r]);
                }
                const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
                for (int r = 0; r < 4; ++r) e += __builtin_amdgcn_exp2f(l[r] - base);
                join(top[o], sum[o], m, e);
            } else {
                const bool in = t < count;
                const float lse2 = in ? p.lse2[t] : 0.0f, weight = in ? p.weight[t] : 0.0f;
                float* to = (float*)p.g + (int64_t)(tile * 16 + 4 * g) * 16 + i;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float q = __builtin_amdgcn_exp2f(fmaf(l[r], scale2, -lse2));
                    to[r * 16] = in && 4 * g + r < left ? weight * (target == r ? q - 1.0f : q) : 0.0f;
                }
            }
        }
        half ^= 1;
        tile += gridDim.x;
    };
    Raw a0[kPiece], a1[kPiece];
    ahead(a0);
    if constexpr (OWN) {
        const int target = lane < p.total ? *row_at<int32_t>(p.targets, lane, p.targets_N) : -1;
        const bool in = (uint32_t)target < (uint32_t)p.V;
        const uint64_t all = __ballot(in);
        const int at = __popcll(all & (((uint64_t)1 << lane) - 1));
        count = __popcll(all);
        if (wave == 0) {
            if (in) own_index[at] = lane, own_target[at] = target;
            if (blockIdx.x == 0) {  // for the join
                if (lane == 0) *p.count = count;
                if (in) {
                    p.index[at] = lane;
                } else if (lane < p.total) {
                    p.loss[lane] = 0.0f;
                    p.lse[lane] = 0.0f;
                }
            }
        }
        if (count == 0) return;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < N; ++j) own_row[j] = row_at<T>(p.x, own_index[16 * j + i < count ? 16 * j + i : count - 1], p.x_N);
    }
    if (pieces == 1) load_b(k0);
    while (true) {
        if (tile >= tiles) break;
        ahead(a1);
        work(a0);
        if (tile >= tiles) break;
        ahead(a0);
        work(a1);
    }
    if constexpr (!GRAD) {
#pragma unroll
        for (int o = 0; o < kOwn; ++o) {
            const int j = o * 4 + wave;
            if (j >= N) break;
            for (int k = 16; k < 64; k *= 2) join(top[o], sum[o], __shfl_xor(top[o], k), __shfl_xor(sum[o], k));
            if (g == 0) p.part[(int64_t)blockIdx.x * p.tokens + t0 + 16 * j + i] = make_float2(top[o], sum[o]);
        }
    }
}

// Gradients of at most N tokens: a wave takes the values of its part one after the
// other, 256 channels of them, adds their share to d_x and makes their rows of d_table.
// Bound by reading and writing the two tables (8 tokens in float32: 72 us for 319 MB); G of a
// value is the same for all lanes.  d_table goes past the caches, which leaves the table there
// for the next call's logits (4 tokens in float32, a call: 115 us through them, 108 so).
template <typename T, int N, bool UNITS> __global__ __launch_bounds__(256) void hyena_loss_few_grads(LossArgs p)
{
    __shared__ f32x4 lds[3][N][64];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int c = (int)blockIdx.y * 256 + lane * 4;
    const int count = (int)*p.count;
    auto load4 = [&](const T* row) {
        f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
        if (UNITS) {
            if (c < p.d) y = Mx<T>::widen(*(const typename Mx<T>::vec4*)(row + c));
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < p.d) y[e] = load_one<T>(row + c + e);
        }
        return y;
    };
    f32x4 x[N], dx[N];
#pragma unroll
    for (int t = 0; t < N; ++t) {
        x[t] = dx[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (t < count && c < p.d) {
            // the gathered rows are matrix operands; here they are read as given
            const T* row = row_at<T>(p.x, p.index[t], p.x_N);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < p.d) x[t][e] = load_one<T>(row + c + e);
        }
    }
    const int parts = (int)gridDim.x * 4, part = (int)blockIdx.x * 4 + wave, each = (p.V + parts - 1) / parts;
    const int v0 = part * each, v1 = v0 + each < p.V ? v0 + each : p.V;
    for (int v4 = v0; v4 < v1; v4 += 4) {
        // G of four values for 16 tokens, an element of it in each lane
        const float g = ((const float*)p.g)[(int64_t)v4 * 16 + lane];
        f32x4 w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = load4((const T*)p.table + (int64_t)(v4 + k < v1 ? v4 + k : v1 - 1) * p.d);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int v = v4 + k;
            if (v >= v1) break;
            f32x4 dw = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int t = 0; t < N; ++t) {
                const float q = t < count ? __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(g), k * 16 + t)) : 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    dx[t][e] = fmaf(q, w[k][e], dx[t][e]);
                    dw[e] = fmaf(q, x[t][e], dw[e]);
                }
            }
            if (p.d_table == nullptr) continue;
            dw *= p.scale;
            T* to = (T*)p.d_table + (int64_t)v * p.d + c;
            if (UNITS) {
                if (c < p.d) __builtin_nontemporal_store(Mx<T>::narrow(dw), (typename Mx<T>::vec4*)to);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e < p.d) store_one<T>(to + e, dw[e]);
            }
        }
    }
    if (p.d_x == nullptr) return;
    if (wave > 0) {
#pragma unroll
        for (int t = 0; t < N; ++t) lds[wave - 1][t][lane] = dx[t];
    }
    __syncthreads();
    if (wave == 0 && c < p.d) {
#pragma unroll
        for (int t = 0; t < N; ++t) {
            if (t >= count) break;
            f32x4 s = dx[t];
#pragma unroll
            for (int w = 0; w < 3; ++w) s += lds[w][t][lane];
            *(f32x4*)(p.acc + ((int64_t)blockIdx.x * p.acc_tokens + t) * p.acc_row + c) = s;
        }
    }
}

// tiles: of this piece of the vocabulary; what came before it is in p.running, unless it is
// the first, and what is behind the last one is the result.  TOKENS of a workgroup, 16, or
// where tiles are few 256 (2^18 tokens, 1 tile: 7 us, with 16 51).
template <typename T, int TOKENS> __global__ __launch_bounds__(1024) void hyena_loss_join(LossArgs p, int tiles, bool last)
{
    constexpr int kLanes = TOKENS < 64 ? TOKENS : 64, kParts = TOKENS < 64 ? 16 : 1024 / TOKENS;  // of a wave's tokens; to be joined at last
    __shared__ float2 lds[kParts][TOKENS];
    const int own = threadIdx.x % TOKENS;
    const int64_t count = *p.count, a = (int64_t)blockIdx.x * TOKENS + own;
    if ((int64_t)blockIdx.x * TOKENS >= count) return;
    float m = -INFINITY, s = 0.0f;
    if (a < p.tokens) {
#pragma unroll 8
        for (int i = threadIdx.x / TOKENS; i < tiles; i += 1024 / TOKENS) {
            const float2 x = p.part[(int64_t)i * p.tokens + a];
            join(m, s, x.x, x.y);
        }
    }
    for (int k = kLanes; k < 64; k *= 2) join(m, s, __shfl_xor(m, k), __shfl_xor(s, k));
    if ((threadIdx.x & 63) < kLanes) lds[TOKENS < 64 ? threadIdx.x >> 6 : threadIdx.x / TOKENS][own] = make_float2(m, s);
    __syncthreads();
    if (threadIdx.x < TOKENS && a < count) {
        for (int i = 1; i < kParts; ++i) join(m, s, lds[i][own].x, lds[i][own].y);
        if (p.first != 0) join(m, s, p.running[a].x, p.running[a].y);
        if (!last) {
            p.running[a] = make_float2(m, s);
            return;
        }
        const float log2s = __builtin_amdgcn_logf(s);
        const int32_t t = p.index[a];
        p.lse[t] = (m + log2s) * kLn2;
        p.loss[t] = ((m - p.hit[a]) + log2s) * kLn2;
    }
}

// 4 channels of d_x of a token, x their sum.
template <typename T> __device__ __forceinline__ void store_dx(const LossArgs& p, int64_t t, int c, f32x4 x)
{
    T* to = (T*)p.d_x + t * p.d + c;
    if (p.d % 4 == 0) {
        *(typename Mx<T>::vec4*)to = Mx<T>::narrow(x);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (c + e < p.d) store_one<T>(to + e, x[e]);
    }
}

// One launch, so that neither product waits for the other's last workgroups.  Tiles of 256
// channels by 128 rows and two workgroups a compute unit: with one term of G three of fewer
// registers spilled 22 and took twice as long, tiles of 256 by 256 in one workgroup 2072 us
// instead of 1905.
//
// The first table_groups workgroups: d_table of kGradRows values of this piece and
// kGradChannels channels, the sum over one of p.table_splits parts of the tokens.  The
// others, shorter ones: a share of d_x of kGradRows tokens, the sum over one of p.splits
// parts of the piece's values; or (p.direct) all of it, as d_x itself.
template <typename T> __global__ __launch_bounds__(LossType<T>::kThreads, 2) void hyena_loss_products(LossArgs p, int table_groups, int channel_tiles)
{
    using E = typename LossType<T>::E;
    constexpr int P = LossType<T>::P, WM = LossType<T>::WM, WN = LossType<T>::WN;
    constexpr int GP = kGradPlanes<T>;
    using Table = MatTile<E, kGradChannels, kGradRows, WM, WN, kInRows, kInRows, P, GP, 2>;
    using Dx = MatTile<E, kGradChannels, kGradRows, WM, WN, kInRows, kInColumns, P, GP, 2>;
    __shared__ __attribute__((aligned(16))) char lds[Table::kLds];
    const int64_t count = *p.count;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4;
    const int wm = wave / WN, wn = wave % WN;
    const int32_t values = p.V - p.first < p.chunk ? p.V - p.first : p.chunk;  // of this piece
    int channel_tile, o;
    if ((int)blockIdx.x < table_groups) {
        if (!deal(blockIdx.x, channel_tiles, (values + kGradRows - 1) / kGradRows * p.table_splits, channel_tile, o)) return;
        const int c0 = channel_tile * kGradChannels, split = o % p.table_splits;
        const int32_t v0 = o / p.table_splits * kGradRows;
        const int steps = (int)((count + 31) / 32), per = (steps + p.table_splits - 1) / p.table_splits;
        const int k0 = split * per, k1 = k0 + per < steps ? k0 + per : steps;
        Table tile;
        if (k0 < k1) {
            const Operand x{p.rows + (int64_t)(c0 >> 5) * p.block + (int64_t)k0 * 2048, p.rows + p.rows_plane, 64, p.block};
            const Operand y{p.g + (int64_t)(v0 >> 5) * p.block + (int64_t)k0 * 2048, p.g + p.g_plane, 64, p.block};
            tile.run(lds, x, p.rows_plane, y, p.g_plane, k1 - k0);
        } else {
            tile.clear();
        }
        const float down = p.norm[1];
#pragma unroll
        for (int j = 0; j < Table::NI; ++j) {
            const int32_t v = v0 + wn * (kGradRows / WN) + 16 * j + (lane & 15);
            if (v >= values) continue;
            T* to = (T*)p.d_table + (int64_t)(p.first + v) * p.d;
#pragma unroll
            for (int i = 0; i < Table::MI; ++i) {
                const int c = c0 + wm * (kGradChannels / WM) + 16 * i + 4 * g;
                if (p.table_splits > 1) {
                    if (c < p.acc_row) *(f32x4*)(p.table_acc + ((int64_t)split * p.chunk + v) * p.acc_row + c) = tile.c[i][j];
                    continue;
                }
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
    if (!deal((int64_t)blockIdx.x - table_groups, channel_tiles, (int)(p.tokens / kGradRows) * p.splits, channel_tile, o)) return;
    const int c0 = channel_tile * kGradChannels, split = o % p.splits;
    const int64_t t0 = (int64_t)(o / p.splits) * kGradRows;
    if (t0 >= count) return;
    // this part's values, whole steps of 32
    const int steps = (values + 31) / 32, per = (steps + p.splits - 1) / p.splits;
    const int k0 = split * per, k1 = k0 + per < steps ? k0 + per : steps;
    if (k0 >= k1 && p.first != 0) return;
    Dx tile;
    if (k0 < k1) {
        const Operand x{p.values + (int64_t)(p.first + 32 * k0) * p.values_row + (int64_t)(c0 >> 5) * p.values_block,
                        p.values + p.values_bytes, p.values_row, p.values_block};
        const Operand y{p.g + (int64_t)k0 * p.block + t0 * 64, p.g + p.g_plane, 64, p.block};
        tile.run(lds, x, p.values_plane, y, p.g_plane, k1 - k0);
    } else {
        tile.clear();
    }
    if (p.direct) {
        const float down = p.norm[1];
#pragma unroll
        for (int j = 0; j < Dx::NI; ++j) {
            const int64_t a = t0 + wn * (kGradRows / WN) + 16 * j + (lane & 15);
            if (a >= count) continue;
            const int32_t t = p.index[a];
#pragma unroll
            for (int i = 0; i < Dx::MI; ++i) {
                const int c = c0 + wm * (kGradChannels / WM) + 16 * i + 4 * g;
                if (c < p.d) store_dx<T>(p, t, c, tile.c[i][j] * down);
            }
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < Dx::NI; ++j) {
        const int64_t t = t0 + wn * (kGradRows / WN) + 16 * j + (lane & 15);
        float* to = p.acc + ((int64_t)split * p.tokens + t) * p.acc_row;
#pragma unroll
        for (int i = 0; i < Dx::MI; ++i) {
            const int c = c0 + wm * (kGradChannels / WM) + 16 * i + 4 * g;
            if (c >= p.acc_row) continue;
            f32x4 r = tile.c[i][j];
            if (p.first != 0) r += *(const f32x4*)(to + c);
            *(f32x4*)(to + c) = r;
        }
    }
}

// A row of d_table of a piece from its sums, 256 channels of it: each of 16 waves some of them.
template <typename T> __global__ __launch_bounds__(1024) void hyena_loss_table(LossArgs p)
{
    __shared__ f32x4 lds[16][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int c = (int)blockIdx.y * 256 + lane * 4;
    const float* from = p.table_acc + (int64_t)blockIdx.x * p.acc_row + c;
    f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c < p.d) {
#pragma unroll 4
        for (int s = wave; s < p.table_splits; s += 16) x += *(const f32x4*)(from + (int64_t)s * p.chunk * p.acc_row);
    }
    lds[wave][lane] = x;
    __syncthreads();
    if (wave != 0 || c >= p.d) return;
#pragma unroll
    for (int w = 1; w < 16; ++w) x += lds[w][lane];
    x *= p.norm[1];
    T* to = (T*)p.d_table + (int64_t)(p.first + blockIdx.x) * p.d + c;
    if (p.d % 4 == 0) {
        *(typename Mx<T>::vec4*)to = Mx<T>::narrow(x);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (c + e < p.d) store_one<T>(to + e, x[e]);
    }
}

// d_x of tokens from their sums, a wave for kTokens tokens.
template <typename T, int kTokens> __global__ __launch_bounds__(256) void hyena_loss_finish(LossArgs p)
{
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const float down = p.norm[1];
    for (int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * kTokens; t0 < p.total; t0 += (int64_t)gridDim.x * 4 * kTokens) {
        int32_t a[kTokens];
#pragma unroll
        for (int k = 0; k < kTokens; ++k) a[k] = t0 + k < p.total ? p.place[t0 + k] : -1;
        for (int c = lane * 4; c < p.d; c += 256) {
            f32x4 x[kTokens];
#pragma unroll
            for (int k = 0; k < kTokens; ++k) x[k] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
            for (int s = 0; s < p.splits; ++s) {
#pragma unroll
                for (int k = 0; k < kTokens; ++k)  // (a token that takes no part has some row's sum and drops it)
                    x[k] += *(const f32x4*)(p.acc + ((int64_t)s * p.tokens + (a[k] < 0 ? 0 : a[k])) * p.acc_row + c);
            }
#pragma unroll
            for (int k = 0; k < kTokens; ++k)
                if (t0 + k < p.total) store_dx<T>(p, t0 + k, c, a[k] < 0 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : x[k] * down);
        }
    }
}

// Zeros for d_x of the tokens that take no part, where the others' is written directly.
template <typename T> __global__ __launch_bounds__(256) void hyena_loss_zeros(LossArgs p)
{
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    for (int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * 64; t0 < p.total; t0 += (int64_t)gridDim.x * 256) {
        uint64_t none = __ballot(t0 + lane < p.total && p.place[t0 + lane] < 0);
        for (; none != 0; none &= none - 1)
            for (int c = lane * 4; c < p.d; c += 256) store_dx<T>(p, t0 + __builtin_ctzll(none), c, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
    }
}

// d_x by 16 waves for each token and 256 channels: few tokens have many sums.
template <typename T> __global__ __launch_bounds__(1024) void hyena_loss_finish_few(LossArgs p)
{
    __shared__ f32x4 lds[16][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, c = (int)blockIdx.y * 256 + lane * 4;
    const float down = p.few ? p.scale : p.norm[1];
    for (int64_t t = blockIdx.x; t < p.total; t += gridDim.x) {
        const int32_t a = p.place[t];
        f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
        if (a >= 0 && c < p.d) {
            const float* from = p.acc + (int64_t)a * p.acc_row + c;
#pragma unroll 4
            for (int s = wave; s < p.splits; s += 16) x += *(const f32x4*)(from + (int64_t)s * p.acc_tokens * p.acc_row);
        }
        lds[wave][lane] = x;
        __syncthreads();
        if (wave == 0 && c < p.d) {
#pragma unroll
            for (int w = 1; w < 16; ++w) x += lds[w][lane];
            store_dx<T>(p, t, c, x * down);
        }
        __syncthreads();
    }
}

// Calls of fewer tokens: a wave of hyena_loss_finish has one token, not four (300 tokens, 2048 values:
// 6.5 us with one, 8.1 with four; 8192 tokens 31 and 30; 16384 tokens, 50257 values 34 and 32).
constexpr int64_t kFinishTokens = 16384;

template <typename T, bool GRAD> hyena_status loss_begin(const LossArgs& a, bool pack, bool units, hipStream_t s)
{
    hyena_status st;
    const dim3 grid((unsigned)((a.total + a.each - 1) / a.each));
    if (units)
        HY_LAUNCH(kernel_label("hyena_loss_gather", type_label<T>(), true, GRAD), (hyena_loss_gather<T, true, GRAD>), grid, dim3(1024), 0, s, a);
    else
        HY_LAUNCH(kernel_label("hyena_loss_gather", type_label<T>(), false, GRAD), (hyena_loss_gather<T, false, GRAD>), grid, dim3(1024), 0, s, a);
    if ((st = launched()) != HYENA_OK || !pack) return st;
    const int64_t need = ((int64_t)a.V + 3) / 4;
    const dim3 pgrid((unsigned)(need < 4096 ? need : 4096));
    if (a.d % kUnit<T> == 0)
        HY_LAUNCH(kernel_label("hyena_loss_pack", type_label<T>(), true), (hyena_loss_pack<T, true>), pgrid, dim3(256), 0, s, a);
    else
        HY_LAUNCH(kernel_label("hyena_loss_pack", type_label<T>(), false), (hyena_loss_pack<T, false>), pgrid, dim3(256), 0, s, a);
    return launched();
}

template <typename T, int N, bool GRAD, bool OWN> hyena_status loss_few(const LossArgs& a, int tiles, hipStream_t s)
{
    const dim3 grid((unsigned)tiles, (unsigned)((a.total + 16 * N - 1) / (16 * N)));
    HY_LAUNCH(kernel_label("hyena_loss_few", type_label<T>(), N, GRAD, OWN), (hyena_loss_few<T, N, GRAD, OWN>), grid, dim3(256), 0, s, a);
    return launched();
}

// Whether the logits' kernel of a forward pass finds the tokens by itself.
template <typename T> bool finds_tokens(const LossArgs& a, bool units) { return a.few && units && a.total <= (LossType<T>::P == 1 ? 32 : 16); }

template <typename T, bool GRAD> hyena_status loss_logits(const LossArgs& a, bool units, int tiles, hipStream_t s)
{
    if (!a.few) {
        const int token_tiles = (int)(a.tokens / (a.small ? kSmallTile : kLossTokens));
        const dim3 grid((unsigned)(deal_tokens(tiles, token_tiles) ? dealt(tiles, token_tiles) : dealt(token_tiles, tiles)));
        if (a.small)
            HY_LAUNCH(kernel_label("hyena_loss_logits", type_label<T>(), GRAD, true), (hyena_loss_logits<T, GRAD, true>), grid, dim3((LogitsTile<T, true>::kThreads)), 0, s, a, tiles);
        else
            HY_LAUNCH(kernel_label("hyena_loss_logits", type_label<T>(), GRAD, false), (hyena_loss_logits<T, GRAD, false>), grid, dim3((LogitsTile<T, false>::kThreads)), 0, s, a, tiles);
        return launched();
    }
    if constexpr (GRAD) {
        return loss_few<T, 1, true, false>(a, tiles, s);
    } else {
        if (finds_tokens<T>(a, units)) {
            if constexpr (LossType<T>::P == 1)
                if (a.total > 16) return loss_few<T, 2, false, true>(a, tiles, s);
            return loss_few<T, 1, false, true>(a, tiles, s);
        }
        if constexpr (LossType<T>::P == 3)
            if (a.total > 32) return loss_few<T, 4, false, false>(a, tiles, s);
        return a.total > 16 ? loss_few<T, 2, false, false>(a, tiles, s) : loss_few<T, 1, false, false>(a, tiles, s);
    }
}

template <typename T, int N> hyena_status loss_few_grads(const LossArgs& a, hipStream_t s)
{
    const dim3 grid((unsigned)a.splits, (unsigned)((a.d + 255) / 256));
    if (a.d % 4 == 0)
        HY_LAUNCH(kernel_label("hyena_loss_few_grads", type_label<T>(), N, true), (hyena_loss_few_grads<T, N, true>), grid, dim3(256), 0, s, a);
    else
        HY_LAUNCH(kernel_label("hyena_loss_few_grads", type_label<T>(), N, false), (hyena_loss_few_grads<T, N, false>), grid, dim3(256), 0, s, a);
    return launched();
}

template <typename T> hyena_status loss_forward(const LossArgs& a, bool pack, bool units, hipStream_t s)
{
    hyena_status st = HYENA_OK;
    if (!finds_tokens<T>(a, units)) st = loss_begin<T, false>(a, pack, units, s);
    if (st != HYENA_OK) return st;
    LossArgs b = a;
    for (int64_t first = 0; first < a.V; first += a.chunk) {
        b.first = (int32_t)first;
        const bool last = first + a.chunk >= a.V;
        const int tiles = a.few ? few_groups(a.V) : loss_tiles(last ? a.V - first : a.chunk, a.small);
        if ((st = loss_logits<T, false>(b, units, tiles, s)) != HYENA_OK) return st;
        if (tiles > 16)
            HY_LAUNCH(kernel_label("hyena_loss_join", type_label<T>(), 16), (hyena_loss_join<T, 16>), dim3((unsigned)((a.total + 15) / 16)), dim3(1024), 0, s, b, tiles, last);
        else
            HY_LAUNCH(kernel_label("hyena_loss_join", type_label<T>(), 256), (hyena_loss_join<T, 256>), dim3((unsigned)((a.total + 255) / 256)), dim3(1024), 0, s, b, tiles, last);
        if ((st = launched()) != HYENA_OK) return st;
    }
    return HYENA_OK;
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
        if ((st = loss_logits<T, true>(b, units, a.few ? few_groups(a.V) : loss_tiles(values, a.small), s)) != HYENA_OK) return st;
        if (a.few) {  // all of the vocabulary is one piece
            if (a.total <= 4) st = loss_few_grads<T, 4>(a, s);
            else if (a.total <= 8) st = loss_few_grads<T, 8>(a, s);
            else if constexpr (LossType<T>::P == 3) st = loss_few_grads<T, 16>(a, s);
            if (st != HYENA_OK) return st;
            break;
        }
        const int64_t table_tiles = a.d_table ? dealt(channel_tiles, (int64_t)((values + kGradRows - 1) / kGradRows) * a.table_splits) : 0;
        const int64_t dx_tiles = a.d_x ? dealt(channel_tiles, a.splits * (a.tokens / kGradRows)) : 0;
        HY_LAUNCH(kernel_label("hyena_loss_products", type_label<T>()), hyena_loss_products<T>, dim3((unsigned)(table_tiles + dx_tiles)),
                  dim3(LossType<T>::kThreads), 0, s, b, (int)table_tiles, channel_tiles);
        if ((st = launched()) != HYENA_OK) return st;
        if (a.d_table == nullptr || a.table_splits == 1) continue;
        HY_LAUNCH(kernel_label("hyena_loss_table", type_label<T>()), hyena_loss_table<T>, dim3((unsigned)values, (unsigned)((a.d + 255) / 256)),
                  dim3(1024), 0, s, b);
        if ((st = launched()) != HYENA_OK) return st;
    }
    if (a.d_x == nullptr) return HYENA_OK;
    if (a.direct) {
        const int64_t groups = (a.total + 255) / 256;
        HY_LAUNCH(kernel_label("hyena_loss_zeros", type_label<T>()), hyena_loss_zeros<T>, dim3((unsigned)(groups < 4096 ? groups : 4096)), dim3(256), 0, s, a);
        return launched();
    }
    const int tokens = a.total < kFinishTokens ? 1 : 4;  // of a wave
    const int64_t need = a.splits <= 8 ? (a.total + 4 * tokens - 1) / (4 * tokens) : a.total;
    const dim3 grid((unsigned)(need < 4096 ? need : 4096));
    if (a.splits <= 8 && tokens == 1)
        HY_LAUNCH(kernel_label("hyena_loss_finish", type_label<T>(), 1), (hyena_loss_finish<T, 1>), grid, dim3(256), 0, s, a);
    else if (a.splits <= 8)
        HY_LAUNCH(kernel_label("hyena_loss_finish", type_label<T>(), 4), (hyena_loss_finish<T, 4>), grid, dim3(256), 0, s, a);
    else
        HY_LAUNCH(kernel_label("hyena_loss_finish_few", type_label<T>()), hyena_loss_finish_few<T>, dim3(grid.x, (unsigned)((a.d + 255) / 256)), dim3(1024), 0, s, a);
    return launched();
}

}  // namespace hy

#define HY_LOSS_INSTANTIATE(T)                                                                  \
    namespace hy {                                                                             \
    template hyena_status loss_forward<T>(const LossArgs&, bool, bool, hipStream_t);            \
    template hyena_status loss_backward<T>(const LossArgs&, bool, bool, hipStream_t);           \
    }
