// recurrence_device.h -- building blocks of the gated linear recurrence's
// kernels: matrix fragments, operand splitting, tile loads and the decays of
// a chunk of tokens.
//
// Matrix products.  Every product runs on 16 x 16 MFMA tiles whose operands
// are fragments of 8 contraction slots per lane: lane l holds row (or column)
// l % 16 and slots 8 (l / 16) + 0..7 of a block of 32.  16-bit types use one
// 16x16x32 instruction per block; float32 uses eight 16x16x4 ones, instruction
// e taking slot e of every lane, so that both have the same fragments and the
// kernels are one template.  A tile of results has row 4 (l / 16) + r and
// column l % 16 in register r.
//
// The order of the slots is free as long as both operands agree.  A pair of
// result tiles (rows 32 b .. 32 b + 31 of, say, the state) is therefore used
// as an operand straight from its registers: lane l holds rows 4g + r and
// 16 + 4g + r (g = l / 16) of its column, and the other operand's channels are
// stored in LDS in that order (perm4 below).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace hy {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

// Storage type T (float, uint16_t for bfloat16, _Float16): fragment and
// 4-vector types, conversions with round to nearest even.
//
// kTerms / split: how many fragments of T carry a float32 operand to float32
// accuracy: 8 bits each for bfloat16 (three), 11 for binary16 (two, the second
// scaled by 2^11 so that it stays above the subnormals).
template <typename T> struct Mx;

template <> struct Mx<float> {
    using frag = f32x8;
    using vec4 = f32x4;
    static constexpr int kTerms = 1;
    static __device__ __forceinline__ f32x4 widen(vec4 x) { return x; }
    static __device__ __forceinline__ vec4 narrow(f32x4 x) { return x; }
    static __device__ __forceinline__ f32x8 widen8(frag x) { return x; }
    static __device__ __forceinline__ frag narrow8(f32x8 x) { return x; }
    static __device__ __forceinline__ f32x4 mma(frag a, frag b, f32x4 c)
    {
#pragma unroll
        for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
        return c;
    }
};

template <> struct Mx<uint16_t> {
    using frag = bf16x8;
    using vec4 = bf16x4;
    static constexpr int kTerms = 3;
    static __device__ __forceinline__ f32x4 widen(vec4 x) { return __builtin_convertvector(x, f32x4); }
    static __device__ __forceinline__ vec4 narrow(f32x4 x) { return __builtin_convertvector(x, bf16x4); }
    static __device__ __forceinline__ f32x8 widen8(frag x) { return __builtin_convertvector(x, f32x8); }
    static __device__ __forceinline__ frag narrow8(f32x8 x) { return __builtin_convertvector(x, bf16x8); }
    static __device__ __forceinline__ f32x4 mma(frag a, frag b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};

template <> struct Mx<_Float16> {
    using frag = f16x8;
    using vec4 = f16x4;
    static constexpr int kTerms = 2;
    static __device__ __forceinline__ f32x4 widen(vec4 x) { return __builtin_convertvector(x, f32x4); }
    static __device__ __forceinline__ vec4 narrow(f32x4 x) { return __builtin_convertvector(x, f16x4); }
    static __device__ __forceinline__ f32x8 widen8(frag x) { return __builtin_convertvector(x, f32x8); }
    static __device__ __forceinline__ frag narrow8(f32x8 x) { return __builtin_convertvector(x, f16x8); }
    static __device__ __forceinline__ f32x4 mma(frag a, frag b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};

// A float32 operand as NT fragments whose sum (binary16: first + 2^-11 second)
// is the operand: NT = kTerms keeps float32 accuracy, NT = 1 rounds to T.
template <typename T, int NT> struct Split {
    typename Mx<T>::frag f[NT];
    __device__ __forceinline__ void set(f32x8 x)
    {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            f[n] = Mx<T>::narrow8(x);
            if (n + 1 < NT) {
                x = x - Mx<T>::widen8(f[n]);
                if constexpr (sizeof(T) == 2 && Mx<T>::kTerms == 2) x = x * 2048.0f;
            }
        }
    }
};

// c + a * s for a split operand (on either side: the tile's orientation is set
// by the argument order, split operand first or second).
template <typename T, int NT, bool FIRST>
__device__ __forceinline__ f32x4 mma_split(const Split<T, NT>& s, typename Mx<T>::frag x, f32x4 c)
{
    if constexpr (Mx<T>::kTerms == 2 && NT == 2) {
        f32x4 t = {0.0f, 0.0f, 0.0f, 0.0f};
        t = FIRST ? Mx<T>::mma(s.f[1], x, t) : Mx<T>::mma(x, s.f[1], t);
        c = FIRST ? Mx<T>::mma(s.f[0], x, c) : Mx<T>::mma(x, s.f[0], c);
        return c + t * 0.00048828125f;
    } else {
#pragma unroll
        for (int n = NT - 1; n >= 0; --n) c = FIRST ? Mx<T>::mma(s.f[n], x, c) : Mx<T>::mma(x, s.f[n], c);
        return c;
    }
}

// s * all + x y^T summed over NB blocks; y is split and, for binary16, without
// the common factor `lead` of its decays, which may be far below its range.
template <typename T, int NT, int NB, typename F>
__device__ __forceinline__ f32x4 update(f32x4 s, float all, float lead, const Split<T, NT> (&y)[NB], F x)
{
    if constexpr (Mx<T>::kTerms == 2) {
        f32x4 t = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < NB; ++j) t = mma_split<T, NT, false>(y[j], x(j), t);
        return s * all + t * lead;
    } else {
        s = s * all;
#pragma unroll
        for (int j = 0; j < NB; ++j) s = mma_split<T, NT, false>(y[j], x(j), s);
        return s;
    }
}

// binary16 holds a state of up to 65504 only: as an operand it is scaled by
// 2^-10 (and always split in two, so that small states lose nothing).
template <typename T> struct StateScale { static constexpr float down = 1.0f, up = 1.0f; };
template <> struct StateScale<_Float16> { static constexpr float down = 0.0009765625f, up = 1024.0f; };

__device__ __forceinline__ f32x8 join8(f32x4 a, f32x4 b)
{
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Place, in a row stored in operand order, of the group of 4 channels 4 c ..
// 4 c + 3: within each block of 32, lane group g = c % 4 finds the channels
// 4g + r and 16 + 4g + r side by side.
__device__ __forceinline__ constexpr int perm4(int c)
{
    return (c >> 3) * 32 + (c & 3) * 8 + ((c >> 2) & 1) * 4;
}

template <typename T> __device__ __forceinline__ float load_one(const T* p)
{
    if constexpr (sizeof(T) == 2 && Mx<T>::kTerms == 3) return __uint_as_float((uint32_t)*p << 16);
    else return (float)*p;
}
template <typename T> __device__ __forceinline__ void store_one(T* p, float x)
{
    if constexpr (sizeof(T) == 2 && Mx<T>::kTerms == 3) *p = __builtin_bit_cast(uint16_t, (__bf16)x);
    else *p = (T)x;
}

// LDS rows are padded by 16 bytes.
template <typename T> constexpr int kPad = 16 / (int)sizeof(T);

// A strided tensor [B][N][heads][width] (strides in elements).
struct RView {
    const void* p;
    int64_t b, t, h;
    int32_t vec;  // rows of 4-channel groups can be read as one vector each
};

// C tokens x D channels of a tensor as blocks of 4 tokens x 4 channels, held
// in registers between the global load and the LDS store.
template <typename T, int C, int D, int THREADS> struct Tile {
    using vec4 = typename Mx<T>::vec4;
    static constexpr int kBlocks = (C / 4) * (D / 4);
    static constexpr int kPer = (kBlocks + THREADS - 1) / THREADS;
    vec4 x[kPer][4];

    // tokens t0 .. t0 + C - 1 of the row whose first element is `base`; tokens
    // at n_valid and after it, and channels at `width` and after it, are zero
    // and not read
    __device__ __forceinline__ void load(const T* base, int64_t stride, int vec, int64_t t0,
                                         int64_t n_valid, int width, int tid)
    {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int b = tid + i * THREADS;
            const int c = 4 * (b % (D / 4));
            const int64_t t = t0 + 4 * (b / (D / 4));
            const bool in = kBlocks % THREADS == 0 || b < kBlocks;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                vec4 v = {};
                if (in && t + r < n_valid && c < width) {
                    const T* q = base + (t + r) * stride + c;
                    if (vec) {
                        v = *(const vec4*)q;
                    } else {
                        T* e = (T*)&v;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (c + j < width) e[j] = q[j];
                    }
                }
                x[i][r] = v;
            }
        }
    }
    // rows[token][channel], channels in operand order (perm4)
    template <int LD> __device__ __forceinline__ void store_rows(T* lds, int tid) const
    {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int b = tid + i * THREADS;
            if (kBlocks % THREADS != 0 && b >= kBlocks) break;
            const int c = perm4(b % (D / 4)), t = 4 * (b / (D / 4));
#pragma unroll
            for (int r = 0; r < 4; ++r) *(vec4*)(lds + (t + r) * LD + c) = x[i][r];
        }
    }
    // cols[channel][token]
    template <int LD> __device__ __forceinline__ void store_cols(T* lds, int tid) const
    {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int b = tid + i * THREADS;
            if (kBlocks % THREADS != 0 && b >= kBlocks) break;
            const int c = 4 * (b % (D / 4)), t = 4 * (b / (D / 4));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                vec4 v = {x[i][0][j], x[i][1][j], x[i][2][j], x[i][3][j]};
                *(vec4*)(lds + (c + j) * LD + t) = v;
            }
        }
    }
};

template <typename T>
__device__ __forceinline__ typename Mx<T>::frag frag_at(const T* lds)
{
    if constexpr (sizeof(T) == 4) return join8(*(const f32x4*)lds, *(const f32x4*)(lds + 4));
    else return *(const typename Mx<T>::frag*)lds;
}

// The decays of one chunk, in LDS.  logs: sum of the log2 decays up to and
// with each token, float64 (differences of sums of up to 64 terms keep float32
// accuracy); count: resets so far (a reset's own log counts as 0; a pair of
// tokens with a reset between them has factor 0); head: from the chunk's start
// through each token; tail: from after each token to the chunk's end; inner:
// from after the chunk's first token through each, head[i] = head[0] inner[i].
template <int C> struct alignas(16) Decays {
    double logs[C];
    int count[C];
    float head[C], tail[C], inner[C];
};

// exp2 of anything below this is no normal float32 (v_exp_f32 gives 0)
constexpr float kResetLog2 = -126.0f;

__device__ __forceinline__ double shfl_up_f64(double x, int d)
{
    const int2 v = __builtin_bit_cast(int2, x);
    return __builtin_bit_cast(double, make_int2(__shfl_up(v.x, d), __shfl_up(v.y, d)));
}

// One wave fills the decays of a chunk from its log decay per lane (lane =
// token, 0 where the token does not exist).
template <int C>
__device__ __forceinline__ void fill_decays(Decays<C>& d, float g, int lane)
{
    const float l2 = g * 1.44269504088896340736f;
    const bool reset = l2 < kResetLog2;
    const unsigned long long resets = __ballot(reset && lane < C);
    double s = reset ? 0.0 : (double)g * 1.44269504088896340736;
#pragma unroll
    for (int k = 1; k < C; k <<= 1) {
        const double o = shfl_up_f64(s, k);
        if (lane >= k) s += o;
    }
    const int2 sv = __builtin_bit_cast(int2, s);
    const double end = __builtin_bit_cast(double, make_int2(__shfl(sv.x, C - 1), __shfl(sv.y, C - 1)));
    const double first = __builtin_bit_cast(double, make_int2(__shfl(sv.x, 0), __shfl(sv.y, 0)));
    const int first_count = (int)(resets & 1);
    const int before = __popcll(resets & (~0ull >> (63 - lane)));
    const int all = __popcll(resets);
    if (lane < C) {
        d.logs[lane] = s;
        d.count[lane] = before;
        d.head[lane] = before == 0 ? __builtin_amdgcn_exp2f((float)s) : 0.0f;
        d.inner[lane] = before == first_count ? __builtin_amdgcn_exp2f((float)(s - first)) : 0.0f;
        d.tail[lane] = before == all ? __builtin_amdgcn_exp2f((float)(end - s)) : 0.0f;
    }
}

// Decay from after token j through token i >= j of a chunk.
template <int C>
__device__ __forceinline__ float pair_decay(const Decays<C>& d, double log_i, int count_i, int j)
{
    return count_i == d.count[j] ? __builtin_amdgcn_exp2f((float)(log_i - d.logs[j])) : 0.0f;
}

__device__ __forceinline__ int64_t valid_tokens(const int32_t* lengths, int64_t b, int64_t N)
{
    if (lengths == nullptr) return N;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : n < N ? n : N;
}

}  // namespace hy
