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
typedef int i32x4 __attribute__((ext_vector_type(4)));
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
// scaled by 2^11 so that it stays above the subnormals; see Fit for its range).
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
// bfloat16 terms before the last are cut, not rounded: the upper half of the
// word, then that of the exact remainder; three cut terms are all 24 bits.
template <typename T, int NT> struct Split {
    typename Mx<T>::frag f[NT];
    __device__ __forceinline__ void set(f32x8 x)
    {
        if constexpr (Mx<T>::kTerms == 3 && NT > 1) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (n + 1 == NT && NT < 3) {
                    f[n] = Mx<T>::narrow8(x);
                    break;
                }
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)  // the upper halves of two words
                    w[e] = __builtin_amdgcn_perm(__float_as_uint(x[2 * e + 1]), __float_as_uint(x[2 * e]), 0x07060302);
                f[n] = __builtin_bit_cast(typename Mx<T>::frag, w);
                if (n + 1 < NT) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] -= __uint_as_float(__float_as_uint(x[e]) & 0xffff0000u);
                }
            }
        } else {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                f[n] = Mx<T>::narrow8(x);
                if (n + 1 < NT) x = (x - Mx<T>::widen8(f[n])) * 2048.0f;
            }
        }
    }
};

// Four values as NT vectors whose sum (binary16: first + 2^-11 second) is the
// values, as above but rounded; stored in LDS `apart` elements from each other.
template <typename T, int NT> struct Split4 {
    typename Mx<T>::vec4 y[NT];
    __device__ __forceinline__ void set(f32x4 x)
    {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            y[n] = Mx<T>::narrow(x);
            if (n + 1 < NT) x = (x - Mx<T>::widen(y[n])) * (Mx<T>::kTerms == 2 ? 2048.0f : 1.0f);
        }
    }
};
template <typename T, int NT> __device__ __forceinline__ void store_split(T* to, int apart, f32x4 x)
{
    Split4<T, NT> s;
    s.set(x);
#pragma unroll
    for (int n = 0; n < NT; ++n) *(typename Mx<T>::vec4*)(to + n * apart) = s.y[n];
}

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

// binary16 holds 2^-24 .. 65504 only, 11 bits from 2^-14 on.  The columns of a
// float32 operand are brought there by a power of two each, made of the column's
// largest magnitude, and their results taken back: what is lost is below 2^-36 of
// that, wherever a state or a decay is.  down leaves the largest in 2^14 .. 2^15;
// up = 1 / down.  Nothing for the other types, whose exponents are float32's.
struct Fit {
    float down, up;
    __device__ __forceinline__ explicit Fit(float largest)
    {
        uint32_t e = __float_as_uint(largest) >> 23;
        e = e < 15 ? 15 : e;  // up is normal
        down = __uint_as_float((268 - e) << 23);
        up = __uint_as_float((e - 14) << 23);
    }
};
template <typename T> constexpr bool kFit = Mx<T>::kTerms == 2;

// Largest over the four lanes l, l ^ 16, l ^ 32, l ^ 48, in each of them: the rows
// of a fragment's column are in these lanes.
__device__ __forceinline__ float max_rows(float x)
{
    typedef uint32_t u32x2_ __attribute__((ext_vector_type(2)));
    u32x2_ s = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
    s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}

// NB fragments of one operand, value(j) the j-th in float32, split; returns what
// the results of their columns (a lane's own) are to be multiplied by.
template <typename T, int NT, int NB, typename F>
__device__ __forceinline__ float split_columns(Split<T, NT> (&y)[NB], F value)
{
    if constexpr (kFit<T>) {
        f32x8 x[NB];
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            x[j] = value(j);
#pragma unroll
            for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[j][e]));
        }
        const Fit fit(max_rows(m));
#pragma unroll
        for (int j = 0; j < NB; ++j) y[j].set(x[j] * fit.down);
        return fit.up;
    } else {
#pragma unroll
        for (int j = 0; j < NB; ++j) y[j].set(value(j));
        return 1.0f;
    }
}

// s * all + x y^T summed over NB blocks; up: of split_columns.
template <typename T, int NT, int NB, typename F>
__device__ __forceinline__ f32x4 update(f32x4 s, float all, float up, const Split<T, NT> (&y)[NB], F x)
{
    if constexpr (kFit<T>) {
        f32x4 t = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < NB; ++j) t = mma_split<T, NT, false>(y[j], x(j), t);
        return s * all + t * up;
    } else {
        s = s * all;
#pragma unroll
        for (int j = 0; j < NB; ++j) s = mma_split<T, NT, false>(y[j], x(j), s);
        return s;
    }
}

// A tile column of a state as an operand: M 16 x 16 tiles of registers, tile(m) the
// m-th.  down: for its operands; up: for results whose rows are its columns.
template <typename T> struct StateFit {
    float down = 1.0f;
    f32x4 up = {1.0f, 1.0f, 1.0f, 1.0f};
    template <int M, typename F> __device__ __forceinline__ void set(F tile, int grp)
    {
        if constexpr (kFit<T>) {
            float m = 0.0f;
#pragma unroll
            for (int x = 0; x < M; ++x)
#pragma unroll
                for (int r = 0; r < 4; ++r) m = fmaxf(m, fabsf(tile(x)[r]));
            const Fit fit(max_rows(m));
            down = fit.down;
#pragma unroll
            for (int r = 0; r < 4; ++r) up[r] = __shfl(fit.up, 4 * grp + r);
        }
    }
    __device__ __forceinline__ f32x8 fitted(f32x8 x) const
    {
        if constexpr (kFit<T>) return x * down;
        else return x;
    }
    // a tile of results times f
    __device__ __forceinline__ f32x4 results(f32x4 x, float f) const
    {
        if constexpr (kFit<T>) return x * (up * f);
        else return x * f;
    }
};

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
    int32_t vec;  // kRowVectors, kRowPairs or kRowElements
};
// What a row is read by: its 16-byte groups are whole, aligned vectors; the same
// of pairs of elements; or anything.  (2 x 4096 tokens, 8 heads of 62 in bf16:
// forward 43 us by elements, 34 by pairs; heads of 64 by vectors 30.)
enum : int32_t { kRowElements = 0, kRowPairs = 1, kRowVectors = 2 };

// Rows of one (batch row, head) of a tensor, read and written through a buffer
// descriptor: an access whose offset is kOutside is dropped (a load gives 0),
// so what a mask leaves out costs a select and no branch, and all loads of a
// tile are under way together.
constexpr uint32_t kOutside = 0xffffffffu;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_at(const void* p)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, 0x7fffffff, 0x00020000);
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <typename T>
__device__ __forceinline__ typename Mx<T>::vec4 load4(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t scalar = 0)
{
    if constexpr (sizeof(T) == 4)
        return __builtin_bit_cast(typename Mx<T>::vec4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, (int)scalar, 0));
    else
        return __builtin_bit_cast(typename Mx<T>::vec4, __builtin_amdgcn_raw_buffer_load_b64(r, (int)off, (int)scalar, 0));
}
// Stores take their whole offset in a vector register: after a 16-byte store
// with a scalar offset the compiler puts no wait before an instruction that
// overwrites the stored registers, and such a store was seen to write the new
// value.
template <typename T>
__device__ __forceinline__ void store4(__amdgpu_buffer_rsrc_t r, uint32_t off, typename Mx<T>::vec4 x)
{
    if constexpr (sizeof(T) == 4)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), r, (int)off, 0, 0);
    else
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, x), r, (int)off, 0, 0);
}
template <typename T> __device__ __forceinline__ T load1(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t scalar = 0)
{
    if constexpr (sizeof(T) == 4) return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, (int)scalar, 0));
    else return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b16(r, (int)off, (int)scalar, 0));
}
// two elements that make an aligned pair
template <typename T> __device__ __forceinline__ void load2(T* e, __amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t scalar = 0)
{
    if constexpr (sizeof(T) == 4) {
        const u32x2 x = __builtin_amdgcn_raw_buffer_load_b64(r, (int)off, (int)scalar, 0);
        e[0] = __builtin_bit_cast(T, (uint32_t)x[0]);
        e[1] = __builtin_bit_cast(T, (uint32_t)x[1]);
    } else {
        const uint32_t x = __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, (int)scalar, 0);
        e[0] = __builtin_bit_cast(T, (uint16_t)(x & 0xffff));
        e[1] = __builtin_bit_cast(T, (uint16_t)(x >> 16));
    }
}
template <typename T> __device__ __forceinline__ void store1(__amdgpu_buffer_rsrc_t r, uint32_t off, T x)
{
    if constexpr (sizeof(T) == 4) __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, x), r, (int)off, 0, 0);
    else __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, x), r, (int)off, 0, 0);
}

// 4 channels from `ch` on of the row at byte `off`; width: the row's channels.
template <typename T>
__device__ __forceinline__ void store_row4(__amdgpu_buffer_rsrc_t r, uint32_t off, bool in, int ch, int width, f32x4 x)
{
    const typename Mx<T>::vec4 y = Mx<T>::narrow(x);
    if ((width & 3) == 0) {
        store4<T>(r, in & (ch < width) ? off + ch * (uint32_t)sizeof(T) : kOutside, y);
    } else if ((width & 1) == 0) {
        const u32x2* e = (const u32x2*)&y;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t at = in & (ch + 2 * j < width) ? off + (ch + 2 * j) * (uint32_t)sizeof(T) : kOutside;
            if constexpr (sizeof(T) == 4) __builtin_amdgcn_raw_buffer_store_b64(e[j], r, (int)at, 0, 0);
            else __builtin_amdgcn_raw_buffer_store_b32((*e)[j], r, (int)at, 0, 0);
        }
    } else {
        const T* e = (const T*)&y;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            store1<T>(r, in & (ch + j < width) ? off + (ch + j) * (uint32_t)sizeof(T) : kOutside, e[j]);
    }
}

// The same value, newly made: what is computed from it stays in the loop it is
// used in, instead of in a register of its own (or in scratch) through all of it.
__device__ __forceinline__ int again(int x)
{
    asm volatile("" : "+v"(x));
    return x;
}
__device__ __forceinline__ int again_uniform(int x)
{
    asm volatile("" : "+s"(x));
    return x;
}

// The rows of one (batch row, head), walked a chunk at a time; step: bytes from
// token to token (token strides are below 2^23 elements).
struct Stream {
    const char* p;
    uint32_t step;
    int32_t vec;
    template <typename T> __device__ __forceinline__ void start(const RView& v, int64_t b, int64_t h, int64_t t)
    {
        p = (const char*)v.p + (b * v.b + h * v.h + t * v.t) * (int64_t)sizeof(T);
        step = (uint32_t)v.t * (uint32_t)sizeof(T);
        vec = v.vec;
    }
    __device__ __forceinline__ void move(int tokens) { p += (int64_t)tokens * (int64_t)step; }
};

// Place of (channel, token) in a transposed tile: rows of C tokens are 128 bytes,
// eight units of 16.  Unit u of a row is kept at u ^ key: eight rows in turn, and
// every fourth of 32, have eight keys, so that the column stores of a tile (every
// fourth row) and the fragment loads (16 rows in turn) spread over the banks.  By units
// (float32) they do not conflict; the 8-byte stores of 16-bit types do: 29% of the
// LDS cycles of hyena_rec_states.
template <typename T, int C> __device__ __forceinline__ int col_at(int channel, int token)
{
    constexpr int U = 16 / (int)sizeof(T);
    static_assert(C * sizeof(T) == 128, "a row is eight units");
    return channel * C + (((token / U) ^ ((channel ^ (channel >> 3)) & 7)) * U) + token % U;
}

// C tokens x D channels of a tensor, held in registers between the global load
// and the LDS store as blocks of R tokens x W channels, W channels being 16
// bytes: lanes follow the rows, so that a load instruction asks for whole
// 128-byte lines (with 64-byte pieces of rows, and 8-byte loads, the reading
// rate fell from 5.8 to 4.0 TB/s).  Blocks of 4 tokens can be stored transposed.
template <typename T, int C, int D, int THREADS, int R> struct Tile {
    using vec4 = typename Mx<T>::vec4;
    static constexpr int W = 16 / (int)sizeof(T), V = W / 4;
    static constexpr int kBlocks = (C / R) * (D / W);
    static constexpr int kPer = (kBlocks + THREADS - 1) / THREADS;
    vec4 x[kPer][R][V];

    static __device__ __forceinline__ int token(int b) { return R * (b / (D / W)); }
    static __device__ __forceinline__ int channel(int b) { return W * (b % (D / W)); }

    // Byte offsets of a thread's blocks from the stream's place: kept through the
    // loop, kOutside where the block's channels do not exist.
    struct Places {
        uint32_t off[kPer];
        __device__ __forceinline__ Places(const Stream& s, int width, int tid)
        {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int b = tid + i * THREADS;
                const bool in = (kBlocks % THREADS == 0 || b < kBlocks) && channel(b) < width;
                off[i] = in ? (uint32_t)token(b) * s.step + (uint32_t)channel(b) * (uint32_t)sizeof(T) : kOutside;
            }
        }
    };

    // The first n tokens of the stream from its place on; tokens at n and after
    // it, and channels at `width` and after it, are zero and not read.  VEC:
    // known to be kRowVectors.
    template <bool VEC> __device__ __forceinline__ void load(const Stream& s, const Places& at, int n, int width, int tid)
    {
        const __amdgpu_buffer_rsrc_t rsrc = rows_at(s.p);
        // each block's rows by `one`, of its registers, byte offset and first channel
        auto blocks = [&](auto one) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int t = token(tid + i * THREADS), c = channel(tid + i * THREADS);
#pragma unroll
                for (int r = 0; r < R; ++r) one(x[i][r], t + r < n ? at.off[i] : kOutside, c, r * s.step);
            }
        };
        if (VEC || s.vec == kRowVectors) {
            blocks([&](vec4* to, uint32_t off, int, uint32_t scalar) {
                *(u32x4*)to = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, (int)off, (int)scalar, 0));
            });
        } else if (s.vec == kRowPairs) {
            blocks([&](vec4* to, uint32_t off, int c, uint32_t scalar) {
                T e[W];
#pragma unroll
                for (int j = 0; j < W; j += 2)
                    load2<T>(e + j, rsrc, (c + j < width) & (off != kOutside) ? off + j * (uint32_t)sizeof(T) : kOutside, scalar);
#pragma unroll
                for (int v = 0; v < V; ++v) to[v] = *(const vec4*)(e + 4 * v);
            });
        } else {
            blocks([&](vec4* to, uint32_t off, int c, uint32_t scalar) {
                T e[W];
#pragma unroll
                for (int j = 0; j < W; ++j)
                    e[j] = load1<T>(rsrc, (c + j < width) & (off != kOutside) ? off + j * (uint32_t)sizeof(T) : kOutside, scalar);
#pragma unroll
                for (int v = 0; v < V; ++v) to[v] = *(const vec4*)(e + 4 * v);
            });
        }
    }
    // rows[token][channel], channels in operand order (perm4)
    template <int LD> __device__ __forceinline__ void store_rows(T* lds, int tid) const
    {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int b = tid + i * THREADS;
            if (kBlocks % THREADS != 0 && b >= kBlocks) break;
            const int c = channel(b), t = token(b);
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int v = 0; v < V; ++v) *(vec4*)(lds + (t + r) * LD + perm4(c / 4 + v)) = x[i][r][v];
        }
    }
    // cols[channel][token], in units of 16 bytes swapped within a row (col_at)
    __device__ __forceinline__ void store_cols(T* lds, int tid) const
    {
        static_assert(R == 4, "a column's piece is a vector");
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int b = tid + i * THREADS;
            if (kBlocks % THREADS != 0 && b >= kBlocks) break;
            const int c = channel(b), t = token(b);
#pragma unroll
            for (int j = 0; j < W; ++j) {
                vec4 v = {x[i][0][j / 4][j % 4], x[i][1][j / 4][j % 4], x[i][2][j / 4][j % 4], x[i][3][j / 4][j % 4]};
                *(vec4*)(lds + col_at<T, C>(c + j, t)) = v;
            }
        }
    }
};

// The elements of a tensor under a tile of results (column = token 16 i + l16,
// rows = channels 16 t + 4 grp ..), read straight into that place.
template <typename T, int IT, int CW> struct UnderResults {
    typename Mx<T>::vec4 x[IT][CW];
    template <bool VEC>
    __device__ __forceinline__ void load(const Stream& s, int n, int width, int l16, int grp, int wave)
    {
        const __amdgpu_buffer_rsrc_t rsrc = rows_at(s.p);
#pragma unroll
        for (int i = 0; i < IT; ++i)
#pragma unroll
            for (int v = 0; v < CW; ++v) {
                const int c = 16 * (wave + 4 * v) + 4 * grp;
                const uint32_t off = (uint32_t)l16 * s.step + (uint32_t)c * (uint32_t)sizeof(T);
                const bool in = 16 * i + l16 < n;
                if (VEC || s.vec == kRowVectors) {
                    x[i][v] = load4<T>(rsrc, in & (c < width) ? off : kOutside, 16 * i * s.step);
                } else if (s.vec == kRowPairs) {
                    T e[4];
#pragma unroll
                    for (int j = 0; j < 4; j += 2)
                        load2<T>(e + j, rsrc, in & (c + j < width) ? off + j * (uint32_t)sizeof(T) : kOutside, 16 * i * s.step);
                    x[i][v] = *(const typename Mx<T>::vec4*)e;
                } else {
                    T e[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        e[j] = load1<T>(rsrc, in & (c + j < width) ? off + j * (uint32_t)sizeof(T) : kOutside, 16 * i * s.step);
                    x[i][v] = *(const typename Mx<T>::vec4*)e;
                }
            }
    }
};

// Fragments of a transposed tile: 8 tokens 32 j + 8 grp .. of the row 16 k + l16.
// Of the key only bits of k and j change from fragment to fragment, so four
// places per lane serve all of them (float32: and their neighbours, unit ^ 1).
template <typename T, int C> struct ColFrags {
    static constexpr int U = 16 / (int)sizeof(T);
    uint32_t at[4];
    __device__ __forceinline__ ColFrags(int l16, int grp)
    {
#pragma unroll
        for (int x = 0; x < 4; ++x)
            at[x] = l16 * C + (((grp * (8 / U)) ^ ((l16 ^ (l16 >> 3)) & 7) ^ (2 * x)) & 7) * U;
    }
    static __device__ __forceinline__ typename Mx<T>::frag load(const T* lds, uint32_t p)
    {
        if constexpr (sizeof(T) == 4) return join8(*(const f32x4*)(lds + p), *(const f32x4*)(lds + (p ^ 4)));
        else return *(const typename Mx<T>::frag*)(lds + p);
    }
    // k and j known to the compiler
    __device__ __forceinline__ typename Mx<T>::frag operator()(const T* lds, int k, int j) const
    {
        return load(lds, at[(k ^ (2 * j)) & 3] + 16 * k * C);
    }
    // any k
    __device__ __forceinline__ typename Mx<T>::frag any(const T* lds, int k, int j) const
    {
        return load(lds, (at[0] ^ (2 * ((k ^ (2 * j)) & 3) * U)) + 16 * k * C);
    }
};

template <typename T>
__device__ __forceinline__ typename Mx<T>::frag frag_at(const T* lds)
{
    if constexpr (sizeof(T) == 4) return join8(*(const f32x4*)lds, *(const f32x4*)(lds + 4));
    else return *(const typename Mx<T>::frag*)lds;
}

// The decays of one chunk, in LDS.  A pair of tokens i >= j of different 16-token
// tiles has the factor within[i] cross[i / 16 - 1][j]: from the tile's start
// through i, and from after j to that start.  Pairs of one tile take the
// difference of logs: sums of the log2 decays from the chunk's start, float64, so
// that differences of up to 64 terms keep float32 accuracy.  A reset's own log
// counts as 0; count is the number of resets so far, and a factor that spans one
// is 0.  head: from the chunk's start through each token; tail: from after each
// token to the chunk's end.
template <int C> struct alignas(16) Decays {
    double logs[C];
    int count[C];
    float head[C], tail[C], within[C];
    float cross[C / 16 - 1][C];
    unsigned long long resets;  // bit per token
};

// exp2 of anything below this is no normal float32 (v_exp_f32 gives 0)
constexpr float kResetLog2 = -126.0f;

// Cross-lane sums by DPP and lane swaps: they cost an instruction or two each,
// where a shuffle through the LDS crossbar costs its latency.
template <int CTRL, int ROWS> __device__ __forceinline__ double dpp_f64(double x)
{
    const int2 v = __builtin_bit_cast(int2, x);
    return __builtin_bit_cast(double, make_int2(__builtin_amdgcn_update_dpp(0, v.x, CTRL, ROWS, 0xf, false),
                                                __builtin_amdgcn_update_dpp(0, v.y, CTRL, ROWS, 0xf, false)));
}
// sum over lanes 0 .. lane
__device__ __forceinline__ double scan_f64(double x)
{
    x += dpp_f64<0x111, 0xf>(x);  // row_shr 1, 2, 4, 8: within 16 lanes
    x += dpp_f64<0x112, 0xf>(x);
    x += dpp_f64<0x114, 0xf>(x);
    x += dpp_f64<0x118, 0xf>(x);
    x += dpp_f64<0x142, 0xa>(x);  // row_bcast 15, 31: the sums of the rows before
    x += dpp_f64<0x143, 0xc>(x);
    return x;
}
// The same over the last `span` lanes up to and with this one, where lanes between two
// borders all sum from the lower border on: a step adds a lower lane's sum if that
// lane is within the span, so what lies before a border is never added.
__device__ __forceinline__ double scan_spans_f64(double x, int span, int lane)
{
    auto add = [&](double y, int apart) { x += span > apart ? y : 0.0; };
    add(dpp_f64<0x111, 0xf>(x), 1);
    add(dpp_f64<0x112, 0xf>(x), 2);
    add(dpp_f64<0x114, 0xf>(x), 4);
    add(dpp_f64<0x118, 0xf>(x), 8);
    add(dpp_f64<0x142, 0xa>(x), (lane & 15) + 1);
    add(dpp_f64<0x143, 0xc>(x), lane - 31);
    return x;
}
__device__ __forceinline__ double lane_f64(double x, int lane)
{
    const int2 v = __builtin_bit_cast(int2, x);
    return __builtin_bit_cast(double, make_int2(__builtin_amdgcn_readlane(v.x, lane), __builtin_amdgcn_readlane(v.y, lane)));
}
template <int CTRL> __device__ __forceinline__ float dpp_f32(float x)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
// sum over the 16 lanes of a row, in each of them
__device__ __forceinline__ float sum16(float x)
{
    x += dpp_f32<0xb1>(x);   // quad_perm 1, 0, 3, 2
    x += dpp_f32<0x4e>(x);   // quad_perm 2, 3, 0, 1
    x += dpp_f32<0x141>(x);  // row_half_mirror
    x += dpp_f32<0x140>(x);  // row_mirror
    return x;
}
// sum over the four lanes l, l ^ 16, l ^ 32, l ^ 48, in each of them
__device__ __forceinline__ float sum_rows(float x)
{
    typedef uint32_t u32x2_ __attribute__((ext_vector_type(2)));
    u32x2_ s = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

// One wave fills the decays of a chunk from its log decay per lane (lane =
// token, 0 where the token does not exist).
template <int C>
__device__ __forceinline__ void fill_decays(Decays<C>& d, float g, int lane)
{
    const bool reset = g * 1.44269504088896340736f < kResetLog2;
    const unsigned long long resets = __ballot(reset && lane < C);
    const double s = scan_f64(reset ? 0.0 : (double)g * 1.44269504088896340736);
    // resets up to and with token t
    auto upto = [&](int t) { return __popcll(resets & (~0ull >> (63 - t))); };
    auto factor = [](bool same, double log) { return same ? __builtin_amdgcn_exp2f((float)log) : 0.0f; };
    const int count = upto(lane);
    double edge[C / 16];
#pragma unroll
    for (int i = 0; i < C / 16; ++i) edge[i] = lane_f64(s, 16 * i + 15);
    double before = 0.0;
    int count_before = 0;
#pragma unroll
    for (int i = 1; i < C / 16; ++i) {
        before = lane >= 16 * i ? edge[i - 1] : before;
        count_before = lane >= 16 * i ? upto(16 * i - 1) : count_before;
    }
    if (lane < C) {
        d.logs[lane] = s;
        d.count[lane] = count;
        d.head[lane] = factor(count == 0, s);
        d.tail[lane] = factor(count == upto(C - 1), edge[C / 16 - 1] - s);
        d.within[lane] = factor(count == count_before, s - before);
#pragma unroll
        for (int i = 1; i < C / 16; ++i)
            d.cross[i - 1][lane] = factor(lane < 16 * i && count == upto(16 * i - 1), edge[i - 1] - s);
        if (lane == 0) d.resets = resets;
    }
}

// The decays of kDecayBatch chunks at a time: wave w < kDecayBatch fills the
// w-th of a batch, so the scan's latency is paid once per batch.
constexpr int kDecayBatch = 2;

// First token of a segment: whole pieces of 64 tokens, spread evenly (segments
// differ by one piece at most, and every m-th segment of a cut into m n is a
// segment of the cut into n).
__device__ __forceinline__ int64_t segment_start(int64_t N, int nseg, int64_t seg)
{
    const int64_t t = seg * ((N + 63) / 64) / nseg * 64;
    return t < N ? t : N;
}

__device__ __forceinline__ int64_t valid_tokens(const int32_t* lengths, int64_t b, int64_t N)
{
    if (lengths == nullptr) return N;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : n < N ? n : N;
}

}  // namespace hy
