// matmul_device.h -- a tile of a matrix product of 16-bit operands on MFMA.
//
// C[m][n] = sum over k of A(m, k) B(n, k): a workgroup of WM x WN waves makes a
// tile of TM x TN, k in steps of 32.  An operand is stored with k or with its own
// axis contiguous; both go through LDS and come back as the fragments of 16x16x32
// instructions (8 values of k for each lane):
//   k contiguous:    an LDS row is 32 values of k, four 16-byte chunks; chunk c of
//                    row m is kept at c ^ ((m >> 1) & 3), so that the eight lanes
//                    that one cycle serves read eight different 16-byte slots;
//   axis contiguous: an LDS row is one k; its 32-byte blocks are kept at
//                    b ^ key(k), so that the four rows that 16 lanes read together
//                    lie in different banks.  ds_read_b64_tr_b16 turns 4 k x 16
//                    values on the way into the registers.
// A lane's results: row 4 (lane / 16) + r of a 16 x 16 tile, column lane % 16.
#pragma once

#include "recurrence_device.h"

namespace hy {

typedef short s16x4 __attribute__((ext_vector_type(4)));

// What a tile reads of one operand: `at` its first byte at k = 0, `end` the end of
// the memory (what lies there and after it is read as 0), `row` the bytes from one
// row of the storage to the next.
struct Operand {
    const char* at;
    const char* end;
    int64_t row;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t operand_rsrc(const char* at, const char* end)
{
    const int64_t left = end - at;
    const int n = left <= 0 ? 0 : left < 0x7fffffff ? (int)left : 0x7fffffff;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(at), (short)0, n, 0x00020000);
}

// One operand of a tile: W rows of the output's axis; KC: k contiguous.
template <int W, int THREADS, bool KC> struct Stage {
    static constexpr int kBytes = W * 64;           // of a step in LDS
    static constexpr int kLoads = W * 4 / THREADS;  // 16-byte loads of a thread
    static_assert(W * 4 % THREADS == 0 && W % 16 == 0, "");
    static constexpr int kRowChunks = KC ? 4 : W / 8;
    static constexpr int kBlocks = W / 16;          // 32-byte blocks of a row (axis contiguous)

    uint32_t off[kLoads];  // bytes from `at`
    u32x4 x[kLoads];

    __device__ __forceinline__ void init(int64_t row)
    {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int n = (int)threadIdx.x + i * THREADS;
            off[i] = (uint32_t)((n / kRowChunks) * (uint32_t)row + (n % kRowChunks) * 16);
        }
    }
    __device__ __forceinline__ void load(const char* at, const char* end)
    {
        const __amdgpu_buffer_rsrc_t r = operand_rsrc(at, end);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) x[i] = __builtin_amdgcn_raw_buffer_load_b128(r, (int)off[i], 0, 0);
    }
    // Bytes from one step's first value to the next one's.
    static __device__ __forceinline__ int64_t step(int64_t row) { return KC ? 64 : 32 * row; }
    static __device__ __forceinline__ int key(int k) { return (k & 3) | ((k >> 3) & 1) << 2; }
    __device__ __forceinline__ void store(char* lds) const
    {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int n = (int)threadIdx.x + i * THREADS, row = n / kRowChunks, c = n % kRowChunks;
            int at;
            if constexpr (KC) at = row * 64 + ((c ^ ((row >> 1) & 3)) * 16);
            else at = row * (W * 2) + ((((c >> 1) ^ (key(row) % kBlocks)) << 5) | (c & 1) << 4);
            *(u32x4*)(lds + at) = x[i];
        }
    }
    // The fragment of the 16 rows at m0.
    template <typename F> static __device__ __forceinline__ F fragment(const char* lds, int m0)
    {
        const int lane = threadIdx.x & 63;
        if constexpr (KC) {
            const int m = m0 + (lane & 15), c = lane >> 4;
            return *(const F*)(lds + m * 64 + ((c ^ ((m >> 1) & 3)) * 16));
        } else {
            typedef __attribute__((address_space(3))) s16x4* at3;
            const int g = lane >> 4, i = lane & 15;
            s16x4 v[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = g * 8 + h * 4 + (i >> 2);
                const char* p = lds + k * (W * 2) + (((m0 >> 4) ^ (key(k) % kBlocks)) << 5) + (i & 3) * 8;
                v[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((at3)p);
            }
            return __builtin_bit_cast(F, v);
        }
    }
};

// Which pieces of the operands are multiplied: with NP planes (float32 as three
// bfloat16 terms, largest first) the six largest of the products of two planes, the
// smallest first; with one plane that.
template <int NP> struct Planes {
    static constexpr int kPairs = NP == 1 ? 1 : 6;
    static __device__ __forceinline__ int a(int i) { return NP == 1 ? 0 : (0x001021 >> (4 * i)) & 15; }
    static __device__ __forceinline__ int b(int i) { return NP == 1 ? 0 : (0x010201 >> (4 * i)) & 15; }
};

// E: uint16_t (bfloat16) or _Float16.
template <typename E, int TM, int TN, int WM, int WN, bool AK, bool BK, int NP> struct MatTile {
    static constexpr int kThreads = WM * WN * 64;
    using A = Stage<TM, kThreads, AK>;
    using B = Stage<TN, kThreads, BK>;
    static constexpr int kStep = A::kBytes + B::kBytes, kLds = 2 * kStep;
    static constexpr int MI = TM / WM / 16, NI = TN / WN / 16;
    using frag = typename Mx<E>::frag;

    f32x4 c[MI][NI];

    // aplane, bplane: bytes between planes.  steps: of 32 values of k, at least 1.
    __device__ __forceinline__ void run(char* lds, const Operand& oa, int64_t aplane, const Operand& ob, int64_t bplane,
                                        int steps)
    {
        const int wave = threadIdx.x >> 6;
        const int m0 = wave / WN * (TM / WM), n0 = wave % WN * (TN / WN);
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) c[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        A a;
        B b;
        a.init(oa.row);
        b.init(ob.row);
        const int64_t astep = A::step(oa.row), bstep = B::step(ob.row);
        const int total = steps * Planes<NP>::kPairs;
        int pair = 0, left = steps;
        auto move = [&](const char*& pa, const char*& ea, const char*& pb, const char*& eb) {
            pa += astep;
            pb += bstep;
            if (NP > 1 && --left == 0 && ++pair < Planes<NP>::kPairs) {
                left = steps;
                pa = oa.at + Planes<NP>::a(pair) * aplane, ea = oa.end + Planes<NP>::a(pair) * aplane;
                pb = ob.at + Planes<NP>::b(pair) * bplane, eb = ob.end + Planes<NP>::b(pair) * bplane;
            }
        };
        const char *pa = oa.at + Planes<NP>::a(0) * aplane, *ea = oa.end + Planes<NP>::a(0) * aplane;
        const char *pb = ob.at + Planes<NP>::b(0) * bplane, *eb = ob.end + Planes<NP>::b(0) * bplane;
        a.load(pa, ea);
        b.load(pb, eb);
        move(pa, ea, pb, eb);
        a.store(lds);
        b.store(lds + A::kBytes);
        __syncthreads();
        for (int s = 0; s < total; ++s) {
            const char* now = lds + (s & 1) * kStep;
            char* next = lds + ((s + 1) & 1) * kStep;
            if (s + 1 < total) {
                a.load(pa, ea);
                b.load(pb, eb);
                move(pa, ea, pb, eb);
            }
            frag fa[MI], fb[NI];
#pragma unroll
            for (int j = 0; j < NI; ++j) fb[j] = B::template fragment<frag>(now + A::kBytes, n0 + 16 * j);
#pragma unroll
            for (int i = 0; i < MI; ++i) fa[i] = A::template fragment<frag>(now, m0 + 16 * i);
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j) c[i][j] = Mx<E>::mma(fa[i], fb[j], c[i][j]);
            if (s + 1 < total) {
                a.store(next);
                b.store(next + A::kBytes);
            }
            __syncthreads();
        }
    }
};

}  // namespace hy
