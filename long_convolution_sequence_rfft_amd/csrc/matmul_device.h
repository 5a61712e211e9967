// matmul_device.h -- a tile of a matrix product of 16-bit operands on MFMA.
//
// C[m][n] = sum over k of A(m, k) B(n, k): a workgroup of WM x WN waves makes a
// tile of TM x TN, k in steps of 32.
//
// Operands lie in blocks of 32 columns, [columns / 32][rows][32]: 64 bytes of a row,
// the rows of a block one after the other.  k is either the columns or the rows:
//   k in the columns: a step of a tile is W rows of one block, W * 64 bytes in a
//       piece; 16-byte chunk c of row m is kept in LDS at c ^ ((m >> 1) & 3), so that
//       the eight lanes that one cycle serves read eight different 16-byte slots
//       (in pairs: two 16-row fragments take 4 rows of 8 in turn, so that a lane's results of
//       the two are 8 rows in a row);
//   k in the rows: a step is 32 rows of W / 32 blocks, 2 KB pieces; the 32-byte half h
//       of row k is kept at h ^ key(k), so that the rows that lanes read together lie
//       in different banks.  ds_read_b64_tr_b16 turns 4 k x 16 columns on the way into
//       the registers.
// Both bring memory to LDS in contiguous KBs.  (An operand whose rows are whole is read in
// the same way by its strides, 64 bytes here and there: products of 16384 x 16384 x
// 768 run at 997 TFLOP/s so, at 1150 to 1390 with blocks.)
//
// Loads go to LDS directly, a step ahead of the products (of a step's 512 cycles of
// matrix instructions per wave little else has to be issued; staged in registers the
// same product ran at 854).  No bank conflicts.
//
// With several planes a step has all planes of both operands, so that each is loaded once for
// the products it takes part in.  Where both have several, the products of less than the first
// planes are summed apart and added last; where only B has (an operand of more bits than its
// type by one that is as given), all are one sum.
// A lane's results: row 4 (lane / 16) + r of a 16 x 16 tile, column lane % 16.
#pragma once

#include "recurrence_device.h"

namespace hy {

typedef short s16x4 __attribute__((ext_vector_type(4)));

// What a tile reads of one operand: `at` its first byte at k = 0, `end` the end of
// the memory (what lies there and after it is read as 0), `row` the bytes from one
// row to the next, `block` from one 32 columns to the next.
struct Operand {
    const char* at;
    const char* end;
    int64_t row, block;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t operand_rsrc(const char* at, const char* end)
{
    const int64_t left = end - at;
    const uint32_t n = left <= 0 ? 0u : left < 0xffffff00 ? (uint32_t)left : 0xffffff00u;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(at), (short)0, (int)n, 0x00020000);
}

// 16 bytes of each lane to LDS, side by side from byte `lds` on.  The compiler does
// not know of these loads: wait_loads before the barrier that publishes them.
__device__ __forceinline__ void load_to_lds(uint32_t lds, uint32_t off, __amdgpu_buffer_rsrc_t r)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(off), "s"(r) : "memory", "m0");
}
template <int N> __device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }

// A barrier of what wait_loads has waited for and of this wave's reads of LDS, which what is
// loaded behind it may overwrite: no other memory access is waited for.
__device__ __forceinline__ void barrier_only()
{
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

enum Form { kInRows, kInColumns, kInColumnsPaired };  // where k is

// One operand of a tile: W rows of the output's axis.
template <int W, int THREADS, Form F> struct Stage {
    static constexpr bool KC = F != kInRows;
    static constexpr int kBytes = W * 64;           // of a step in LDS
    static constexpr int kLoads = W * 4 / THREADS;  // of a thread, 16 bytes each
    static_assert(W * 4 % THREADS == 0 && W % 32 == 0, "");

    uint32_t off[kLoads];  // bytes from `at`

    static __device__ __forceinline__ int key(int k) { return ((k >> 1) ^ (k >> 3)) & 1; }
    static __device__ __forceinline__ int chunk_key(int row)
    {
        return F == kInColumnsPaired ? ((row >> 1) & 1) | ((row >> 3) & 1) << 1 : (row >> 1) & 3;
    }
    __device__ __forceinline__ void init(const Operand& o)
    {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int n = (int)threadIdx.x + i * THREADS, s = n & 3;  // the 16 bytes of LDS that it fills
            if constexpr (KC) {
                const int row = n >> 2;
                off[i] = (uint32_t)row * (uint32_t)o.row + (uint32_t)((s ^ chunk_key(row)) * 16);
            } else {
                const int k = (n >> 2) & 31;
                off[i] = (uint32_t)(n >> 7) * (uint32_t)o.block + (uint32_t)k * (uint32_t)o.row +
                         (uint32_t)((((s >> 1) ^ key(k)) << 1 | (s & 1)) * 16);
            }
        }
    }
    __device__ __forceinline__ void load(uint32_t lds, const char* at, const char* end) const
    {
        const __amdgpu_buffer_rsrc_t r = operand_rsrc(at, end);
        const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) load_to_lds(lds + i * THREADS * 16 + wave * 1024, off[i], r);
    }
    // Bytes from one step's first value to the next one's.
    static __device__ __forceinline__ int64_t step(const Operand& o) { return KC ? o.block : 32 * o.row; }
    // The fragment of the 16 rows at m0 (paired: of 16 of the 32 rows around it).
    template <typename V> static __device__ __forceinline__ V fragment(const char* lds, int m0)
    {
        const int lane = threadIdx.x & 63;
        if constexpr (KC) {
            const int i = lane & 15, c = lane >> 4;
            const int m = F == kInColumnsPaired ? (m0 & ~31) + 8 * (i >> 2) + ((m0 >> 4) & 1) * 4 + (i & 3) : m0 + i;
            return *(const V*)(lds + m * 64 + ((c ^ chunk_key(m)) * 16));
        } else {
            typedef __attribute__((address_space(3))) s16x4* at3;
            const int g = lane >> 4, i = lane & 15;
            s16x4 v[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = g * 8 + h * 4 + (i >> 2);
                const char* p = lds + (m0 >> 5) * 2048 + k * 64 + ((((m0 >> 4) & 1) ^ key(k)) << 5) + (i & 3) * 8;
                v[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((at3)p);
            }
            return __builtin_bit_cast(V, v);
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

// E: uint16_t (bfloat16) or _Float16.  NP planes of A, NB of B.  STAGES - 1 steps are under way.
template <typename E, int TM, int TN, int WM, int WN, Form AF, Form BF, int NP, int NB, int STAGES> struct MatTile {
    static_assert(NP == 1 || NB == NP, "");
    static constexpr int kThreads = WM * WN * 64;
    using A = Stage<TM, kThreads, AF>;
    using B = Stage<TN, kThreads, BF>;
    static constexpr int kStep = NP * A::kBytes + NB * B::kBytes, kLds = STAGES * kStep;
    static constexpr int MI = TM / WM / 16, NI = TN / WN / 16;
    using frag = typename Mx<E>::frag;

    f32x4 c[MI][NI];

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) c[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    // One step's products of one plane of A, the smaller ones first.
    __device__ __forceinline__ void products(const char* at, int m0, int n0)
    {
        frag fa[MI], fb[NB][NI];
#pragma unroll
        for (int n = NB - 1; n >= 0; --n)
#pragma unroll
            for (int j = 0; j < NI; ++j) fb[n][j] = B::template fragment<frag>(at + A::kBytes + n * B::kBytes, n0 + 16 * j);
#pragma unroll
        for (int i = 0; i < MI; ++i) fa[i] = A::template fragment<frag>(at, m0 + 16 * i);
#pragma unroll
        for (int n = NB - 1; n >= 0; --n)
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j) c[i][j] = Mx<E>::mma(fa[i], fb[n][j], c[i][j]);
    }

    // aplane, bplane: bytes between planes.  steps: of 32 values of k, at least 1.
    // Ends behind a barrier after the last read of lds.
    __device__ __forceinline__ void run(char* lds, const Operand& oa, int64_t aplane, const Operand& ob, int64_t bplane,
                                        int steps)
    {
        const int wave = threadIdx.x >> 6;
        const int m0 = wave / WN * (TM / WM), n0 = wave % WN * (TN / WN);
        clear();
        A a;
        B b;
        a.init(oa);
        b.init(ob);
        const int64_t astep = A::step(oa), bstep = B::step(ob);
        const uint32_t base = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds);
        const char *pa = oa.at, *pb = ob.at;
        auto issue = [&](int stage) {
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                if (n < NP) a.load(base + stage * kStep + n * A::kBytes, pa + n * aplane, oa.end + n * aplane);
                b.load(base + stage * kStep + NP * A::kBytes + n * B::kBytes, pb + n * bplane, ob.end + n * bplane);
            }
            pa += astep;
            pb += bstep;
        };
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i)
            if (i < steps) issue(i);
        // (with several planes the smaller products have sums of their own)
        f32x4 low[NP == 1 ? 1 : MI][NP == 1 ? 1 : NI];
        if constexpr (NP > 1) {
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j) low[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        int now = 0, into = STAGES - 1;
        for (int s = 0; s < steps; ++s) {
            // this step's loads are done: those of later steps may be under way
            if (STAGES > 2 && s + STAGES - 1 <= steps) wait_loads<(STAGES - 2) * (NP * A::kLoads + NB * B::kLoads)>();
            else wait_loads<0>();
            barrier_only();
            if (s + STAGES - 1 < steps) issue(into);
            const char* at = lds + now * kStep;
            if constexpr (NP == 1) {
                products(at, m0, n0);
            } else {
                frag fb[NP][NI];
#pragma unroll
                for (int n = 0; n < NP; ++n)
#pragma unroll
                    for (int j = 0; j < NI; ++j)
                        fb[n][j] = B::template fragment<frag>(at + NP * A::kBytes + n * B::kBytes, n0 + 16 * j);
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    frag fa[NP];
#pragma unroll
                    for (int n = 0; n < NP; ++n) fa[n] = A::template fragment<frag>(at + n * A::kBytes, m0 + 16 * i);
#pragma unroll
                    for (int q = 0; q < Planes<NP>::kPairs; ++q)
#pragma unroll
                        for (int j = 0; j < NI; ++j) {
                            f32x4& to = q + 1 == Planes<NP>::kPairs ? c[i][j] : low[i][j];
                            to = Mx<E>::mma(fa[Planes<NP>::a(q)], fb[Planes<NP>::b(q)][j], to);
                        }
                }
            }
            now = now + 1 == STAGES ? 0 : now + 1;
            into = into + 1 == STAGES ? 0 : into + 1;
        }
        if constexpr (NP > 1) {
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j) c[i][j] += low[i][j];
        }
        barrier_only();
    }
};

}  // namespace hy
