// recurrence_kernels.h -- kernels of the gated linear recurrence
//   S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
// and of its backward pass.
//
// A chunk of C tokens is handled by matrix products (the sum over the tokens
// of the chunk as scores between tokens, weighted by the decays between them;
// everything before the chunk through the state), so the state is touched once
// per C tokens and stays in registers.  The chunks of a segment run one after
// the other; segments run in parallel, each from the state that
// hyena_rec_states and hyena_rec_scan have put before it.
//
// With A_i the product of the decays from the chunk's start through token i, the
// decay between tokens j <= i of a chunk is w_ij = A_i / A_j, made of differences
// of logs (see Decays), and with S the state before the chunk
//   o_i = scale (A_i S^T q_i + sum_{j <= i} w_ij (q_i . k_j) v_j),
//   S <- A_last S + sum_j (A_last / A_j) k_j v_j^T.
// Chunks are 64 tokens (32 in float32, whose operands take twice the LDS), so a
// row of a transposed tile is 128 bytes.  Two passes over k and v, one for the
// segments' states and one for the outputs, are the price of walking a long
// sequence in parallel: at 65536 tokens of 12 heads of 64 in bfloat16 the three
// kernels take 165 to 175 us for 663 MB (403 without the first pass and the
// states), 4 TB/s, where a large copy reaches 5.1.
#pragma once

#include <type_traits>

#include "recurrence.h"
#include "timing.h"

namespace hy {

template <typename T>
__device__ __forceinline__ const T* row_base(const RView& v, int64_t b, int64_t h)
{
    return (const T*)v.p + b * v.b + h * v.h;
}

template <typename T> using DecaysOf = Decays<kRecChunk<T>>;

// Waves per SIMD that the registers leave room for: with 64 x 64 states three,
// with 128 x 128 ones and binary16's second accumulators one (with two, 112 to 136
// spilled registers: 8192 tokens of 8 heads forward 102 us, backward 242, with one
// 98 and 216; 128 x 64 with two 45 and 124, with one 62 and 126).  Two leave some
// spilled still: at 128 x 128 18 in bfloat16's outputs and 45 in its dq, 19 and 16 in
// float32's; 32 in binary16's dq with heads of 128 keys and 64 values; in dk and dv
// (eight waves, 128 x 128) 53, 8 and 85 in bfloat16, float32 and binary16.
constexpr int rec_waves(int d0, int d1, bool light) { return d0 * d1 <= 64 * 64 && light ? 3 : 2; }
template <typename T> constexpr int rec_out_waves(int d0, int d1, bool trans)
{
    return Mx<T>::kTerms == 2 && d0 * d1 == 128 * 128 ? 1 : rec_waves(d0, d1, !trans && sizeof(T) == 2);
}

// Wide states: nothing moves across, so that the operands of one part of a
// chunk's work are not all fetched during the one before (which spilled).
template <bool HOLD> __device__ __forceinline__ void hold_schedule()
{
    if constexpr (HOLD) __builtin_amdgcn_sched_barrier(0);
}

// A state in front of a reset has no part in what comes after it, whatever it
// holds: zero times an infinity would not be zero.  restarts: the chunk has a reset
// (the same for all lanes).
template <typename D> __device__ __forceinline__ bool restarts(const D& d, int last)
{
    return __builtin_amdgcn_readfirstlane(d.count[last]) != 0;
}
// the state's part of a tile of results whose column is the lane's token
__device__ __forceinline__ f32x4 unless_zero(f32x4 x, float factor)
{
    return factor != 0.0f ? x : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
}

// *out(16 i + l16) = sum over the four lanes of a column of x[i]
template <int IT, typename F> __device__ __forceinline__ void store_token_sums(F out, const float (&x)[IT], int lane, int grp)
{
    float y = sum_rows(x[0]);
#pragma unroll
    for (int i = 1; i < IT; ++i) {
        const float z = sum_rows(x[i]);
        y = grp == i ? z : y;
    }
    if (lane < 16 * IT) *out(lane) = y;
}

// ---------------------------------------------------------------------------
// Local states of the segments.  One workgroup per (row, head, segment, role);
// wave w owns every fourth 16-column tile of the state.  Bound by memory: 53 us
// at 65536 tokens of 12 heads of 64 in bfloat16 (217 MB, 4.4 TB/s without the
// 4 us that any launch takes), 31 us with both roles at 2 x 8192 (118 MB).
// ---------------------------------------------------------------------------
template <typename T, int DK, int DV, bool VEC>
__global__ __launch_bounds__(256, rec_waves(DK, DV, true)) void hyena_rec_states(RecStateArgs p)
{
    constexpr int C = kRecChunk<T>, NT = Mx<T>::kTerms;
    constexpr int KT = DK / 16, VW = DV / 64;
    using frag = typename Mx<T>::frag;
    __shared__ __attribute__((aligned(16))) T xt[(DK > DV ? DK : DV) * C];
    __shared__ __attribute__((aligned(16))) T yt[(DK > DV ? DK : DV) * C];
    __shared__ DecaysOf<T> decays[kDecayBatch];

    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, grp = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const ColFrags<T, C> cols_of(l16, grp);
    const int64_t bh = blockIdx.x / p.nseg, seg = blockIdx.x % p.nseg;
    const int role = blockIdx.y;
    const int64_t b = bh / p.heads, h = bh % p.heads;
    const int64_t nv = valid_tokens(p.lengths, b, p.N);
    const int64_t t0 = segment_start(p.N, p.nseg, seg), tN = segment_start(p.N, p.nseg, seg + 1);
    const int64_t t1 = tN < nv ? tN : nv;
    const int nchunk = t1 > t0 ? (int)((t1 - t0 + C - 1) / C) : 0;

    f32x4 S[KT][VW] = {};
    float total = 1.0f;
    // the chunks are walked forward (role 0) or from the last one back; two
    // waves bring in x, two y
    const bool is_x = wave < 2;
    constexpr int DM = DK > DV ? DK : DV;
    using Half = Tile<T, C, DM, 128, 4>;
    Half tile;
    Stream xs, gs;
    const int64_t first = t0 + (role ? (int64_t)(nchunk - 1) * C : 0);
    const int way = role ? -C : C;
    xs.start<T>(is_x ? p.x[role] : p.y[role], b, h, first);
    gs.start<float>(p.g, b, h, first + wave * way);
    const int width = is_x ? p.dk : p.dv, half = tid & 127;
    const typename Half::Places place(xs, width, half);
    const int len = (int)(t1 - t0);
    // tokens of the c-th chunk walked
    auto tokens = [&](int c) { return len - (role ? nchunk - 1 - c : c) * C; };
    auto fetch = [&](int c) {
        tile.template load<VEC>(xs, place, tokens(c), width, half);
        xs.move(way);
    };
    float g = 0.0f;
    auto fetch_g = [&](int c) {
        g = load1<float>(rows_at(gs.p), lane < C && c < nchunk && lane < tokens(c) ? lane * gs.step : kOutside);
        gs.move(kDecayBatch * way);
    };
    if (nchunk > 0) {
        fetch_g(wave);
        fetch(0);
    }
    for (int c = 0; c < nchunk; ++c) {
        const int slot = c % kDecayBatch;
        if (slot == 0 && wave < kDecayBatch) fill_decays<C>(decays[wave], g, lane);
        const DecaysOf<T>& dec = decays[slot];
        tile.store_cols(is_x ? xt : yt, half);
        __syncthreads();
        if (c + 1 < nchunk) {
            fetch(c + 1);
            if (slot == 0) fetch_g(c + kDecayBatch + wave);
        }
        const float all = dec.head[C - 1];
        const bool fresh = restarts(dec, C - 1);
        const float* f = role ? dec.head : dec.tail;
        total = fresh || total == 0.0f ? 0.0f : total * all;  // (all may not be a number)
        if (fresh) {
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
                for (int v = 0; v < VW; ++v) S[k][v] = f32x4{};
        }
#pragma unroll
        for (int v = 0; v < VW; ++v) {
            const int vt = wave + 4 * v;
            Split<T, NT> y[C / 32];
            const float up = split_columns<T>(y, [&](int j) {
                const f32x8 w = join8(*(const f32x4*)(f + 32 * j + 8 * grp),
                                      *(const f32x4*)(f + 32 * j + 8 * grp + 4));
                return Mx<T>::widen8(cols_of.any(yt, vt, j)) * w;
            });
#pragma unroll
            for (int k = 0; k < KT; ++k)
                S[k][v] = update<T>(S[k][v], all, up, y,
                                    [&](int j) { return cols_of(xt, k, j); });
        }
        __syncthreads();
    }
    const float scale = role ? p.scale : 1.0f;
    const int64_t per = (int64_t)p.dk * p.dv;
    float* out = p.local[role] + (bh * (p.nseg + 1) + seg + (role ? 0 : 1)) * per;
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int v = 0; v < VW; ++v)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int kk = 16 * k + 4 * grp + r, vv = 16 * (wave + 4 * v) + l16;
                if (kk < p.dk && vv < p.dv) out[kk * p.dv + vv] = S[k][v][r] * scale;
            }
    if (role == 0 && tid == 0) p.decay[bh * p.nseg + seg] = total;
}

// Scores of 16-bit types are split operands of two terms, and no state is read as one,
// so that a result's own rounding is the only one of 8 (binary16: 11) bits.  With
// scores, and bfloat16 states, of one term a result's error was 1.4 times that, and
// 65536 tokens of 12 heads of 64 took 93 instead of 105 us, 2 x 8192 of 6 heads of
// 128 43.5 instead of 50; of 12 heads of 64 dq 41 instead of 44.5, dk and dv 65
// instead of 71.5.
template <typename T> constexpr int kScoreTerms = sizeof(T) == 2 ? 2 : 1;

// LDS of the two kernels below.
template <typename T, int DA, int DC> constexpr size_t rec_out_lds()
{
    constexpr int C = kRecChunk<T>, DM = DA > DC ? DA : DC, LA = DA + kPad<T>, LB = DM + kPad<T>, LC = C + kPad<T>;
    return sizeof(T) * (size_t)(C * LA + C * LB + 2 * DM * C + C * LC) + kDecayBatch * sizeof(DecaysOf<T>);
}

// Chunks whose terms of dg are held before they are summed up.
constexpr int kGradHold = 16;

template <typename T, int D> constexpr size_t rec_grad_lds()
{
    constexpr int C = kRecChunk<T>, LD = D + kPad<T>, LC = C + kPad<T>;
    return sizeof(T) * (size_t)(4 * C * LD + 2 * D * C + 2 * kScoreTerms<T> * C * LC) + kDecayBatch * sizeof(DecaysOf<T>) +
           sizeof(float) * (size_t)(2 * (C / 16) * C + 4 * C + kDecayBatch * C + kGradHold * C) + kGradHold * 16;
}

// ---------------------------------------------------------------------------
// Outputs of one direction of reading: out_i = scale (f_i a_i . S + sum_j w_ij
// (a_i . b_j) c_j).  a = q, b = k, c = v gives o; a = do, b = v, c = k gives dq
// (TRANS: the state's rows are then the channels of c).  TRANS also writes
// rq_i = r_i . (the state's part of out_i), with the state as a split operand
// so that it keeps float32 accuracy.  So does the state itself through the segment:
// with updates of two bfloat16 terms what is left of values that cancel would be
// lost, and o would depend on whether the final state is asked for (65536 tokens
// of 12 heads of 64 in bfloat16 91 us so, 93 with three; 2 x 8192 of 6 heads of 128
// 41 and 43.5).
//
// One workgroup of four waves per (row, head, segment).  Waves share the score
// tiles of a chunk (written to LDS as terms of storage type) and each owns every fourth
// 16-channel tile of c: its part of the state never leaves its registers.
//
// Bound by the instructions of a chunk and the LDS beside memory: 65536 tokens of 12
// heads of 64 in bfloat16 in 105 to 112 us (420 MB, 4 TB/s without the launch; vector
// units busy for 62% of the time, the LDS for 61%, 39% of that bank conflicts,
// matrix units for 27%, three waves per SIMD); with two waves per SIMD 2 x 8192
// tokens of 6 heads of 128 in 48 us (134 MB; 36%, 36%, 22%) and dq of 12 heads of 64
// in 45 us (137 MB; 45%, 34%, 17%; 720 vector instructions per wave and chunk).  In
// float32 matrix instructions bound it: dq of 4 x 2048 tokens in 47 us, matrix units
// 54%.
// ---------------------------------------------------------------------------
template <typename T, int DA, int DC, bool TRANS, bool VEC>
__global__ __launch_bounds__(256, rec_out_waves<T>(DA, DC, TRANS)) void hyena_rec_out(RecArgs p)
{
    constexpr int C = kRecChunk<T>, DM = DA > DC ? DA : DC, LA = DA + kPad<T>, LB = DM + kPad<T>, LC = C + kPad<T>;
    constexpr int NT = Mx<T>::kTerms;  // state update
    constexpr int NS = TRANS || Mx<T>::kTerms < 2 ? Mx<T>::kTerms : 2;  // state as an operand
    constexpr int NP = kScoreTerms<T>;
    constexpr int AT = DA / 16, CW = DC / 64, IT = C / 16;
    using frag = typename Mx<T>::frag;
    using vec4 = typename Mx<T>::vec4;
    __shared__ __attribute__((aligned(16))) char smem[rec_out_lds<T, DA, DC>()];
    T* ar = (T*)smem;              // [C][LA]
    T* br = ar + C * LA;           // [C][LB]
    T* bt = br + C * LB;           // [DM][C] transposed
    T* ct = bt + DM * C;           // [DM][C] transposed
    T* ps = ct + DM * C;           // [C][LC] scores; their second terms over the rows of b, whose last use they are
    constexpr int kApart = -(C * LB + 2 * DM * C);  // from ps to br
    static_assert(LB >= LC, "second terms fit");
    DecaysOf<T>* const decays = (DecaysOf<T>*)(ps + C * LC);
    // [C][4], TRANS: a wave's sum of a token in the padding behind its scores
    auto part = [&](int token) { return (float*)(ps + token * LC + C); };
    static_assert(kPad<T> * sizeof(T) == 4 * sizeof(float), "a sum for each wave");

    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, grp = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const ColFrags<T, C> cols_of(l16, grp);
    const int64_t bh = blockIdx.x / p.nseg, seg = blockIdx.x % p.nseg;
    const int64_t b = bh / p.heads, h = bh % p.heads;
    const int64_t nv = valid_tokens(p.lengths, b, p.N);
    const int64_t t0 = segment_start(p.N, p.nseg, seg), tN = segment_start(p.N, p.nseg, seg + 1);
    const int64_t t1 = tN < nv ? tN : nv;
    const int nchunk = t1 > t0 ? (int)((t1 - t0 + C - 1) / C) : 0;
    T* const op = (T*)p.out + (b * p.N * p.heads + h) * p.dc;
    const int64_t ostride = p.heads * (int64_t)p.dc;
    const uint32_t ostep = (uint32_t)ostride * (uint32_t)sizeof(T);

    // the state before this segment
    f32x4 S[AT][CW];
    const int64_t per = (int64_t)p.da * p.dc;
    const float* sp = p.state ? p.state + (bh * p.state_n + seg) * per : nullptr;
#pragma unroll
    for (int k = 0; k < AT; ++k)
#pragma unroll
        for (int v = 0; v < CW; ++v)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int aa = 16 * k + 4 * grp + r, cc = 16 * (wave + 4 * v) + l16;
                const int64_t at = TRANS ? (int64_t)cc * p.da + aa : (int64_t)aa * p.dc + cc;
                S[k][v][r] = sp && aa < p.da && cc < p.dc ? sp[at] : 0.0f;
            }

    // all waves bring in a, two b and two c
    const bool is_b = wave < 2;
    using Rows = Tile<T, C, DA, 256, 1>;
    using Half = Tile<T, C, DM, 128, 4>;
    Rows ta;
    Half tile;
    UnderResults<T, IT, CW> under;
    Stream as, xs, rs, gs;
    as.start<T>(p.a, b, h, t0);
    xs.start<T>(is_b ? p.b : p.c, b, h, t0);
    if constexpr (TRANS) rs.start<T>(p.r, b, h, t0);
    gs.start<float>(p.g, b, h, t0 + wave * C);
    const int width = is_b ? p.da : p.dc, half = tid & 127;
    const typename Rows::Places pa(as, p.da, tid);
    const typename Half::Places px(xs, width, half);
    const int len = (int)(t1 - t0);
    auto fetch = [&](int c) {
        const int n = len - c * C;
        ta.template load<VEC>(as, pa, n, p.da, tid);
        tile.template load<VEC>(xs, px, n, width, half);
        as.move(C);
        xs.move(C);
    };
    float g = 0.0f;
    auto fetch_g = [&](int c) {
        g = load1<float>(rows_at(gs.p), lane < C && lane < len - c * C ? lane * gs.step : kOutside);
        gs.move(kDecayBatch * C);
    };
    if (nchunk > 0) {
        fetch_g(wave);
        fetch(0);
    }
    for (int c = 0; c < nchunk; ++c) {
        const int slot = c % kDecayBatch;
        if (slot == 0 && wave < kDecayBatch) fill_decays<C>(decays[wave], g, lane);
        const DecaysOf<T>& dec = decays[slot];
        ta.template store_rows<LA>(ar, tid);
        if (is_b) tile.template store_rows<LB>(br, half);
        tile.store_cols(is_b ? bt : ct, half);
        if constexpr (TRANS) {
            // used at the end of this chunk: a load ahead of the next chunk's
            under.template load<VEC>(rs, len - c * C, p.dc, l16, grp, wave);
            rs.move(C);
        }
        __syncthreads();
        const int64_t tb0 = t0 + (int64_t)c * C;
        const __amdgpu_buffer_rsrc_t orows = rows_at(op + tb0 * ostride);
        const int left = t1 - tb0 < C ? (int)(t1 - tb0) : C;
        if (c + 1 < nchunk) {
            fetch(c + 1);
            if (slot == 0) fetch_g(c + kDecayBatch + wave);
        }

        // scores of the tokens of tile `wave` against all before them and their
        // own tile; tiles right of that are zero (and their products not used).
        // C = 32 has two tiles: the other waves repeat the work of the first two.
        {
            const int it = again_uniform(wave) % IT, ti = 16 * it + l16, to = 16 * it + 4 * grp;
            const double li = dec.logs[ti];
            double lj[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) lj[r] = dec.logs[to + r];
            const int ci = dec.count[ti];
            const i32x4 cj = *(const i32x4*)(dec.count + to);
            const float wi = it > 0 ? p.scale : 0.0f;
            const float within = wi * dec.within[ti];
            const float* cross = dec.cross[it > 0 ? it - 1 : 0];
            f32x4 cw[IT - 1];
#pragma unroll
            for (int j = 0; j < IT - 1; ++j) cw[j] = *(const f32x4*)(cross + 16 * j + 4 * grp);
            frag af[DA / 32];
#pragma unroll
            for (int k = 0; k < DA / 32; ++k) af[k] = frag_at<T>(ar + ti * LA + 32 * k + 8 * grp);
            auto tile = [&](int j) {
                f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int k = 0; k < DA / 32; ++k)
                    s = Mx<T>::mma(frag_at<T>(br + (16 * j + l16) * LB + 32 * k + 8 * grp), af[k], s);
                return s;
            };
            f32x4 own = tile(it), s[IT - 1];
#pragma unroll
            for (int j = 0; j < IT - 1; ++j) s[j] = tile(j);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const bool in = (to + r <= ti) & (cj[r] == ci);
                const float w = p.scale * __builtin_amdgcn_exp2f((float)(li - lj[r]));
                own[r] = in ? own[r] * w : 0.0f;
            }
            Split4<T, NP> w[IT];
#pragma unroll
            for (int j = 0; j < IT - 1; ++j) w[j].set(s[j] * (cw[j] * within));
            w[IT - 1].set(own);
            if constexpr (NP > 1) __syncthreads();  // the rows of b are done with
            // the tile right of the last own one is not among the s; the own tile itself comes last
#pragma unroll
            for (int n = 0; n < NP; ++n) {
                T* const row = ps + n * kApart + ti * LC;
#pragma unroll
                for (int j = 0; j < IT - 1; ++j) *(vec4*)(row + 16 * j + 4 * grp) = w[j].y[n];
                *(vec4*)(row + 16 * (IT - 1) + 4 * grp) = vec4{};
                *(vec4*)(row + to) = w[IT - 1].y[n];
            }
        }
        __syncthreads();

        const float all = dec.head[C - 1];
        const bool fresh = restarts(dec, C - 1);
        float rdot[IT] = {};
#pragma unroll
        for (int v = 0; v < CW; ++v) {
            const int vt = wave + 4 * v;
            frag cf[C / 32];
#pragma unroll
            for (int j = 0; j < C / 32; ++j) cf[j] = cols_of.any(ct, vt, j);
            const uint32_t orow = (uint32_t)again(l16) * ostep;
            // outputs: column = token, rows = 4 channels
            f32x4 so[IT] = {};
            StateFit<T> fit;
            fit.template set<AT>([&](int k) { return S[k][v]; }, grp);
#pragma unroll
            for (int k = 0; k < DA / 32; ++k) {
                Split<T, NS> sf;
                sf.set(fit.fitted(join8(S[2 * k][v], S[2 * k + 1][v])));
#pragma unroll
                for (int i = 0; i < IT; ++i)
                    so[i] = mma_split<T, NS, true>(sf, frag_at<T>(ar + (16 * i + l16) * LA + 32 * k + 8 * grp), so[i]);
            }
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int ti = 16 * i + l16;
                if (fresh) so[i] = unless_zero(so[i], dec.head[ti]);
                f32x4 o = fit.results(so[i], p.scale * dec.head[ti]);
                if constexpr (TRANS) {
                    const f32x4 r = Mx<T>::widen(under.x[i][v]);
                    rdot[i] += o[0] * r[0] + o[1] * r[1] + o[2] * r[2] + o[3] * r[3];
                }
#pragma unroll
                for (int j = 0; j <= i / 2; ++j) {
                    Split<T, NP> w;
#pragma unroll
                    for (int n = 0; n < NP; ++n) w.f[n] = frag_at<T>(ps + n * kApart + ti * LC + 32 * j + 8 * grp);
                    o = mma_split<T, NP, false>(w, cf[j], o);
                }
                store_row4<T>(orows, orow + 16 * i * ostep, ti < left, 16 * vt + 4 * grp, p.dc, o);
            }
            // the state after this chunk
            hold_schedule<(DA * DC > 64 * 64)>();
            if (fresh) {
#pragma unroll
                for (int k = 0; k < AT; ++k) S[k][v] = f32x4{};
            }
            Split<T, NT> y[C / 32];
            const float up = split_columns<T>(y, [&](int j) {
                const f32x8 w = join8(*(const f32x4*)(dec.tail + 32 * j + 8 * grp),
                                      *(const f32x4*)(dec.tail + 32 * j + 8 * grp + 4));
                return Mx<T>::widen8(cf[j]) * w;
            });
#pragma unroll
            for (int k = 0; k < AT; ++k)
                S[k][v] = update<T>(S[k][v], all, up, y,
                                    [&](int j) { return cols_of(bt, k, j); });
            hold_schedule<(DA * DC > 64 * 64)>();
        }
        if constexpr (TRANS) store_token_sums<IT>([&](int token) { return part(token) + wave; }, rdot, lane, grp);
        __syncthreads();
        if constexpr (TRANS) {
            if (tid < C && tb0 + tid < t1) {
                const f32x4 y = *(const f32x4*)part(tid);
                p.rq[bh * p.N + tb0 + tid] = (y[0] + y[1]) + (y[2] + y[3]);
            }
        }
    }
    // rows of a padded batch past the length
    for (int64_t i = tid; i < (tN - (t1 > t0 ? t1 : t0)) * p.dc; i += 256) {
        const int64_t t = (t1 > t0 ? t1 : t0) + i / p.dc;
        op[t * ostride + i % p.dc] = T(0);
    }
    if (p.last != nullptr) {
        float* out = p.last + bh * per;
#pragma unroll
        for (int k = 0; k < AT; ++k)
#pragma unroll
            for (int v = 0; v < CW; ++v)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int aa = 16 * k + 4 * grp + r, cc = 16 * (wave + 4 * v) + l16;
                    if (aa < p.da && cc < p.dc)
                        out[TRANS ? (int64_t)cc * p.da + aa : (int64_t)aa * p.dc + cc] = S[k][v][r];
                }
    }
}

// ---------------------------------------------------------------------------
// dk, dv and dg of a segment, its chunks from the last to the first.
//   dk_j = sum_i w_ij (do_i . v_j) q_i + tail_j dS v_j
//   dv_j = sum_i w_ij (q_i . k_j) do_i + tail_j dS^T k_j      (q, do times scale)
// Eight waves: four own tiles of dk (their part of dS has the channels of v as
// rows) and bring in q and k, four own tiles of dv (the other way round) and
// bring in do and v.
//
// dg_t = <S_end, dS_end> + sum_{s >= t} (q_s . dq_s - k_s . dk_s), s up to the
// segment's end, without a token's own pair in either product: both are made of
// float32 values (scores weighted by both products before any rounding, the states' parts
// from split operands) and kept in LDS for kGradHold chunks, then summed up in
// float64 by all waves.  Over a whole sequence the sum is zero, so at a reset it
// starts anew: a sequence's dg holds no rounding of those after it.
//
// Bound by a chunk's instructions and the waits between them, with two waves per
// SIMD: 72 to 76 us at 2 x 8192 tokens of 12 heads of 64 in bfloat16 (166 MB), 82 us at
// 4 x 2048 in float32.  In bfloat16 660 vector instructions per wave and chunk keep
// the vector units busy for 45% of the time, the LDS is for 35% (41% of that bank
// conflicts), the matrix units for 16%; in float32 20%, 19% and 46%.  With scores of
// one term, where it took 66 us, two workgroups per compute unit, with 128 registers and
// 81 KB of LDS each, came to 64, two chunks in LDS with the next one's scores made
// beside this one's gradients to 66: not kept.  dk and dv are padded apart: with both
// at 128 heads of 40 and 72 in float16 (3 x 4100 tokens, 5 heads) took 69 us, then
// 41, now 44.
// ---------------------------------------------------------------------------
template <typename T, int DK, int DV, bool VEC>
__global__ __launch_bounds__(512) void hyena_rec_grad(RecGradArgs p)
{
    constexpr int D = DK > DV ? DK : DV;
    constexpr int C = kRecChunk<T>, LD = D + kPad<T>, LC = C + kPad<T>;
    constexpr int NT = Mx<T>::kTerms;
    constexpr int NP = kScoreTerms<T>;
    constexpr int IT = C / 16, kCells = (DK / 16) * (DV / 64);
    using frag = typename Mx<T>::frag;
    using vec4 = typename Mx<T>::vec4;
    __shared__ __attribute__((aligned(16))) char smem[rec_grad_lds<T, D>()];
    T* qr = (T*)smem;              // [C][LD]
    T* kr = qr + C * LD;           // [C][LD]
    T* dr = kr + C * LD;           // [C][LD]
    T* vr = dr + C * LD;           // [C][LD]
    T* qt = vr + C * LD;           // [D][C] transposed
    T* dt = qt + D * C;            // [D][C] transposed
    T* pa = dt + D * C;            // [C][LC] row j, column i: w_ij (q_i . k_j)
    T* pd = pa + NP * C * LC;      // [C][LC] w_ij (do_i . v_j)
    char* rest = (char*)(pd + NP * C * LC);
    DecaysOf<T>* const decays = (DecaysOf<T>*)rest;
    float* rows = (float*)(rest + kDecayBatch * sizeof(DecaysOf<T>));  // [IT][C] by j tile: sum over its j, per i
    float* cols = rows + IT * C;                       // [IT][C] by i tile: sum over its i, per j
    float* part = cols + IT * C;                       // [4][C] k . (state's part of dk), per wave
    float* rqs = part + 4 * C;                         // [kDecayBatch][C]
    float* hold = rqs + kDecayBatch * C;               // [kGradHold][C] q . dq - k . dk
    double* sums = (double*)(hold + kGradHold * C);    // [kGradHold] their sums, [8] at the start
    unsigned long long* resets = (unsigned long long*)(sums + kGradHold);  // [kGradHold]

    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, grp = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const ColFrags<T, C> cols_of(l16, grp);
    const bool own_k = wave < 4;
    const int w4 = wave & 3, half = tid & 127;
    const int64_t bh = blockIdx.x / p.nseg, seg = blockIdx.x % p.nseg;
    const int64_t b = bh / p.heads, h = bh % p.heads;
    const int64_t nv = valid_tokens(p.lengths, b, p.N);
    const int64_t t0 = segment_start(p.N, p.nseg, seg), tN = segment_start(p.N, p.nseg, seg + 1);
    const int64_t t1 = tN < nv ? tN : nv;
    const int nchunk = t1 > t0 ? (int)((t1 - t0 + C - 1) / C) : 0;
    T* const kout = (T*)p.dk_out + (b * p.N * p.heads + h) * p.dk;
    T* const vout = (T*)p.dv_out + (b * p.N * p.heads + h) * p.dv;

    // gradient of the state after this segment, and its product with the state
    // (waves of dk: [DV / 16][DK / 64] tiles, of dv: [DK / 16][DV / 64])
    f32x4 S[kCells];
    const int64_t per = (int64_t)p.dk * p.dv;
    const int64_t entry = (bh * ((int64_t)p.nseg * p.every + 1) + (seg + 1) * p.every) * per;
    const float* ep = p.end ? p.end + entry : nullptr;
    const float* sp = p.start ? p.start + entry : nullptr;
    float cross = 0.0f;
#pragma unroll
    for (int x = 0; x < kCells; ++x)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 16 * (own_k ? x / (DK / 64) : x / (DV / 64)) + 4 * grp + r;
            const int col = 16 * (w4 + 4 * (own_k ? x % (DK / 64) : x % (DV / 64))) + l16;
            const int kk = own_k ? col : row, vv = own_k ? row : col;
            const bool in = kk < p.dk && vv < p.dv;
            S[x][r] = ep && in ? ep[kk * p.dv + vv] : 0.0f;
            if (own_k && ep && sp && in) cross += S[x][r] * sp[kk * p.dv + vv];
        }
    cross = sum_rows(sum16(cross));
    if (lane == 0) sums[wave] = own_k ? (double)cross : 0.0;
    __syncthreads();
    double over = ((sums[0] + sums[1]) + (sums[2] + sums[3]));  // <S, dS> after the chunks held, or their sum up to a reset
    __syncthreads();

    // two waves bring in each tensor: q and do are also needed transposed
    const bool is_x = w4 < 2;
    using Half = Tile<T, C, D, 128, 4>;
    Half tile;
    Stream xs, gs;
    const int64_t last = t0 + (int64_t)(nchunk - 1) * C;
    xs.start<T>(own_k ? is_x ? p.q : p.k : is_x ? p.o : p.v, b, h, last);
    static_assert(kDecayBatch == 2, "two waves fill a batch");
    gs.start<float>(p.g, b, h, last - (w4 - 2) * C);
    const int width = own_k ? p.dk : p.dv;
    T* const xr = own_k ? is_x ? qr : kr : is_x ? dr : vr;
    T* const xt = own_k ? qt : dt;
    const typename Half::Places px(xs, width, half);
    const int len = (int)(t1 - t0);
    auto fetch = [&](int c) {
        const int n = len - (nchunk - 1 - c) * C;
        tile.template load<VEC>(xs, px, n, width, half);
        xs.move(-C);
    };
    // of the waves with less to store, 2 + w fills the decays of the w-th chunk of
    // a batch and 6 + w hands over the state's part of q . dq
    float g = 0.0f;
    auto fetch_g = [&](int c) {
        const int n = c < nchunk ? len - (nchunk - 1 - c) * C : 0;
        const bool in = !is_x & (lane < C) & (lane < n);
        if (own_k) g = load1<float>(rows_at(gs.p), in ? lane * gs.step : kOutside);
        else g = load1<float>(rows_at(p.rq + bh * p.N + t0 + (int64_t)(nchunk - 1 - c) * C), in ? lane * 4 : kOutside);
        gs.move(-kDecayBatch * C);
    };
    if (nchunk > 0) {
        fetch_g(w4 - 2);
        fetch(0);
    }
    for (int c = 0; c < nchunk; ++c) {
        const int slot = c % kDecayBatch;
        if (slot == 0 && !is_x) {
            if (own_k) fill_decays<C>(decays[w4 - 2], g, lane);
            else if (lane < C) rqs[(w4 - 2) * C + lane] = g;
        }
        const DecaysOf<T>& dec = decays[slot];
        const int at = D > 64 ? again(half) : half;
        tile.template store_rows<LD>(xr, at);
        if (is_x) tile.store_cols(xt, at);
        __syncthreads();
        const int64_t tb0 = t0 + (int64_t)(nchunk - 1 - c) * C;
        const int left = t1 - tb0 < C ? (int)(t1 - tb0) : C;
        if (c + 1 < nchunk) {
            fetch(c + 1);
            if (slot == 0) fetch_g(c + kDecayBatch + w4 - 2);
        }
        // what the last wave adds up below, read before others may refill it
        float rq_now = 0.0f;
        unsigned long long resets_now = 0;
        if (wave == 7) {
            rq_now = rqs[slot * C + lane % C];
            resets_now = dec.resets;
        }

        // both scores of each pair of tiles: rows i, columns j <= i.  Waves 0 to 3
        // take the tiles of one's own (an exp2 per pair), 4 and 5 those left of
        // an odd one, 6 and 7 the two left of tiles 2 and 3 (their decays are
        // products of two factors); with two tiles, wave 2 takes (1, 0)
        if (wave < IT) {
            const int l16 = D > 64 ? again(lane & 15) : lane & 15, grp = D > 64 ? again(lane >> 4) : lane >> 4;
            const int at = again_uniform(wave);
            const int tj = 16 * at + l16, ti = 16 * at + 4 * grp;
            const double lj = dec.logs[tj];
            const int cj = dec.count[tj];
            double li[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) li[r] = dec.logs[ti + r];
            const i32x4 ci = *(const i32x4*)(dec.count + ti);
            f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f}, d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                if (k < DK / 32)
                    s = Mx<T>::mma(frag_at<T>(qr + tj * LD + 32 * k + 8 * grp), frag_at<T>(kr + tj * LD + 32 * k + 8 * grp), s);
                if (k < DV / 32)
                    d = Mx<T>::mma(frag_at<T>(dr + tj * LD + 32 * k + 8 * grp), frag_at<T>(vr + tj * LD + 32 * k + 8 * grp), d);
            }
            f32x4 w;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                w[r] = (tj <= ti + r) & (ci[r] == cj) ? p.scale * __builtin_amdgcn_exp2f((float)(li[r] - lj)) : 0.0f;
            // (products that a mask leaves out may not be finite)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                s[r] = tj <= ti + r ? s[r] * w[r] : 0.0f;
                d[r] = tj <= ti + r ? d[r] : 0.0f;
            }
            // (a token's own pair has no part in the gradient of g; it would cancel in
            // q . dq - k . dk, but only after either sum was rounded at its size)
            f32x4 both;
#pragma unroll
            for (int r = 0; r < 4; ++r) both[r] = tj < ti + r ? s[r] * d[r] : 0.0f;
            d = d * w;
            store_split<T, NP>(pa + tj * LC + ti, C * LC, s);
            store_split<T, NP>(pd + tj * LC + ti, C * LC, d);
            if (at & 1) {  // the tile above an odd own one is read with it
#pragma unroll
                for (int n = 0; n < NP; ++n) {
                    *(vec4*)(pa + n * C * LC + tj * LC + ti - 16) = vec4{};
                    *(vec4*)(pd + n * C * LC + tj * LC + ti - 16) = vec4{};
                }
            }
            // every lane of a row or column writes the same sum
            cols[at * C + tj] = sum_rows((both[0] + both[1]) + (both[2] + both[3]));
            f32x4 row;
#pragma unroll
            for (int r = 0; r < 4; ++r) row[r] = sum16(both[r]);
            *(f32x4*)(rows + at * C + ti) = row;
        } else if (IT == 4 ? wave >= 4 : wave == 2) {
            const int l16 = D > 64 ? again(lane & 15) : lane & 15, grp = D > 64 ? again(lane >> 4) : lane >> 4;
            const int at = again_uniform(wave);
            // (1, 0), (3, 2), (2, 0) and (2, 1), (3, 0) and (3, 1)
            const int i = IT == 2 || at == 4 ? 1 : at == 6 ? 2 : 3, j0 = at == 5 ? 2 : 0;
            const bool two = at >= 6;
            const int ti = 16 * i + 4 * grp, tr = 16 * i + l16;
            const f32x4 within = *(const f32x4*)(dec.within + ti) * p.scale;
            f32x4 s[2] = {}, d[2] = {};
            float crossed[2];
#pragma unroll
            for (int n = 0; n < 2; ++n) crossed[n] = dec.cross[i - 1][16 * (j0 + n) + l16];
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                frag qf, df;
                if (k < DK / 32) qf = frag_at<T>(qr + tr * LD + 32 * k + 8 * grp);
                if (k < DV / 32) df = frag_at<T>(dr + tr * LD + 32 * k + 8 * grp);
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    if (n == 1 && !two) break;
                    const int tj = 16 * (j0 + n) + l16;
                    if (k < DK / 32) s[n] = Mx<T>::mma(qf, frag_at<T>(kr + tj * LD + 32 * k + 8 * grp), s[n]);
                    if (k < DV / 32) d[n] = Mx<T>::mma(df, frag_at<T>(vr + tj * LD + 32 * k + 8 * grp), d[n]);
                }
            }
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                if (n == 1 && !two) break;
                const int j = j0 + n, tj = 16 * j + l16;
                const f32x4 w = within * crossed[n];
                s[n] = s[n] * w;
                const f32x4 both = s[n] * d[n];
                d[n] = d[n] * w;
                store_split<T, NP>(pa + tj * LC + ti, C * LC, s[n]);
                store_split<T, NP>(pd + tj * LC + ti, C * LC, d[n]);
                cols[i * C + tj] = sum_rows((both[0] + both[1]) + (both[2] + both[3]));
                f32x4 row;
#pragma unroll
                for (int r = 0; r < 4; ++r) row[r] = sum16(both[r]);
                *(f32x4*)(rows + j * C + ti) = row;
            }
        }
        __syncthreads();

        const float all = dec.head[C - 1];
        const bool fresh = restarts(dec, C - 1);
        // across: rows that dS multiplies (v or k); scores and fold: out_j += scores_ij fold_i; add: the other
        // tensor of dS's update
        auto work = [&](auto is_dk, const T* across, const T* scores, const T* fold, const T* add, T* out) {
            constexpr bool kSums = decltype(is_dk)::value;
            constexpr int kAcross = kSums ? DV : DK, MT = kAcross / 16, MW = (kSums ? DK : DV) / 64;
            const int l16 = D > 64 ? again(lane & 15) : lane & 15, grp = D > 64 ? again(lane >> 4) : lane >> 4;
            constexpr int NS = kSums || NT < 2 ? NT : 2;  // dS as an operand
            const __amdgpu_buffer_rsrc_t orows = rows_at(out + tb0 * p.heads * width);
            const uint32_t ostep = (uint32_t)p.heads * (uint32_t)width * (uint32_t)sizeof(T);
            const uint32_t orow = (uint32_t)again(l16) * ostep;
            float kdot[IT] = {};
#pragma unroll
            for (int n = 0; n < MW; ++n) {
                const int nt = w4 + 4 * n;
                frag ff[C / 32];
#pragma unroll
                for (int i = 0; i < C / 32; ++i) ff[i] = cols_of.any(fold, nt, i);
                f32x4 sx[IT] = {};
                StateFit<T> fit;
                fit.template set<MT>([&](int m) { return S[m * MW + n]; }, grp);
#pragma unroll
                for (int k = 0; k < kAcross / 32; ++k) {
                    Split<T, NS> sf;
                    sf.set(fit.fitted(join8(S[2 * k * MW + n], S[(2 * k + 1) * MW + n])));
#pragma unroll
                    for (int j = 0; j < IT; ++j)
                        sx[j] = mma_split<T, NS, true>(sf, frag_at<T>(across + (16 * j + l16) * LD + 32 * k + 8 * grp), sx[j]);
                }
#pragma unroll
                for (int j = 0; j < IT; ++j) {
                    const int tj = 16 * j + l16;
                    if (fresh) sx[j] = unless_zero(sx[j], dec.tail[tj]);
                    f32x4 x = fit.results(sx[j], dec.tail[tj]);
                    if constexpr (kSums) {
                        const f32x4 kk = Mx<T>::widen(*(const vec4*)(kr + tj * LD + perm4(4 * nt + grp)));
                        kdot[j] += x[0] * kk[0] + x[1] * kk[1] + x[2] * kk[2] + x[3] * kk[3];
                    }
#pragma unroll
                    for (int i = j / 2; i < C / 32; ++i) {
                        Split<T, NP> w;
#pragma unroll
                        for (int n = 0; n < NP; ++n) w.f[n] = frag_at<T>(scores + n * C * LC + tj * LC + 32 * i + 8 * grp);
                        x = mma_split<T, NP, false>(w, ff[i], x);
                    }
                    store_row4<T>(orows, orow + 16 * j * ostep, tj < left, 16 * nt + 4 * grp, width, x);
                }
                hold_schedule<(DK * DV > 64 * 64)>();
                if (fresh) {
#pragma unroll
                    for (int m = 0; m < MT; ++m) S[m * MW + n] = f32x4{};
                }
                Split<T, NT> y[C / 32];
                const float up = split_columns<T>(y, [&](int i) {
                    const f32x8 w = join8(*(const f32x4*)(dec.head + 32 * i + 8 * grp), *(const f32x4*)(dec.head + 32 * i + 8 * grp + 4));
                    return Mx<T>::widen8(ff[i]) * (w * p.scale);
                });
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    S[m * MW + n] = update<T>(S[m * MW + n], all, up, y, [&](int i) { return cols_of(add, m, i); });
                hold_schedule<(DK * DV > 64 * 64)>();
            }
            if constexpr (kSums) store_token_sums<IT>([&](int token) { return part + w4 * C + token; }, kdot, lane, grp);
        };
        if (own_k) work(std::true_type{}, vr, pd, qt, dt, kout);
        else work(std::false_type{}, kr, pa, dt, qt, vout);
        __syncthreads();

        const int held = c % kGradHold;
        if (wave == 7 && lane < C) {
            float r = rq_now, k = (part[lane] + part[C + lane]) + (part[2 * C + lane] + part[3 * C + lane]);
            const int it = lane >> 4;
#pragma unroll
            for (int x = 0; x < IT; ++x) {
                const float rx = rows[x * C + lane], cx = cols[x * C + lane];
                r += x <= it ? rx : 0.0f;
                k += x >= it ? cx : 0.0f;
            }
            hold[held * C + lane] = r - k;
            if (lane == 0) resets[held] = resets_now;
        }
        if (held == kGradHold - 1 || c == nchunk - 1) {
            // chunk held - h (h from 0: the first of them in time) follows all later held ones; lane l has
            // the chunk's token C - 1 - l and sums from it to the next reset or the chunk's end
            __syncthreads();
            const int t = lane < C ? C - 1 - lane : 0;
            auto later = [&](int x) { return resets[x] >> t >> 1; };  // resets after the lane's token
            auto scan = [&](int x) {
                const unsigned long long next = later(x);
                return scan_spans_f64(lane < C ? (double)hold[x * C + t] : 0.0, next ? __builtin_ctzll(next) + 1 : C, lane);
            };
            // what the tokens before chunk y add, if `after` is what follows the chunk
            auto across = [&](double after, int y) { return (resets[y] ? 0.0 : after) + sums[y]; };
            for (int x = wave; x <= held; x += 8) {
                const double s = scan(x);
                if (lane == C - 1) sums[x] = resets[x] & 1 ? 0.0 : s;
            }
            __syncthreads();
            for (int x = wave; x <= held; x += 8) {
                double after = over;
                for (int y = 0; y < x; ++y) after = across(after, y);
                const double s = scan(x);
                const int64_t tc = t0 + (int64_t)(nchunk - 1 - (c - held + x)) * C + t;
                if (lane < C && tc < t1)
                    p.dg[(b * p.N + tc) * p.heads + h] = resets[x] >> t & 1 ? 0.0f : (float)((later(x) ? 0.0 : after) + s);
            }
            for (int y = 0; y <= held; ++y) over = across(over, y);
            __syncthreads();
        }
    }
    const int64_t tz = t1 > t0 ? t1 : t0;
    for (int64_t i = tid; i < (tN - tz) * p.dk; i += 512) kout[(tz + i / p.dk) * p.heads * p.dk + i % p.dk] = T(0);
    for (int64_t i = tid; i < (tN - tz) * p.dv; i += 512) vout[(tz + i / p.dv) * p.heads * p.dv + i % p.dv] = T(0);
    for (int64_t i = tid; i < tN - tz; i += 512) p.dg[(b * p.N + tz + i) * p.heads + h] = 0.0f;
}

// ---------------------------------------------------------------------------
// One token: S <- exp(g) S + k v^T in place, o = scale S^T q.  One workgroup per
// (row, head); a thread owns VEC columns and every (256 / columns)th row.  Where g
// starts a new sequence the old state is not read: it may be what memory held.  Bound
// by memory, for few rows by the launch: 256 requests of 12 heads of 64 in 17 us
// (101 MB of states read and written, in part from the last-level cache), one
// request in 6 us on the device.
// ---------------------------------------------------------------------------
template <typename T, int VEC>
__global__ __launch_bounds__(256) void hyena_rec_step(RecStepArgs p)
{
    __shared__ float qs[128], ks[128], acc[256 * VEC];
    const int tid = threadIdx.x;
    const int64_t b = blockIdx.x / p.heads, h = blockIdx.x % p.heads;
    const int64_t slot = p.slots ? p.slots[b] : b;
    T* o = (T*)p.o + (b * p.heads + h) * p.dv;
    if (slot < 0 || slot >= p.n_slots) {
        if (tid < p.dv) o[tid] = T(0);
        return;
    }
    const T* q = row_base<T>(p.q, b, h);
    const T* k = row_base<T>(p.k, b, h);
    const T* v = row_base<T>(p.v, b, h);
    if (tid < p.dk) {
        qs[tid] = load_one<T>(q + tid) * p.scale;
        ks[tid] = load_one<T>(k + tid);
    }
    const float g = *row_base<float>(p.g, b, h), a = expf(g);
    const bool fresh = g * 1.44269504088896340736f < kResetLog2;  // a new sequence, whatever the state holds
    const int cols = (p.dv + VEC - 1) / VEC, groups = 256 / cols;
    const int col = tid % cols, row0 = tid / cols;
    float* s = p.states + ((slot * p.heads + h) * p.dk) * p.dv + col * VEC;
    float vv[VEC], sum[VEC] = {};
#pragma unroll
    for (int j = 0; j < VEC; ++j) vv[j] = load_one<T>(v + col * VEC + j);
    __syncthreads();
    if (row0 < groups) {
        auto rows = [&](auto old) {
            for (int r = row0; r < p.dk; r += groups) {
                alignas(16) float x[VEC];
                if constexpr (!decltype(old)::value) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) x[j] = ks[r] * vv[j];
                } else {
                    if constexpr (VEC == 4) *(f32x4*)x = *(const f32x4*)(s + (int64_t)r * p.dv);
                    else x[0] = s[(int64_t)r * p.dv];
#pragma unroll
                    for (int j = 0; j < VEC; ++j) x[j] = fmaf(a, x[j], ks[r] * vv[j]);
                }
#pragma unroll
                for (int j = 0; j < VEC; ++j) sum[j] = fmaf(qs[r], x[j], sum[j]);
                if constexpr (VEC == 4) *(f32x4*)(s + (int64_t)r * p.dv) = *(const f32x4*)x;
                else s[(int64_t)r * p.dv] = x[0];
            }
        };
        if (fresh) rows(std::false_type{});
        else rows(std::true_type{});
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc[(row0 * cols + col) * VEC + j] = sum[j];
    }
    __syncthreads();
    if (tid < p.dv) {
        float x = 0.0f;
        for (int r = 0; r < groups; ++r) x += acc[r * cols * VEC + tid];
        store_one<T>(o + tid, x);
    }
}

}  // namespace hy
