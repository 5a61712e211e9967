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

// ---------------------------------------------------------------------------
// Local states of the segments.  One workgroup per (row, head, segment, role);
// wave w owns every fourth 16-column tile of the state.
// ---------------------------------------------------------------------------
template <typename T, int DK, int DV>
__global__ __launch_bounds__(256) void hyena_rec_states(RecStateArgs p)
{
    constexpr int C = kRecChunk<T>, LC = C + kPad<T>, NT = Mx<T>::kTerms;
    constexpr int KT = DK / 16, VW = DV / 64;
    using frag = typename Mx<T>::frag;
    __shared__ __attribute__((aligned(16))) T xt[DK * LC];
    __shared__ __attribute__((aligned(16))) T yt[DV * LC];
    __shared__ Decays<C> dec;

    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, grp = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t bh = blockIdx.x / p.nseg, seg = blockIdx.x % p.nseg;
    const int role = blockIdx.y;
    const int64_t b = bh / p.heads, h = bh % p.heads;
    const RView& xv = p.x[role];
    const RView& yv = p.y[role];
    const T* xp = row_base<T>(xv, b, h);
    const T* yp = row_base<T>(yv, b, h);
    const float* gp = row_base<float>(p.g, b, h);
    const int64_t nv = valid_tokens(p.lengths, b, p.N);
    const int64_t t0 = seg * (int64_t)p.seg;
    const int64_t t1 = t0 + p.seg < nv ? t0 + p.seg : nv;
    const int nchunk = t1 > t0 ? (int)((t1 - t0 + C - 1) / C) : 0;

    f32x4 S[KT][VW] = {};
    float total = 1.0f;
    Tile<T, C, DK, 256> tx;
    Tile<T, C, DV, 256> ty;
    float g = 0.0f;
    auto fetch = [&](int c) {
        const int64_t t = t0 + (int64_t)(role ? nchunk - 1 - c : c) * C;
        tx.load(xp, xv.t, xv.vec, t, t1, p.dk, tid);
        ty.load(yp, yv.t, yv.vec, t, t1, p.dv, tid);
        g = wave == 0 && lane < C && t + lane < t1 ? gp[(t + lane) * p.g.t] : 0.0f;
    };
    if (nchunk > 0) fetch(0);
    for (int c = 0; c < nchunk; ++c) {
        tx.template store_cols<LC>(xt, tid);
        ty.template store_cols<LC>(yt, tid);
        if (wave == 0) fill_decays<C>(dec, g, lane);
        __syncthreads();
        if (c + 1 < nchunk) fetch(c + 1);
        const float all = dec.head[C - 1];
        constexpr bool kLead = Mx<T>::kTerms == 2;
        const float* f = role ? (kLead ? dec.inner : dec.head) : dec.tail;
        const float lead = kLead && role ? dec.head[0] : 1.0f;
        total *= all;
#pragma unroll
        for (int v = 0; v < VW; ++v) {
            const int vt = wave + 4 * v;
            Split<T, NT> y[C / 32];
#pragma unroll
            for (int j = 0; j < C / 32; ++j) {
                const f32x8 w = join8(*(const f32x4*)(f + 32 * j + 8 * grp),
                                      *(const f32x4*)(f + 32 * j + 8 * grp + 4));
                y[j].set(Mx<T>::widen8(frag_at<T>(yt + (16 * vt + l16) * LC + 32 * j + 8 * grp)) * w);
            }
#pragma unroll
            for (int k = 0; k < KT; ++k)
                S[k][v] = update<T>(S[k][v], all, lead, y,
                                    [&](int j) { return frag_at<T>(xt + (16 * k + l16) * LC + 32 * j + 8 * grp); });
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

// LDS of the two kernels below.
template <typename T, int DA, int DC, bool TRANS> constexpr size_t rec_out_lds()
{
    constexpr int C = kRecChunk<T>, LA = DA + kPad<T>, LR = DC + kPad<T>, LC = C + kPad<T>;
    return sizeof(T) * (size_t)(2 * C * LA + DA * LC + DC * LC + C * LC + (TRANS ? C * LR : 0)) +
           sizeof(Decays<C>) + (TRANS ? 4 * C * sizeof(float) : 0);
}

template <typename T, int DK, int DV> constexpr size_t rec_grad_lds()
{
    constexpr int C = kRecChunk<T>, LK = DK + kPad<T>, LV = DV + kPad<T>, LC = C + kPad<T>;
    return sizeof(T) * (size_t)(2 * C * LK + 2 * C * LV + DK * LC + DV * LC + 2 * C * LC) +
           sizeof(Decays<C>) + sizeof(float) * (size_t)(2 * (C / 16) * C + 4 * C + 8);
}

// ---------------------------------------------------------------------------
// Outputs of one direction of reading: out_i = scale (f_i a_i . S + sum_j w_ij
// (a_i . b_j) c_j).  a = q, b = k, c = v gives o; a = do, b = v, c = k gives dq
// (TRANS: the state's rows are then the channels of c).  TRANS also writes
// rq_i = r_i . (the state's part of out_i), with the state as a split operand
// so that it keeps float32 accuracy.
//
// One workgroup of four waves per (row, head, segment).  Waves share the score
// tiles of a chunk (written to LDS in storage type) and each owns every fourth
// 16-channel tile of c: its part of the state never leaves its registers.
// ---------------------------------------------------------------------------
template <typename T, int DA, int DC, bool TRANS>
__global__ __launch_bounds__(256) void hyena_rec_out(RecArgs p)
{
    constexpr int C = kRecChunk<T>, LA = DA + kPad<T>, LR = DC + kPad<T>, LC = C + kPad<T>;
    constexpr int NT = Mx<T>::kTerms;                              // state update
    constexpr int NS = TRANS ? NT : NT == 2 ? 2 : 1;               // state as an operand
    constexpr int AT = DA / 16, CW = DC / 64, IT = C / 16;
    using frag = typename Mx<T>::frag;
    using vec4 = typename Mx<T>::vec4;
    __shared__ __attribute__((aligned(16))) char smem[rec_out_lds<T, DA, DC, TRANS>()];
    T* ar = (T*)smem;              // [C][LA]
    T* br = ar + C * LA;           // [C][LA]
    T* bt = br + C * LA;           // [DA][LC]
    T* ct = bt + DA * LC;          // [DC][LC]
    T* ps = ct + DC * LC;          // [C][LC]
    T* rr = ps + C * LC;           // [C][LR], TRANS
    char* tail = (char*)(rr + (TRANS ? C * LR : 0));
    Decays<C>& dec = *(Decays<C>*)tail;
    float* part = (float*)(tail + sizeof(Decays<C>));  // [4][C], TRANS

    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, grp = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t bh = blockIdx.x / p.nseg, seg = blockIdx.x % p.nseg;
    const int64_t b = bh / p.heads, h = bh % p.heads;
    const T* ap = row_base<T>(p.a, b, h);
    const T* bp = row_base<T>(p.b, b, h);
    const T* cp = row_base<T>(p.c, b, h);
    const T* rp = TRANS ? row_base<T>(p.r, b, h) : nullptr;
    const float* gp = row_base<float>(p.g, b, h);
    const int64_t nv = valid_tokens(p.lengths, b, p.N);
    const int64_t t0 = seg * (int64_t)p.seg;
    const int64_t tN = t0 + p.seg < p.N ? t0 + p.seg : p.N;
    const int64_t t1 = tN < nv ? tN : nv;
    const int nchunk = t1 > t0 ? (int)((t1 - t0 + C - 1) / C) : 0;
    T* const op = (T*)p.out + (b * p.N * p.heads + h) * p.dc;
    const int64_t ostride = p.heads * (int64_t)p.dc;
    const bool ovec = (p.dc & 3) == 0;

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

    Tile<T, C, DA, 256> ta, tb;
    Tile<T, C, DC, 256> tc, tr;
    float g = 0.0f;
    auto fetch = [&](int c) {
        const int64_t t = t0 + (int64_t)c * C;
        ta.load(ap, p.a.t, p.a.vec, t, t1, p.da, tid);
        tb.load(bp, p.b.t, p.b.vec, t, t1, p.da, tid);
        tc.load(cp, p.c.t, p.c.vec, t, t1, p.dc, tid);
        if constexpr (TRANS) tr.load(rp, p.r.t, p.r.vec, t, t1, p.dc, tid);
        g = wave == 0 && lane < C && t + lane < t1 ? gp[(t + lane) * p.g.t] : 0.0f;
    };
    if (nchunk > 0) fetch(0);
    for (int c = 0; c < nchunk; ++c) {
        ta.template store_rows<LA>(ar, tid);
        tb.template store_rows<LA>(br, tid);
        tb.template store_cols<LC>(bt, tid);
        tc.template store_cols<LC>(ct, tid);
        if constexpr (TRANS) tr.template store_rows<LR>(rr, tid);
        if (wave == 0) fill_decays<C>(dec, g, lane);
        __syncthreads();
        const int64_t tb0 = t0 + (int64_t)c * C;
        if (c + 1 < nchunk) fetch(c + 1);

        // scores: lower triangle of IT x IT tiles, in turn by the waves; the
        // tile right of a diagonal tile in an even row is read too: zero it
        {
            int n = 0;
#pragma unroll
            for (int i = 0; i < IT; ++i)
#pragma unroll
                for (int j = 0; j <= i; ++j, ++n) {
                    if ((n & 3) != wave) continue;
                    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int k = 0; k < DA / 32; ++k)
                        s = Mx<T>::mma(frag_at<T>(br + (16 * j + l16) * LA + 32 * k + 8 * grp),
                                       frag_at<T>(ar + (16 * i + l16) * LA + 32 * k + 8 * grp), s);
                    const int ti = 16 * i + l16, tj = 16 * j + 4 * grp;
                    const double li = dec.logs[ti];
                    const int ci = dec.count[ti];
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        s[r] = tj + r <= ti ? s[r] * (p.scale * pair_decay<C>(dec, li, ci, tj + r)) : 0.0f;
                    *(vec4*)(ps + ti * LC + tj) = Mx<T>::narrow(s);
                    if (i == j && (i & 1) == 0) {
                        const vec4 z = {};
                        *(vec4*)(ps + ti * LC + tj + 16) = z;
                    }
                }
        }
        __syncthreads();

        const float all = dec.head[C - 1];
#pragma unroll
        for (int v = 0; v < CW; ++v) {
            const int vt = wave + 4 * v;
            frag cf[C / 32];
#pragma unroll
            for (int j = 0; j < C / 32; ++j) cf[j] = frag_at<T>(ct + (16 * vt + l16) * LC + 32 * j + 8 * grp);
            Split<T, NS> sf[DA / 32];
#pragma unroll
            for (int k = 0; k < DA / 32; ++k)
                sf[k].set(join8(S[2 * k][v], S[2 * k + 1][v]) * StateScale<T>::down);
            // outputs: column = token, rows = 4 channels
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int ti = 16 * i + l16;
                f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int k = 0; k < DA / 32; ++k)
                    o = mma_split<T, NS, true>(sf[k], frag_at<T>(ar + ti * LA + 32 * k + 8 * grp), o);
                o = o * (p.scale * StateScale<T>::up * dec.head[ti]);
                if constexpr (TRANS) {
                    const f32x4 r = Mx<T>::widen(*(const vec4*)(rr + ti * LR + perm4(4 * vt + grp)));
                    float q = o[0] * r[0] + o[1] * r[1] + o[2] * r[2] + o[3] * r[3];
                    q += __shfl_xor(q, 16);
                    q += __shfl_xor(q, 32);
                    if (grp == 0) {
                        if (v == 0) part[wave * C + ti] = q;
                        else part[wave * C + ti] += q;
                    }
                }
#pragma unroll
                for (int j = 0; j <= i / 2; ++j)
                    o = Mx<T>::mma(cf[j], frag_at<T>(ps + ti * LC + 32 * j + 8 * grp), o);
                const int ch = 16 * vt + 4 * grp;
                if (tb0 + ti < t1 && ch < p.dc) {
                    T* q = op + (tb0 + ti) * ostride + ch;
                    const vec4 x = Mx<T>::narrow(o);
                    if (ovec) {
                        *(vec4*)q = x;
                    } else {
                        const T* e = (const T*)&x;
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (ch + r < p.dc) q[r] = e[r];
                    }
                }
            }
            // the state after this chunk
            Split<T, NT> y[C / 32];
#pragma unroll
            for (int j = 0; j < C / 32; ++j) {
                const f32x8 w = join8(*(const f32x4*)(dec.tail + 32 * j + 8 * grp),
                                      *(const f32x4*)(dec.tail + 32 * j + 8 * grp + 4));
                y[j].set(Mx<T>::widen8(cf[j]) * w);
            }
#pragma unroll
            for (int k = 0; k < AT; ++k)
                S[k][v] = update<T>(S[k][v], all, 1.0f, y,
                                    [&](int j) { return frag_at<T>(bt + (16 * k + l16) * LC + 32 * j + 8 * grp); });
        }
        __syncthreads();
        if constexpr (TRANS) {
            if (tid < C && tb0 + tid < t1)
                p.rq[bh * p.N + tb0 + tid] = (part[tid] + part[C + tid]) + (part[2 * C + tid] + part[3 * C + tid]);
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
// rows), four own tiles of dv (the other way round).
//
// dg_t = <S_end, dS_end> + sum_{s >= t} (q_s . dq_s - k_s . dk_s), s up to the
// segment's end: both dot products are made of float32 values (scores weighted
// by both products before any rounding, the states' parts from split operands).
// ---------------------------------------------------------------------------
template <typename T, int DK, int DV>
__global__ __launch_bounds__(512) void hyena_rec_grad(RecGradArgs p)
{
    constexpr int C = kRecChunk<T>, LK = DK + kPad<T>, LV = DV + kPad<T>, LC = C + kPad<T>;
    constexpr int NT = Mx<T>::kTerms;
    constexpr int IT = C / 16;
    using vec4 = typename Mx<T>::vec4;
    __shared__ __attribute__((aligned(16))) char smem[rec_grad_lds<T, DK, DV>()];
    T* qr = (T*)smem;              // [C][LK]
    T* kr = qr + C * LK;           // [C][LK]
    T* vr = kr + C * LK;           // [C][LV]
    T* dr = vr + C * LV;           // [C][LV]
    T* qt = dr + C * LV;           // [DK][LC]
    T* dt = qt + DK * LC;          // [DV][LC]
    T* pa = dt + DV * LC;          // [C][LC] row j, column i: w_ij (q_i . k_j)
    T* pd = pa + C * LC;           // [C][LC] w_ij (do_i . v_j)
    char* rest = (char*)(pd + C * LC);
    Decays<C>& dec = *(Decays<C>*)rest;
    float* rows = (float*)(rest + sizeof(Decays<C>));  // [IT][C] by j tile: sum over its j, per i
    float* cols = rows + IT * C;                       // [IT][C] by i tile: sum over its i, per j
    float* part = cols + IT * C;                       // [4][C] k . (state's part of dk), per wave
    float* xs = part + 4 * C;                          // [8]

    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, grp = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool own_k = wave < 4;
    const int w4 = wave & 3;
    const int64_t bh = blockIdx.x / p.nseg, seg = blockIdx.x % p.nseg;
    const int64_t b = bh / p.heads, h = bh % p.heads;
    const T* qp = row_base<T>(p.q, b, h);
    const T* kp = row_base<T>(p.k, b, h);
    const T* vp = row_base<T>(p.v, b, h);
    const T* dp = row_base<T>(p.o, b, h);
    const float* gp = row_base<float>(p.g, b, h);
    const int64_t nv = valid_tokens(p.lengths, b, p.N);
    const int64_t t0 = seg * (int64_t)p.seg;
    const int64_t tN = t0 + p.seg < p.N ? t0 + p.seg : p.N;
    const int64_t t1 = tN < nv ? tN : nv;
    const int nchunk = t1 > t0 ? (int)((t1 - t0 + C - 1) / C) : 0;
    T* const kout = (T*)p.dk_out + (b * p.N * p.heads + h) * p.dk;
    T* const vout = (T*)p.dv_out + (b * p.N * p.heads + h) * p.dv;

    // gradient of the state after this segment; xs: its product with the state
    constexpr int MT = (DK > DV ? DK : DV) / 16, MW = (DK > DV ? DK : DV) / 64;
    f32x4 S[MT][MW];
    const int64_t per = (int64_t)p.dk * p.dv;
    const float* ep = p.end ? p.end + (bh * (p.nseg + 1) + seg + 1) * per : nullptr;
    const float* sp = p.start ? p.start + (bh * (p.nseg + 1) + seg + 1) * per : nullptr;
    float cross = 0.0f;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < MW; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * m + 4 * grp + r, col = 16 * (w4 + 4 * n) + l16;
                const int kk = own_k ? col : row, vv = own_k ? row : col;
                const bool in = kk < p.dk && vv < p.dv;
                S[m][n][r] = ep && in ? ep[kk * p.dv + vv] : 0.0f;
                if (own_k && ep && sp && in) cross += S[m][n][r] * sp[kk * p.dv + vv];
            }
#pragma unroll
    for (int k = 32; k > 0; k >>= 1) cross += __shfl_xor(cross, k);
    if (lane == 0) xs[wave] = cross;
    __syncthreads();
    double over = 0.0;  // wave 0: <S, dS> after the chunk at hand
    if (wave == 0) over = ((double)xs[0] + (double)xs[1]) + ((double)xs[2] + (double)xs[3]);

    Tile<T, C, DK, 512> tq, tk;
    Tile<T, C, DV, 512> tv, td;
    float g = 0.0f, rq = 0.0f;
    auto fetch = [&](int c) {
        const int64_t t = t0 + (int64_t)(nchunk - 1 - c) * C;
        tq.load(qp, p.q.t, p.q.vec, t, t1, p.dk, tid);
        tk.load(kp, p.k.t, p.k.vec, t, t1, p.dk, tid);
        tv.load(vp, p.v.t, p.v.vec, t, t1, p.dv, tid);
        td.load(dp, p.o.t, p.o.vec, t, t1, p.dv, tid);
        const bool in = wave == 0 && lane < C && t + lane < t1;
        g = in ? gp[(t + lane) * p.g.t] : 0.0f;
        rq = in ? p.rq[bh * p.N + t + lane] : 0.0f;
    };
    if (nchunk > 0) fetch(0);
    for (int c = 0; c < nchunk; ++c) {
        tq.template store_rows<LK>(qr, tid);
        tk.template store_rows<LK>(kr, tid);
        tv.template store_rows<LV>(vr, tid);
        td.template store_rows<LV>(dr, tid);
        tq.template store_cols<LC>(qt, tid);
        td.template store_cols<LC>(dt, tid);
        const float rq_now = rq, g_now = g;
        if (wave == 0) fill_decays<C>(dec, g, lane);
        __syncthreads();
        const int64_t tb0 = t0 + (int64_t)(nchunk - 1 - c) * C;
        if (c + 1 < nchunk) fetch(c + 1);

        // both scores of each pair of tiles: rows i, columns j <= i
        {
            int n = 0;
#pragma unroll
            for (int i = 0; i < IT; ++i)
#pragma unroll
                for (int j = 0; j <= i; ++j, ++n) {
                    if ((n & 7) != wave) continue;
                    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f}, d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int k = 0; k < DK / 32; ++k)
                        s = Mx<T>::mma(frag_at<T>(qr + (16 * i + l16) * LK + 32 * k + 8 * grp),
                                       frag_at<T>(kr + (16 * j + l16) * LK + 32 * k + 8 * grp), s);
#pragma unroll
                    for (int k = 0; k < DV / 32; ++k)
                        d = Mx<T>::mma(frag_at<T>(dr + (16 * i + l16) * LV + 32 * k + 8 * grp),
                                       frag_at<T>(vr + (16 * j + l16) * LV + 32 * k + 8 * grp), d);
                    const int tj = 16 * j + l16, ti = 16 * i + 4 * grp;
                    const double lj = dec.logs[tj];
                    const int cj = dec.count[tj];
                    f32x4 both;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const bool in = tj <= ti + r && dec.count[ti + r] == cj;
                        const float w = p.scale * __builtin_amdgcn_exp2f((float)(dec.logs[ti + r] - lj));
                        const float sw = s[r] * w;
                        both[r] = in ? sw * d[r] : 0.0f;
                        s[r] = in ? sw : 0.0f;
                        d[r] = in ? d[r] * w : 0.0f;
                    }
                    *(vec4*)(pa + tj * LC + ti) = Mx<T>::narrow(s);
                    *(vec4*)(pd + tj * LC + ti) = Mx<T>::narrow(d);
                    if (i == j && (j & 1) == 1) {
                        const vec4 z = {};
                        *(vec4*)(pa + tj * LC + ti - 16) = z;
                        *(vec4*)(pd + tj * LC + ti - 16) = z;
                    }
                    float col = (both[0] + both[1]) + (both[2] + both[3]);
                    col += __shfl_xor(col, 16);
                    col += __shfl_xor(col, 32);
                    if (grp == 0) cols[i * C + tj] = col;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        float x = both[r];
                        x += __shfl_xor(x, 1);
                        x += __shfl_xor(x, 2);
                        x += __shfl_xor(x, 4);
                        x += __shfl_xor(x, 8);
                        if (l16 == 0) rows[j * C + ti + r] = x;
                    }
                }
        }
        __syncthreads();

        const float all = dec.head[C - 1];
        auto work = [&](auto own, const T* across, int la, const T* scores, const T* fold, const T* add,
                        T* out, int width) {
            // own (0: dk, 1: dv); across: rows that dS multiplies (v or k);
            // scores and fold: dk_j += scores_ij fold_i; add: the other tensor of dS's update
            constexpr int O = decltype(own)::value;
            constexpr int DM = O == 0 ? DV : DK, DN = O == 0 ? DK : DV;  // dS rows, columns
            constexpr int NS = O == 0 ? NT : NT == 2 ? 2 : 1;
#pragma unroll
            for (int n = 0; n < DN / 64; ++n) {
                const int nt = w4 + 4 * n;
                typename Mx<T>::frag ff[C / 32];
#pragma unroll
                for (int i = 0; i < C / 32; ++i)
                    ff[i] = frag_at<T>(fold + (16 * nt + l16) * LC + 32 * i + 8 * grp);
                Split<T, NS> sf[DM / 32];
#pragma unroll
                for (int k = 0; k < DM / 32; ++k)
                    sf[k].set(join8(S[2 * k][n], S[2 * k + 1][n]) * StateScale<T>::down);
#pragma unroll
                for (int j = 0; j < IT; ++j) {
                    const int tj = 16 * j + l16;
                    f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int k = 0; k < DM / 32; ++k)
                        x = mma_split<T, NS, true>(sf[k], frag_at<T>(across + tj * la + 32 * k + 8 * grp), x);
                    x = x * (StateScale<T>::up * dec.tail[tj]);
                    if constexpr (O == 0) {
                        const f32x4 kk = Mx<T>::widen(*(const vec4*)(kr + tj * LK + perm4(4 * nt + grp)));
                        float q = x[0] * kk[0] + x[1] * kk[1] + x[2] * kk[2] + x[3] * kk[3];
                        q += __shfl_xor(q, 16);
                        q += __shfl_xor(q, 32);
                        if (grp == 0) {
                            if (n == 0) part[w4 * C + tj] = q;
                            else part[w4 * C + tj] += q;
                        }
                    }
#pragma unroll
                    for (int i = j / 2; i < C / 32; ++i)
                        x = Mx<T>::mma(ff[i], frag_at<T>(scores + tj * LC + 32 * i + 8 * grp), x);
                    const int ch = 16 * nt + 4 * grp;
                    if (tb0 + tj < t1 && ch < width) {
                        T* q = out + (tb0 + tj) * p.heads * width + ch;
                        const vec4 y = Mx<T>::narrow(x);
                        if ((width & 3) == 0) {
                            *(vec4*)q = y;
                        } else {
                            const T* e = (const T*)&y;
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                if (ch + r < width) q[r] = e[r];
                        }
                    }
                }
                constexpr bool kLead = Mx<T>::kTerms == 2;
                const float* f = kLead ? dec.inner : dec.head;
                const float lead = kLead ? p.scale * dec.head[0] : 1.0f;
                Split<T, NT> y[C / 32];
#pragma unroll
                for (int i = 0; i < C / 32; ++i) {
                    const f32x8 w = join8(*(const f32x4*)(f + 32 * i + 8 * grp), *(const f32x4*)(f + 32 * i + 8 * grp + 4));
                    y[i].set(Mx<T>::widen8(ff[i]) * (kLead ? w : w * p.scale));
                }
#pragma unroll
                for (int m = 0; m < DM / 16; ++m)
                    S[m][n] = update<T>(S[m][n], all, lead, y,
                                        [&](int i) { return frag_at<T>(add + (16 * m + l16) * LC + 32 * i + 8 * grp); });
            }
        };
        if (own_k) work(std::integral_constant<int, 0>{}, vr, LV, pd, qt, dt, kout, p.dk);
        else work(std::integral_constant<int, 1>{}, kr, LK, pa, dt, qt, vout, p.dv);
        __syncthreads();

        if (wave == 0) {
            // per token: q . dq - k . dk, then the sum from each token to the chunk's end
            double x = 0.0;
            if (lane < C) {
                float r = rq_now, k = (part[lane] + part[C + lane]) + (part[2 * C + lane] + part[3 * C + lane]);
                const int it = lane >> 4;
                for (int j = 0; j <= it; ++j) r += rows[j * C + lane];
                for (int i = it; i < IT; ++i) k += cols[i * C + lane];
                x = (double)r - (double)k;
            }
#pragma unroll
            for (int k = 1; k < C; k <<= 1) {
                const int2 v = __builtin_bit_cast(int2, x);
                const double o = __builtin_bit_cast(double, make_int2(__shfl_down(v.x, k), __shfl_down(v.y, k)));
                if (lane + k < C) x += o;
            }
            const int2 v = __builtin_bit_cast(int2, x);
            const double first = __builtin_bit_cast(double, make_int2(__shfl(v.x, 0), __shfl(v.y, 0)));
            if (lane < C && tb0 + lane < t1) {
                const bool reset = g_now * 1.44269504088896340736f < kResetLog2;
                p.dg[(b * p.N + tb0 + lane) * p.heads + h] = reset ? 0.0f : (float)(over + x);
            }
            over += first;
        }
    }
    const int64_t tz = t1 > t0 ? t1 : t0;
    for (int64_t i = tid; i < (tN - tz) * p.dk; i += 512) kout[(tz + i / p.dk) * p.heads * p.dk + i % p.dk] = T(0);
    for (int64_t i = tid; i < (tN - tz) * p.dv; i += 512) vout[(tz + i / p.dv) * p.heads * p.dv + i % p.dv] = T(0);
    for (int64_t i = tid; i < tN - tz; i += 512) p.dg[(b * p.N + tz + i) * p.heads + h] = 0.0f;
    if (p.d_state != nullptr && !own_k) {
        float* out = p.d_state + bh * per;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < MW; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int kk = 16 * m + 4 * grp + r, vv = 16 * (w4 + 4 * n) + l16;
                    if (kk < p.dk && vv < p.dv) out[kk * p.dv + vv] = S[m][n][r];
                }
    }
}

// ---------------------------------------------------------------------------
// One token: S <- exp(g) S + k v^T in place, o = scale S^T q.  One workgroup per
// (row, head); a thread owns VEC columns and every (256 / columns)th row.
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
    const float a = expf(*row_base<float>(p.g, b, h));
    const int cols = (p.dv + VEC - 1) / VEC, groups = 256 / cols;
    const int col = tid % cols, row0 = tid / cols;
    float* s = p.states + ((slot * p.heads + h) * p.dk) * p.dv + col * VEC;
    float vv[VEC], sum[VEC] = {};
#pragma unroll
    for (int j = 0; j < VEC; ++j) vv[j] = load_one<T>(v + col * VEC + j);
    __syncthreads();
    if (row0 < groups) {
        for (int r = row0; r < p.dk; r += groups) {
            alignas(16) float x[VEC];
            if constexpr (VEC == 4) *(f32x4*)x = *(const f32x4*)(s + (int64_t)r * p.dv);
            else x[0] = s[(int64_t)r * p.dv];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                x[j] = fmaf(a, x[j], ks[r] * vv[j]);
                sum[j] = fmaf(qs[r], x[j], sum[j]);
            }
            if constexpr (VEC == 4) *(f32x4*)(s + (int64_t)r * p.dv) = *(const f32x4*)x;
            else s[(int64_t)r * p.dv] = x[0];
        }
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
