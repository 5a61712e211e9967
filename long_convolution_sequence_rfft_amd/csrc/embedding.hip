// embedding.hip -- rows of a table by token, times a factor, and the table's
// gradient by sorted tokens (include/hyena.h).
//
// Forward is a gather: 4 bytes of a token, then its row, read and written once.
//
// Backward.  Sums in an order that atomics decide would differ from call to call,
// so tokens are sorted first, in their order within each value:
//   hyena_embedding_sort   workgroup g has the values v with v % groups = g (the
//       frequent tokens of a text have low numbers and would all be one
//       workgroup's in a cut by ranges).  It reads all tokens twice: counts its
//       values (each wave its own part of the tokens), which with the count of the
//       tokens of lower groups gives every value a place, then writes its tokens
//       there, in order.  One launch, and no workgroup waits for another.
//   hyena_embedding_sums   teams of lanes take runs of the sorted list of one
//       length, so a value that is everywhere is shared out like any other.  A
//       value that lies within one run is done: its row is written.  One that
//       reaches over a run's end leaves its sum there.  Other workgroups of the
//       same launch write the zeros of values without tokens.
//   hyena_embedding_joins  adds the pieces of values that reach over runs.
// Bound by memory: each gradient row is read once, each row of the table written
// once.
#include "rows.h"

namespace hy {

namespace {

constexpr const char* kWho = "embedding";
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kSortGroups = 256;   // at least; more where a group would have more values than kSortValues
constexpr int kSortValues = 768;   // counters of a wave: 48 KB of LDS in all
constexpr int kSortTokens = 8;     // loads of a wave under way
constexpr int kSumRows = 4;        // gradient rows of a team under way
constexpr int64_t kSumTeams = 8192;  // runs are no shorter than kSumRows, and as short as this many of them allow

struct EmbedArgs {
    Rows tokens, rows;   // rows: d_out
    const void* table;
    void* out;           // backward: d_table
    int64_t total;       // B * N
    uint32_t N, rows_N;  // row_at, of the tokens and of the rows
    int32_t V, d;
    int32_t lanes, per;  // lanes of a team, units of a lane
    int32_t pairs;
    int32_t accumulate;
    float scale;
    int32_t groups;      // of the sort, a power of two
    int32_t run;         // tokens of a run
    int32_t sum_groups;  // workgroups of the sums, fill_groups behind them
    int32_t fill_groups;
    int32_t* counts;     // [V]
    int2* sorted;        // [total] value and token, in order; [total].x the number of tokens that take part
    float* part;         // [runs][2][d]: sums that reach over a run's start and over its end
};

__device__ __forceinline__ int token_at(const EmbedArgs& p, int64_t t) { return *row_at<int32_t>(p.tokens, t, p.N); }

template <typename T, bool VEC> __global__ __launch_bounds__(256) void hyena_embedding_gather(EmbedArgs p)
{
    constexpr int K = kUnit<T>;
    const int teams = 256 / p.lanes, team = threadIdx.x / p.lanes, tl = threadIdx.x % p.lanes;
    for (int64_t t = (int64_t)blockIdx.x * teams + team; t < p.total; t += (int64_t)gridDim.x * teams) {
        const int v = token_at(p, t);
        const bool in = (uint32_t)v < (uint32_t)p.V;
        const T* row = (const T*)p.table + (int64_t)(in ? v : 0) * p.d;
        T* out = (T*)p.out + t * p.d;
        for (int c = tl * K; c < p.d; c += p.lanes * K) {
            float x[K];
#pragma unroll
            for (int i = 0; i < K; ++i) x[i] = 0.0f;
            if (in) load_unit<T, VEC>(row, c, p.d, p.pairs, x);
#pragma unroll
            for (int i = 0; i < K; ++i) x[i] = in ? x[i] * p.scale : 0.0f;
            store_unit<T, VEC>(out, c, p.d, p.pairs, x);
        }
    }
}

// Sum of one value over a workgroup's threads.
__device__ __forceinline__ int workgroup_sum(int x, int* lds)
{
    for (int m = 1; m < 64; m *= 2) x += __shfl_xor(x, m);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    x = 0;
    for (int w = 0; w < kSortWaves; ++w) x += lds[w];
    return x;
}

__global__ __launch_bounds__(kSortThreads) void hyena_embedding_sort(EmbedArgs p)
{
    extern __shared__ int counters[];  // [values][waves]
    __shared__ int lds[kSortWaves];
    const int group = blockIdx.x, shift = __builtin_ctz(p.groups);
    const int values = (p.V - group + p.groups - 1) >> shift;  // v = group + groups * i, i < values
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    // each wave a part of the tokens, whole 64s of them
    const int64_t each = ((p.total + 64 * kSortWaves - 1) / (64 * kSortWaves)) * 64;
    const int64_t first = each * wave, last = first + each < p.total ? first + each : p.total;

    for (int i = threadIdx.x; i < values * kSortWaves; i += kSortThreads) counters[i] = 0;
    __syncthreads();
    int lower = 0, all = 0;
    for (int64_t t0 = first; t0 < last; t0 += 64 * kSortTokens) {
        int v[kSortTokens];
#pragma unroll
        for (int k = 0; k < kSortTokens; ++k) {
            const int64_t t = t0 + 64 * k + lane;
            v[k] = t < last ? token_at(p, t) : -1;
        }
#pragma unroll
        for (int k = 0; k < kSortTokens; ++k) {
            const bool in = (uint32_t)v[k] < (uint32_t)p.V;
            const int g = v[k] & (p.groups - 1);
            all += in;
            lower += in && g < group;
            if (in && g == group) atomicAdd(&counters[(v[k] >> shift) * kSortWaves + wave], 1);
        }
    }
    lower = workgroup_sum(lower, lds);
    all = workgroup_sum(all, lds);
    __syncthreads();
    // counts to places: thread i has the counters of the values [i n, (i + 1) n)
    const int n = (values + kSortThreads - 1) / kSortThreads;
    int mine = 0;
    for (int k = 0; k < n; ++k) {
        const int i = threadIdx.x * n + k;
        if (i >= values) break;
        int c = 0;
        for (int w = 0; w < kSortWaves; ++w) c += counters[i * kSortWaves + w];
        p.counts[group + (int64_t)p.groups * i] = c;
        mine += c;
    }
    int before = mine;  // inclusive sum over the wave, then over the waves
    for (int m = 1; m < 64; m *= 2) {
        const int up = __shfl_up(before, m);
        if (lane >= m) before += up;
    }
    __syncthreads();
    if (lane == 63) lds[wave] = before;
    __syncthreads();
    before -= mine;
    for (int w = 0; w < wave; ++w) before += lds[w];
    before += lower;
    for (int k = 0; k < n; ++k) {
        const int i = threadIdx.x * n + k;
        if (i >= values) break;
        for (int w = 0; w < kSortWaves; ++w) {
            const int c = counters[i * kSortWaves + w];
            counters[i * kSortWaves + w] = before;
            before += c;
        }
    }
    __syncthreads();
    if (group == 0 && threadIdx.x == 0) p.sorted[p.total] = make_int2(all, 0);
    // the same tokens again, each to its value's place; a wave's are in order
    for (int64_t t0 = first; t0 < last; t0 += 64 * kSortTokens) {
        int v[kSortTokens];
#pragma unroll
        for (int k = 0; k < kSortTokens; ++k) {
            const int64_t t = t0 + 64 * k + lane;
            v[k] = t < last ? token_at(p, t) : -1;
        }
#pragma unroll
        for (int k = 0; k < kSortTokens; ++k) {
            const bool own = (uint32_t)v[k] < (uint32_t)p.V && (v[k] & (p.groups - 1)) == group;
            uint64_t left = __ballot(own);
            while (left != 0) {  // one value of these 64 tokens after the other
                const int one = __builtin_amdgcn_readlane(v[k], __builtin_ctzll(left));
                const bool same = own && v[k] == one;
                const uint64_t all_same = __ballot(same);
                int* counter = &counters[(one >> shift) * kSortWaves + wave];
                const int place = *counter;
                if (same) {
                    const int at = place + __popcll(all_same & (((uint64_t)1 << lane) - 1));
                    p.sorted[at] = make_int2(one, (int)(t0 + 64 * k + lane));
                }
                *counter = place + __popcll(all_same);  // every lane the same value
                left &= ~all_same;
            }
        }
    }
}

// The unit at channel c of a row of the table's gradient: x times the scale, or
// added to what is there.
template <typename T, bool VEC>
__device__ __forceinline__ void write_sum(const EmbedArgs& p, int v, int c, float (&x)[kUnit<T>])
{
    constexpr int K = kUnit<T>;
    T* row = (T*)p.out + (int64_t)v * p.d;
    if (p.accumulate) {
        float old[K];
        load_unit<T, VEC>(row, c, p.d, p.pairs, old);
#pragma unroll
        for (int i = 0; i < K; ++i) x[i] = fmaf(x[i], p.scale, old[i]);
    } else {
#pragma unroll
        for (int i = 0; i < K; ++i) x[i] *= p.scale;
    }
    store_unit<T, VEC>(row, c, p.d, p.pairs, x);
}

// U units of a lane at a time; blockIdx.y: which of the row's blocks of U * lanes units.
template <typename T, bool VEC, int U> __global__ __launch_bounds__(256) void hyena_embedding_sums(EmbedArgs p)
{
    constexpr int K = kUnit<T>;
    const int teams = 256 / p.lanes, team = threadIdx.x / p.lanes, tl = threadIdx.x % p.lanes;
    const int c0 = (int)blockIdx.y * U * p.lanes * K;
    float zero[K];
#pragma unroll
    for (int i = 0; i < K; ++i) zero[i] = 0.0f;
    if ((int)blockIdx.x >= p.sum_groups) {
        // zeros where no token is
        const int64_t step = (int64_t)p.fill_groups * teams;
        for (int64_t v = (int64_t)((int)blockIdx.x - p.sum_groups) * teams + team; v < p.V; v += step) {
            if (p.counts[v] != 0) continue;
            T* row = (T*)p.out + v * p.d;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + (tl + u * p.lanes) * K;
                if (c < p.d) store_unit<T, VEC>(row, c, p.d, p.pairs, zero);
            }
        }
        return;
    }
    const int64_t n = p.sorted[p.total].x;  // tokens that take part
    const int64_t run = (int64_t)blockIdx.x * teams + team, first = run * p.run;
    if (first >= n) return;
    const int64_t last = first + p.run < n ? first + p.run : n;
    float s[U][K];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < K; ++i) s[u][i] = 0.0f;
    bool open = first > 0 && p.sorted[first - 1].x == p.sorted[first].x;  // the value began before this run
    const int next_value = last < n ? p.sorted[last].x : -1;
    for (int64_t i0 = first; i0 < last; i0 += kSumRows) {
        int2 e[kSumRows + 1];
        float x[kSumRows][U][K];
#pragma unroll
        for (int k = 0; k < kSumRows; ++k) {
            const int64_t i = i0 + k < last ? i0 + k : last - 1;
            e[k] = p.sorted[i];
        }
        e[kSumRows] = i0 + kSumRows < last ? p.sorted[i0 + kSumRows] : make_int2(next_value, 0);
#pragma unroll
        for (int k = 0; k < kSumRows; ++k) {
            const T* row = row_at<T>(p.rows, e[k].y, p.rows_N);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + (tl + u * p.lanes) * K;
                if (c < p.d) load_unit<T, VEC>(row, c, p.d, p.pairs, x[k][u]);
            }
        }
#pragma unroll
        for (int k = 0; k < kSumRows; ++k) {
            if (i0 + k >= last) break;
            const bool at_end = i0 + k + 1 == last;
            const int following = at_end ? next_value : e[k + 1].x;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < K; ++i) s[u][i] += x[k][u][i];
            if (following == e[k].x && !at_end) continue;
            // a value's last token here: its row, or a piece of it
            const bool on = following == e[k].x;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + (tl + u * p.lanes) * K;
                if (c < p.d) {
                    if (open || on) {
                        float* part = p.part + (run * 2 + (open ? 0 : 1)) * p.d;
#pragma unroll
                        for (int i = 0; i < K; ++i)
                            if (VEC || c + i < p.d) part[c + i] = s[u][i];
                    } else {
                        write_sum<T, VEC>(p, e[k].x, c, s[u]);
                    }
                }
#pragma unroll
                for (int i = 0; i < K; ++i) s[u][i] = 0.0f;
            }
            open = false;
        }
    }
}

// A workgroup for each run: the value that begins in it and goes on in the next
// ones, 64 units of its row at a time, every wave some of the pieces.
template <typename T, bool VEC> __global__ __launch_bounds__(256) void hyena_embedding_joins(EmbedArgs p)
{
    constexpr int K = kUnit<T>;
    __shared__ float lds[4][64 * K];
    const int64_t n = p.sorted[p.total].x;
    const int64_t run = blockIdx.x, first = run * p.run, end = first + p.run;
    if (end >= n) return;  // nothing comes after it
    const int v = p.sorted[end - 1].x;
    if (p.sorted[end].x != v) return;
    const int count = p.counts[v];
    // where it began: in this run, or this workgroup has nothing to do
    if (first > 0 && p.sorted[first - 1].x == v) return;
    int64_t begin = first;
    while (p.sorted[begin].x != v) ++begin;
    const int64_t pieces = (begin + count - 1) / p.run - run;  // runs after this one
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    for (int c0 = 0; c0 < p.d; c0 += 64 * K) {
        const int c = c0 + lane * K;
        float s[K];
#pragma unroll
        for (int i = 0; i < K; ++i) s[i] = 0.0f;
        if (c < p.d) {
            if (wave == 0) {
                const float* part = p.part + (run * 2 + 1) * p.d;
#pragma unroll
                for (int i = 0; i < K; ++i)
                    if (VEC || c + i < p.d) s[i] = part[c + i];
            }
#pragma unroll 4
            for (int64_t k = 1 + wave; k <= pieces; k += 4) {
                const float* part = p.part + (run + k) * 2 * p.d;
#pragma unroll
                for (int i = 0; i < K; ++i)
                    if (VEC || c + i < p.d) s[i] += part[c + i];
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < K; ++i) lds[wave][i * 64 + lane] = s[i];
        __syncthreads();
        if (wave == 0 && c < p.d) {
#pragma unroll
            for (int i = 0; i < K; ++i) s[i] = lds[0][i * 64 + lane] + lds[1][i * 64 + lane] + lds[2][i * 64 + lane] + lds[3][i * 64 + lane];
            write_sum<T, VEC>(p, v, c, s);
        }
    }
}

hyena_status refuse(const char* what) { return fail(HYENA_ERR_INVALID_ARGUMENT, std::string(kWho) + ": " + what); }

hyena_status embed_sizes(const hyena_embedding* op)
{
    if (op == nullptr) return refuse("the description is NULL");
    if (op->B < 1 || op->N < 1 || op->V < 1 || op->d < 1) return refuse("B, N, V and d must be at least 1");
    if (op->V > 1 << 24 || op->d > 65536) return fail(HYENA_ERR_UNSUPPORTED, "embedding: V at most 2^24 and d at most 65536");
    if (op->B > 1 << 30 || op->N > 1 << 30 || op->B * op->N > 1 << 30)
        return fail(HYENA_ERR_UNSUPPORTED, "embedding: at most 2^30 tokens");
    return check_io(kWho, op->io_dtype);
}

struct EmbedSpace {
    int64_t run, runs;
    size_t sorted, counts, part, total;  // byte offsets and the size
};

EmbedSpace embed_space(const hyena_embedding* op)
{
    EmbedSpace w;
    const int64_t T = op->B * op->N;
    const int64_t most = (T + kSumTeams - 1) / kSumTeams;
    w.run = most < kSumRows ? kSumRows : (most + kSumRows - 1) / kSumRows * kSumRows;
    w.runs = (T + w.run - 1) / w.run;
    auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
    w.sorted = 0;
    w.counts = up((size_t)(T + 1) * sizeof(int2));
    w.part = w.counts + up((size_t)op->V * 4);
    w.total = w.part + (size_t)w.runs * 2 * (size_t)op->d * 4;
    return w;
}

void team_shape(EmbedArgs& a, size_t element)
{
    // as many lanes of a wave as leave the fewest idle with at most 4 units each
    const int units = (int)((a.d * element + 15) / 16);
    int best = 64;
    for (int n = 64; n >= 1; n /= 2) {
        const int per = (units + n - 1) / n;
        if (per > 4) break;
        if (per * n < ((units + best - 1) / best) * best) best = n;
    }
    a.lanes = best;
    a.per = (units + best - 1) / best;
}

template <typename T, int U> hyena_status launch_sums(const EmbedArgs& a, bool vec, hipStream_t s)
{
    const int block = U * a.lanes * kUnit<T>;
    const dim3 grid((unsigned)(a.sum_groups + a.fill_groups), (unsigned)((a.d + block - 1) / block));
    if (vec)
        HY_LAUNCH(kernel_label("hyena_embedding_sums", type_label<T>(), true, U), (hyena_embedding_sums<T, true, U>), grid, dim3(256), 0, s, a);
    else
        HY_LAUNCH(kernel_label("hyena_embedding_sums", type_label<T>(), false, U), (hyena_embedding_sums<T, false, U>), grid, dim3(256), 0, s, a);
    return launched();
}

template <typename T> hyena_status embed_backward(const EmbedArgs& a, bool vec, int64_t runs, hipStream_t s)
{
    hyena_status st;
    HY_LAUNCH(kernel_label("hyena_embedding_sort"), hyena_embedding_sort, dim3((unsigned)a.groups), dim3(kSortThreads),
              (size_t)((a.V + a.groups - 1) / a.groups) * kSortWaves * 4, s, a);
    if ((st = launched()) != HYENA_OK) return st;
    const int u = a.per < 4 ? a.per : 4;
    st = u == 1 ? launch_sums<T, 1>(a, vec, s) : u == 2 ? launch_sums<T, 2>(a, vec, s) : u == 3 ? launch_sums<T, 3>(a, vec, s) : launch_sums<T, 4>(a, vec, s);
    if (st != HYENA_OK || runs < 2) return st;
    if (vec)
        HY_LAUNCH(kernel_label("hyena_embedding_joins", type_label<T>(), true), (hyena_embedding_joins<T, true>), dim3((unsigned)(runs - 1)), dim3(256), 0, s, a);
    else
        HY_LAUNCH(kernel_label("hyena_embedding_joins", type_label<T>(), false), (hyena_embedding_joins<T, false>), dim3((unsigned)(runs - 1)), dim3(256), 0, s, a);
    return launched();
}

EmbedArgs embed_args(const hyena_embedding* op)
{
    EmbedArgs a{};
    hyena_rows tokens = plain_rows(op->tokens, op->B, op->N);
    int64_t N = op->N;
    hyena_rows* one[1] = {&tokens};
    flatten_rows(one, 1, op->B, &N);
    a.tokens = Rows{tokens.data, tokens.batch, tokens.token};
    a.N = (uint32_t)N;
    a.total = op->B * op->N;
    a.V = (int32_t)op->V;
    a.d = (int32_t)op->d;
    a.scale = op->scale;
    team_shape(a, element_bytes(op->io_dtype));
    return a;
}

}  // namespace
}  // namespace hy

using namespace hy;

extern "C" {

hyena_status hyena_embedding_forward(const hyena_embedding* op, const void* table, void* out, void* stream)
{
    hyena_status st = embed_sizes(op);
    if (st != HYENA_OK) return st;
    const size_t e = element_bytes(op->io_dtype);
    if ((st = check_rows(kWho, op->tokens, "tokens", 4)) != HYENA_OK) return st;
    if (table == nullptr || out == nullptr) return refuse("table or out is NULL");
    if ((uintptr_t)table % e != 0 || (uintptr_t)out % e != 0) return refuse("table or out is not aligned to its element");
    EmbedArgs a = embed_args(op);
    const Span ins[2] = {rows_span(plain_rows(op->tokens, op->B, op->N), op->B, op->N, 1, 4),
                         Span{table, (size_t)(op->V * op->d) * e}};
    const Named outs[1] = {{Span{out, (size_t)a.total * (size_t)op->d * e}, "out"}};
    if ((st = check_apart(kWho, ins, 2, outs, 1)) != HYENA_OK) return st;
    RowShape made(op->d, e);
    made.dense(table);
    made.dense(out);
    a.pairs = made.made_of() >= kMadeOfPairs;
    a.table = table;
    a.out = out;
    const int64_t teams = 256 / a.lanes, need = (a.total + teams - 1) / teams, most = (int64_t)1 << 20;
    const dim3 grid((unsigned)(need < most ? need : most));
    const bool vec = made.made_of() == kMadeOfUnits;
    const hipStream_t s = (hipStream_t)stream;
    return by_io(op->io_dtype, [&](auto* t) {
        using T = std::remove_pointer_t<decltype(t)>;
        if (vec)
            HY_LAUNCH(kernel_label("hyena_embedding_gather", type_label<T>(), true), (hyena_embedding_gather<T, true>), grid, dim3(256), 0, s, a);
        else
            HY_LAUNCH(kernel_label("hyena_embedding_gather", type_label<T>(), false), (hyena_embedding_gather<T, false>), grid, dim3(256), 0, s, a);
        return launched();
    });
}

hyena_status hyena_embedding_scratch_bytes(const hyena_embedding* op, size_t* bytes)
{
    const hyena_status st = embed_sizes(op);
    if (st != HYENA_OK) return st;
    if (bytes == nullptr) return refuse("bytes is NULL");
    *bytes = embed_space(op).total;
    return HYENA_OK;
}

hyena_status hyena_embedding_backward(const hyena_embedding* op, const hyena_rows* d_out, void* d_table, int32_t accumulate,
                                      void* scratch, void* stream)
{
    hyena_status st = embed_sizes(op);
    if (st != HYENA_OK) return st;
    const size_t e = element_bytes(op->io_dtype);
    if (d_out == nullptr) return refuse("d_out is NULL");
    if ((st = check_rows(kWho, op->tokens, "tokens", 4)) != HYENA_OK || (st = check_rows(kWho, *d_out, "d_out", e)) != HYENA_OK)
        return st;
    if (d_table == nullptr || (uintptr_t)d_table % e != 0) return refuse("d_table is NULL or not aligned to its element");
    if (scratch == nullptr || (uintptr_t)scratch % 16 != 0) return refuse("scratch is NULL or not 16-byte aligned");
    EmbedArgs a = embed_args(op);
    hyena_rows rows = plain_rows(*d_out, op->B, op->N);
    const EmbedSpace w = embed_space(op);
    const Span ins[2] = {rows_span(plain_rows(op->tokens, op->B, op->N), op->B, op->N, 1, 4),
                         rows_span(rows, op->B, op->N, op->d, e)};
    const Named outs[2] = {{Span{d_table, (size_t)(op->V * op->d) * e}, "d_table"}, {Span{scratch, w.total}, "scratch"}};
    if ((st = check_apart(kWho, ins, 2, outs, 2)) != HYENA_OK) return st;
    RowShape made(op->d, e);
    made.add(rows);
    made.dense(d_table);
    a.pairs = made.made_of() >= kMadeOfPairs;
    int64_t N = op->N;
    hyena_rows* one[1] = {&rows};
    flatten_rows(one, 1, op->B, &N);
    a.rows = Rows{rows.data, rows.batch, rows.token};
    a.rows_N = (uint32_t)N;
    a.out = d_table;
    a.accumulate = accumulate != 0;
    a.groups = kSortGroups;
    while ((a.V + a.groups - 1) / a.groups > kSortValues) a.groups *= 2;
    a.run = (int32_t)w.run;
    a.sorted = (int2*)((char*)scratch + w.sorted);
    a.counts = (int32_t*)((char*)scratch + w.counts);
    a.part = (float*)((char*)scratch + w.part);
    const int64_t teams = 256 / a.lanes;
    a.sum_groups = (int32_t)((w.runs + teams - 1) / teams);
    const int64_t fill = (a.V + teams - 1) / teams;
    a.fill_groups = a.accumulate ? 0 : (int32_t)(fill < 2048 ? fill : 2048);
    const bool vec = made.made_of() == kMadeOfUnits;
    return by_io(op->io_dtype, [&](auto* t) {
        return embed_backward<std::remove_pointer_t<decltype(t)>>(a, vec, w.runs, (hipStream_t)stream);
    });
}

}  // extern "C"
