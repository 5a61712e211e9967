// embedding.hip -- rows of a table by token, times a factor, and the table's
// gradient by sorted tokens (include/hyena.h).
//
// Forward is a gather: 4 bytes of a token, then its row, read and written once (16384 tokens of
// width 768 in bf16 8.4 us, the table's rows mostly from the last-level cache; 32 tokens 3.0).
//
// Backward.  Sums in an order that atomics decide would differ from call to call,
// so tokens are sorted first, in their order within each value:
//   hyena_embedding_sort   workgroup g has the values v with v % groups = g (the
//       frequent tokens of a text have low numbers and would all be one
//       workgroup's in a cut by ranges).  It reads all tokens twice: counts its
//       values (each wave its own part of the tokens), which with the count of the
//       tokens of lower groups gives every value a place, then writes its tokens
//       there, in order.  One launch, and no workgroup waits for another.  Of many
//       tokens hyena_embedding_deal first makes lists: each workgroup deals its 4096
//       tokens out to the groups, which then read what is theirs only.
//   hyena_embedding_sums   teams of lanes take runs of the sorted list of one
//       length, so a value that is everywhere is shared out like any other.  A
//       value that lies within one run is done: its row is written.  One that
//       reaches over a run's end leaves its sum there.  Other workgroups of the
//       same launch write the zeros of values without tokens.
//       The runs of a workgroup that is all one value's leave one sum.
//   hyena_embedding_joins  adds the pieces of values that reach over runs (65536 tokens of one value:
//       8 us, 36 with a piece for each run).
// A table of few values needs no sorting: in hyena_embedding_few each team of lanes has its
// tokens, one after the other, and sums of all values in LDS, which
// hyena_embedding_few_join adds up (2^18 tokens, 16 values, width 256: 64 us so, 130 sorted;
// 2^20 tokens, 4 values, width 64: 63 and 899).
// Bound by memory: each gradient row is read once, each row of the table written
// once.  8192 tokens of 31999 values, width 770 in float32: sort 8.2, sums 27.0 (119 MB, most
// of it zeros), joins 5.5 us.  65536 tokens of a text of 50257 values, width 768 in bf16, added to a
// gradient: 20.0, 40.2 (161 MB), 9.6 us; the sort is bound by all groups reading all tokens from
// the L2.
#include "rows.h"

namespace hy {

namespace {

constexpr const char* kWho = "embedding";
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kSortGroups = 256;   // at least; more where a group would have more values than kSortValues
constexpr int kSortValues = 384;   // counters of a wave: 24 KB of LDS in all
// From kDealGroups groups on, which all read all tokens, they have up to this many (16384 tokens of 10^6
// values: the sort takes 35 us so, 92 with 4096 groups): 96 KB.
constexpr int kSortMostValues = 1536;
constexpr int kPlaceBits = 21;
static_assert(kSortMostValues <= 1 << (32 - kPlaceBits), "");
constexpr int kSortTokens = 16;    // of a lane, in four loads
constexpr int kDealTokens = 4096;  // of a workgroup that deals
constexpr int kDealGroups = 1024;  // at most; the lists of more of the sort's groups are one, of those with the same lower bits
// Calls of fewer tokens are not dealt (values of a text in a vocabulary of 50257, dealt and
// sorted, against sorted only: 65536 tokens 20 and 19 us, 2^20 tokens 129 and 410; 2^20 of 1600000 values, of
// which two groups share a list, 199 and 820).
constexpr int64_t kDealCalls = 131072;
constexpr int kSortKept = 512;     // tokens of its values that a wave keeps: 32 KB of LDS in all
// Gradient rows of a team under way (gradient of 65536 tokens of a text, width 768 in bf16, added to one that is
// there, inputs that come from memory, in all: 8 73.0 us, 4 68.8).
constexpr int kSumRows = 4;
// Runs are no shorter than kSumRows, and as short as this many of them allow: fewer leave the
// sums waiting, more the joins (the same gradient: 2048 77.3, 4096 68.8, 8192 73.3 us; sums 51, 41 and 41,
// joins 10, 12 and 17).  4096 of width 768 in bf16 are one round of six waves a SIMD.
constexpr int64_t kSumTeams = 4096;
constexpr int kFewValues = 32;     // tables of no more values than this
constexpr int kFewRows = 8;        // gradient rows of a team under way
constexpr int kFewGroups = 512;    // workgroups at most
constexpr int kJoinThreads = 512, kJoinWaves = kJoinThreads / 64;

struct EmbedArgs {
    Rows tokens, rows;   // rows: d_out
    const void* table;
    void* out;           // backward: d_table
    int64_t total;       // B * N
    uint32_t N, rows_N;  // row_at, of the tokens and of the rows
    int32_t V, d;
    int32_t lanes;       // of a team, a power of two
    int32_t accumulate;
    float scale;
    int32_t groups;      // of the sort, a power of two
    int32_t run;         // tokens of a run, a power of two
    int32_t sum_groups;  // workgroups of the sums, fill_groups behind them
    int32_t fill_groups;
    int32_t* counts;     // [V]; few values: [few_groups] which of them a workgroup has tokens of, by bits
    int2* sorted;        // [total] value and token, in order; [total].x the number of tokens that take part
    int4* joins;         // [V] values that reach over runs, where they begin, tokens: group g's from g * values on
    int32_t* join_counts;  // [groups]
    int2* dealt;         // [blocks of kDealTokens] value and token, by lists; NULL: the sort reads the tokens
    int32_t* deal_starts;  // [deal_groups + 1][blocks] where a list begins in a block
    int32_t deal_groups;   // lists, a power of two
    int32_t deal_blocks;
    float* part;         // [runs][2][d4]: sums that reach over a run's start and over its end
    int32_t d4;          // d rounded up to 4
    int32_t few_groups;  // few values: workgroups, each with a part [V][d4]
};

__device__ __forceinline__ int token_at(const EmbedArgs& p, int64_t t) { return *row_at<int32_t>(p.tokens, t, p.N); }

struct __attribute__((packed, aligned(4))) Four {
    int v[4];
};

// A lane's kSortTokens tokens of a block: token t0 + 256 (k / 4) + 4 lane + k % 4 in
// v[k], -1 at last and after it.
template <bool DENSE> __device__ __forceinline__ void load_tokens(const EmbedArgs& p, int64_t t0, int64_t last, int (&v)[kSortTokens])
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int k = 0; k < kSortTokens; k += 4) {
        const int64_t t = t0 + 64 * k + 4 * lane;
        if (DENSE && t + 4 <= last) {
            const Four x = *(const Four*)((const int32_t*)p.tokens.p + t);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[k + j] = x.v[j];
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[k + j] = t + j < last ? token_at(p, t + j) : -1;
        }
    }
}

template <typename T, bool UNITS> __global__ __launch_bounds__(256) void hyena_embedding_gather(EmbedArgs p)
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
            if (in) load_unit<T, UNITS>(row, c, p.d, x);
#pragma unroll
            for (int i = 0; i < K; ++i) x[i] = in ? x[i] * p.scale : 0.0f;
            store_unit<T, UNITS>(out, c, p.d, x);
        }
    }
}

// The lanes of a wave pass values to each other through LDS: what lies before this is done for
// all of them, and nothing behind it is moved ahead.  (A wave's LDS accesses are done in
// order; this holds the compiler to theirs.)
__device__ __forceinline__ void wave_exchange()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
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

// kDealTokens tokens by lists (of value v: v % deal_groups), in the order they are read within each.
template <bool DENSE> __global__ __launch_bounds__(kSortThreads) void hyena_embedding_deal(EmbedArgs p)
{
    extern __shared__ int counters[];  // [waves][groups]
    __shared__ int lds[kSortWaves];
    const int groups = p.deal_groups;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, bits = __builtin_ctz(groups);
    const int64_t first = (int64_t)blockIdx.x * kDealTokens;
    int* own = counters + wave * groups;
    for (int i = threadIdx.x; i < groups * kSortWaves; i += kSortThreads) counters[i] = 0;
    __syncthreads();
    static_assert(kDealTokens == 4 * kSortThreads, "");
    int v[4], at[4];
    const int64_t t0 = first + wave * 256 + 4 * lane;
    if (DENSE && t0 + 4 <= p.total) {
        const Four x = *(const Four*)((const int32_t*)p.tokens.p + t0);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = x.v[k];
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = t0 + k < p.total ? token_at(p, t0 + k) : -1;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const bool in = (uint32_t)v[k] < (uint32_t)p.V;
        const int group = v[k] & (groups - 1);
        uint64_t same = __ballot(in);  // the lanes of one group
        for (int b = 0; b < bits; ++b) {
            const uint64_t ones = __ballot(group >> b & 1);
            same &= group >> b & 1 ? ones : ~ones;
        }
        const int before = in ? own[group] : 0, rank = __popcll(same & (((uint64_t)1 << lane) - 1));
        at[k] = before + rank;
        wave_exchange();  // every lane has read before one writes
        if (in && rank == 0) own[group] = before + __popcll(same);
        wave_exchange();
    }
    __syncthreads();
    // counts to places: thread i has group i
    const int i = threadIdx.x;
    int mine = 0;
    if (i < groups)
        for (int w = 0; w < kSortWaves; ++w) {
            const int c = counters[w * groups + i];
            counters[w * groups + i] = mine;
            mine += c;
        }
    int before = mine;
    for (int m = 1; m < 64; m *= 2) {
        const int up = __shfl_up(before, m);
        if (lane >= m) before += up;
    }
    if (lane == 63) lds[wave] = before;
    __syncthreads();
    before -= mine;
    int all = 0;
    for (int w = 0; w < kSortWaves; ++w) {
        if (w < wave) before += lds[w];
        all += lds[w];
    }
    if (i < groups) {
        for (int w = 0; w < kSortWaves; ++w) counters[w * groups + i] += before;
        p.deal_starts[(int64_t)i * p.deal_blocks + blockIdx.x] = before;
    }
    if (i == 0) p.deal_starts[(int64_t)groups * p.deal_blocks + blockIdx.x] = all;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if ((uint32_t)v[k] < (uint32_t)p.V)
            p.dealt[first + own[v[k] & (groups - 1)] + at[k]] = make_int2(v[k], (int)(t0 + k));
}

template <bool DENSE> __global__ __launch_bounds__(kSortThreads) void hyena_embedding_sort(EmbedArgs p)
{
    extern __shared__ int counters[];  // [waves][values]
    __shared__ int lds[kSortWaves], join_count;
    __shared__ uint32_t kept[kSortWaves][kSortKept];
    const int group = blockIdx.x, shift = __builtin_ctz(p.groups);
    const int values = (p.V - group + p.groups - 1) >> shift;  // v = group + groups * i, i < values
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    // each wave a part of the tokens (whole 64s of them) or of the blocks that were dealt out
    const int blocks = (p.deal_blocks + kSortWaves - 1) / kSortWaves;
    const int b0 = blocks * wave, b1 = b0 + blocks < p.deal_blocks ? b0 + blocks : p.deal_blocks;
    const int64_t each = p.dealt != nullptr ? (int64_t)blocks * kDealTokens : ((p.total + 64 * kSortWaves - 1) / (64 * kSortWaves)) * 64;
    const int64_t first = each * wave, last = first + each < p.total ? first + each : p.total;

    for (int i = threadIdx.x; i < values * kSortWaves; i += kSortThreads) counters[i] = 0;
    if (threadIdx.x == 0) join_count = 0;
    __syncthreads();
    int lower = 0, all = 0;
    // this wave's dealt tokens of the group's list, 64 at a time: f(there is one, value, token)
    const int list_of = group & (p.deal_groups - 1);
    auto each_dealt = [&](auto f) {
        const int32_t *lo = p.deal_starts + (int64_t)list_of * p.deal_blocks, *hi = lo + p.deal_blocks;
        for (int b = b0; b < b1; ++b) {
            const int n = hi[b] - lo[b];
            const int2* list = p.dealt + (int64_t)b * kDealTokens + lo[b];
            for (int k0 = 0; k0 < n; k0 += 256) {
                int2 e[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) e[k] = k0 + 64 * k + lane < n ? list[k0 + 64 * k + lane] : make_int2(0, 0);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k0 + 64 * k < n) f(k0 + 64 * k + lane < n, e[k].x, (int64_t)e[k].y);
            }
        }
    };
    int n_own = 0;  // this wave's tokens of the group's values; the first kSortKept are kept: i << kPlaceBits | place in its part
    if (p.dealt != nullptr) {
        // lower groups: those of lower lists, and of its own list the lower ones
        const int32_t *lo = p.deal_starts + (int64_t)list_of * p.deal_blocks, *end = p.deal_starts + (int64_t)p.deal_groups * p.deal_blocks;
        for (int b = threadIdx.x; b < p.deal_blocks; b += kSortThreads) {
            lower += lo[b];
            all += end[b];
        }
        each_dealt([&](bool there, int v, int64_t t) {
            const int i = v >> shift;
            const bool own = there && (v & (p.groups - 1)) == group;
            lower += there && (v & (p.groups - 1)) < group;
            const uint64_t who = __ballot(own);
            if (who == 0) return;
            // (of one value all at once: 131072 tokens of one value 89 us so, 162 with an atomic of each lane)
            int* to = &counters[wave * values + i];
            const int one = __builtin_ctzll(who), at = n_own + __popcll(who & (((uint64_t)1 << lane) - 1));
            if (__ballot(own && i != __builtin_amdgcn_readlane(i, one)) == 0) {
                if (lane == one) atomicAdd(to, __popcll(who));
            } else if (own) {
                atomicAdd(to, 1);
            }
            if (own && at < kSortKept) kept[wave][at] = (uint32_t)i << kPlaceBits | (uint32_t)(t - first);
            n_own += __popcll(who);
        });
    } else
    for (int64_t t0 = first; t0 < last; t0 += 64 * kSortTokens) {
        int v[kSortTokens];
        load_tokens<DENSE>(p, t0, last, v);
#pragma unroll
        for (int k = 0; k < kSortTokens; k += 4) {
            bool any = false;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool in = (uint32_t)v[k + j] < (uint32_t)p.V;
                const int g = v[k + j] & (p.groups - 1);
                all += in;
                lower += in && g < group;
                any = any || (in && g == group);
            }
            if (__ballot(any) == 0) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool own = (uint32_t)v[k + j] < (uint32_t)p.V && (v[k + j] & (p.groups - 1)) == group;
                const uint64_t who = __ballot(own);
                const int at = n_own + __popcll(who & (((uint64_t)1 << lane) - 1)), i = v[k + j] >> shift;
                if (own) {
                    atomicAdd(&counters[wave * values + i], 1);
                    if (at < kSortKept) kept[wave][at] = (uint32_t)i << kPlaceBits | (uint32_t)(t0 - first + 64 * k + 4 * lane + j);
                }
                n_own += __popcll(who);
            }
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
        for (int w = 0; w < kSortWaves; ++w) c += counters[w * values + i];
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
    const int run_shift = __builtin_ctz(p.run), most = (p.V + p.groups - 1) >> shift;
    for (int k = 0; k < n; ++k) {
        const int i = threadIdx.x * n + k;
        if (i >= values) break;
        const int start = before;
        for (int w = 0; w < kSortWaves; ++w) {
            const int c = counters[w * values + i];
            counters[w * values + i] = before;
            before += c;
        }
        // (which of the list's places a value takes does not matter)
        if (before > start && start >> run_shift != (before - 1) >> run_shift)
            p.joins[(int64_t)group * most + atomicAdd(&join_count, 1)] = make_int4(group + p.groups * i, start, before - start, 0);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        p.join_counts[group] = join_count;
        if (group == 0) p.sorted[p.total] = make_int2(all, 0);
    }
    // this wave's tokens, in the order they were read, each to its value's place
    auto put = [&](bool own, int i, int64_t t) {
        uint64_t left = __ballot(own);
        while (left != 0) {  // one value of 64 tokens after the other
            const int one = __builtin_amdgcn_readlane(i, __builtin_ctzll(left));
            const bool same = own && i == one;
            const uint64_t all_same = __ballot(same);
            int* counter = &counters[wave * values + one];
            const int place = *counter;
            wave_exchange();  // every lane has read before one writes
            if (same) p.sorted[place + __popcll(all_same & (((uint64_t)1 << lane) - 1))] = make_int2(group + p.groups * i, (int)t);
            if (lane == 0) *counter = place + __popcll(all_same);
            wave_exchange();
            left &= ~all_same;
        }
    };
    if (n_own <= kSortKept && each <= 1 << kPlaceBits) {
        for (int k = 0; k < n_own; k += 64) {
            const bool own = k + lane < n_own;
            const uint32_t x = own ? kept[wave][k + lane] : 0;
            put(own, (int)(x >> kPlaceBits), first + (x & ((1 << kPlaceBits) - 1)));
        }
        return;
    }
    // too many to keep: the tokens again
    if (p.dealt != nullptr) {
        each_dealt([&](bool there, int v, int64_t t) { put(there && (v & (p.groups - 1)) == group, v >> shift, t); });
        return;
    }
    for (int64_t t0 = first; t0 < last; t0 += 64 * kSortTokens) {
        int v[kSortTokens];
        load_tokens<DENSE>(p, t0, last, v);
#pragma unroll
        for (int k = 0; k < kSortTokens; ++k)
            put((uint32_t)v[k] < (uint32_t)p.V && (v[k] & (p.groups - 1)) == group, v[k] >> shift, t0 + 64 * (k & ~3) + 4 * lane + (k & 3));
    }
}

// blockIdx.y: which of the row's blocks of `lanes` units.
template <typename T, bool UNITS> __global__ __launch_bounds__(256) void hyena_embedding_sums(EmbedArgs p)
{
    constexpr int K = kUnit<T>;
    const int teams = 256 / p.lanes, team = threadIdx.x / p.lanes, tl = threadIdx.x % p.lanes;
    const int c = ((int)blockIdx.y * p.lanes + tl) * K;
    if ((int)blockIdx.x >= p.sum_groups) {
        // zeros where no token is, whole rows
        const int64_t step = (int64_t)p.fill_groups * gridDim.y * teams;
        for (int64_t v = ((int64_t)((int)blockIdx.x - p.sum_groups) * gridDim.y + blockIdx.y) * teams + team; v < p.V; v += step) {
            if (p.counts[v] != 0) continue;
            T* row = (T*)p.out + v * p.d;
            // by aligned 16 bytes, and elements at both ends, past the caches, which the rows of a
            // large table would only run through (8192 tokens, 31999 values, width 770 in float32, five
            // gradients in turn: 58 us with the rows' ordinary stores, 50 aligned, 42 so)
            const int head = UNITS ? 0 : (int)(-(uintptr_t)row & 15) / (int)sizeof(T);
            if (!UNITS)
                for (int i = tl; i < head && i < p.d; i += p.lanes) store_one<T>(row + i, 0.0f);
            int at = head + tl * K;
            for (; at + K <= p.d; at += p.lanes * K) __builtin_nontemporal_store(u32x4{0, 0, 0, 0}, (u32x4*)(row + at));
            if (!UNITS)
                for (int i = at; i < at + K && i < p.d; ++i) store_one<T>(row + i, 0.0f);
        }
        return;
    }
    const int n = p.sorted[p.total].x;  // tokens that take part
    const int run = (int)blockIdx.x * teams + team, first = run * p.run;
    // a workgroup whose runs all lie inside one value leaves one sum: at its first run's start
    __shared__ float inside[256][K + 1];
    const int before = (int)blockIdx.x * teams * p.run - 1, behind = before + 1 + teams * p.run;
    const bool whole = before >= 0 && behind < n && p.sorted[before].x == p.sorted[behind].x;
    if (first >= n) return;
    const int last = first + p.run < n ? first + p.run : n;
    float s[K];
#pragma unroll
    for (int i = 0; i < K; ++i) s[i] = 0.0f;
    bool open = first > 0 && p.sorted[first - 1].x == p.sorted[first].x;  // the value began before this run
    const int next_value = last < n ? p.sorted[last].x : -1;
    for (int i0 = first; i0 < last; i0 += kSumRows) {
        int2 e[kSumRows + 1];
#pragma unroll
        for (int k = 0; k < kSumRows; ++k) {
            const int i = i0 + k < last ? i0 + k : last - 1;
            e[k] = p.sorted[i];
        }
        e[kSumRows] = i0 + kSumRows < last ? p.sorted[i0 + kSumRows] : make_int2(next_value, 0);
        // the last token of a value ends it, here or (at this run's end) in a later run
        bool ends[kSumRows], on[kSumRows];
#pragma unroll
        for (int k = 0; k < kSumRows; ++k) {
            const bool at_end = i0 + k + 1 >= last;
            on[k] = (at_end ? next_value : e[k + 1].x) == e[k].x;
            ends[k] = i0 + k < last && (at_end || !on[k]);
        }
        // (loads past the caches are faster by 8% for 100 MB that come from memory, and slower by a third
        // for rows that the caches hold, as those of a backward pass mostly are)
        Unit<T, UNITS> x[kSumRows], old[kSumRows];
#pragma unroll
        for (int k = 0; k < kSumRows; ++k) {
            const T* row = row_at<T>(p.rows, e[k].y, p.rows_N);
            const T* there = (const T*)p.out + (int64_t)e[k].x * p.d;
            x[k].load(row, c, p.d);
            if (p.accumulate && ends[k]) old[k].load(there, c, p.d);
        }
#pragma unroll
        for (int k = 0; k < kSumRows; ++k) {
            if (i0 + k >= last) break;
            float y[K];
            x[k].widen(y);
#pragma unroll
            for (int i = 0; i < K; ++i) s[i] += y[i];
            if (!ends[k]) continue;
            if (whole) {
#pragma unroll
                for (int i = 0; i < K; ++i) inside[threadIdx.x][i] = s[i];
            } else if (open || on[k]) {  // a piece
                float* part = p.part + ((int64_t)run * 2 + (open ? 0 : 1)) * p.d4 + c;
#pragma unroll
                for (int i = 0; i < K; i += 4)
                    if (c + i < p.d4) *(f32x4*)(part + i) = f32x4{s[i], s[i + 1], s[i + 2], s[i + 3]};
            } else {
                if (p.accumulate) old[k].widen(y);
#pragma unroll
                for (int i = 0; i < K; ++i) y[i] = p.accumulate ? fmaf(s[i], p.scale, y[i]) : s[i] * p.scale;
                store_unit<T, UNITS>((T*)p.out + (int64_t)e[k].x * p.d, c, p.d, y);
            }
#pragma unroll
            for (int i = 0; i < K; ++i) s[i] = 0.0f;
            open = false;
        }
    }
    if (!whole) return;
    __syncthreads();
    if (team != 0) return;
    for (int k = 0; k < teams; ++k)  // (s is 0 behind a piece)
#pragma unroll
        for (int i = 0; i < K; ++i) s[i] += inside[k * p.lanes + tl][i];
    float* part = p.part + (int64_t)run * 2 * p.d4 + c;
#pragma unroll
    for (int i = 0; i < K; i += 4)
        if (c + i < p.d4) *(f32x4*)(part + i) = f32x4{s[i], s[i + 1], s[i + 2], s[i + 3]};
}

// The values of one group of the sort that reach over runs, 256 channels of them.
// Of few pieces: each wave its own values.  Of many: all waves some of the pieces, the
// first wave the waves' sums.
template <typename T> __global__ __launch_bounds__(kJoinThreads) void hyena_embedding_joins(EmbedArgs p)
{
    __shared__ f32x4 lds[kJoinWaves][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int c = (int)blockIdx.y * 256 + lane * 4;
    const int n = p.join_counts[blockIdx.x];
    const int4* list = p.joins + (int64_t)blockIdx.x * ((p.V + p.groups - 1) / p.groups);
    // a value's pieces: runs up to the first workgroup of the sums that is all its own, such
    // workgroups, and the runs behind them
    const int run_shift = __builtin_ctz(p.run), group_shift = run_shift + __builtin_ctz(256 / p.lanes);
    struct Pieces {
        int first, runs, group, groups, rest, all;
    };
    auto pieces_of = [&](int4 e) {
        const int first = e.y >> run_shift, last = (e.y + e.z - 1) >> run_shift, wide = group_shift - run_shift;
        // workgroup g is all its own where the tokens before and behind it are, too
        const int g0 = (e.y >> group_shift) + 1, g1 = (e.y + e.z - 1) >> group_shift;
        Pieces q;
        q.first = first;
        q.groups = g1 > g0 ? g1 - g0 : 0;
        q.group = g0 << wide;
        q.runs = q.groups ? q.group - first : last - first + 1;
        q.rest = q.groups ? g1 << wide : 0;
        q.all = q.groups ? q.runs + q.groups + (last - q.rest + 1) : q.runs;
        return q;
    };
    auto sum = [&](const Pieces& q, int from, int step) {
        const float* part = p.part + c;
        const int wide = group_shift - run_shift;
        f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
        // the first piece is its run's last, the others their runs' first
#pragma unroll 8
        for (int k = from; k < q.all; k += step) {
            const int in = k - q.runs, run = in < 0 ? q.first + k : in < q.groups ? q.group + (in << wide) : q.rest + in - q.groups;
            s += *(const f32x4*)(part + ((int64_t)run * 2 + (k == 0)) * p.d4);
        }
        return s;
    };
    auto write = [&](int4 e, f32x4 s) {
        T* row = (T*)p.out + (int64_t)e.x * p.d + c;
        float old[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (p.accumulate) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c + i < p.d) old[i] = load_one<T>(row + i);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i < p.d) store_one<T>(row + i, fmaf(s[i], p.scale, old[i]));
    };
    for (int i = wave; i < n; i += kJoinWaves) {
        const int4 e = list[i];
        const Pieces q = pieces_of(e);
        if (q.all <= kJoinWaves && c < p.d) write(e, sum(q, 0, 1));
    }
    for (int i = 0; i < n; ++i) {
        const int4 e = list[i];
        const Pieces q = pieces_of(e);
        if (q.all <= kJoinWaves) continue;
        f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
        if (c < p.d) s = sum(q, wave, kJoinWaves);
        lds[wave][lane] = s;
        __syncthreads();
        if (wave == 0 && c < p.d) {
#pragma unroll
            for (int w = 1; w < kJoinWaves; ++w) s += lds[w][lane];
            write(e, s);
        }
        __syncthreads();
    }
}

// Tokens of a team of p.lanes lanes, four channels each; blockIdx.y: which 256 channels.
template <typename T, bool UNITS> __global__ __launch_bounds__(256) void hyena_embedding_few(EmbedArgs p)
{
    extern __shared__ f32x4 few_sums[];  // [teams][V][lanes]
    __shared__ uint32_t any;             // bit v: value v has a token
    static_assert(kFewValues <= 32, "");
    if (threadIdx.x == 0) any = 0;
    uint32_t seen = 0;
    const int teams = 256 / p.lanes, team = threadIdx.x / p.lanes, tl = threadIdx.x % p.lanes;
    const int c = (int)blockIdx.y * 256 + tl * 4;
    f32x4* own = few_sums + (size_t)team * p.V * p.lanes + tl;
    for (int v = 0; v < p.V; ++v) own[v * p.lanes] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int64_t parts = (int64_t)gridDim.x * teams, each = (p.total + parts - 1) / parts;
    const int64_t first = ((int64_t)blockIdx.x * teams + team) * each, last = first + each < p.total ? first + each : p.total;
    // kFewRows rows are under way while those before them are added, and the tokens behind them
    struct Rows8 {
        int v[kFewRows];
        typename Mx<T>::vec4 x[kFewRows];
    } a, b;
    auto tokens = [&](int64_t t0, Rows8& r) {
#pragma unroll
        for (int k = 0; k < kFewRows; ++k) r.v[k] = t0 + k < last ? token_at(p, t0 + k) : -1;
    };
    auto rows = [&](int64_t t0, Rows8& r) {
#pragma unroll
        for (int k = 0; k < kFewRows; ++k) {
            r.x[k] = typename Mx<T>::vec4{};
            if ((uint32_t)r.v[k] >= (uint32_t)p.V) continue;
            const T* row = row_at<T>(p.rows, t0 + k, p.rows_N) + c;
            if (UNITS) {
                if (c < p.d) r.x[k] = *(const typename Mx<T>::vec4*)row;
            } else {
                T* e = (T*)&r.x[k];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c + i < p.d) e[i] = row[i];
            }
        }
    };
    auto add = [&](const Rows8& r) {
#pragma unroll
        for (int k = 0; k < kFewRows; ++k)
            if ((uint32_t)r.v[k] < (uint32_t)p.V) {
                own[r.v[k] * p.lanes] += Mx<T>::widen(r.x[k]);
                seen |= 1u << r.v[k];
            }
    };
    tokens(first, a);
    rows(first, a);
    tokens(first + kFewRows, b);
    for (int64_t t0 = first; t0 < last; t0 += 2 * kFewRows) {
        rows(t0 + kFewRows, b);
        add(a);
        tokens(t0 + 2 * kFewRows, a);
        rows(t0 + 2 * kFewRows, a);
        add(b);
        tokens(t0 + 3 * kFewRows, b);
    }
    __syncthreads();
    if (tl == 0) atomicOr(&any, seen);
    // the teams' sums in their order
    for (int i = threadIdx.x; i < p.V * p.lanes; i += 256) {
        f32x4 sum = few_sums[i];
        for (int k = 1; k < teams; ++k) sum += few_sums[(size_t)k * p.V * p.lanes + i];
        const int at = (int)blockIdx.y * 256 + i % p.lanes * 4;
        if (at < p.d) *(f32x4*)(p.part + ((int64_t)blockIdx.x * p.V + i / p.lanes) * p.d4 + at) = sum;
    }
    __syncthreads();
    if (threadIdx.x == 0 && blockIdx.y == 0) p.counts[blockIdx.x] = (int32_t)any;
}

// blockIdx.x: the value, blockIdx.y: which 256 channels; each of 16 waves some of the parts.
template <typename T> __global__ __launch_bounds__(1024) void hyena_embedding_few_join(EmbedArgs p)
{
    __shared__ f32x4 lds[16][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int c = (int)blockIdx.y * 256 + lane * 4;
    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c < p.d) {
#pragma unroll 8
        for (int g = wave; g < p.few_groups; g += 16) s += *(const f32x4*)(p.part + ((int64_t)g * p.V + blockIdx.x) * p.d4 + c);
    }
    lds[wave][lane] = s;
    __syncthreads();
    if (wave != 0) return;
    uint32_t seen = 0;
    for (int g = lane; g < p.few_groups; g += 64) seen |= (uint32_t)p.counts[g];
    const bool some = __any(seen >> blockIdx.x & 1);
    if (!some && p.accumulate) return;
#pragma unroll
    for (int w = 1; w < 16; ++w) s += lds[w][lane];
    T* row = (T*)p.out + (int64_t)blockIdx.x * p.d + c;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (c + i < p.d) store_one<T>(row + i, !some ? 0.0f : p.accumulate ? fmaf(s[i], p.scale, load_one<T>(row + i)) : s[i] * p.scale);
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
    size_t sorted, counts, joins, join_counts, dealt, deal_starts, part, total;  // byte offsets and the size
    int32_t deal_blocks;  // 0: not dealt
    int32_t groups, deal_groups, d4;
    int32_t few_groups, few_lanes;  // 0: the tokens are sorted
};

EmbedSpace embed_space(const hyena_embedding* op)
{
    EmbedSpace w{};
    const int64_t T = op->B * op->N;
    w.d4 = (int32_t)((op->d + 3) / 4 * 4);
    w.few_groups = w.few_lanes = 0;
    if (op->V <= kFewValues) {
        // lanes of a team: a power of two, as many as channels ask for
        w.few_lanes = 64;
        while (w.few_lanes > 8 && w.few_lanes / 2 * 4 >= w.d4) w.few_lanes /= 2;
        const int64_t teams = 256 / w.few_lanes, need = (T + teams * 2 * kFewRows - 1) / (teams * 2 * kFewRows);
        w.few_groups = (int32_t)(need < kFewGroups ? need : kFewGroups);
        w.counts = 0;
        w.part = (size_t)(w.few_groups + 63) / 64 * 256;
        w.total = w.part + (size_t)w.few_groups * (size_t)op->V * (size_t)w.d4 * 4;
        return w;
    }
    const int64_t most = (T + kSumTeams - 1) / kSumTeams;
    w.run = kSumRows;
    while (w.run < most) w.run *= 2;
    w.runs = (T + w.run - 1) / w.run;
    auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
    w.sorted = 0;
    w.counts = up((size_t)(T + 1) * sizeof(int2));
    w.groups = kSortGroups;
    while ((op->V + w.groups - 1) / w.groups > (w.groups < kDealGroups ? kSortValues : kSortMostValues)) w.groups *= 2;
    w.joins = w.counts + up((size_t)op->V * 4);
    w.join_counts = w.joins + up((size_t)((op->V + w.groups - 1) / w.groups * w.groups) * sizeof(int4));
    w.deal_groups = w.groups < kDealGroups ? w.groups : kDealGroups;
    w.deal_blocks = T >= kDealCalls ? (int32_t)((T + kDealTokens - 1) / kDealTokens) : 0;
    w.dealt = w.join_counts + up((size_t)w.groups * 4);
    w.deal_starts = w.dealt + up((size_t)w.deal_blocks * kDealTokens * sizeof(int2));
    w.part = w.deal_starts + up((size_t)(w.deal_groups + 1) * (size_t)w.deal_blocks * 4);
    w.total = w.part + (size_t)w.runs * 2 * (size_t)w.d4 * 4;
    return w;
}

// Lanes of a team, which hold a unit each: 64, or 32 if that leaves fewer of them idle
// over a row, or as few as a narrow row has (2^20 rows of 64 in bf16: 30 us so, 98 by 32).
void team_shape(EmbedArgs& a, size_t element)
{
    const int units = (int)((a.d * element + 15) / 16);
    auto used = [&](int n) { return (units + n - 1) / n * n; };
    a.lanes = 64;
    if (used(32) < used(64)) a.lanes = 32;
    while (a.lanes > 4 && a.lanes / 2 >= units) a.lanes /= 2;
}

template <typename T> hyena_status embed_backward(const EmbedArgs& a, bool units, int64_t runs, hipStream_t s)
{
    hyena_status st;
    const bool dense = a.N == 0 && a.tokens.t == 1;
    const dim3 few_grid((unsigned)a.few_groups, (unsigned)((a.d + 255) / 256));
    if (a.few_groups > 0) {
        st = by_units(units, [&](auto u) {
            constexpr bool UNITS = decltype(u)::value;
            HY_LAUNCH(kernel_label("hyena_embedding_few", type_label<T>(), UNITS), (hyena_embedding_few<T, UNITS>), few_grid, dim3(256), (size_t)a.V * 4096, s, a);
            return launched();
        });
        if (st != HYENA_OK) return st;
        HY_LAUNCH(kernel_label("hyena_embedding_few_join", type_label<T>()), hyena_embedding_few_join<T>, dim3((unsigned)a.V, few_grid.y), dim3(1024), 0, s, a);
        return launched();
    }
    if (a.dealt != nullptr) {
        const dim3 grid((unsigned)a.deal_blocks);
        const size_t lds = (size_t)a.deal_groups * kSortWaves * 4;
        if (dense)
            HY_LAUNCH(kernel_label("hyena_embedding_deal", true), hyena_embedding_deal<true>, grid, dim3(kSortThreads), lds, s, a);
        else
            HY_LAUNCH(kernel_label("hyena_embedding_deal", false), hyena_embedding_deal<false>, grid, dim3(kSortThreads), lds, s, a);
        if ((st = launched()) != HYENA_OK) return st;
    }
    const dim3 sort_grid((unsigned)a.groups);
    const size_t sort_lds = (size_t)((a.V + a.groups - 1) / a.groups) * kSortWaves * 4;
    if (dense)
        HY_LAUNCH(kernel_label("hyena_embedding_sort", true), hyena_embedding_sort<true>, sort_grid, dim3(kSortThreads), sort_lds, s, a);
    else
        HY_LAUNCH(kernel_label("hyena_embedding_sort", false), hyena_embedding_sort<false>, sort_grid, dim3(kSortThreads), sort_lds, s, a);
    if ((st = launched()) != HYENA_OK) return st;
    const int block = a.lanes * kUnit<T>;
    const dim3 grid((unsigned)(a.sum_groups + a.fill_groups), (unsigned)((a.d + block - 1) / block));
    st = by_units(units, [&](auto u) {
        constexpr bool UNITS = decltype(u)::value;
        HY_LAUNCH(kernel_label("hyena_embedding_sums", type_label<T>(), UNITS), (hyena_embedding_sums<T, UNITS>), grid, dim3(256), 0, s, a);
        return launched();
    });
    if (st != HYENA_OK || runs < 2) return st;
    HY_LAUNCH(kernel_label("hyena_embedding_joins", type_label<T>()), hyena_embedding_joins<T>,
              dim3((unsigned)a.groups, (unsigned)((a.d + 255) / 256)), dim3(kJoinThreads), 0, s, a);
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
    a.table = table;
    a.out = out;
    const int64_t teams = 256 / a.lanes, need = (a.total + teams - 1) / teams, most = (int64_t)1 << 20;
    const dim3 grid((unsigned)(need < most ? need : most));
    const hipStream_t s = (hipStream_t)stream;
    return by_io(op->io_dtype, [&](auto* t) {
        using T = std::remove_pointer_t<decltype(t)>;
        return by_units(made.units(), [&](auto u) {
            constexpr bool UNITS = decltype(u)::value;
            HY_LAUNCH(kernel_label("hyena_embedding_gather", type_label<T>(), UNITS), (hyena_embedding_gather<T, UNITS>), grid, dim3(256), 0, s, a);
            return launched();
        });
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
    int64_t N = op->N;
    hyena_rows* one[1] = {&rows};
    flatten_rows(one, 1, op->B, &N);
    a.rows = Rows{rows.data, rows.batch, rows.token};
    a.rows_N = (uint32_t)N;
    a.out = d_table;
    a.accumulate = accumulate != 0;
    a.d4 = w.d4;
    a.part = (float*)((char*)scratch + w.part);
    a.counts = (int32_t*)((char*)scratch + w.counts);
    a.few_groups = w.few_groups;
    const hipStream_t s = (hipStream_t)stream;
    if (w.few_groups > 0) {
        a.lanes = w.few_lanes;
        return by_io(op->io_dtype, [&](auto* t) { return embed_backward<std::remove_pointer_t<decltype(t)>>(a, made.units(), 0, s); });
    }
    a.groups = w.groups;
    a.joins = (int4*)((char*)scratch + w.joins);
    a.join_counts = (int32_t*)((char*)scratch + w.join_counts);
    a.run = (int32_t)w.run;
    a.sorted = (int2*)((char*)scratch + w.sorted);
    a.deal_blocks = w.deal_blocks;
    a.deal_groups = w.deal_groups;
    a.dealt = w.deal_blocks ? (int2*)((char*)scratch + w.dealt) : nullptr;
    a.deal_starts = (int32_t*)((char*)scratch + w.deal_starts);
    const int64_t teams = 256 / a.lanes;
    a.sum_groups = (int32_t)((w.runs + teams - 1) / teams);
    const int64_t fill = (a.V + teams - 1) / teams;
    a.fill_groups = a.accumulate ? 0 : (int32_t)(fill < 2048 ? fill : 2048);
    return by_io(op->io_dtype, [&](auto* t) {
        return embed_backward<std::remove_pointer_t<decltype(t)>>(a, made.units(), w.runs, s);
    });
}

}  // extern "C"
