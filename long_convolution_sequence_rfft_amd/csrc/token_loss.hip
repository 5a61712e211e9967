// token_loss.hip -- entry points of the loss over a vocabulary (include/hyena.h):
// checks, the scratch, and the pieces of the vocabulary.
#include "token_loss.h"

namespace hy {
namespace {

constexpr const char* kWho = "token loss";

// G of a piece of the vocabulary takes about this much, or a tile of values if that
// is more (gradients of 16384 tokens, a quarter masked, 50257 values, width 768: in pieces of 256 MB 5105,
// 512 MB 5050, 1 GiB 4540, 2 GiB 4255 us; the last 6% are not worth as much scratch again).
constexpr int64_t kGradBytes = (int64_t)1024 << 20;
// The sums of a piece's tiles, forward: larger ones would be written to memory and read back,
// and a launch could have more than 2^32 threads.
constexpr int64_t kPartBytes = (int64_t)256 << 20;
// Logits of no more tiles than this are made in small ones (width 1024, of 2, 32, 128 and 256 tiles:
// in 16 bits 19, 20, 29 and 44 us so, 31, 32, 34 and 35 us in large ones; in float32 32, 31, 64
// and 115 us so, 72, 73, 76 and 82 us in large ones; width 256 in 16 bits: 14, 14, 17, 23 and 18, 20, 19, 20).
constexpr int64_t kSmallTiles = 128;
// Rows that the blocks of gathered rows and of G are apart from each other beyond their tokens: at a power
// of two a step's pieces of all of a tile's blocks would share one place in the caches (the same
// gradients' logits: 1400 us without, 1378 so).
constexpr int64_t kBlockRows = 32;
// Workgroups that d_x's sums are cut for, and into which part of their time: they come last,
// and the shorter they are the sooner the last one ends, but each adds to d_x's sums (the
// same gradients: 1 part 4700, 2 4380, 4 4480, 6 4390 us; of 2048 tokens, 31999 values in float32
// 1725, 1630, 1497 and 1488).
constexpr int64_t kSplitGroups = 512, kSplitParts = 4;
// Steps of 32 tokens that a part of d_table's sums has at least.  They are cut so that no part takes
// longer than a workgroup's share of the piece's work (16384 tokens, 2048 values: 315 us so, of
// twice the share 325, of half of it 336; 65536 tokens, 16 values: 154, 188 and 154).
constexpr int64_t kTableSteps = 4;

hyena_status refuse(const char* what) { return fail(HYENA_ERR_INVALID_ARGUMENT, std::string(kWho) + ": " + what); }

hyena_status loss_sizes(const hyena_token_loss* op)
{
    if (op == nullptr) return refuse("the description is NULL");
    if (op->B < 1 || op->N < 1 || op->V < 1 || op->d < 1) return refuse("B, N, V and d must be at least 1");
    if (op->V > 1 << 22 || op->d > 16384) return fail(HYENA_ERR_UNSUPPORTED, "token loss: V at most 2^22 and d at most 16384");
    if (op->B > 1 << 22 || op->N > 1 << 22 || op->B * op->N > 1 << 22)
        return fail(HYENA_ERR_UNSUPPORTED, "token loss: at most 2^22 tokens");
    return check_io(kWho, op->io_dtype);
}

// Calls of at most this many tokens have their own kernels: forward, in 16 bits and in
// float32 (whose table is read as given then), and backward.  With 50257 values of width 768,
// by them and by the others: forward in 16 bits 4 tokens 21 and 39 us, 32 23 and 40; in float32 8 38 and
// 153, 64 121 and 157 (128 186 and 159); backward in 16 bits 4 tokens 69 and 108, 8 88 and 108 (12 169 and
// 108, for twice the sums in the registers); in float32 8 120 and 315, 16 177 and 315.
constexpr int64_t kFewTokens = 32, kFewTokensF32 = 64, kFewTokensGrad = 8, kFewTokensGradF32 = 16;
// Workgroups of 256 channels, backward: more have more loads under way, and more sums of d_x
// behind them (256 and 512: 4 tokens in 16 bits 74 and 69 us, 8 88 and 96; 8 in float32 123 and 131).
constexpr int32_t kFewGroups = 256, kFewGroupsHalf = 512;
constexpr int64_t kFewGroupsTokens = 4;  // in 16 bits, at most: kFewGroupsHalf
// Others of more tokens than this bring the table into the matrix operands' form first (in that
// form and as given, forward: 1024 tokens 128 and 103 us, 4096 314 and 304, 8192 573 and 575, 16384 1062
// and 1117; backward 460 and 446, 1473 and 1465, 2840 and 2856, 5890 and 6023).
constexpr int64_t kPackTokens = 4096;

bool is_few(const hyena_token_loss* op, bool grad)
{
    const bool f32 = op->io_dtype == HYENA_F32;
    return op->B * op->N <= (grad ? (f32 ? kFewTokensGradF32 : kFewTokensGrad) : f32 ? kFewTokensF32 : kFewTokens);
}

bool needs_pack(const hyena_token_loss* op, bool grad)
{
    if (op->io_dtype == HYENA_F32) return !is_few(op, grad);
    // 16-byte loads need rows that are made of them (float32's any 4-byte address)
    return op->d % 8 != 0 || (!is_few(op, grad) && op->B * op->N > kPackTokens);
}

// Tiles of values of a piece, if `fit` of all are to be one: pieces of about one size, of as
// many tiles for each XCD.
int64_t even_pieces(int64_t all, int64_t fit)
{
    if (fit >= all) return all;
    const int64_t pieces = fit < 1 ? all : (all + fit - 1) / fit, tiles = (all + pieces - 1) / pieces;
    return tiles <= 8 ? tiles : (tiles + 7) / 8 * 8;
}

// Sizes, and with a scratch the addresses in it; returns the bytes.
size_t lay_out(const hyena_token_loss* op, bool grad, void* scratch, LossArgs& a)
{
    const int64_t planes = op->io_dtype == HYENA_F32 ? 3 : 1, grad_planes = planes == 3 ? 3 : 2;  // kGradPlanes
    a.total = op->B * op->N;
    a.V = (int32_t)op->V;
    a.d = (int32_t)op->d;
    a.kd = (int32_t)((op->d + 31) / 32 * 32);
    a.few = is_few(op, grad);
    a.small = !a.few && (int64_t)loss_tiles(a.V) * ((a.total + kLossTokens - 1) / kLossTokens) <= kSmallTiles;
    a.tokens = a.few && grad ? 32 : (a.total + kLossTokens - 1) / kLossTokens * kLossTokens;
    a.scale = op->scale;
    a.table = op->table;
    // a workgroup of the gather for 64 tokens, or at most 512 of them
    const int64_t each = (a.total + 511) / 512;
    a.each = (int32_t)(each < 64 ? 64 : each);
    size_t at = 0;
    auto take = [&](size_t n) {
        char* p = scratch ? (char*)scratch + at : nullptr;
        at += (n + 255) & ~(size_t)255;
        return p;
    };
    const size_t tokens = (size_t)a.tokens;
    a.count = (int64_t*)take(8);
    a.norm = (float*)take(8);
    a.index = (int32_t*)take(tokens * 4);
    a.target = (int32_t*)take(tokens * 4);
    a.block = (a.tokens + kBlockRows) * 64;
    a.rows_plane = a.kd / 32 * a.block;
    a.rows = take((size_t)(planes * a.rows_plane));
    if (needs_pack(op, grad)) {
        a.values_row = 64;
        a.values_block = (int64_t)a.V * 64;
        a.values_bytes = a.values_plane = a.kd / 32 * a.values_block;
        a.values = take((size_t)(planes * a.values_plane));
    } else {
        a.values_row = (int64_t)a.d * (int64_t)element_bytes(op->io_dtype);
        a.values_block = 64;
        a.values_plane = 0;
        a.values_bytes = (int64_t)a.V * a.values_row;
        a.values = (const char*)op->table;
    }
    if (!grad) a.hit = (float*)take(tokens * 4);
    const int64_t whole = loss_tiles(a.V);
    if (!grad && a.small) {
        a.chunk = a.V;
        a.part = (float2*)take((size_t)loss_tiles(a.V, true) * tokens * 8);
        return at;
    }
    if (!grad) {
        const int64_t fit = kPartBytes / (a.tokens * 8), tiles = a.few ? few_groups(a.V) : even_pieces(whole, fit);
        a.chunk = a.few ? a.V : (int32_t)(tiles * kLossValues);
        a.part = (float2*)take((size_t)tiles * tokens * 8);
        a.running = (float2*)take(tiles < whole && !a.few ? tokens * 8 : 0);
        return at;
    }
    a.place = (int32_t*)take((size_t)a.total * 4);
    a.weight = (float*)take(tokens * 4);
    a.lse2 = (float*)take(tokens * 4);
    a.acc_row = (int32_t)((a.d + 3) / 4 * 4);
    if (a.few) {
        a.chunk = a.V;
        a.g = take((size_t)((a.V + 15) / 16 * 16 + 3) * 16 * 4);  // (read four values at a time)
        a.splits = planes == 1 && a.total <= kFewGroupsTokens ? kFewGroupsHalf : kFewGroups;
        a.acc_tokens = a.total;
        a.acc = (float*)take((size_t)a.splits * (size_t)a.total * (size_t)a.acc_row * 4);
        return at;
    }
    const int64_t tiles = even_pieces(whole, kGradBytes / (a.tokens * 2 * grad_planes * kLossValues));
    a.chunk = (int32_t)(tiles * kLossValues);
    a.g_plane = a.chunk / 32 * a.block;
    a.g = take((size_t)(grad_planes * a.g_plane));
    // d_x's sums over a piece are cut so that their workgroups, which come last, take a part
    // of what all of the piece's work takes on kSplitGroups of them
    const int64_t channel_tiles = (a.d + kGradChannels - 1) / kGradChannels, dx_tiles = a.tokens / kGradRows * channel_tiles;
    const int64_t dx_steps = a.chunk / 32, table_steps = a.tokens / 32, table_tiles = a.chunk / kGradRows * channel_tiles;
    const int64_t all = (dx_tiles * dx_steps + table_tiles * table_steps) / kSplitGroups, share = all < 1 ? 1 : all;
    int64_t splits = (kSplitParts * dx_steps + share - 1) / share;
    const int64_t most = a.chunk / 512 < 1 ? 1 : a.chunk / 512;  // a part has 512 values at least
    const int64_t cap = a.tokens <= 1024 ? 64 : 16;
    splits = splits < 1 ? 1 : splits > most ? most : splits > cap ? cap : splits;
    a.splits = (int32_t)splits;
    // (2^18 tokens, 16 values, width 256: 345 us so, 457 through a sum)
    a.acc_tokens = a.tokens;
    a.direct = splits == 1 && a.chunk >= a.V;
    a.acc = (float*)take(a.direct ? 0 : (size_t)splits * tokens * (size_t)a.acc_row * 4);
    // d_table's over the tokens, where one of them would take longer than that
    const int64_t part = planes == 3 ? 2 * share : share;  // (float32: a compute unit holds one workgroup, not two)
    const int64_t table_splits = (table_steps + part - 1) / part, table_most = table_steps / kTableSteps;
    a.table_splits = (int32_t)(table_splits <= 1 || table_most <= 1 ? 1 : table_splits < table_most ? table_splits : table_most);
    a.table_acc = (float*)take(a.table_splits == 1 ? 0 : (size_t)a.table_splits * (size_t)a.chunk * (size_t)a.acc_row * 4);
    return at;
}

hyena_status loss_args(const hyena_token_loss* op, void* scratch, bool grad, const hyena_rows* d_loss, LossArgs& a, Span* ins,
                       bool* units, size_t* bytes)
{
    hyena_status st = loss_sizes(op);
    if (st != HYENA_OK) return st;
    const size_t e = element_bytes(op->io_dtype);
    if ((st = check_rows(kWho, op->x, "x", e)) != HYENA_OK || (st = check_rows(kWho, op->targets, "targets", 4)) != HYENA_OK ||
        (d_loss != nullptr && (st = check_rows(kWho, *d_loss, "d_loss", 4)) != HYENA_OK))
        return st;
    if (op->table == nullptr || (uintptr_t)op->table % 16 != 0) return refuse("table is NULL or not 16-byte aligned");
    if (scratch == nullptr || (uintptr_t)scratch % 16 != 0) return refuse("scratch is NULL or not 16-byte aligned");
    *bytes = lay_out(op, grad, scratch, a);
    hyena_rows x = plain_rows(op->x, op->B, op->N), targets = plain_rows(op->targets, op->B, op->N),
               dl = d_loss ? plain_rows(*d_loss, op->B, op->N) : hyena_rows{nullptr, 0, 0};
    ins[0] = rows_span(x, op->B, op->N, op->d, e);
    ins[1] = rows_span(targets, op->B, op->N, 1, 4);
    ins[2] = Span{op->table, (size_t)(op->V * op->d) * e};
    ins[3] = d_loss ? rows_span(dl, op->B, op->N, 1, 4) : Span{nullptr, 0};
    RowShape made(op->d, e);
    made.add(x);
    *units = made.units();
    hyena_rows* v[3] = {&x, &targets, &dl};
    uint32_t* n[3] = {&a.x_N, &a.targets_N, &a.d_loss_N};
    Rows* to[3] = {&a.x, &a.targets, &a.d_loss};
    for (int i = 0; i < 3; ++i) {
        int64_t N = op->N;
        flatten_rows(&v[i], 1, op->B, &N);
        *n[i] = (uint32_t)N;
        *to[i] = Rows{v[i]->data, v[i]->batch, v[i]->token};
    }
    return HYENA_OK;
}

}  // namespace
}  // namespace hy

using namespace hy;

extern "C" {

hyena_status hyena_token_loss_scratch_bytes(const hyena_token_loss* op, size_t* forward_bytes, size_t* backward_bytes)
{
    const hyena_status st = loss_sizes(op);
    if (st != HYENA_OK) return st;
    LossArgs a{};
    if (forward_bytes) *forward_bytes = lay_out(op, false, nullptr, a);
    if (backward_bytes) *backward_bytes = lay_out(op, true, nullptr, a);
    return HYENA_OK;
}

hyena_status hyena_token_loss_forward(const hyena_token_loss* op, float* loss, float* lse, void* scratch, void* stream)
{
    LossArgs a{};
    Span ins[4];
    bool units;
    size_t bytes;
    hyena_status st = loss_args(op, scratch, false, nullptr, a, ins, &units, &bytes);
    if (st != HYENA_OK) return st;
    if (loss == nullptr || lse == nullptr || (uintptr_t)loss % 4 != 0 || (uintptr_t)lse % 4 != 0)
        return refuse("loss or lse is NULL or not aligned to its element");
    const Named outs[3] = {{Span{loss, (size_t)a.total * 4}, "loss"}, {Span{lse, (size_t)a.total * 4}, "lse"}, {Span{scratch, bytes}, "scratch"}};
    if ((st = check_apart(kWho, ins, 4, outs, 3)) != HYENA_OK) return st;
    a.loss = loss;
    a.lse = lse;
    return by_io(op->io_dtype, [&](auto* t) {
        return loss_forward<std::remove_pointer_t<decltype(t)>>(a, needs_pack(op, false), units, (hipStream_t)stream);
    });
}

hyena_status hyena_token_loss_backward(const hyena_token_loss* op, const hyena_rows* d_loss, const float* lse, void* d_x,
                                       void* d_table, void* scratch, void* stream)
{
    LossArgs a{};
    Span ins[5];
    bool units;
    size_t bytes;
    if (d_loss == nullptr) return refuse("d_loss is NULL");
    hyena_status st = loss_args(op, scratch, true, d_loss, a, ins, &units, &bytes);
    if (st != HYENA_OK) return st;
    if (lse == nullptr || (uintptr_t)lse % 4 != 0) return refuse("lse is NULL or not aligned to its element");
    if (d_x == nullptr && d_table == nullptr) return refuse("neither d_x nor d_table is wanted");
    if ((uintptr_t)d_x % 16 != 0 || (uintptr_t)d_table % 16 != 0) return refuse("d_x or d_table is not 16-byte aligned");
    const size_t e = element_bytes(op->io_dtype);
    ins[4] = Span{lse, (size_t)a.total * 4};
    const Named outs[3] = {{Span{d_x, (size_t)(a.total * op->d) * e}, "d_x"}, {Span{d_table, (size_t)(op->V * op->d) * e}, "d_table"},
                           {Span{scratch, bytes}, "scratch"}};
    if ((st = check_apart(kWho, ins, 5, outs, 3)) != HYENA_OK) return st;
    a.lse_in = lse;
    a.d_x = d_x;
    a.d_table = d_table;
    return by_io(op->io_dtype, [&](auto* t) {
        return loss_backward<std::remove_pointer_t<decltype(t)>>(a, needs_pack(op, true), units, (hipStream_t)stream);
    });
}

}  // extern "C"
