// token_loss.h -- arguments and scratch of the loss over a vocabulary.
#pragma once

#include "rows.h"

namespace hy {

// Tokens and values of the vocabulary of a tile of logits; channels and rows of a
// tile of the gradients.
constexpr int kLossTokens = 128, kLossValues = 256;
// The same where whole tiles are few.
constexpr int kSmallTile = 64;
// Workgroups of the logits of few tokens, which take tiles of 16 values in turn (768 and 1024 are
// slower by 1 us of 20: the registers let a compute unit have two).
constexpr int kFewLogits = 512;
inline int loss_tiles(int64_t V, bool small = false)
{
    const int tile = small ? kSmallTile : kLossValues;
    return (int)((V + tile - 1) / tile);
}
inline int few_groups(int64_t V) { return (V + 15) / 16 < kFewLogits ? (int)((V + 15) / 16) : kFewLogits; }
constexpr int kGradRows = 128, kGradChannels = 256;

struct LossArgs {
    Rows x, targets, d_loss;
    uint32_t x_N, targets_N, d_loss_N;  // row_at
    int64_t total;         // B * N
    int32_t V, d;
    int32_t kd;            // d rounded up to 32: the width of gathered rows
    int32_t each;          // tokens of a workgroup of the gather
    int32_t few;           // few tokens: their own kernels
    int32_t small;         // tiles of logits of kSmallTile
    float scale;
    const void* table;     // as given
    const float* lse_in;
    float* loss;
    float* lse;
    void* d_x;
    void* d_table;

    // scratch
    int64_t* count;        // tokens that take part
    float* norm;           // [0] what G is multiplied by, [1] what undoes it
    int32_t* index;        // [tokens] which token of the call
    int32_t* place;        // [B * N] which gathered row, or -1
    int32_t* target;       // [tokens]
    float* weight;         // [tokens] d_loss
    float* lse2;           // [tokens] lse / ln 2
    char* rows;            // gathered x: [planes][kd / 32][tokens rounded up][32], 16-bit
    int64_t block;         // bytes from 32 channels (values) of rows (g) to the next
    int64_t rows_plane;    // bytes
    const char* values;    // the table as matrix operand: itself, or [planes][kd / 32][V][32]
    int64_t values_row, values_block, values_plane, values_bytes;  // bytes: of a row, 32 channels, a plane; the first plane's
    float2* part;          // [tiles of a piece's values][tokens rounded up]: largest, sum
    float2* running;       // [tokens] the same of the pieces before, where there is more than one
    float* hit;            // [tokens] forward: the target's logit
    char* g;               // [planes][chunk / 32][tokens rounded up][32]; of few tokens float32 [values rounded up][16]
    int64_t g_plane;
    float* acc;            // [splits][acc_tokens][acc_row] d_x
    int64_t acc_tokens;    // tokens rounded up; of few tokens as many as there are
    int64_t tokens;        // rounded up
    int32_t acc_row;
    int32_t chunk;         // values of a piece of the vocabulary
    int32_t first;         // of this piece
    int32_t splits;        // of the sum over a piece's values, for d_x
    int32_t direct;        // one piece, one part: d_x is not summed up but written
    int32_t table_splits;  // of the sum over the tokens, for d_table
    float* table_acc;      // [table_splits][chunk][acc_row] d_table of a piece, where there is more than one
};

// Launches of one call; P: planes (float32: three bfloat16 terms).
template <typename T> hyena_status loss_forward(const LossArgs& a, bool pack, bool units, hipStream_t s);
template <typename T> hyena_status loss_backward(const LossArgs& a, bool pack, bool units, hipStream_t s);
#define HY_LOSS_EXTERN(T)                                                                                  \
    extern template hyena_status loss_forward<T>(const LossArgs&, bool, bool, hipStream_t);                \
    extern template hyena_status loss_backward<T>(const LossArgs&, bool, bool, hipStream_t);
HY_LOSS_EXTERN(float)
HY_LOSS_EXTERN(uint16_t)
HY_LOSS_EXTERN(_Float16)

}  // namespace hy
