// Interface between the host-side ABI layer of the loss operators
// (zero_loss_abi.cpp: validation, piece sizes, workspace layout) and their
// gfx950 kernels (zero_loss.hip). Plain C++, no HIP types.
#pragma once

#include <cstddef>
#include <cstdint>

namespace zloss {

enum Dtype { kF32 = 0, kBF16 = 1, kF16 = 2 };

// Tile extents every padded size below is a multiple of.
constexpr int64_t kRowPad = 256;  // token rows
constexpr int64_t kVocPad = 256;  // vocabulary rows of a piece
constexpr int64_t kDimPad = 64;   // the products' inner step
// Vocabulary rows one entry of the softmax partials covers.
constexpr int64_t kStatRows = 128;
// Up to here the tiles of dhidden and dweight are made for few tokens.
constexpr int kFewTokens = 64;

// Sizes and workspace offsets of one call, made by the ABI layer.
struct Plan {
  int64_t tokens, vocab, dim;
  int dtype;
  int planes;        // 16-bit parts per value: 3 for fp32, else 1
  bool grad;
  bool pack_w;       // the weight goes through an aligned, padded copy, piece by piece
  int64_t rows;      // tokens padded to kRowPad
  int64_t dimp;      // dim padded to kDimPad
  int64_t piece;     // vocabulary rows per piece, a multiple of kVocPad
  int tile_m, tile_n; // the logits' tiles: vocabulary rows (256 or 128), tokens (256 or 64)
  int64_t stat_cols; // softmax partials per token
  int acc_tiles;     // tiles that the slabs of dhidden's sum have room for
  // workspace offsets, bytes
  size_t o_head;     // Head: live count, runs, scale
  size_t o_rowmap;   // int32[rows]: live position -> token
  size_t o_pos;      // int32[tokens]: token -> live position, -1 empty, -2 bad
  size_t o_state;    // uint8[tokens]: distillation's row states
  size_t o_h;        // 16-bit [planes][rows][dimp]: the live rows of hidden
  size_t o_w;        // 16-bit [planes][piece][dimp] when pack_w
  size_t o_stat;     // float2 [rows][stat_cols] (forward)
  size_t o_sum;      // float [rows][stat_cols] (forward): sums of the logits
  size_t o_entry;    // float [tokens] (cross entropy, forward): the targets' logits
  size_t o_rowp;     // RowParam[rows] (gradient)
  size_t o_g;        // 16-bit [planes][rows][piece] (gradient)
  size_t o_acc;      // float [splits][live rows][dimp] (gradient)
  size_t total;
};

// One call's arguments, validated.
struct Call {
  Plan plan;
  const void* hidden;
  int64_t hidden_stride;
  const void* weight;
  int64_t weight_stride;
  char* ws;
  // targets: k == 0 is cross entropy
  const void* target;      // tokens values, or the teacher's indices
  int index64;             // 1: 64-bit indices
  int64_t ignore_index;
  float smoothing, z_loss;
  int k;
  int64_t index_stride, logit_stride;
  const void* teacher;
  int teacher_dtype;
  float temperature;       // 1 for cross entropy
  // forward
  float* loss;
  float* lse;
  float* logit;
  // gradient
  const float* lse_in;
  const float* logit_in;
  const float* upstream;
  int64_t upstream_stride;
  void* dhidden;
  int64_t dhidden_stride;
  void* dweight;
  int64_t dweight_stride;
};

// Each returns nullptr on success, or the HIP runtime's error string.
const char* launch_loss(const Call& c, void* stream);
const char* launch_grad(const Call& c, void* stream);

}  // namespace zloss
