// Launch descriptors of the operators around the optimizer step: embedding,
// layer norm, 8-bit activation checkpoints and the weight gradient.
#pragma once
#include "common.hpp"

namespace ma {

// storage code of an operand held as an 8-bit checkpoint (kernel templates only)
constexpr int DT_ACT8 = 2;

// ---- embedding ----
struct EmbedFwdArgs {
  const void* table;
  const void* tokens;
  void* out;
  int64_t rows, n_tokens;
  int32_t cols, wide;   // wide: 8-byte tokens
  float scale;
};
hipError_t launch_embed_fwd(const EmbedFwdArgs& a, int table_dt, int out_dt, hipStream_t s);

// Runs of the sorted tokens longer than this are summed in pieces of as many
// sorted positions, one wave each, and joined in order. Short pieces shorten the
// longest wave, long ones the join (5003 tokens x 333 fp32: sums 7.5 us with 16,
// 10.5 with 32, join 4.2 both; 49152 x 1024 bf16: join 10.3 and 7.3, sums alike).
constexpr int64_t kEmbedShortPieces = 16384;   // tokens
constexpr int embed_piece(int64_t n_tokens) { return n_tokens <= kEmbedShortPieces ? 16 : 32; }
// Up to this many tokens the rows' waves look for their tokens themselves, in
// one launch in place of three (bf16 into 1000 x 1024: 1000 tokens 15 us against
// 5.8 + 8.5 + 3.7 and two launches, 2000 tokens 24 against 6 + 8.2 + 4.6; into
// 50304 x 1024: 35 against 6 + 37 + 4.7).
constexpr int kEmbedDirect = 1024;
struct EmbedBwdArgs {
  const void* dout;
  const void* tokens;
  float* grad;
  int64_t rows, n_tokens;
  int32_t cols, wide, accumulate;
  float scale;
  // workspace: the number of valid tokens, start / count of every row's run in
  // the sorted order (by slot, see k_embed_bin), the positions and slots in that
  // order, and two partial rows for each piece
  int32_t *n_valid, *start, *count, *order, *keys;
  float* partial;
  int32_t log2nb, per_block;   // the sort's blocks (2^log2nb) and rows per block
  int32_t piece;               // embed_piece(n_tokens)
};
size_t embed_bwd_workspace(int64_t rows, int64_t cols, int64_t n_tokens);
void embed_bwd_carve(EmbedBwdArgs& a, unsigned char* ws);
hipError_t launch_embed_bwd(const EmbedBwdArgs& a, int dout_dt, hipStream_t s);

// ---- layer norm ----
constexpr int64_t kMaxNormCols = 16384;   // what 1024 lanes hold in registers
struct NormFwdArgs {
  const void* x;
  const float *gain, *bias;   // either may be null
  void* y;
  float* stats;               // 2 per row: mean, 1 / sqrt(var + eps)
  uint8_t *q, *qscale;        // checkpoint of x, or null
  int64_t rows;
  int32_t cols;
  float eps;
};
hipError_t launch_norm_fwd(const NormFwdArgs& a, int x_dt, int y_dt, hipStream_t s);

struct NormBwdArgs {
  const void* dy;
  const void* x;              // or q / qscale
  const uint8_t *q, *qscale;
  const float *stats, *gain;
  void* dx;
  float *dgain, *dbias;       // either may be null
  float* partial;             // [2][cols / 32][blocks][32]; null if not kept
  int64_t rows;
  int32_t cols, accumulate, blocks;
};
int norm_bwd_blocks(int64_t rows, int64_t cols);
bool norm_bwd_direct(int64_t rows);
hipError_t launch_norm_bwd(const NormBwdArgs& a, int x_dt, int dy_dt, int dx_dt, hipStream_t s);

// ---- 8-bit activation checkpoints ----
struct ActArgs {
  const void* x;
  void* out;
  uint8_t *q, *qscale;
  int64_t rows;
  int32_t cols;
};
hipError_t launch_act_pack(const ActArgs& a, int x_dt, hipStream_t s);
hipError_t launch_act_unpack(const ActArgs& a, int out_dt, hipStream_t s);

// ---- weight gradient out of a checkpoint ----
struct WgradArgs {
  const void* dy;             // tokens x outs
  const uint8_t *q, *qscale;  // tokens x ins
  void* grad;                 // outs x ins
  float* partial;             // [splits][wgrad_partial], splits > 1
  int64_t tokens;
  int32_t outs, ins, accumulate, splits, big;   // splits, big: wgrad_plan's
};
struct WgradPlan { bool big; int splits; };
// elements of one split's partial products (whole cache lines)
__host__ __device__ constexpr int64_t wgrad_partial(int64_t outs, int64_t ins) { return round_up(outs * ins, 64); }
WgradPlan wgrad_plan(int64_t tokens, int64_t outs, int64_t ins, int dy_dt);
hipError_t launch_wgrad(const WgradArgs& a, int dy_dt, int grad_dt, hipStream_t s);

}  // namespace ma
