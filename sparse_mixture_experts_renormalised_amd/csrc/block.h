// Launchers of the residual block's kernels and of dropout (block.hip,
// dropout.hip).  Not part of the public interface.
#pragma once

#include "moe_common.h"
#include "philox.h"

namespace moe {

enum { kNormNone = 0, kNormRms = 1, kNormLayer = 2 };
constexpr int kMaxBlockWidth = 16384;   // elements of a row that a workgroup holds

struct BlockJoin {
  bool act_bf16, res_bf16;
  int64_t T;
  int d, K, n_shared, norm_out, norm_in;
  float eps, scale;
  Dropout drop;
  const void *residual;         // [T][d] stream type
  const void *branch;           // [T][d] act or null
  const void *y_rows;           // act rows or null; then with slot_row, topk_gate
  const int32_t *slot_row;      // [T][K]
  const float *topk_gate;       // [T][K]
  const void *shared_out;       // [n_shared][T][d] act
  const float *gate;            // [T] or null
  const float *w_out, *b_out, *w_in, *b_in;   // [d] or null
  void *out, *next, *branch_out;
};

struct BlockJoinGrad {
  bool act_bf16, res_bf16;
  int64_t T;
  int d, K, norm_out, norm_in;
  float eps, scale;
  Dropout drop;
  const void *d_out, *d_next, *h, *branch, *y_rows;
  const int32_t *slot_row;
  const float *topk_gate, *gate, *w_out, *b_out, *w_in;
  void *d_residual, *d_branch, *d_y_rows;
  float *d_gate, *d_topk_gate;
  float *sum[4];                // d_w_in, d_b_in, d_w_out, d_b_out: [d] or null
  float *part;                  // workspace (null where no sum is asked for)
};

hipError_t launch_block_join(const BlockJoin &a, hipStream_t s);
size_t block_join_grad_workspace_bytes(int64_t T, int d);
hipError_t launch_block_join_grad(const BlockJoinGrad &a, hipStream_t s);

// y[i] = x[i] keep or 0 for the elements of the first min(rows, *n_rows) rows.
hipError_t launch_dropout(bool bf16, const void *x, void *y, int64_t rows, int64_t d,
                          const int32_t *n_rows, const Dropout &drop, hipStream_t s);

}  // namespace moe
