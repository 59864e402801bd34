// Launchers of the products grouped by expert and of the 4-bit products (defined
// in pe_grouped.hip), and of what stands around them: the order by expert, the
// weighted sum back to tokens and its gradients.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "pe_dense.h"

namespace pe {

// A product whose rows belong to experts: rows offsets[e] .. offsets[e + 1] - 1 of the output take expert e's weights.
// Without offsets all of the d.T rows take the one matrix.
struct GroupedArgs {
  DenseArgs d;               // d.b, d.bias: the first expert's.  Products of rows: d.T = R.  Weight gradients: the
                             // output has d.T rows of d.N columns for each expert, d.K is not used
  const int32_t* offsets;    // [E + 1] or nullptr
  const int32_t* rows;       // [R] the row of x (d.a; of weight gradients d.b) that each row takes, or nullptr: its own
  int E, R;
  int x_rows;                // rows of x
  const void* ws;            // 4-bit weights' scales: fp16 [E, rows, K / 128] or E8M0 [E, rows, K / 32]
};

struct GroupRowsArgs {
  const int32_t* ids;        // [n]
  int n, k, E;
  int32_t* offsets;          // [E + 1]
  int32_t* rows;             // [n]
  int32_t* places;           // [n]
};

struct CombineArgs {
  const uint16_t* y;         // bf16 [R, H], rows ldy apart
  int64_t ldy;
  const int32_t* places;     // [T, k]
  const float* w;            // [T, k] or nullptr: 1
  const uint16_t* residual;  // bf16 [T, H] or nullptr
  int64_t ldr;
  int T, k, H, R;
  uint16_t* out;             // bf16 [T, H]
  int64_t ldo;
};

struct CombineBackArgs {
  const uint16_t* dout;      // bf16 [T, H]
  int64_t lddo;
  const int32_t* places;     // [T, k]
  const float* w;            // [T, k] or nullptr: 1
  const uint16_t* y;         // bf16 [R, H]; with dw
  int64_t ldy;
  int T, k, H, R;
  uint16_t* dy;              // bf16 [R, H] or nullptr
  int64_t lddy;
  float* dw;                 // [T, k] or nullptr
};

// wtype: PE_W_BF16, PE_W_INT4_G128 or PE_W_MXFP4_B32.
void launch_grouped(DenseOp op, int wtype, const GroupedArgs& a, hipStream_t s);
// dh, dg and du from dy (DENSE_DGLU), and dx from those (DENSE_LINEAR): w k-slow
void launch_grouped_back(DenseOp op, const GroupedArgs& a, hipStream_t s);
// weight gradients: the sums over each expert's rows
void launch_grouped_weights(const GroupedArgs& a, hipStream_t s);
void launch_group_rows(const GroupRowsArgs& a, hipStream_t s);
void launch_combine(const CombineArgs& a, hipStream_t s);
void launch_combine_back(const CombineBackArgs& a, hipStream_t s);

}  // namespace pe
