// tmoe_grouped.hpp -- launch arguments of the products grouped by expert.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tmoe {

enum GroupedOp { kGroupedLinear = 0, kGroupedGradX = 1, kGroupedGradW = 2 };

// out[row][col] = sum over the depth of R[row] C[col]; group e holds rows [offsets[e], offsets[e + 1]) of R_total.
//   linear  R = x [rows][K]      C = w_e [N][K]      depth K, cols N
//   grad_x  R = dy [rows][N]     C = w_e [N][K]      depth N, cols K   (C's depth runs along its rows)
//   grad_w  R = dy [rows][N]     C = x [rows][K]     depth: the group's rows (of both), out_rows N, cols K
struct GroupedArgs {
  const void* r;
  const void* c;
  const uint8_t* rs;         // MXFP8: scale bytes [rows][K / 32] and [E][N][K / 32]
  const uint8_t* cs;
  const void* offsets;       // [E + 1]
  int off64;
  int experts;
  int rows;                  // R_total
  int depth;                 // grad_w: unused
  int cols;
  int out_rows;              // grad_w: N
  void* y;
};

// op: GroupedOp; dtype: TMOE_BF16 or TMOE_F16; out_f32: y is fp32, else of dtype. False: more workgroups than a launch holds.
bool launch_grouped_bf16(const GroupedArgs& a, int op, bool out_f32, hipStream_t s);
bool launch_grouped_f16(const GroupedArgs& a, int op, bool out_f32, hipStream_t s);
bool launch_grouped_mxfp8(const GroupedArgs& a, bool out_f32, hipStream_t s);   // linear; y bf16 or fp32

}  // namespace tmoe
