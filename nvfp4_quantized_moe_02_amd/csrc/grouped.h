// Launchers of the products with 8- and 16-bit weights (grouped.hip) and of the expert
// combine (combine.hip). Argument validation is the C-ABI layer's job (api_grouped.hip).
#pragma once
#include "common.h"

namespace nvfp4 {

// One grouped product. Rows r of the sorted order belong to expert e when
// offsets[e] <= r < offsets[e+1]; offsets == nullptr: one expert with all P rows.
struct GroupedArgs {
  const void* a;          // forward: x [xrows][K]; dx, dw: dy [P][N]
  const void* b;          // forward, dx: w [E][N][K]; dw: x [xrows][K]
  const float* a_scale;   // int8: one per row of x
  const float* b_scale;   // int8: [E][N]
  const int32_t* offsets; // [E+1]
  const int32_t* pairs;   // sorted pairs, or nullptr: row r of x is row r
  int topk;
  int xrows;              // rows of x (bounds the rows that pairs name)
  int E, P, N, K;
  void* out;
  int out_dtype;          // nvfp4_dtype
};

// type: 0 bf16, 1 fp16, 2 int8 (forward only)
hipError_t launch_grouped_fwd(int type, const GroupedArgs& g, hipStream_t st);
hipError_t launch_grouped_dx(int type, const GroupedArgs& g, hipStream_t st);
hipError_t launch_grouped_dw(int type, const GroupedArgs& g, hipStream_t st);

// combine.hip. inv: workspace of P = T * topk ints (any contents); none up to kSmallPairs.
constexpr int kSmallPairs = 1024;
struct CombineArgs {
  const int32_t* pairs;  // sorted pairs [P], -1 for dropped ones
  const float* w;        // [T][topk] or nullptr (1)
  int32_t* inv;
  int T, topk, H;
};
// out[t] = sum over slots j in order of w[t][j] * y[position of pair t*topk+j]
hipError_t launch_combine_rows(const CombineArgs& c, const void* y, int y_dtype, void* out, int out_dtype,
                               hipStream_t st);
// dy[position] = w * dout[t]; dw[t][j] = dout[t] . y[position] (dw == nullptr: not computed, y unused)
hipError_t launch_combine_grad(const CombineArgs& c, const void* dout, const void* y, int dtype, void* dy, float* dw,
                               hipStream_t st);

}  // namespace nvfp4
