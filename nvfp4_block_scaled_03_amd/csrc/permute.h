// Host entry points of the movement of rows by expert (permute.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nvfp4 {

// Row widths W in elements; every row is a whole number of 16-byte pieces.
struct PermuteArgs {
  int T, topk, shared, slots;
  int64_t W;
  const int32_t* offsets;   // [slots + 1]
  const int32_t* inv_pos;   // [P]
  const float* w;           // [T][topk], or null: 1
};
// rows[inv_pos[f]] = x[token of f]; with zero_tail the rows behind the last kept one are cleared.
hipError_t launch_permute(const PermuteArgs& a, const void* x, bool f32, int64_t ldx, void* rows, bool zero_tail,
                          hipStream_t s);
// out[t] = sum of w rows[inv_pos[f]] over the pairs f of token t.
hipError_t launch_unpermute(const PermuteArgs& a, const void* rows, bool f32, void* out, bool out_f32, hipStream_t s);
// d_rows[inv_pos[f]] = w d_out[t]; d_w[t][j] = <d_out[t], rows[inv_pos[f]]>; either may be null.
hipError_t launch_unpermute_backward(const PermuteArgs& a, const void* d_out, bool out_f32, const void* rows, bool f32,
                                     void* d_rows, float* d_w, bool zero_tail, hipStream_t s);

}  // namespace nvfp4
