// ep_experts_w4.cuh -- what the two kernels of the experts' products with
// 4-bit weights share: the arguments and the split between them.
//
// An expert with at most kFewRows rows is bound by reading its weights and
// goes to the register kernel (ep_experts_w4.cu); one with more goes to the
// tcgen05 kernel (ep_experts_w4_tc.cu).  The counts are on the device, so
// each kernel skips the other's experts.  Measured on 256 experts of 7168 ->
// 2048 channels, register against tcgen05 kernel: about 2 rows each 457 against
// 772 us, 4 rows 550 against 878, 6 rows 635 against 879, 8 rows (some experts
// have more) 711 against 879; E4M3 rows: 2 rows 409 against 607, 6 rows 565
// against 690.  A form of the register kernel for up to 32 rows took 983 us at
// 10 rows and 2144 at 20, where the tcgen05 kernel of that time took 831 and 985.
#pragma once

#include <cuda_bf16.h>

#include "ep_common.cuh"

namespace ep {

constexpr int kFewRows = 8;

struct ExpertsArgs {
  const uint8_t* x;  // bf16 or E4M3 rows
  const float* x_scales;
  int I;  // input channels
  const int32_t* count;
  int E;
  int64_t cap;
  const uint8_t* q;
  const __nv_bfloat16* scales;
  const uint8_t* zeros;
  int N;      // output channels
  int rows;   // weight rows per expert (N, or 2 N for swiglu)
  int tiles;  // tiles of output channels per expert
  __nv_bfloat16* y;
  int32_t* err;
  int stall;  // test hook: a step of x that block 0 does not load (-1: off)
};

// g / (1 + exp(-g)) * up with the exponential of -|g|, which cannot overflow: the
// results of very negative gates stay numbers until exp(g) itself is 0 (below
// -103).  A few units in the last place of float32, rounded to bf16 next.
__device__ __forceinline__ float silu_times(float g, float up) {
  const float e = expf(-fabsf(g));
  return __fdividef(g < 0.0f ? g * e : g, 1.0f + e) * up;
}

// Experts with more than kFewRows rows (nothing is launched if the capacity
// rules them out).
ep_status_t launch_experts_many(const ExpertsArgs& a, bool fp8, bool swiglu, int group,
                                cudaStream_t st);

}  // namespace ep
