// Host interface of the bf16 products grouped by expert (internal to liblmoe.so).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "lmoe_internal.cuh"

namespace lmoe {

constexpr long long kMaxGroupedRows = 1ll << 27;
constexpr int kMaxGroupedDim = 65536;

// Expert e owns rows offsets[e] .. offsets[e+1] - 1 of the row matrices.
struct GroupedLinear {
  const uint16_t* rows_in;     // x [R, K] (forward) or grad_out [R, N] (backward)
  const uint16_t* w;           // [E, N, K]
  const int32_t* offsets;      // [E + 1], on the device
  uint16_t* rows_out;          // [R, N] (forward) or [R, K] (backward)
  long long R;
  int E, N, K;
};

struct GroupedWeightGrad {
  const uint16_t* dy;          // [R, N]
  const uint16_t* x;           // [R, K]
  const int32_t* offsets;
  const float* add;            // [E, N, K] or NULL, with dw
  float* dw;                   // [E, N, K], or NULL and
  uint16_t* dw_bf16;           // [E, N, K]
  long long R;
  int E, N, K;
};

// ... for few rows in all (grouped_stream.cu); launch_grouped_linear calls it
long long grouped_stream_ctas(const GroupedLinear& g, bool backward);
cudaError_t launch_grouped_stream(const GroupedLinear& g, bool backward, cudaStream_t s);
cudaError_t launch_grouped_linear(const GroupedLinear& g, bool backward, cudaStream_t s);
cudaError_t launch_grouped_weight_grad(const GroupedWeightGrad& g, cudaStream_t s);

}  // namespace lmoe
