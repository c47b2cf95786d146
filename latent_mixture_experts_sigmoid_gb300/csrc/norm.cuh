// Host interface of the residual + RMSNorm kernels (internal to liblmoe.so).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "lmoe_internal.cuh"

namespace lmoe {

constexpr int kMaxNormDim = 16384;

struct NormForward {
  const uint16_t* x;           // [T, H]
  const uint16_t* residual;    // [T, H] or NULL (zeros)
  const uint16_t* w;           // [H] or NULL (ones)
  uint16_t* h;                 // [T, H] or NULL: bf16(x + residual)
  uint16_t* out;               // [T, H] or NULL
  uint8_t* codes;              // [T, H] or NULL
  float* scales;               // [T, ceil(H / 128)], with codes
  int T, H;
  float eps;
};

struct NormBackward {
  const uint16_t* dy;          // [T, H]
  const uint16_t* h;           // [T, H]
  const uint16_t* w;           // [H] or NULL (ones)
  const uint16_t* dres;        // [T, H] or NULL (zeros)
  uint16_t* dh;                // [T, H]
  float* dw;                   // [H] or NULL
  float* partial;              // workspace, with dw
  int T, H;
  float eps;
  int* err;                    // the device error word
};

size_t norm_backward_workspace_bytes(int T, int H);
cudaError_t launch_norm(const NormForward& n, cudaStream_t s);
cudaError_t launch_norm_backward(const NormBackward& n, cudaStream_t s);

}  // namespace lmoe
