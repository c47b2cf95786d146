// Host interface of the 8-bit (e4m3) kernels (internal to liblmoe.so).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "lmoe_internal.cuh"

namespace lmoe {

constexpr int kFp8Block = 128;   // elements along K (and weight rows) that share a scale

inline int fp8_blocks(long long n) { return (int)((n + kFp8Block - 1) / kFp8Block); }

// One block-scaled product over token rows X and weight rows W, both e4m3 with
// K contiguous:  y[t, n] = sum_kb xs[t, kb] ws[n / 128, kb] sum_{c in kb} X[t, c] W[n, c].
struct Fp8Gemm {
  const uint8_t* X;          // [rows, K]
  const float* xs;           // [rows, ceil(K / 128)]
  const uint8_t* W;          // [groups, feat, K]
  const float* ws;           // [groups, ceil(feat / 128), ceil(K / 128)]
  long long rows;
  int groups, feat, K;
  const int32_t* offsets;    // [groups + 1] first row of each group (device), or NULL: one group
  const uint16_t* add;       // bf16 [rows, feat] or NULL
  uint16_t* out;             // bf16 [rows, feat]
  // SituGLU: feat = 2 d, gate rows first; writes e4m3 act [rows, d] and its
  // scales [rows, d / 128] in the place of out (d % 128 == 0)
  uint8_t* act;
  float* act_s;
  float beta, linear_beta;
  // few rows an expert: the activations in fp32 [rows, d] between the two
  // products, the first's output (instead of act) and the second's input
  // (instead of X and xs), which quantises them by the same rule
  float* act_f32;
  const float* act_in;
  // grouped: only groups of more than min_rows rows (the tensor-core kernel), of up to
  // max_rows (the streaming kernel; 0: any number)
  int min_rows, max_rows;
  // the kernel launched before this one writes nothing that this one reads, and has waited
  // for all work before it: this one waits at its end only, so that its own end says
  // that both are complete
  int beside;
};

// Dense products of up to this many token rows stream their weights through
// registers (fp8_stream.cu).
constexpr int kStreamRows = 16;

cudaError_t launch_fp8_gemm(const Fp8Gemm& g, cudaStream_t s);
// ... for few token rows (grouped: with act_f32 or act_in)
cudaError_t launch_fp8_stream(const Fp8Gemm& g, cudaStream_t s);
// ... dense, for many tiles of 256 x 256
cudaError_t launch_fp8_pair(const Fp8Gemm& g, cudaStream_t s);

// codes / scales of bf16 x [rows, K], one scale per block_rows (1 or 128) rows x 128 columns
cudaError_t launch_quantize_fp8(const uint16_t* x, uint8_t* codes, float* scales, long long rows,
                                int K, int block_rows, cudaStream_t s);

// The rows of Z [T, L] bf16 (L % 128 == 0) quantised per 128 columns and copied to
// the k rows row_of[t, :] of codes [T k, L] and scales [T k, L / 128].
cudaError_t launch_quantize_scatter_fp8(const uint16_t* Z, int T, int L, int k,
                                        const int32_t* row_of, uint8_t* codes, float* scales,
                                        cudaStream_t s);

}  // namespace lmoe
