// Host interface of the router's training kernels (internal to liblmoe.so).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace lmoe {

// A batch of router decisions: T tokens over E experts, k chosen each, in S
// sequences [seq[s], seq[s+1]) (seq NULL: one sequence of all tokens); mask
// NULL or nonzero where the token counts.
struct RouterBatch {
  const float* logits;      // [T, E]
  const int32_t* ids;       // [T, k]
  const uint8_t* mask;      // [T] or NULL
  const int32_t* seq;       // [S + 1] or NULL
  int T, E, k, S;
};

size_t balance_workspace_bytes(int T);

cudaError_t launch_balance_loss(const RouterBatch& b, float alpha, float* loss, int32_t* counts,
                                int32_t* tokens, void* workspace, cudaStream_t s);

// grad [T, E] = the gradient through the routing weights (grad_w [T, k], or
// NULL) plus the balance loss's (grad_loss [1] with counts and tokens, or NULL)
cudaError_t launch_router_backward(const RouterBatch& b, const float* grad_w, int renorm, float rsf,
                                   const float* grad_loss, const int32_t* counts,
                                   const int32_t* tokens, float alpha, float* grad, cudaStream_t s);

}  // namespace lmoe
