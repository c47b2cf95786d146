// bf16 products of rows grouped by expert and their gradients:
//   forward   out[r] = W_e x[r]
//   backward  grad_x[r] = W_e^T grad_out[r],   grad_W_e = sum over r of grad_out[r] x[r]^T
// for the rows r of expert e, offsets[e] .. offsets[e+1] - 1; products summed in fp32 and rounded
// once.
//
// The simplest form: a CTA a 64 x 64 tile, operands through shared memory, fp32 FMAs.
#include "grouped.cuh"

namespace lmoe {
namespace {

constexpr int kT = 64, kD = 16, kThreads = 256;

// sum over k < depth of A(m, k) B(n, k), A(m, k) at a[m am + k ak]; the caller's thread gets rows
// 4 ty .. and columns 4 tx .. of the tile
__device__ void tile_product(const uint16_t* a, long long am, long long ak, int mv, const uint16_t* b,
                             long long bn, long long bk, int nv, int depth, float (&acc)[4][4]) {
  __shared__ float as[kD][kT + 1], bs[kD][kT + 1];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
  for (int k0 = 0; k0 < depth; k0 += kD) {
    __syncthreads();
    for (int i = threadIdx.x; i < kT * kD; i += kThreads) {
      const int k = i % kD, m = i / kD;
      const bool in = k0 + k < depth;
      as[k][m] = in && m < mv ? __uint_as_float((uint32_t)a[m * am + (k0 + k) * ak] << 16) : 0.0f;
      bs[k][m] = in && m < nv ? __uint_as_float((uint32_t)b[m * bn + (k0 + k) * bk] << 16) : 0.0f;
    }
    __syncthreads();
    for (int k = 0; k < kD; ++k)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(as[k][4 * ty + i], bs[k][4 * tx + j], acc[i][j]);
  }
}

__device__ __forceinline__ int2 group_rows(const int32_t* offsets, int e, long long R) {
  const int a = min(max(__ldg(offsets + e), 0), (int)R);
  return make_int2(a, min(max(__ldg(offsets + e + 1), a), (int)R));
}

__global__ void __launch_bounds__(kThreads)
linear_kernel(GroupedLinear p, bool backward) {
  pdl_trigger();
  pdl_wait();
  const int e = blockIdx.y, in = backward ? p.N : p.K, out = backward ? p.K : p.N;
  const int2 r = group_rows(p.offsets, e, p.R);
  const int c0 = blockIdx.x * kT;
  const uint16_t* w = p.w + (long long)e * p.N * p.K + (long long)c0 * (backward ? 1 : p.K);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (long long r0 = r.x; r0 < r.y; r0 += kT) {
    float acc[4][4];
    tile_product(p.rows_in + r0 * in, in, 1, (int)min((long long)kT, r.y - r0), w,
                 backward ? 1 : p.K, backward ? p.K : 1, out - c0, in, acc);
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j) {
        const long long row = r0 + 4 * ty + i;
        const int c = c0 + 4 * tx + j;
        if (row < r.y && c < out) p.rows_out[row * out + c] = to_bf16(acc[i][j]);
      }
  }
}

__global__ void __launch_bounds__(kThreads)
weight_grad_kernel(GroupedWeightGrad p) {
  pdl_trigger();
  pdl_wait();
  const int e = blockIdx.z, n0 = blockIdx.y * kT, k0 = blockIdx.x * kT;
  const int2 r = group_rows(p.offsets, e, p.R);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4];
  tile_product(p.dy + (long long)r.x * p.N + n0, 1, p.N, p.N - n0, p.x + (long long)r.x * p.K + k0, 1,
               p.K, p.K - k0, r.y - r.x, acc);
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + 4 * ty + i, k = k0 + 4 * tx + j;
      if (n >= p.N || k >= p.K) continue;
      const long long at = ((long long)e * p.N + n) * p.K + k;
      if (p.dw) p.dw[at] = p.add ? p.add[at] + acc[i][j] : acc[i][j];
      else p.dw_bf16[at] = to_bf16(acc[i][j]);
    }
}

}  // namespace

cudaError_t launch_grouped_linear(const GroupedLinear& g, bool backward, cudaStream_t s) {
  return launch_k(linear_kernel, dim3(ceil_div(backward ? g.K : g.N, kT), g.E), dim3(kThreads), 0, s, g,
                  backward);
}

cudaError_t launch_grouped_weight_grad(const GroupedWeightGrad& g, cudaStream_t s) {
  return launch_k(weight_grad_kernel, dim3(ceil_div(g.K, kT), ceil_div(g.N, kT), g.E), dim3(kThreads), 0,
                  s, g);
}

}  // namespace lmoe
