// SituGLU gated activation, dense and masked (batched MoE) layouts.
//
// vLLM PR #50088, commit 2:
//   gate_out = beta * tanh(gate / beta) * sigmoid(gate)
//   up_out   = linear_beta * tanh(up / linear_beta)   (linear_beta > 0)
//   out      = gate_out * up_out
// commit 3: linear_beta <= 0 means unset and up passes through.  Arithmetic is
// fp32 and results go straight to the output buffer.  The masked kernel reads
// expert_num_tokens and never touches padded rows.
//
// Bandwidth-bound: every thread moves 16-byte vectors (8 bf16); the scalar
// math (one hardware 2^x per exponential, one reciprocal per element, relative
// error about 1e-6) lives with the other SituGLU users in lmoe_internal.cuh.
#include "lmoe_internal.cuh"

namespace lmoe {
namespace {

__device__ __forceinline__ uint4 situ8(const uint4& g, const uint4& u, const SituParams& p) {
  uint4 o;
  o.x = situ2(g.x, u.x, p);
  o.y = situ2(g.y, u.y, p);
  o.z = situ2(g.z, u.z, p);
  o.w = situ2(g.w, u.w, p);
  return o;
}

__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

// Rows [row0, row0 + nrows) of a [*, 2d] -> [*, d] problem, vpr = d / 8.
__device__ __forceinline__ void situ_rows(const uint16_t* __restrict__ in, uint16_t* __restrict__ out,
                                          long long row0, int nrows, int d, int vpr,
                                          const SituParams& p) {
  const int total = nrows * vpr;
  for (int j0 = threadIdx.x; j0 < total; j0 += kUnroll * kThreads) {
    uint4 g[kUnroll], u[kUnroll];
    long long oi[kUnroll];
#pragma unroll
    for (int q = 0; q < kUnroll; ++q) {
      const int j = j0 + q * kThreads;
      oi[q] = -1;
      if (j < total) {
        const int r = j / vpr;
        const int c = j - r * vpr;
        const long long row = row0 + r;
        const uint16_t* src = in + row * (2LL * d) + (long long)c * 8;
        g[q] = ld_stream(reinterpret_cast<const uint4*>(src));
        u[q] = ld_stream(reinterpret_cast<const uint4*>(src + d));
        oi[q] = row * d + (long long)c * 8;
      }
    }
#pragma unroll
    for (int q = 0; q < kUnroll; ++q)
      if (oi[q] >= 0) *reinterpret_cast<uint4*>(out + oi[q]) = situ8(g[q], u[q], p);
  }
}

__global__ void __launch_bounds__(kThreads)
situ_dense_kernel(const uint16_t* __restrict__ in, uint16_t* __restrict__ out, long long N,
                  int d, int rows_per_block, SituParams p) {
  pdl_trigger();
  pdl_wait();
  const long long row0 = (long long)blockIdx.x * rows_per_block;
  if (row0 >= N) return;
  const int nrows = (int)min((long long)rows_per_block, N - row0);
  situ_rows(in, out, row0, nrows, d, d / 8, p);
}

__global__ void __launch_bounds__(kThreads)
situ_masked_kernel(const uint16_t* __restrict__ in, uint16_t* __restrict__ out,
                   const int32_t* __restrict__ counts, int T_max, int d, int rows_per_block,
                   SituParams p) {
  pdl_trigger();
  pdl_wait();
  const int e = blockIdx.y;
  const int n = min(max(__ldg(counts + e), 0), T_max);
  const int r0 = blockIdx.x * rows_per_block;
  if (r0 >= n) return;
  const int nrows = min(rows_per_block, n - r0);
  situ_rows(in, out, (long long)e * T_max + r0, nrows, d, d / 8, p);
}

int rows_for(int d) {
  // about 4096 16-byte vectors (64 KiB of input) per block
  const int vpr = d / 8;
  return vpr >= 4096 ? 1 : 4096 / vpr;
}

// ---------------------------------------------------------------------------
// Gradient.  With z = g / beta, s = sigmoid(g), v = u / linear_beta and the factors
//   a = beta tanh(z) s,  b = linear_beta tanh(v)  (or u):   out = a b,
//   grad_gate = dy b [ sech^2(z) s + beta tanh(z) s (1 - s) ],
//   grad_up   = dy a sech^2(v)  (or dy a).
// All of it comes from three exponentials of non-positive arguments and one reciprocal:
//   q = e^{-2|z|}:  |tanh z| = (1 - q) / (1 + q),  sech^2 z = 4 q / (1 + q)^2
//   p = e^{-|g|}:   s (1 - s) = p / (1 + p)^2,     s = 1 / (1 + p)  (g < 0: p / (1 + p))
//   k = e^{-2|v|}:  as q
// and 1 / ((1 + q)(1 + p)(1 + k)), whose divisor lies in [1, 8].  sech^2 = 1 - tanh^2 would
// cancel where the activation saturates; these keep their relative accuracy.  1 - q cancels
// for small z, where its cubic stands in.
// ---------------------------------------------------------------------------

// |tanh x| from m = |x|, q = e^{-2m} and r = 1 / (1 + q).  Below 2^-5 the first two terms of
// the series (the third is 2 m^4 / 15 < 2^-22 of the first); from there on 1 - q has lost at
// most five bits to cancellation.
__device__ __forceinline__ float tanh_of(float m, float q, float r) {
  return m < 0.03125f ? fmaf(m * m, m * -0.33333334f, m) : (1.0f - q) * r;
}

template <bool kLinear>
__device__ __forceinline__ float2 situ_grad(float g, float u, float dy, const SituParams& c) {
  constexpr float kLog2e = 1.4426950408889634f;
  const float z = fabsf(g) * c.inv_beta;
  const float q = ex2_fast(z * (-2.0f * kLog2e)), p = ex2_fast(fabsf(g) * -kLog2e);
  const float q1 = 1.0f + q, p1 = 1.0f + p;
  float rq, rp, b = u, db = 1.0f;
  if constexpr (kLinear) {
    const float v = fabsf(u) * c.inv_lbeta;
    const float k = ex2_fast(v * (-2.0f * kLog2e)), k1 = 1.0f + k;
    const float qp = q1 * p1;
    const float r = rcp_fast(qp * k1);
    const float rk = r * qp, rqp = r * k1;
    rq = rqp * p1;
    rp = rqp * q1;
    b = copysignf(c.lbeta * tanh_of(v, k, rk), u);
    db = 4.0f * k * rk * rk;
  } else {
    const float r = rcp_fast(q1 * p1);
    rq = r * p1;
    rp = r * q1;
  }
  const float t = tanh_of(z, q, rq);                       // |tanh z|
  const float s = g < 0.0f ? p * rp : rp;                  // sigmoid
  const float sb = c.beta * t;
  // beta tanh(z) s (1 - s), of g's sign, and sech^2(z) s
  const float da = fmaf(4.0f * q * rq * rq, s, copysignf(sb * p * rp * rp, g));
  return make_float2(dy * b * da, dy * copysignf(sb * s, g) * db);
}

// Eight elements a step: 48 bytes read, 32 written.  Bound by memory.
template <bool kLinear>
__global__ void __launch_bounds__(kThreads)
situ_backward_kernel(const uint16_t* __restrict__ in, const uint16_t* __restrict__ dy,
                     uint16_t* __restrict__ dx, long long total, int vpr, SituParams p) {
  pdl_trigger();
  pdl_wait();
  const long long j = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (j >= total) return;
  const long long row = j / vpr;
  const int c = (int)(j - row * vpr);
  const long long at = (row * 2 * vpr + c) * 8;
  const uint4 g = ld_stream(reinterpret_cast<const uint4*>(in + at));
  const uint4 u = ld_stream(reinterpret_cast<const uint4*>(in + at + 8ll * vpr));
  const uint4 d = ld_stream(reinterpret_cast<const uint4*>(dy + j * 8));
  const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w}, dw[4] = {d.x, d.y, d.z, d.w};
  uint32_t og[4], ou[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 lo = situ_grad<kLinear>(bf16_lo(gw[i]), bf16_lo(uw[i]), bf16_lo(dw[i]), p);
    const float2 hi = situ_grad<kLinear>(bf16_hi(gw[i]), bf16_hi(uw[i]), bf16_hi(dw[i]), p);
    og[i] = pack_bf16x2(lo.x, hi.x);
    ou[i] = pack_bf16x2(lo.y, hi.y);
  }
  *reinterpret_cast<uint4*>(dx + at) = make_uint4(og[0], og[1], og[2], og[3]);
  *reinterpret_cast<uint4*>(dx + at + 8ll * vpr) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
}

}  // namespace

cudaError_t launch_situ(const uint16_t* in, uint16_t* out, long long N, int d, float beta,
                        float lbeta, cudaStream_t s) {
  if (N <= 0) return cudaSuccess;
  // at least two blocks per SM when there are enough rows
  const long long spread = (N + 2LL * num_sms() - 1) / (2LL * num_sms());
  const int rpb = (int)(spread < rows_for(d) ? (spread < 1 ? 1 : spread) : rows_for(d));
  const long long blocks = (N + rpb - 1) / rpb;
  return launch_k(situ_dense_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, s, in, out, N, d,
                  rpb, make_situ_params(beta, lbeta));
}

cudaError_t launch_masked_situ(const uint16_t* in, uint16_t* out, const int32_t* counts, int E,
                               int T_max, int d, float beta, float lbeta, cudaStream_t s) {
  if (E <= 0 || T_max <= 0) return cudaSuccess;
  const int rpb = min(rows_for(d), T_max);
  dim3 grid((unsigned)ceil_div(T_max, rpb), (unsigned)E);
  return launch_k(situ_masked_kernel, grid, dim3(kThreads), 0, s, in, out, counts, T_max, d, rpb,
                  make_situ_params(beta, lbeta));
}

cudaError_t launch_situ_backward(const uint16_t* in, const uint16_t* dy, uint16_t* dx, long long N,
                                 int d, float beta, float lbeta, cudaStream_t s) {
  if (N <= 0) return cudaSuccess;
  const SituParams p = make_situ_params(beta, lbeta);
  const long long total = N * (d / 8);
  const dim3 grid((unsigned)((total + kThreads - 1) / kThreads)), block(kThreads);
  return p.has_lbeta
             ? launch_k(situ_backward_kernel<true>, grid, block, 0, s, in, dy, dx, total, d / 8, p)
             : launch_k(situ_backward_kernel<false>, grid, block, 0, s, in, dy, dx, total, d / 8, p);
}

}  // namespace lmoe
