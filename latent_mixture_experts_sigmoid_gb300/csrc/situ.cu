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

// the same of memory that the kernel may write
__device__ __forceinline__ uint4 ld_in_place(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
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
//   A = beta tanh(z),  b = linear_beta tanh(v)  (or u):   out = A s b,
//   grad_gate = dy s b [ sech^2(z) + A (1 - s) ],
//   grad_up   = dy s A sech^2(v)  (or dy s A).
// Besides the two hardware tanh (as the forward's) all of it comes from three exponentials of
// non-positive arguments and one reciprocal:
//   q = e^{-2|z|}:  sech^2 z = 4 q / (1 + q)^2;   k = e^{-2|v|}: as q
//   p = e^{-|g|}:   s and 1 - s are 1 / (1 + p) and p / (1 + p), the other way round for g < 0
// and 1 / ((1 + q)(1 + p)(1 + k)), whose divisor lies in [1, 8].  sech^2 = 1 - tanh^2 and
// 1 - s would cancel where the activation saturates; these keep their relative accuracy.
// ---------------------------------------------------------------------------
struct SituGradParams {
  float beta, inv_beta, lbeta, inv_lbeta;
  float ez, ev;                // -2 log2(e) / beta, / linear_beta: 2^(ez |g|) = q
};

struct GradPair {
  f32x2 gate, up;
};
// two elements: gate, up and grad_out as bf16 pairs
template <bool kLinear>
__device__ __forceinline__ GradPair situ_grad2(uint32_t g2, uint32_t u2, uint32_t dy2,
                                               const SituGradParams& c) {
  auto wide = [](uint32_t w) { return f2_make(w << 16, w & 0xFFFF0000u); };
  const f32x2 one = f2_splat(1.0f);
  const f32x2 g = wide(g2), ag = wide(g2 & 0x7FFF7FFFu), dy = wide(dy2);
  const f32x2 q = LMOE_F2_APPLY(ex2_fast, f2_mul(ag, f2_splat(c.ez)));
  const f32x2 p = LMOE_F2_APPLY(ex2_fast, f2_mul(ag, f2_splat(-1.4426950408889634f)));
  const f32x2 q1 = f2_add(q, one), p1 = f2_add(p, one), qp = f2_mul(q1, p1);
  f32x2 b = wide(u2), db = one, rqp;
  if constexpr (kLinear) {
    const f32x2 k = LMOE_F2_APPLY(ex2_fast, f2_mul(wide(u2 & 0x7FFF7FFFu), f2_splat(c.ev)));
    const f32x2 k1 = f2_add(k, one);
    const f32x2 r = LMOE_F2_APPLY(rcp_fast, f2_mul(qp, k1));
    const f32x2 rk = f2_mul(r, qp), twice = f2_add(rk, rk);
    rqp = f2_mul(r, k1);
    db = f2_mul(f2_mul(twice, twice), k);
    b = f2_mul(LMOE_F2_APPLY(tanh_fast, f2_mul(b, f2_splat(c.inv_lbeta))), f2_splat(c.lbeta));
  } else {
    rqp = LMOE_F2_APPLY(rcp_fast, qp);
  }
  const f32x2 rq = f2_mul(rqp, p1), rp = f2_mul(rqp, q1), pr = f2_mul(p, rp);
  const f32x2 twice = f2_add(rq, rq);
  const f32x2 sech2 = f2_mul(f2_mul(twice, twice), q);
  const bool lo = f2_lo(g) < 0.0f, hi = f2_hi(g) < 0.0f;
  const f32x2 s = f2_make(__float_as_uint(lo ? f2_lo(pr) : f2_lo(rp)), __float_as_uint(hi ? f2_hi(pr) : f2_hi(rp)));
  const f32x2 t = f2_make(__float_as_uint(lo ? f2_lo(rp) : f2_lo(pr)), __float_as_uint(hi ? f2_hi(rp) : f2_hi(pr)));
  const f32x2 A = f2_mul(LMOE_F2_APPLY(tanh_fast, f2_mul(g, f2_splat(c.inv_beta))), f2_splat(c.beta));
  const f32x2 ds = f2_mul(dy, s);
  GradPair o;
  // (the small factors first: grad_out times up, which may be unbounded, leaves fp32 where the result does not)
  o.gate = f2_mul(f2_mul(ds, f2_fma(A, t, sech2)), b);
  o.up = kLinear ? f2_mul(f2_mul(ds, db), A) : f2_mul(ds, A);
  return o;
}

// Eight elements a thread: 48 bytes read, 32 written; a CTA blockDim.y rows (blockIdx.x) of
// 8 blockDim.x columns (blockIdx.y).  dx may be in: a thread writes what it alone has read.
// Memory bound: [65536, 2 x 512] 53 us (336 MB, 6.3 TB/s; each factor by its own exponential, one
// element at a time, took 73: bound by issue).
template <bool kLinear>
__global__ void __launch_bounds__(kThreads)
situ_backward_kernel(const uint16_t* in, const uint16_t* __restrict__ dy, uint16_t* dx, long long N, int d,
                     SituGradParams p) {
  pdl_trigger();
  const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  const int c = (int)(blockIdx.y * blockDim.x + threadIdx.x) * 8;
  pdl_wait();
  if (row >= N || c >= d) return;
  const long long at = row * 2 * d + c;
  // (up, used last, is asked for first: without linear_beta 50.7 us, the other way round 54.5)
  const uint4 u = ld_in_place(reinterpret_cast<const uint4*>(in + at + d));
  const uint4 g = ld_in_place(reinterpret_cast<const uint4*>(in + at));
  const uint4 y = ld_stream(reinterpret_cast<const uint4*>(dy + row * d + c));
  const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w}, yw[4] = {y.x, y.y, y.z, y.w};
  uint32_t og[4], ou[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const GradPair o = situ_grad2<kLinear>(gw[i], uw[i], yw[i], p);
    og[i] = pack_bf16x2(f2_lo(o.gate), f2_hi(o.gate));
    ou[i] = pack_bf16x2(f2_lo(o.up), f2_hi(o.up));
  }
  *reinterpret_cast<uint4*>(dx + at) = make_uint4(og[0], og[1], og[2], og[3]);
  *reinterpret_cast<uint4*>(dx + at + d) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
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
  const SituParams f = make_situ_params(beta, lbeta);
  const float twice = -2.0f * 1.4426950408889634f;
  const SituGradParams p{f.beta, f.inv_beta, f.lbeta, f.inv_lbeta, twice * f.inv_beta, twice * f.inv_lbeta};
  const int vpr = d / 8, cols = ceil_div(vpr, kThreads), tx = ceil_div(vpr, cols);
  const dim3 block(tx, kThreads / tx), grid((unsigned)((N + block.y - 1) / block.y), cols);
  return f.has_lbeta ? launch_k(situ_backward_kernel<true>, grid, block, 0, s, in, dy, dx, N, d, p)
                     : launch_k(situ_backward_kernel<false>, grid, block, 0, s, in, dy, dx, N, d, p);
}

}  // namespace lmoe
