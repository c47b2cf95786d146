// Residual addition and RMSNorm in one pass, with a bf16 and an e4m3 output, and
// the gradient of both.
//
//   h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  y = h r w        (fp32)
//   out = bf16(y);  codes, scales: the rule of fp8_quant.cuh on y, a row and 128 columns a block
// Gradient, with g = grad_out w and n = h r:
//   grad_h = grad_residual + r (g - n mean(g n)),   grad_w = sum over rows of grad_out n
//
// Both are bound by memory: a row is read once, stays in registers between its sum of squares
// and its outputs, and is written once.  h is not rounded before it is normalised.
#include <float.h>

#include "fp8_quant.cuh"
#include "norm.cuh"

namespace lmoe {
namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;

__device__ __forceinline__ uint4 ld_stream(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ void widen(const uint4& v, float (&f)[8]) {
  f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
  f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}

__device__ __forceinline__ uint4 narrow(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

constexpr uint4 kOnes = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};   // bf16 1.0

// Sums over a row of two values at a time: a warp's rows by shuffles alone, a block's through
// one slot a warp (the caller alternates two slots, so that one barrier a sum is enough).
template <bool kWarpRow>
__device__ __forceinline__ float2 row_sum(float2 v, float2* slots) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    v.x += __shfl_xor_sync(kAll, v.x, o);
    v.y += __shfl_xor_sync(kAll, v.y, o);
  }
  if (kWarpRow) return v;
  const int lane = threadIdx.x & 31, warps = (int)blockDim.x >> 5;
  if (lane == 0) slots[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? slots[lane] : make_float2(0.0f, 0.0f);
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    v.x += __shfl_xor_sync(kAll, v.x, o);
    v.y += __shfl_xor_sync(kAll, v.y, o);
  }
  return v;
}

// Where the squares of a row leave the range of fp32, the row is scaled by a power of two first:
// its sum of squares overflows (down by 2^80), or it is so small that squares are lost and eps
// does not hide them (up by 2^80).  NaN and infinite rows take the branch, too, and stay so.
__device__ __forceinline__ float range_scale(float sum, float H, float eps) {
  if (!(sum <= FLT_MAX)) return 8.271806125530277e-25f;                       // 2^-80
  if (sum < H * 8.077935669463161e-28f && eps < 8.077935669463161e-28f)      // 2^-90
    return 1.2089258196146292e24f;                                            // 2^80
  return 1.0f;
}

// kVec: 16-byte vectors a thread, vector i at column 8 (i threads + thread).  kWarpRow: a warp a
// row, blockDim.x / 32 rows a CTA; else a CTA a row.
template <int kVec, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 256 : kVec == 4 ? 512 : 1024)
norm_kernel(const NormForward p) {
  __shared__ float2 slots[2][32];
  pdl_trigger();
  const int nt = kWarpRow ? 32 : (int)blockDim.x;
  const int t = kWarpRow ? (int)threadIdx.x & 31 : (int)threadIdx.x;
  const long long row = kWarpRow ? (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)
                                 : (long long)blockIdx.x;
  pdl_wait();
  if (row >= p.T) return;                        // (a warp, or none of a CTA)
  const int nvec = p.H >> 3;
  const long long base = row * p.H;
  uint4 a[kVec], b[kVec], wv[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int j = i * nt + t;
    a[i] = b[i] = wv[i] = make_uint4(0, 0, 0, 0);
    if (j < nvec) {
      a[i] = ld_stream(p.x + base + 8 * j);
      if (p.residual) b[i] = ld_stream(p.residual + base + 8 * j);
      wv[i] = p.w ? *reinterpret_cast<const uint4*>(p.w + 8 * j) : kOnes;
    }
  }
  float h[kVec][8];
  float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    float r[8];
    widen(a[i], h[i]);
    widen(b[i], r);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (p.residual) h[i][e] += r[e];           // (not -0 + 0)
      sum.x = fmaf(h[i][e], h[i][e], sum.x);
    }
    const int j = i * nt + t;
    if (p.h && j < nvec) *reinterpret_cast<uint4*>(p.h + base + 8 * j) = narrow(h[i]);
  }
  sum = row_sum<kWarpRow>(sum, slots[0]);
  const float H = (float)p.H;
  float eps = p.eps;
  const float s = range_scale(sum.x, H, eps);    // (one for the row)
  if (s != 1.0f) {
    sum = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kVec; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[i][e] *= s;
        sum.x = fmaf(h[i][e], h[i][e], sum.x);
      }
    sum = row_sum<kWarpRow>(sum, slots[1]);
    eps = eps * s * s;
  }
  const float r = 1.0f / sqrtf(sum.x / H + eps);
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int j = i * nt + t;
    float w[8];
    widen(wv[i], w);
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[i][e] = h[i][e] * r * w[e];
      m = max(m, abs_bits(h[i][e]));
    }
    if (p.out && j < nvec) *reinterpret_cast<uint4*>(p.out + base + 8 * j) = narrow(h[i]);
    if (p.codes) {
      if (j >= nvec) m = 0;
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) m = max(m, __shfl_xor_sync(kAll, m, o));
      const BlockScale bs = block_scale(m);
      if (j < nvec) {
        uint2 c;
        c.x = pack_e4m3x4(h[i][0] * bs.inv, h[i][1] * bs.inv, h[i][2] * bs.inv, h[i][3] * bs.inv);
        c.y = pack_e4m3x4(h[i][4] * bs.inv, h[i][5] * bs.inv, h[i][6] * bs.inv, h[i][7] * bs.inv);
        *reinterpret_cast<uint2*>(p.codes + base + 8 * j) = c;
        if ((j & 15) == 0) p.scales[row * ((p.H + 127) >> 7) + (j >> 4)] = bs.scale;
      }
    }
  }
}

// The gradient.  CTAs walk the rows; a thread keeps its columns' part of grad_w in registers and
// leaves it in the workspace, one row of it a CTA (kWarpRow: a warp), summed in order by the
// second kernel.
template <int kVec, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 256 : 512)
norm_backward_kernel(const NormBackward p) {
  __shared__ float2 slots[4][32];
  pdl_trigger();
  const int nt = kWarpRow ? 32 : (int)blockDim.x;
  const int t = kWarpRow ? (int)threadIdx.x & 31 : (int)threadIdx.x;
  const int per = kWarpRow ? (int)blockDim.x >> 5 : 1;
  const int walker = kWarpRow ? (int)blockIdx.x * per + (int)(threadIdx.x >> 5) : (int)blockIdx.x;
  const int walkers = (int)gridDim.x * per;
  const int nvec = p.H >> 3;
  pdl_wait();
  float acc[kVec][8];
  uint4 wv[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int j = i * nt + t;
    wv[i] = make_uint4(0, 0, 0, 0);
    if (j < nvec) wv[i] = p.w ? *reinterpret_cast<const uint4*>(p.w + 8 * j) : kOnes;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[i][e] = 0.0f;
  }
  const float H = (float)p.H;
  int flip = 0;
  for (long long row = walker; row < p.T; row += walkers, flip ^= 1) {
    const long long base = row * p.H;
    uint4 dv[kVec], hv[kVec], rv[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int j = i * nt + t;
      dv[i] = hv[i] = rv[i] = make_uint4(0, 0, 0, 0);
      if (j < nvec) {
        hv[i] = ld_stream(p.h + base + 8 * j);
        dv[i] = ld_stream(p.dy + base + 8 * j);
        if (p.dres) rv[i] = ld_stream(p.dres + base + 8 * j);
      }
    }
    float2 sum = make_float2(0.0f, 0.0f);        // of h^2 and of g h
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      float h[8], d[8], w[8];
      widen(hv[i], h);
      widen(dv[i], d);
      widen(wv[i], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum.x = fmaf(h[e], h[e], sum.x);
        sum.y = fmaf(d[e] * w[e], h[e], sum.y);
      }
    }
    sum = row_sum<kWarpRow>(sum, slots[flip]);
    float eps = p.eps;
    const float s = range_scale(sum.x, H, eps);
    if (s != 1.0f) {
      sum = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        float h[8], d[8], w[8];
        widen(hv[i], h);
        widen(dv[i], d);
        widen(wv[i], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float v = h[e] * s;
          sum.x = fmaf(v, v, sum.x);
          sum.y = fmaf(d[e] * w[e], v, sum.y);
        }
      }
      sum = row_sum<kWarpRow>(sum, slots[2 + flip]);
      eps = eps * s * s;
    }
    const float r = 1.0f / sqrtf(sum.x / H + eps);
    const float k = sum.y * r / H, sr = s * r;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int j = i * nt + t;
      float h[8], d[8], w[8], q[8];
      widen(hv[i], h);
      widen(dv[i], d);
      widen(wv[i], w);
      widen(rv[i], q);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = h[e] * s * r;
        acc[i][e] = fmaf(d[e], n, acc[i][e]);
        q[e] = fmaf(sr, fmaf(-n, k, d[e] * w[e]), q[e]);
      }
      if (j < nvec) *reinterpret_cast<uint4*>(p.dh + base + 8 * j) = narrow(q);
    }
  }
  if (!p.dw) return;
  float* part = p.partial + (long long)walker * p.H;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int j = i * nt + t;
    if (j < nvec) {
      *reinterpret_cast<float4*>(part + 8 * j) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
      *reinterpret_cast<float4*>(part + 8 * j + 4) = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
    }
  }
}

// grad_w: 32 columns a CTA, each of its warps a run of the partial rows, then the warps' sums in order.
constexpr int kJoinWarps = 16;
__global__ void __launch_bounds__(kJoinWarps * 32)
norm_join_kernel(const float* __restrict__ partial, int parts, int H, float* __restrict__ dw) {
  __shared__ float sums[kJoinWarps][32];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = blockIdx.x * 32 + lane;
  const int each = (parts + kJoinWarps - 1) / kJoinWarps;
  const int p0 = warp * each, p1 = min(p0 + each, parts);
  float v = 0.0f;
  if (col < H) {
#pragma unroll 8
    for (int p = p0; p < p1; ++p) v += partial[(long long)p * H + col];
  }
  sums[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && col < H) {
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < kJoinWarps; ++i) v += sums[i][lane];
    dw[col] = v;
  }
}

int round32(int n) { return (n + 31) / 32 * 32; }

constexpr int kRowWarps = 8;                     // rows of a CTA with a warp a row
constexpr int kWarpRowVec = 4;                   // vectors a lane up to which a warp takes a row

// CTAs of the backward kernel (kWarpRow: kRowWarps walkers each)
int backward_blocks(int T, int H) {
  const bool warp_row = H <= 8 * 32 * kWarpRowVec;
  const long long rows = warp_row ? ceil_div(T, kRowWarps) : T;
  const long long most = 4ll * num_sms();
  return (int)(rows < most ? rows : most);
}

}  // namespace

size_t norm_backward_workspace_bytes(int T, int H) {
  const int per = H <= 8 * 32 * kWarpRowVec ? kRowWarps : 1;
  const size_t n = (size_t)backward_blocks(T, H) * per * H * sizeof(float);
  return (n + 255) & ~size_t(255);
}

cudaError_t launch_norm(const NormForward& n, cudaStream_t s) {
  const int nvec = n.H / 8;
  if (nvec <= 32 * kWarpRowVec) {
    const dim3 grid((unsigned)ceil_div(n.T, kRowWarps)), block(32 * kRowWarps);
    if (nvec <= 32) return launch_k(norm_kernel<1, true>, grid, block, 0, s, n);
    if (nvec <= 64) return launch_k(norm_kernel<2, true>, grid, block, 0, s, n);
    return launch_k(norm_kernel<4, true>, grid, block, 0, s, n);
  }
  const dim3 grid((unsigned)n.T);
  if (n.T <= 2 * num_sms())
    return nvec <= 1024 ? launch_k(norm_kernel<1, false>, grid, dim3(round32(nvec)), 0, s, n)
                        : launch_k(norm_kernel<2, false>, grid, dim3(round32((nvec + 1) / 2)), 0, s, n);
  return launch_k(norm_kernel<4, false>, grid, dim3(round32((nvec + 3) / 4)), 0, s, n);
}

cudaError_t launch_norm_backward(const NormBackward& n, cudaStream_t s) {
  const int nvec = n.H / 8, blocks = backward_blocks(n.T, n.H);
  int parts = blocks;
  cudaError_t e;
  if (nvec <= 32 * kWarpRowVec) {
    const dim3 block(32 * kRowWarps);
    parts *= kRowWarps;
    if (nvec <= 32) e = launch_k(norm_backward_kernel<1, true>, dim3(blocks), block, 0, s, n);
    else if (nvec <= 64) e = launch_k(norm_backward_kernel<2, true>, dim3(blocks), block, 0, s, n);
    else e = launch_k(norm_backward_kernel<4, true>, dim3(blocks), block, 0, s, n);
  } else if (nvec <= 512) {
    e = launch_k(norm_backward_kernel<1, false>, dim3(blocks), dim3(round32(nvec)), 0, s, n);
  } else if (nvec <= 1024) {
    e = launch_k(norm_backward_kernel<2, false>, dim3(blocks), dim3(round32((nvec + 1) / 2)), 0, s, n);
  } else {
    e = launch_k(norm_backward_kernel<4, false>, dim3(blocks), dim3(round32((nvec + 3) / 4)), 0, s, n);
  }
  if (e != cudaSuccess || !n.dw) return e;
  return launch_k(norm_join_kernel, dim3(ceil_div(n.H, 32)), dim3(kJoinWarps * 32), 0, s,
                  (const float*)n.partial, parts, n.H, n.dw);
}

}  // namespace lmoe
