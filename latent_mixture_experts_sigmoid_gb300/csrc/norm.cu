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

#include <atomic>

#include "fp8_quant.cuh"
#include "norm.cuh"
#include "tc_ptx.cuh"

namespace lmoe {
namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;

__device__ __forceinline__ uint4 ld_stream(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// a load that is not moved ahead of what is written before it
__device__ __forceinline__ uint4 ld_here(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

// eight bf16 as four packed pairs of fp32, and back
__device__ __forceinline__ void widen(const uint4& v, f32x2 (&f)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = f2_make(w[i] << 16, w[i] & 0xFFFF0000u);
}
__device__ __forceinline__ uint4 narrow(const f32x2 (&f)[4]) {
  return make_uint4(pack_bf16x2(f2_lo(f[0]), f2_hi(f[0])), pack_bf16x2(f2_lo(f[1]), f2_hi(f[1])),
                    pack_bf16x2(f2_lo(f[2]), f2_hi(f[2])), pack_bf16x2(f2_lo(f[3]), f2_hi(f[3])));
}
// the larger magnitude, NaN if one is
__device__ __forceinline__ float max_abs(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(fabsf(a)), "f"(fabsf(b)));
  return m;
}

constexpr uint4 kOnes = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};   // bf16 1.0

// Sums over a row of kN values at a time: those of a row of kLanes lanes by shuffles alone, of a
// CTA's row (kLanes = 0) through one slot a warp (the caller alternates two slots, so that one
// barrier a sum is enough).
template <int kLanes, int kN>
__device__ __forceinline__ void row_sum(float (&v)[kN], float (*slots)[2]) {
#pragma unroll
  for (int o = (kLanes ? kLanes : 32) / 2; o; o >>= 1)
#pragma unroll
    for (int n = 0; n < kN; ++n) v[n] += __shfl_xor_sync(kAll, v[n], o);
  if constexpr (kLanes == 0) {
    const int lane = threadIdx.x & 31, warps = (int)blockDim.x >> 5;
    if (lane == 0)
#pragma unroll
      for (int n = 0; n < kN; ++n) slots[threadIdx.x >> 5][n] = v[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < kN; ++n) v[n] = lane < warps ? slots[lane][n] : 0.0f;
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
      for (int n = 0; n < kN; ++n) v[n] += __shfl_xor_sync(kAll, v[n], o);
  }
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

constexpr int kMaxRing = 16;                     // rows of the gradient's ring

// A bounded wait, about two seconds.
__device__ __forceinline__ bool wait_row(uint32_t bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  for (int n = 0; n < (1 << 21); ++n)
    if (mbar_try_wait_ns(bar, parity, 1000u)) return true;
  return false;
}

// kVec: 16-byte vectors a thread, vector i at column 8 (i threads + thread).  kLanes: lanes a row,
// blockDim.x / kLanes rows a CTA; 0: a CTA a row.
// A row's loads are one burst, so that CTAs in number hide its latencies; packed fp32 throughout (one
// by one, at 29 instructions an element, the kernel was bound by their issue).
// [4096, 7168] with residual and both outputs: 41 us (265 MB, 6.4 TB/s), codes alone without a residual
// 23 us (their floor is 13: 64 registers a thread leave room for four rows an SM, and without a residual each
// has half the bytes on their way); [1, 7168]: 2.2 us.  Rows walked by few CTAs through a ring of copies as
// in the gradient: 49 us.
template <int kVec, int kLanes, bool kRes>
__global__ void __launch_bounds__(kLanes ? 256 : kVec == 4 ? 512 : 1024, kLanes == 0 && kVec == 4 ? 2 : 1)
norm_kernel(const NormForward p) {
  __shared__ float slots[2][32][2];
  pdl_trigger();
  const int nt = kLanes ? kLanes : (int)blockDim.x;
  const int t = kLanes ? (int)threadIdx.x % nt : (int)threadIdx.x;
  const long long row = kLanes ? (long long)blockIdx.x * (blockDim.x / nt) + threadIdx.x / nt
                               : (long long)blockIdx.x;
  // (lanes of a row that is not there stay for the shuffles)
  const int nvec = row < p.T ? p.H >> 3 : 0;
  const long long base = row * p.H + 8 * t;
  pdl_wait();
  uint4 a[kVec], b[kVec], wv[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    a[i] = b[i] = make_uint4(0, 0, 0, 0);
    if (i * nt + t < nvec) {
      a[i] = ld_stream(p.x + base + 8 * i * nt);
      if (kRes) b[i] = ld_stream(p.residual + base + 8 * i * nt);
    }
  }
  auto load_weights = [&] {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      wv[i] = i * nt + t >= nvec ? make_uint4(0, 0, 0, 0) : p.w ? ld_here(p.w + 8 * (i * nt + t)) : kOnes;
  };
  if (kLanes) load_weights();
  f32x2 h[kVec][4], squares = 0ull;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    widen(a[i], h[i]);
    f32x2 r[4];
    widen(b[i], r);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (kRes) h[i][e] = f2_add(h[i][e], r[e]);
      squares = f2_fma(h[i][e], h[i][e], squares);
    }
    if (p.h && i * nt + t < nvec) *reinterpret_cast<uint4*>(p.h + base + 8 * i * nt) = narrow(h[i]);
  }
  // (asked for here: the registers of x and the residual are free again)
  if (!kLanes) load_weights();
  float sum[1] = {f2_lo(squares) + f2_hi(squares)};
  row_sum<kLanes, 1>(sum, slots[0]);
  const float H = (float)p.H, inv_H = 1.0f / H;
  float eps = p.eps;
  const float s = range_scale(sum[0], H, eps);   // (one for the row)
  const bool scaled = s != 1.0f;
  if (kLanes == 32 || kLanes == 0 ? scaled : __any_sync(kAll, scaled)) {
    squares = 0ull;
#pragma unroll
    for (int i = 0; i < kVec; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[i][e] = f2_mul(h[i][e], f2_splat(s));
        squares = f2_fma(h[i][e], h[i][e], squares);
      }
    sum[0] = f2_lo(squares) + f2_hi(squares);
    row_sum<kLanes, 1>(sum, slots[1]);
    eps = eps * s * s;
  }
  const f32x2 r = f2_splat(rsqrtf(fmaf(sum[0], inv_H, eps)));
  float m[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    f32x2 w[4];
    widen(wv[i], w);
    m[i] = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      h[i][e] = f2_mul(f2_mul(h[i][e], r), w[e]);
      m[i] = max_abs(m[i], max_abs(f2_lo(h[i][e]), f2_hi(h[i][e])));
    }
    if (i * nt + t >= nvec) m[i] = 0.0f;
    if (p.out && i * nt + t < nvec) *reinterpret_cast<uint4*>(p.out + base + 8 * i * nt) = narrow(h[i]);
  }
  if (!p.codes) return;
  // sixteen lanes (or the row's) hold the blocks that their vectors belong to; lane i of them takes
  // the divisions of block i for all
  constexpr int kGroup = kLanes && kLanes < 16 ? kLanes : 16;
  float mine = 0.0f;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
#pragma unroll
    for (int o = 1; o < kGroup; o <<= 1) m[i] = max_abs(m[i], __shfl_xor_sync(kAll, m[i], o));
    if (i == 0 || t % kGroup == i) mine = m[i];
  }
  const BlockScale bs = block_scale(__float_as_uint(mine));
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const f32x2 inv = f2_splat(__shfl_sync(kAll, bs.inv, (threadIdx.x & 31 & ~(kGroup - 1)) + i));
    f32x2 c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = f2_mul(h[i][e], inv);
    if (i * nt + t < nvec)
      *reinterpret_cast<uint2*>(p.codes + base + 8 * i * nt) =
          make_uint2(pack_e4m3x4(f2_lo(c[0]), f2_hi(c[0]), f2_lo(c[1]), f2_hi(c[1])),
                     pack_e4m3x4(f2_lo(c[2]), f2_hi(c[2]), f2_lo(c[3]), f2_hi(c[3])));
  }
  // lane i: the scale of its group's block in vector i
  const int i = t % kGroup, j = i * nt + (t - i);
  if (i < kVec && j < nvec) p.scales[row * ((p.H + 127) >> 7) + (j >> 4)] = bs.scale;
}

// The gradient.  CTAs (of short rows: groups of lanes) take every so-manieth row; a thread keeps its
// columns' part of grad_w in registers, each CTA leaves a row of it in the workspace, and the join
// sums those in order.

// a thread's sums of h^2 and of g h, h scaled by s
template <int kVec>
__device__ __forceinline__ void sums_of(float (&sum)[2], const uint4 (&hv)[kVec], const uint4 (&dv)[kVec],
                                        const uint4 (&wv)[kVec], float s) {
  f32x2 hh = 0ull, gh = 0ull;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    f32x2 h[4], d[4], w[4];
    widen(hv[i], h);
    widen(dv[i], d);
    widen(wv[i], w);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (s != 1.0f) h[e] = f2_mul(h[e], f2_splat(s));
      hh = f2_fma(h[e], h[e], hh);
      gh = f2_fma(f2_mul(d[e], w[e]), h[e], gh);
    }
  }
  sum[0] = f2_lo(hh) + f2_hi(hh);
  sum[1] = f2_lo(gh) + f2_hi(gh);
}

// n = (h s) r; grad_h = grad_residual + s (r (g - n k)), k = mean(g n).  (Never s r, which may leave the
// range where the squares did: of rows below 2^-128 it is infinite, and 0 times it NaN.  The multiplication
// more shows in no time.)
struct RowFactors {
  float s, r, k;
};
template <int kVec, int kLanes>
__device__ __forceinline__ RowFactors factors_of(const uint4 (&hv)[kVec], const uint4 (&dv)[kVec],
                                                 const uint4 (&wv)[kVec], float H, float inv_H,
                                                 float eps, float (*slots)[2], float (*more_slots)[2]) {
  float sum[2];
  sums_of<kVec>(sum, hv, dv, wv, 1.0f);
  row_sum<kLanes, 2>(sum, slots);
  const float s = range_scale(sum[0], H, eps);   // (one for the row)
  const bool scaled = s != 1.0f;
  if (kLanes == 32 || kLanes == 0 ? scaled : __any_sync(kAll, scaled)) {
    sums_of<kVec>(sum, hv, dv, wv, s);
    row_sum<kLanes, 2>(sum, more_slots);
    eps = eps * s * s;
  }
  const float r = rsqrtf(fmaf(sum[0], inv_H, eps));
  return {s, r, sum[1] * inv_H * r};
}

__device__ __forceinline__ uint4 grad_of(const uint4& hv, const uint4& dv, const uint4& wv, const uint4& rv,
                                         const RowFactors& f, f32x2 (&acc)[4]) {
  f32x2 h[4], d[4], w[4], q[4];
  widen(hv, h);
  widen(dv, d);
  widen(wv, w);
  widen(rv, q);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (f.s != 1.0f) h[e] = f2_mul(h[e], f2_splat(f.s));
    const f32x2 n = f2_mul(h[e], f2_splat(f.r));
    acc[e] = f2_fma(d[e], n, acc[e]);
    f32x2 v = f2_fma(n, f2_splat(-f.k), f2_mul(d[e], w[e]));
    v = f2_mul(v, f2_splat(f.r));
    q[e] = f2_fma(f2_splat(f.s), v, q[e]);
  }
  return narrow(q);
}

// Short rows: kLanes lanes a row.
template <int kVec, int kLanes>
__global__ void __launch_bounds__(256)
norm_backward_short_kernel(const NormBackward p) {
  pdl_trigger();
  const int t = (int)threadIdx.x % kLanes, per = (int)blockDim.x / kLanes, nvec = p.H >> 3;
  const int walker = (int)blockIdx.x * per + (int)threadIdx.x / kLanes, walkers = (int)gridDim.x * per;
  const int first = (int)blockIdx.x * per + (int)(threadIdx.x & ~31u) / kLanes;   // the warp's first walker
  pdl_wait();
  const float inv_H = 1.0f / (float)p.H;
  f32x2 acc[kVec][4] = {};
  uint4 wv[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int j = i * kLanes + t;
    wv[i] = j >= nvec ? make_uint4(0, 0, 0, 0) : p.w ? *reinterpret_cast<const uint4*>(p.w + 8 * j) : kOnes;
  }
  for (long long r0 = first; r0 < p.T; r0 += walkers) {
    const long long row = r0 + (walker - first), base = row * p.H;
    const bool there = row < p.T;                // (the lanes of other rows of the warp go on)
    uint4 dv[kVec], hv[kVec], rv[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int j = i * kLanes + t;
      dv[i] = hv[i] = rv[i] = make_uint4(0, 0, 0, 0);
      if (there && j < nvec) {
        hv[i] = ld_stream(p.h + base + 8 * j);
        dv[i] = ld_stream(p.dy + base + 8 * j);
        if (p.dres) rv[i] = ld_stream(p.dres + base + 8 * j);
      }
    }
    const RowFactors f = factors_of<kVec, kLanes>(hv, dv, wv, (float)p.H, inv_H, p.eps, nullptr, nullptr);
    if (!there) continue;                        // (with eps = 0 its zeros would be NaN)
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int j = i * kLanes + t;
      const uint4 o = grad_of(hv[i], dv[i], wv[i], rv[i], f, acc[i]);
      if (j < nvec) *reinterpret_cast<uint4*>(p.dh + base + 8 * j) = o;
    }
  }
  // the CTA's rows of sums as one, in order
  if (!p.dw) return;
  constexpr int kCols = kVec * kLanes * 8;
  __shared__ __align__(16) float sums[256 / kLanes][kCols];
#pragma unroll
  for (int i = 0; i < kVec; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *reinterpret_cast<f32x2*>(&sums[threadIdx.x / kLanes][(i * kLanes + t) * 8 + 2 * e]) = acc[i][e];
  __syncthreads();
  for (int c = threadIdx.x; c < p.H; c += 256) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < 256 / kLanes; ++w) v += sums[w][c];
    p.partial[(long long)blockIdx.x * p.H + c] = v;
  }
}

// Few rows: one launch.  A cluster of eight CTAs takes all of them, a warp a row; the warps' parts of
// grad_w are summed in shared memory, the CTAs' over the cluster, in order.
// On the GPU about as long as the two launches ([16, 1024] 3.3 us for 3.7, [64, 1024] 4.2 for 3.8, [128, 1024]
// 5.3 for 4.6), but a call, which the host bounds, takes one launch less: 2.7 us of 9.
constexpr int kFewWarps = 8, kFewCtas = 8;

__device__ __forceinline__ float ld_cluster(const float* p, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr(smem_u32(p), rank)) : "memory");
  return v;
}

template <int kVec>
__global__ void __launch_bounds__(kFewWarps * 32)
norm_backward_few_kernel(const NormBackward p) {
  extern __shared__ __align__(16) float sums[];  // [kFewWarps][H]
  pdl_trigger();
  const int warp = (int)threadIdx.x >> 5, t = (int)threadIdx.x & 31, nvec = p.H >> 3;
  const float inv_H = 1.0f / (float)p.H;
  pdl_wait();
  f32x2 acc[kVec][4] = {};
  for (int row = (int)blockIdx.x + warp * kFewCtas; row < p.T; row += kFewCtas * kFewWarps) {
    const long long base = (long long)row * p.H;
    uint4 dv[kVec], hv[kVec], rv[kVec], wv[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int j = i * 32 + t;
      dv[i] = hv[i] = rv[i] = wv[i] = make_uint4(0, 0, 0, 0);
      if (j < nvec) {
        hv[i] = ld_stream(p.h + base + 8 * j);
        dv[i] = ld_stream(p.dy + base + 8 * j);
        if (p.dres) rv[i] = ld_stream(p.dres + base + 8 * j);
        wv[i] = p.w ? *reinterpret_cast<const uint4*>(p.w + 8 * j) : kOnes;
      }
    }
    const RowFactors f = factors_of<kVec, 32>(hv, dv, wv, (float)p.H, inv_H, p.eps, nullptr, nullptr);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int j = i * 32 + t;
      const uint4 o = grad_of(hv[i], dv[i], wv[i], rv[i], f, acc[i]);
      if (j < nvec) *reinterpret_cast<uint4*>(p.dh + base + 8 * j) = o;
    }
  }
  if (!p.dw) return;
#pragma unroll
  for (int i = 0; i < kVec; ++i)
    if (i * 32 + t < nvec)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<f32x2*>(sums + warp * p.H + (i * 32 + t) * 8 + 2 * e) = acc[i][e];
  __syncthreads();
  for (int c = threadIdx.x; c < p.H; c += kFewWarps * 32) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) v += sums[w * p.H + c];
    sums[c] = v;                                 // (this thread's column alone)
  }
  cluster_sync();
  for (int c = (int)blockIdx.x * kFewWarps * 32 + (int)threadIdx.x; c < p.H; c += kFewCtas * kFewWarps * 32) {
    float v = 0.0f;
#pragma unroll
    for (int r = 0; r < kFewCtas; ++r) v += ld_cluster(sums + c, (uint32_t)r);
    p.dw[c] = v;
  }
  cluster_sync();                                // (the sums stay until all have read them)
}

// Long rows: a CTA a row.  Its next rows (of h, grad_out and grad_residual) are on their way into a
// ring in shared memory meanwhile, as bulk copies that one thread issues: their bytes in flight do
// not depend on how many warps the registers leave room for.  The barrier of a row's sums says that
// the slot of the row before has been read.
// [16384, 7168] with grad_residual: 147 us with the join (940 MB, 6.4 TB/s); one CTA an SM without the
// ring took 229.  [16384, 2048]: 66 us for 40 us of bytes, [8192, 16384] 243 for 158: a row's chain of
// latencies on the 512 threads an SM that the registers leave room for.
template <int kVec>
__global__ void __launch_bounds__(512)
norm_backward_kernel(const NormBackward p, int stages) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float slots[4][32][2];
  __shared__ uint64_t bars[kMaxRing];
  __shared__ int abort_flag;
  pdl_trigger();
  const int nt = (int)blockDim.x, t = (int)threadIdx.x, nvec = p.H >> 3;
  const uint32_t row_bytes = (uint32_t)p.H * 2, slot_bytes = row_bytes * (p.dres ? 3 : 2);
  if (t == 0) {
    for (int i = 0; i < stages; ++i) mbar_init(smem_u32(&bars[i]), 1);
    abort_flag = 0;
    fence_proxy_async_smem();
  }
  pdl_wait();
  __syncthreads();
  long long next = blockIdx.x;                   // the next row to copy (thread 0)
  auto copy = [&](int s) {
    const uint32_t bar = smem_u32(&bars[s]), at = smem_u32(ring) + (uint32_t)s * slot_bytes;
    mbar_arrive_expect_tx(bar, slot_bytes);
    bulk_load(at, p.h + next * p.H, row_bytes, bar);
    bulk_load(at + row_bytes, p.dy + next * p.H, row_bytes, bar);
    if (p.dres) bulk_load(at + 2 * row_bytes, p.dres + next * p.H, row_bytes, bar);
    next += gridDim.x;
  };
  if (t == 0)
    for (int s = 0; s < stages && next < p.T; ++s) copy(s);
  const float inv_H = 1.0f / (float)p.H;
  f32x2 acc[kVec][4] = {};
  uint4 wv[kVec];
  auto load_weights = [&] {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int j = i * nt + t;
      wv[i] = j >= nvec ? make_uint4(0, 0, 0, 0) : p.w ? *reinterpret_cast<const uint4*>(p.w + 8 * j) : kOnes;
    }
  };
  load_weights();
  int s = 0, flip = 0;
  uint32_t ph = 0;
  for (long long row = blockIdx.x; row < p.T; row += gridDim.x, flip ^= 1) {
    if (!wait_row(smem_u32(&bars[s]), ph)) {
      atomicCAS(p.err, 0, kErrNormRow);
      *(volatile int*)&abort_flag = 1;
    }
    const uint4* slot = reinterpret_cast<const uint4*>(ring + (size_t)s * slot_bytes);
    uint4 dv[kVec], hv[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int j = i * nt + t;
      dv[i] = hv[i] = make_uint4(0, 0, 0, 0);
      if (j < nvec) {
        hv[i] = slot[j];
        dv[i] = slot[nvec + j];
      }
    }
    if constexpr (kVec == 4) load_weights();     // (kept, 384 bytes a thread spill; as it is, 248)
    const RowFactors f = factors_of<kVec, 0>(hv, dv, wv, (float)p.H, inv_H, p.eps, slots[flip], slots[2 + flip]);
    if (*(volatile int*)&abort_flag) break;      // (set ahead of the barrier in factors_of: for all)
    const int last = s ? s - 1 : stages - 1;
    if (t == 0 && row != blockIdx.x && next < p.T) copy(last);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int j = i * nt + t;
      if (j < nvec) {
        const uint4 rv = p.dres ? slot[2 * nvec + j] : make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(p.dh + row * p.H + 8 * j) = grad_of(hv[i], dv[i], wv[i], rv, f, acc[i]);
      }
    }
    if (++s == stages) { s = 0; ph ^= 1u; }
  }
  if (abort_flag) {
    // copies may still be under way: the CTA does not leave before they have landed, or a bound
    for (int i = 0; i < stages; ++i) wait_row(smem_u32(&bars[i]), i < s ? ph ^ 1u : ph);
    return;
  }
  if (!p.dw) return;
  float* part = p.partial + (long long)blockIdx.x * p.H;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int j = i * nt + t;
    if (j < nvec)
#pragma unroll
      for (int e = 0; e < 4; ++e) *reinterpret_cast<f32x2*>(part + 8 * j + 2 * e) = acc[i][e];
  }
}

// grad_w: 32 columns a CTA, eight lanes of them four each, each quarter of its warps a run of the
// partial rows; then the quarters' sums in order.
constexpr int kJoinWarps = 16;
__global__ void __launch_bounds__(kJoinWarps * 32)
norm_join_kernel(const float* __restrict__ partial, int parts, int H, float* __restrict__ dw) {
  __shared__ float4 sums[kJoinWarps * 4][8];
  pdl_trigger();
  pdl_wait();
  const int run = threadIdx.x >> 3, c = threadIdx.x & 7;
  const int col = blockIdx.x * 32 + c * 4;
  const int each = (parts + kJoinWarps * 4 - 1) / (kJoinWarps * 4);
  const int p0 = run * each, p1 = min(p0 + each, parts);
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (col < H) {
    for (int p = p0; p < p1; p += 8) {           // eight loads at a time, also of a run that is shorter
      float4 a[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        a[i] = p + i < p1 ? *reinterpret_cast<const float4*>(partial + (long long)(p + i) * H + col)
                          : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v.x += a[i].x; v.y += a[i].y; v.z += a[i].z; v.w += a[i].w;
      }
    }
  }
  sums[run][c] = v;
  __syncthreads();
  if (threadIdx.x < 32 && blockIdx.x * 32 + threadIdx.x < H) {
    float a = 0.0f;
#pragma unroll 16
    for (int i = 0; i < kJoinWarps * 4; ++i) a += reinterpret_cast<const float*>(sums[i])[threadIdx.x];
    dw[blockIdx.x * 32 + threadIdx.x] = a;
  }
}

constexpr int round32(int n) { return (n + 31) / 32 * 32; }

constexpr int kShortThreads = 256;               // a CTA of several short rows
// lanes that a short row takes, vectors a lane (of H <= 512; the forward's up to 1024)
struct ShortRow {
  int lanes, vec;
};
ShortRow short_row(int nvec) {
  if (nvec <= 8) return {8, 1};
  if (nvec <= 16) return {16, 1};
  return {32, nvec <= 32 ? 1 : nvec <= 64 ? 2 : 4};
}
constexpr int kForwardShort = 128, kBackwardShort = 64;      // vectors

// Long rows of the gradient: as many CTAs of 512 threads together as the registers (128 a thread) leave
// room for, if their rings have three rows each.  The rings take up to 216 KB of an SM's 228, less where
// many CTAs have 2.3 KB each beside them (their sums and barriers, and 1 KB that the system keeps): the grid
// is the CTAs that fit, each with an equal share of the rows, and one that did not would run alone
// behind them ([16384, 768] with grad_residual 26.6 us, 39.6 with seven of eight CTAs resident).
constexpr int kSmSmem = 228 * 1024, kRingSmem = 216 * 1024, kRingBeside = 1280 + 1024;
struct RingPlan {
  int vec, threads, per_sm, stages;
  size_t smem;
};
constexpr RingPlan ring_plan(int H, bool residual) {
  RingPlan r{};
  const int nvec = H / 8, slot = H * 2 * (residual ? 3 : 2);
  r.vec = nvec <= 1024 ? 2 : 4;
  r.threads = round32((nvec + r.vec - 1) / r.vec);
  int most = 0;
  for (r.per_sm = 512 / r.threads;; --r.per_sm) {
    most = kRingSmem / r.per_sm;
    if (most > kSmSmem / r.per_sm - kRingBeside) most = kSmSmem / r.per_sm - kRingBeside;
    if (r.per_sm == 1 || most >= 3 * slot) break;
  }
  r.stages = most / slot < kMaxRing ? most / slot : kMaxRing;
  r.smem = (size_t)r.stages * slot;
  return r;
}
constexpr bool rings_fit() {
  for (int H = kBackwardShort * 8 + 8; H <= kMaxNormDim; H += 8)
    for (int residual = 0; residual < 2; ++residual) {
      const RingPlan r = ring_plan(H, residual != 0);
      if (r.stages < 2 || r.per_sm * (r.smem + kRingBeside) > kSmSmem) return false;
    }
  return true;
}
static_assert(rings_fit(), "the grid's CTAs are resident together");

// How the gradient's kernel is launched.  Short rows: four CTAs an SM, of which the registers let three be
// resident (two of rows of 264 and more), not fitted yet: times in us with four / three / two, with
// grad_residual: [65536, 64] 11.3 / 11.0 / 10.8, [65536, 128] 17.3 / 13.1 / 16.6, [65536, 256]
// 35.7 / 28.0 / 34.7, [65536, 512] 48.8 / 55.0 / 47.4.
struct BackwardPlan {
  int lanes, vec;              // lanes 0: long rows
  int threads, blocks, stages;
  size_t smem;
};
BackwardPlan backward_plan(int T, int H, bool residual) {
  BackwardPlan b{};
  const int nvec = H / 8;
  long long rows = T, per_sm = 4;
  if (nvec <= kBackwardShort) {
    const ShortRow r = short_row(nvec);
    b.lanes = r.lanes;
    b.vec = r.vec;
    b.threads = kShortThreads;
    rows = ceil_div(T, kShortThreads / r.lanes);
  } else {
    const RingPlan r = ring_plan(H, residual);
    b.vec = r.vec;
    b.threads = r.threads;
    b.stages = r.stages;
    b.smem = r.smem;
    per_sm = r.per_sm;
  }
  const long long blocks = per_sm * num_sms();
  b.blocks = (int)(rows < blocks ? rows : blocks);
  return b;
}

// Dynamic shared memory of a kernel beyond the default limit, set once a device.
template <auto kKernel>
cudaError_t allow_smem(int bytes) {
  static std::atomic<bool> set[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!set[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    set[dev].store(true, std::memory_order_release);
  }
  return cudaSuccess;
}

template <int kVec>
cudaError_t launch_long(const NormBackward& n, const BackwardPlan& b, cudaStream_t s) {
  const cudaError_t e = allow_smem<norm_backward_kernel<kVec>>(216 * 1024);
  if (e != cudaSuccess) return e;
  return launch_k(norm_backward_kernel<kVec>, dim3(b.blocks), dim3(b.threads), b.smem, s, n, b.stages);
}

constexpr int kFewRows = 64, kFewDim = 1024;
// Few enough rows for the one launch.
bool takes_few(const NormBackward& n) {
  return n.H <= kFewDim && n.T <= kFewRows;
}

template <int kVec>
cudaError_t launch_few_as(const NormBackward& n, cudaStream_t s) {
  return launch_k_cluster(norm_backward_few_kernel<kVec>, dim3(kFewCtas), dim3(kFewWarps * 32),
                          (size_t)kFewWarps * n.H * sizeof(float), s, kFewCtas, n);
}
cudaError_t launch_few(const NormBackward& n, cudaStream_t s) {
  const int vec = (n.H / 8 + 31) / 32;
  return vec == 1 ? launch_few_as<1>(n, s) : vec == 2 ? launch_few_as<2>(n, s) : launch_few_as<4>(n, s);
}

cudaError_t launch_backward(const NormBackward& n, const BackwardPlan& b, cudaStream_t s) {
  const dim3 grid(b.blocks), block(b.threads);
  if (b.lanes == 8) return launch_k(norm_backward_short_kernel<1, 8>, grid, block, 0, s, n);
  if (b.lanes == 16) return launch_k(norm_backward_short_kernel<1, 16>, grid, block, 0, s, n);
  if (b.lanes == 32)
    return b.vec == 1 ? launch_k(norm_backward_short_kernel<1, 32>, grid, block, 0, s, n)
                      : launch_k(norm_backward_short_kernel<2, 32>, grid, block, 0, s, n);
  return b.vec == 2 ? launch_long<2>(n, b, s) : launch_long<4>(n, b, s);
}

}  // namespace

size_t norm_backward_workspace_bytes(int T, int H) {
  // (without grad_residual there may be more CTAs)
  const int a = backward_plan(T, H, false).blocks, b = backward_plan(T, H, true).blocks;
  return ((size_t)(a > b ? a : b) * H * sizeof(float) + 255) & ~size_t(255);
}

template <int kVec, int kLanes>
static cudaError_t launch_norm_as(const NormForward& n, dim3 grid, int threads, cudaStream_t s) {
  return n.residual ? launch_k(norm_kernel<kVec, kLanes, true>, grid, dim3(threads), 0, s, n)
                    : launch_k(norm_kernel<kVec, kLanes, false>, grid, dim3(threads), 0, s, n);
}

cudaError_t launch_norm(const NormForward& n, cudaStream_t s) {
  const int nvec = n.H / 8;
  if (nvec <= kForwardShort) {
    const ShortRow r = short_row(nvec);
    const dim3 grid((unsigned)ceil_div(n.T, kShortThreads / r.lanes));
    if (r.lanes == 8) return launch_norm_as<1, 8>(n, grid, kShortThreads, s);
    if (r.lanes == 16) return launch_norm_as<1, 16>(n, grid, kShortThreads, s);
    return r.vec == 1   ? launch_norm_as<1, 32>(n, grid, kShortThreads, s)
           : r.vec == 2 ? launch_norm_as<2, 32>(n, grid, kShortThreads, s)
                        : launch_norm_as<4, 32>(n, grid, kShortThreads, s);
  }
  const dim3 grid((unsigned)n.T);
  // Up to two rows an SM: as many threads a row as it has vectors, beyond that a quarter of them with four
  // each, so that more rows fit (us, many threads / four vectors, both outputs with a residual:
  // [16, 7168] 2.1 / 2.4, [304, 7168] 3.25 / 3.23, [608, 7168] 5.8 / 4.7, [4096, 7168] 45.5 / 40.7;
  // [16, 2048] 1.6 / 2.1, [304, 2048] 2.0 / 2.2, [1024, 2048] 3.6 / 4.7, [4096, 2048] 9.8 / 8.1;
  // [152, 16384] 3.6 / 3.7, [304, 16384] 7.0 / 5.4, [608, 16384] 14.0 / 10.8).
  if (n.T <= 2 * num_sms())
    return nvec <= 1024 ? launch_norm_as<1, 0>(n, grid, round32(nvec), s)
                        : launch_norm_as<2, 0>(n, grid, round32((nvec + 1) / 2), s);
  return launch_norm_as<4, 0>(n, grid, round32((nvec + 3) / 4), s);
}

cudaError_t launch_norm_backward(const NormBackward& n, cudaStream_t s) {
  if (takes_few(n)) return launch_few(n, s);
  const BackwardPlan b = backward_plan(n.T, n.H, n.dres != nullptr);
  const cudaError_t e = launch_backward(n, b, s);
  if (e != cudaSuccess || !n.dw) return e;
  return launch_k(norm_join_kernel, dim3(ceil_div(n.H, 32)), dim3(kJoinWarps * 32), 0, s,
                  (const float*)n.partial, b.blocks, n.H, n.dw);
}

}  // namespace lmoe
