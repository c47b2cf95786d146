// bf16 products grouped by expert for few rows in all (grouped.cu has the formulas and the form for
// more): the weights stream from memory to registers and warp-level MMAs.
//
// Bound by the weights' bytes and by latency: a token's expert is 4 MB at 1024 x 2048, which pairs of
// SMs in tiles of 256 x 2048 would read with four pairs of 76.  Here a CTA takes 16 features (forward)
// or 32 columns (rows' gradient) of one expert and up to 16 of its rows, and its warps split the sum.
// Nothing goes through shared memory on the way: a thread's 16 bytes of weights are its part of the
// MMA operands, since the order of a sum's terms is free as long as both operands share it.
//   forward   B = W: a thread has 8 consecutive k of feature g, used as the MMA's k = 2t, 2t + 1,
//             2t + 8, 2t + 9 of two MMAs; its 8 k of token rows g and g + 8 are A likewise
//   rows      B = W^T: a thread has 4 consecutive columns of the four weight rows 4t .. 4t + 3 of 16;
//             column j of each thread's four makes MMA j (pairs of rows packed by byte permutes)
// The warps' partial sums meet in shared memory and are added in order.
// One row, 1024 x 2048: forward 4.8 us, rows 5.3; 2048 x 512: 2.8 and 5.6; 256 x 128: 2.0 and 2.3 (tiles of
// 256: 12.2, 9.2, 7.2, 12.1, 5.0, 5.3); rows with 64 columns and eight parts of N a CTA: 7.8 us.  Rows of
// many experts: 5.2 TB/s forward, 4 TB/s for the rows' gradient, whose pieces of a weight row are 64 bytes.
#include "grouped.cuh"

namespace lmoe {
namespace {

constexpr int kTok = 16;                        // token rows of a CTA
constexpr int kFeat = 16, kFeatSplit = 4;       // forward: features of a CTA (8 a warp), parts of K
constexpr int kForwardThreads = 2 * kFeatSplit * 32;
constexpr int kCols = 32, kColSplit = 16;       // rows: columns of a CTA, parts of N
constexpr int kRowsThreads = kColSplit * 32;

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// (a row's next 64-byte pieces come to L2 with the first: 64 rows of 64 experts, 1024 x 2048, 58 -> 51 us)
__device__ __forceinline__ uint4 ld_weights(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ uint2 ld_weights2(const uint16_t* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// The expert that owns row r and its rows; -1 if none does.  By all threads, each with its run of the
// offsets, asked for at once.  (At most 2^12 rows get here: a row number takes 16 bits.)
template <int kThreads>
__device__ __forceinline__ int owner(const GroupedLinear& p, int r, int2* rows, unsigned long long* found) {
  constexpr int kPer = 1024 / kThreads;
  if (threadIdx.x == 0) *found = 0;
  const int R = (int)p.R, e0 = threadIdx.x * kPer;
  int at[kPer + 1];
#pragma unroll
  for (int i = 0; i <= kPer; ++i) at[i] = __ldg(p.offsets + min(e0 + i, p.E));
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int a = min(max(at[i], 0), R), b = min(max(at[i + 1], a), R);
    if (e0 + i < p.E && a <= r && r < b)         // (of one expert, where the offsets ascend)
      atomicMax(found, (unsigned long long)(e0 + i + 1) << 32 | (unsigned)(a << 16 | b));
  }
  __syncthreads();
  const unsigned long long f = *found;
  *rows = make_int2((int)(f >> 16 & 0xFFFF), (int)(f & 0xFFFF));
  return (int)(f >> 32) - 1;
}

// grid: x strips of features or columns, y token rows; the CTAs of the rows that begin a tile of kTok
// of their expert's work
__global__ void __launch_bounds__(kForwardThreads)
stream_forward_kernel(const GroupedLinear p) {
  __shared__ float part[kFeatSplit][kTok][kFeat];
  __shared__ unsigned long long found;
  pdl_trigger();
  pdl_wait();
  int2 rows;
  const int r0 = blockIdx.y, e = owner<kForwardThreads>(p, r0, &rows, &found);
  if (e < 0 || (r0 - rows.x) % kTok) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int valid = min(kTok, rows.y - r0);
  const int f = blockIdx.x * kFeat + (warp & 1) * 8 + g, slice = warp >> 1;
  // this warp's part of K, in steps of 64
  const int steps = (p.K + 63) / 64, s0 = steps * slice / kFeatSplit, s1 = steps * (slice + 1) / kFeatSplit;
  const uint16_t* w = p.w + ((long long)e * p.N + f) * p.K;
  const uint16_t* x = p.rows_in + (long long)(r0 + g) * p.K;
  const uint16_t* x8 = x + 8ll * p.K;
  const bool wv = f < p.N, xv = g < valid, xv8 = g + 8 < valid;
  const uint4 none = make_uint4(0, 0, 0, 0);
  float c[4] = {};
#pragma unroll 8
  for (int s = s0; s < s1; ++s) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = s * 64 + i * 32 + t * 8;
      const bool in = k < p.K;                  // (K % 8 == 0)
      const uint4 b = wv && in ? ld_weights(w + k) : none;
      const uint4 a = xv && in ? *reinterpret_cast<const uint4*>(x + k) : none;
      const uint4 a8 = xv8 && in ? *reinterpret_cast<const uint4*>(x8 + k) : none;
      mma_bf16(c, a.x, a8.x, a.y, a8.y, b.x, b.y);
      mma_bf16(c, a.z, a8.z, a.w, a8.w, b.z, b.w);
    }
  }
  float* to = &part[slice][g][(warp & 1) * 8 + 2 * t];
  *reinterpret_cast<float2*>(to) = make_float2(c[0], c[1]);
  *reinterpret_cast<float2*>(to + 8 * kFeat) = make_float2(c[2], c[3]);
  __syncthreads();
  const int tok = threadIdx.x / (kFeat / 2), c2 = threadIdx.x % (kFeat / 2) * 2;
  const int col = blockIdx.x * kFeat + c2;
  if (tok < valid && col < p.N) {
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int s = 0; s < kFeatSplit; ++s) {
      lo += part[s][tok][c2];
      hi += part[s][tok][c2 + 1];
    }
    *reinterpret_cast<uint32_t*>(p.rows_out + (long long)(r0 + tok) * p.N + col) = pack_bf16x2(lo, hi);
  }
}

__global__ void __launch_bounds__(kRowsThreads)
stream_rows_kernel(const GroupedLinear p) {
  __shared__ __align__(16) float part[kColSplit][kTok][kCols + 4];    // (a quarter warp's stores meet no bank twice)
  __shared__ unsigned long long found;
  pdl_trigger();
  pdl_wait();
  int2 rows;
  const int r0 = blockIdx.y, e = owner<kRowsThreads>(p, r0, &rows, &found);
  if (e < 0 || (r0 - rows.x) % kTok) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int valid = min(kTok, rows.y - r0);
  const int col = blockIdx.x * kCols + g * 4;
  const int steps = (p.N + 15) / 16, s0 = steps * warp / kColSplit, s1 = steps * (warp + 1) / kColSplit;
  const uint16_t* w = p.w + (long long)e * p.N * p.K + col;
  const uint16_t* d = p.rows_in + (long long)(r0 + g) * p.N;
  const uint16_t* d8 = d + 8ll * p.N;
  const bool cv = col < p.K, dv = g < valid, dv8 = g + 8 < valid;     // (K % 8 == 0)
  float c[4][4] = {};
#pragma unroll 4
  for (int s = s0; s < s1; ++s) {
    const int n = s * 16 + t * 4;
    const bool in = n < p.N;                    // (N % 8 == 0: all four rows or none)
    uint2 b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      b[i] = cv && in ? ld_weights2(w + (long long)(n + i) * p.K) : make_uint2(0, 0);
    const uint2 a = dv && in ? *reinterpret_cast<const uint2*>(d + n) : make_uint2(0, 0);
    const uint2 a8 = dv8 && in ? *reinterpret_cast<const uint2*>(d8 + n) : make_uint2(0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      auto word = [&](const uint2& v) { return j < 2 ? v.x : v.y; };
      const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
      mma_bf16(c[j], a.x, a8.x, a.y, a8.y, __byte_perm(word(b[0]), word(b[1]), sel),
               __byte_perm(word(b[2]), word(b[3]), sel));
    }
  }
  // c[j]: rows g and g + 8, columns 4 (2t) + j and 4 (2t + 1) + j
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int k = 0; k < 2; ++k)
      *reinterpret_cast<float4*>(&part[warp][g + 8 * i][8 * t + 4 * k]) =
          make_float4(c[0][2 * i + k], c[1][2 * i + k], c[2][2 * i + k], c[3][2 * i + k]);
  __syncthreads();
  const int tok = threadIdx.x / kCols, c1 = threadIdx.x % kCols, out = blockIdx.x * kCols + c1;
  static_assert(kTok * kCols == kRowsThreads, "an output a thread");
  if (tok < valid && out < p.K) {
    float v = 0.0f;
#pragma unroll
    for (int s = 0; s < kColSplit; ++s) v += part[s][tok][c1];
    p.rows_out[(long long)(r0 + tok) * p.K + out] = to_bf16(v);
  }
}

}  // namespace

long long grouped_stream_ctas(const GroupedLinear& g, bool backward) {
  return g.R * (backward ? ceil_div(g.K, kCols) : ceil_div(g.N, kFeat));
}

cudaError_t launch_grouped_stream(const GroupedLinear& g, bool backward, cudaStream_t s) {
  if (backward)
    return launch_k(stream_rows_kernel, dim3(ceil_div(g.K, kCols), (unsigned)g.R), dim3(kRowsThreads), 0, s, g);
  return launch_k(stream_forward_kernel, dim3(ceil_div(g.N, kFeat), (unsigned)g.R), dim3(kForwardThreads), 0,
                  s, g);
}

}  // namespace lmoe
