// Block-scaled 8-bit products: bf16 -> e4m3 quantisation and the matrix product
// of e4m3 operands whose scales are fp32, one per token row and 128 columns and
// one per 128 x 128 block of weights.
//
// Quantisation of a block with largest magnitude m:
//   a = max(m, 2^-100),  scale = a / 448,  code = e4m3(x * (448 / a))
// each operation in fp32 and rounded once (448 is the largest e4m3 value; the
// floor keeps 448 / a finite, so an all-zero block gets codes 0).
//
// Product:
//   y[t, n] = sum_kb xs[t, kb] * ws[n/128, kb] * P_kb[t, n],
//   P_kb[t, n] = sum_{c in block kb} X[t, c] W[n, c]
// The scales change from one K block to the next, so P_kb cannot stay in the
// tensor core's accumulator: each K block is one accumulation there (K = 128:
// four MMAs), read back from TMEM and added in fp32 registers with its scale.
// With tokens on the MMA's M side a thread owns one token row, so that factor
// is one scalar per thread and 128 columns.
#include <cuda.h>

#include <type_traits>

#include "fp8.cuh"
#include "fp8_epilogue.cuh"
#include "fp8_quant.cuh"
#include "tc_ptx.cuh"

namespace lmoe {
namespace {

__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// A load that stays where it is written: ahead of the waits that follow it.
__device__ __forceinline__ float ld_ahead(const float* p) {
  float v;
  asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}

// largest magnitude of eight bf16 values, as the bits of a bf16 (magnitudes
// order like their bit patterns)
__device__ __forceinline__ uint32_t absmax8(const uint4& v) {
  const uint32_t m = 0x7FFF7FFFu;
  const uint32_t a = __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
  return max(a & 0xFFFFu, a >> 16);
}

__device__ __forceinline__ uint2 quant8(const uint4& v, float inv) {
  uint2 o;
  o.x = pack_e4m3x4(__fmul_rn(bf16_lo(v.x), inv), __fmul_rn(bf16_hi(v.x), inv),
                    __fmul_rn(bf16_lo(v.y), inv), __fmul_rn(bf16_hi(v.y), inv));
  o.y = pack_e4m3x4(__fmul_rn(bf16_lo(v.z), inv), __fmul_rn(bf16_hi(v.z), inv),
                    __fmul_rn(bf16_lo(v.w), inv), __fmul_rn(bf16_hi(v.w), inv));
  return o;
}

constexpr int kQuantThreads = 256;

// One scale per row and 128 columns: eight lanes a block, 16 elements a lane
// (a lane's elements are all inside the row or all outside: K % 16 == 0).
// Memory bound: each element is read once (2 bytes) and written once (1).  One block a group
// of lanes and many CTAs: two or four blocks each, their loads all ahead, were slower
// ([4096, 7168] 14.9 us, 14.5 with one: 6.1 TB/s; [8192, 7168] 27.1 us, 6.6 TB/s; [8, 7168]
// 1.3 us, the launch).
__global__ void __launch_bounds__(kQuantThreads)
quantize_rows_kernel(const uint16_t* __restrict__ x, uint8_t* __restrict__ codes,
                     float* __restrict__ scales, uint32_t nblocks, uint32_t nkb, int K) {
  pdl_trigger();
  pdl_wait();
  const uint32_t sub = threadIdx.x & 7;
  const uint32_t b = blockIdx.x * (kQuantThreads / 8) + (threadIdx.x >> 3);
  long long at = -1;
  if (b < nblocks) {
    if ((uint32_t)K == nkb * kFp8Block) {
      at = (long long)b * kFp8Block + sub * 16;
    } else {
      const uint32_t row = b / nkb, col = (b - row * nkb) * kFp8Block + sub * 16;
      if (col < (uint32_t)K) at = (long long)row * K + col;
    }
  }
  uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
  if (at >= 0) {
    v0 = ld_stream(x + at);
    v1 = ld_stream(x + at + 8);
  }
  uint32_t m = max(absmax8(v0), absmax8(v1));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  const BlockScale bs = block_scale(m << 16);
  if (at >= 0) {
    const uint2 lo = quant8(v0, bs.inv), hi = quant8(v1, bs.inv);
    *reinterpret_cast<uint4*>(codes + at) = make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
  if (sub == 0 && b < nblocks) scales[b] = bs.scale;
}

// One scale per 128 rows x 128 columns: a CTA a block, eight lanes a row, the block in
// registers between its maximum and its codes.  Memory bound ([8192, 7168] 27.2 us, 6.5 TB/s).
__global__ void __launch_bounds__(kQuantThreads)
quantize_blocks_kernel(const uint16_t* __restrict__ x, uint8_t* __restrict__ codes,
                       float* __restrict__ scales, long long rows, uint32_t nkb, int K) {
  constexpr int kSteps = kFp8Block / (kQuantThreads / 8);
  __shared__ uint32_t warp_max[kQuantThreads / 32];
  pdl_trigger();
  pdl_wait();
  const uint32_t rb = blockIdx.x / nkb, kb = blockIdx.x - rb * nkb;
  const uint32_t col = kb * kFp8Block + (threadIdx.x & 7) * 16;
  const long long row0 = (long long)rb * kFp8Block + (threadIdx.x >> 3);
  uint4 v[kSteps][2];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const long long row = row0 + i * (kQuantThreads / 8);
    v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
    if (row < rows && col < (uint32_t)K) {
      v[i][0] = ld_stream(x + row * K + col);
      v[i][1] = ld_stream(x + row * K + col + 8);
    }
    m = max(m, max(absmax8(v[i][0]), absmax8(v[i][1])));
  }
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kQuantThreads / 32; ++i) m = max(m, warp_max[i]);
  const BlockScale bs = block_scale(m << 16);
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const long long row = row0 + i * (kQuantThreads / 8);
    if (row < rows && col < (uint32_t)K) {
      const uint2 lo = quant8(v[i][0], bs.inv), hi = quant8(v[i][1], bs.inv);
      *reinterpret_cast<uint4*>(codes + row * K + col) = make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
  }
  if (threadIdx.x == 0) scales[blockIdx.x] = bs.scale;
}

// A token's row quantised once and written to its k expert-major rows: a CTA a
// token and 4096 columns, 16 columns a thread, eight lanes a block.  Bound by the writes
// (T = 4096, L = 2048, k = 16: 159 MB in 23.3 us, 6.8 TB/s, part of it still in L2).
__global__ void __launch_bounds__(kQuantThreads)
quantize_scatter_kernel(const uint16_t* __restrict__ Z, const int32_t* __restrict__ row_of, int L,
                        int k, uint8_t* __restrict__ codes, float* __restrict__ scales) {
  pdl_trigger();
  pdl_wait();
  const int t = blockIdx.x;
  const int col = (blockIdx.y * kQuantThreads + threadIdx.x) * 16;
  const bool in = col < L;                 // the same for a block's eight lanes
  uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
  if (in) {
    const uint16_t* src = Z + (long long)t * L + col;
    v0 = ld_stream(src);
    v1 = ld_stream(src + 8);
  }
  uint32_t m = max(absmax8(v0), absmax8(v1));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if (!in) return;
  const BlockScale bs = block_scale(m << 16);
  const uint2 lo = quant8(v0, bs.inv), hi = quant8(v1, bs.inv);
  for (int j = 0; j < k; ++j) {
    const long long row = __ldg(row_of + (long long)t * k + j);
    *reinterpret_cast<uint4*>(codes + row * L + col) = make_uint4(lo.x, lo.y, hi.x, hi.y);
    if ((threadIdx.x & 7) == 0) scales[row * (L / kFp8Block) + col / kFp8Block] = bs.scale;
  }
}

// ---------------------------------------------------------------------------
// The product: a persistent kernel of twelve warps a CTA.
//   warp 0      TMA producer: 128 K columns of 128 token rows and of kNH x 128
//               weight rows a stage (128-byte rows, 128-byte swizzle);
//   warp 1      allocates TMEM; one thread issues the MMAs (kind::f8f6f4,
//               M = 128 tokens, N = 128 kNH weight rows, K = 32), a K block
//               into each of the TMEM accumulators in turn;
//   warps 4..11 read the finished K block from TMEM (warp w: the 32 token rows
//               of lane quarter w % 4, half h = (w - 4) / 4 of the columns),
//               scale and add it in registers, and write the tile.
// Few rows an expert: bound by the weights' bytes; many: by the epilogue, in which a K block
// takes about 1050 cycles where its MMAs take 512 (kNH = 2): a TMEM load waits for the MMA in
// progress, then 128 columns are added up, and the accumulator goes back through a barrier.
// The wide tile (kNH = 2) halves the token bytes a product reads and the barriers.  SituGLU,
// four special functions an output, costs a tile another 4500 cycles, in which the tensor core
// runs two K blocks ahead and the ring fills.
// 65536 rows over 806 of 896 experts, latent 2048, inter 512: first product 362 us (1.84 GB,
// 5.1 TB/s), second 198 us (1.13 GB, 5.7 TB/s).
// Every wait is bounded: on expiry the code goes to the device error word, the
// CTA drains its copies and MMAs, frees its TMEM and returns.
// ---------------------------------------------------------------------------
constexpr int kEpiWarp0 = 4;                   // the first epilogue warp
constexpr int kEpiWarps = 8;
constexpr int kThreads = (kEpiWarp0 + kEpiWarps) * 32;
constexpr int BM = 128;                       // token rows of a tile
constexpr int kBK = 128;                      // K columns (bytes) of a stage
constexpr uint32_t kBoxBytes = 128 * kBK;     // a 128-row operand box
constexpr int kSmallTok = 16;                 // token rows of the small token box
constexpr long long kWaitCycles = 1ll << 32;  // ~2 s at 2 GHz
constexpr int kMaxGroups = 1024;

// device error word codes, as in the bf16 GEMM
enum : int { kErrProducer = 1, kErrMmaFull = 2, kErrMmaTmem = 3, kErrEpilogue = 4,
             kErrDrain = 5, kErrDone = 6 };

struct Fp8Params {
  int feat, nkb, groups, nfeat, stages, ws_rows;
  int wide_store, wide_add;    // rows of out / of add start on 32 bytes
  int min_rows;      // groups of up to this many rows are another kernel's
  int splits;        // > 1: clusters of this many CTAs share a tile's K blocks (one tile a cluster)
  long long rows;
  const int32_t* offsets;
  const float* xs;
  const float* ws;
  const uint16_t* add;
  uint16_t* out;
  uint8_t* act;
  float* act_s;
  int* err;
  SituParams sp;
};

__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                       int* err, int code) {
  const long long t0 = clock64();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > kWaitCycles) {
      atomicCAS(err, 0, code);
      *abort_flag = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                           int* err, int code) {
  return mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort_flag, err, code);
}

// K-major operand, 128-byte rows with the 128-byte swizzle, 8-row groups 1024 bytes apart
__device__ __forceinline__ uint64_t sdesc(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// kind::f8f6f4: fp32 accumulator, e4m3 A and B (format code 0), both K-major
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

struct Tile {
  int group, feat_tile;
  long long row0;   // first token row
  int nvalid;       // token rows of the tile that exist (1..128)
};

// Tiles of one CTA's walk: units of (token tile, feature tile), the feature
// tile changing fastest, so that neighbouring CTAs share a token tile.
// prefix [G + 1]: token tiles before each group; first / end rows per group.
__device__ __forceinline__ Tile tile_of(const Fp8Params& p, const int* prefix, const int* first,
                                        const int* end, int u) {
  Tile x;
  const int t = u / p.nfeat;
  x.feat_tile = u - t * p.nfeat;
  if (p.offsets == nullptr) {
    x.group = 0;
    x.row0 = (long long)t * BM;
    x.nvalid = (int)min((long long)BM, p.rows - x.row0);
    return x;
  }
  int lo = 0, hi = p.groups - 1;   // the last group whose prefix is <= t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= t) lo = mid; else hi = mid - 1;
  }
  x.group = lo;
  x.row0 = (long long)first[lo] + (long long)(t - prefix[lo]) * BM;
  x.nvalid = (int)min((long long)BM, (long long)end[lo] - x.row0);
  return x;
}

// tile_of by a whole warp: the group from two votes of 32 (kMaxGroups = 32 * 32).
__device__ __forceinline__ Tile tile_of_warp(const Fp8Params& p, const int* prefix, const int* first,
                                             const int* end, int u, int lane) {
  if (p.offsets == nullptr) return tile_of(p, prefix, first, end, u);
  Tile x;
  const int t = u / p.nfeat;
  x.feat_tile = u - t * p.nfeat;
  const int b = __popc(__ballot_sync(0xFFFFFFFFu, lane * 32 < p.groups && prefix[lane * 32] <= t)) - 1;
  const int g = b * 32 + lane;
  x.group = b * 32 + __popc(__ballot_sync(0xFFFFFFFFu, g < p.groups && prefix[g] <= t)) - 1;
  x.row0 = (long long)first[x.group] + (long long)(t - prefix[x.group]) * BM;
  x.nvalid = (int)min((long long)BM, (long long)end[x.group] - x.row0);
  return x;
}

// prefix / first / end of the groups from their offsets, by all threads of the
// CTA.  Offsets are clamped to [0, rows] and to be ascending within a group, so
// that no offset can lead outside the buffers.
__device__ void build_groups(const Fp8Params& p, int* prefix, int* first, int* end, int* warp_sum) {
  constexpr int kPer = (kMaxGroups + kThreads - 1) / kThreads;
  const int g0 = threadIdx.x * kPer;
  const int R = (int)p.rows;
  int tiles[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int g = g0 + i;
    tiles[i] = 0;
    if (g < p.groups) {
      const int a = min(max(__ldg(p.offsets + g), 0), R);
      const int b = min(max(__ldg(p.offsets + g + 1), a), R);
      first[g] = a;
      end[g] = b;
      tiles[i] = b - a > p.min_rows ? (b - a + BM - 1) / BM : 0;
    }
    sum += tiles[i];
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int run = incl - sum;
  for (int w = 0; w < warp; ++w) run += warp_sum[w];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int g = g0 + i;
    if (g <= p.groups) prefix[g] = run;
    run += tiles[i];
  }
}

// Split K: a cluster's CTAs leave their partial tiles in shared memory, rows
// kPartPad floats longer than the tile (so that a warp's 16-byte stores, a row a
// lane, meet no bank twice), and each then sums its share of the tile over the
// cluster in rank order.
constexpr int kPartPad = 4;
constexpr int kMaxSplits = 4;

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr, uint32_t rank) {
  uint32_t a;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// Forms of the product.  kFormSitu (kNH == 2): the weight boxes are the gate and
// the up rows of the same 128 features.  kFormSplit: split K, one tile a cluster.
enum : int { kFormPlain = 0, kFormSitu = 1, kFormSplit = 2 };

// kNH: 128-row weight boxes a tile (MMA N = 128 kNH).
template <int kNH, int kForm>
__global__ void __launch_bounds__(kThreads, 1)
fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmXs,
                const __grid_constant__ CUtensorMap tmW, const Fp8Params p) {
  constexpr bool kSitu = kForm == kFormSitu;
  constexpr bool kSplit = kForm == kFormSplit;
  constexpr int kBN = 128 * kNH;
  constexpr int kAcc = 512 / kBN;            // TMEM accumulators
  constexpr int kCols = kBN / 2;             // columns an epilogue thread owns
  constexpr uint32_t kStageBytes = kBoxBytes * (1 + kNH);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const int S = p.stages;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + (size_t)S * kStageBytes);
  // full[S], empty[S], tfull[kAcc], tempty[kAcc], done
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 2 * S + 2 * kAcc + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  uint32_t* amax_ex = tmem_holder + 2;   // [2][2][128] (SituGLU)
  int* warp_sum = reinterpret_cast<int*>(amax_ex + 512);        // [kThreads / 32]
  int* prefix = warp_sum + kThreads / 32;                       // [G + 1]
  int* first = prefix + p.groups + 1;                           // [G]
  int* end = first + p.groups;                                  // [G]

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bar0 + 8u * ((uint32_t)S + s); };
  auto tfull_bar = [&](uint32_t a) { return bar0 + 8u * (2u * S + a); };
  auto tempty_bar = [&](uint32_t a) { return bar0 + 8u * (2u * S + kAcc + a); };
  const uint32_t done_bar = bar0 + 8u * (2u * S + 2u * kAcc);

  // Operands, scales and offsets may come from the preceding kernel: nothing is read before
  // the wait.  (Grouped: nothing after this kernel starts before it either, see Fp8Gemm::beside.)
  if (p.offsets) {
    pdl_wait();
    pdl_trigger();
    build_groups(p, prefix, first, end, warp_sum);
    __syncthreads();
    if (prefix[p.groups] == 0) return;     // no group of this kernel's
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < kAcc; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), kEpiWarps);
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_holder)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (!p.offsets) {
    pdl_trigger();
    pdl_wait();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const int ntok = p.offsets ? prefix[p.groups] : (int)((p.rows + BM - 1) / BM);
  const int U = ntok * p.nfeat;
  // this CTA's tiles and K blocks
  const int rank = kSplit ? (int)cluster_rank() : 0;
  const int u0 = kSplit ? (int)blockIdx.x / p.splits : (int)blockIdx.x;
  const int ustep = kSplit ? U : (int)gridDim.x;
  const int kb0 = kSplit ? p.nkb * rank / p.splits : 0;
  const int kb1 = kSplit ? p.nkb * (rank + 1) / p.splits : p.nkb;

  // the launch's 168 registers a thread, split anew: 168 * 384 = 40 * 128 + 232 * 256
  if (warp < kEpiWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0 && lane == 0) {
      // ---------------- TMA producer ----------------
      uint32_t it = 0, s = 0, ph = 0;
      bool ok = true;
      for (int u = u0; u < U && ok; u += ustep) {
        const Tile x = tile_of(p, prefix, first, end, u);
        const bool small = x.nvalid <= kSmallTok;
        // weight rows of the boxes; a second box past the last feature is left out
        const int w0 = x.group * p.feat + x.feat_tile * (kSitu ? 128 : kBN);
        const int w1 = w0 + (kSitu ? p.feat / 2 : 128);
        const bool two = kNH == 2 && (kSitu || x.feat_tile * kBN + 128 < p.feat);
        const uint32_t bytes = (small ? kSmallTok * kBK : kBoxBytes) + (two ? 2u : 1u) * kBoxBytes;
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          if (!wait_phase(empty_bar(s), ph ^ 1u, abort_flag, p.err, kErrProducer)) { ok = false; break; }
          const uint32_t bar = full_bar(s);
          const uint32_t sa = smem_u32(smem) + s * kStageBytes;
          mbar_arrive_expect_tx(bar, bytes);
          tma_load_2d(&tmW, sa + kBoxBytes, bar, kb * kBK, w0);
          if (two) tma_load_2d(&tmW, sa + 2 * kBoxBytes, bar, kb * kBK, w1);
          tma_load_2d(small ? &tmXs : &tmX, sa, bar, kb * kBK, (int)x.row0);
          if (++s == (uint32_t)S) { s = 0; ph ^= 1u; }
        }
      }
      // every copy this thread issued has landed before the CTA exits
      const uint32_t from = it > (uint32_t)S ? it - (uint32_t)S : 0u;
      for (uint32_t j = from; j < it; ++j) {
        volatile int never = 0;
        if (!wait_phase(full_bar(j % (uint32_t)S), (j / (uint32_t)S) & 1u, &never, p.err, kErrDrain))
          break;
      }
    } else if (warp == 1 && lane == 0) {
      // ---------------- MMA issuer ----------------
      constexpr uint32_t idesc = idesc_e4m3(BM, kBN);
      const uint64_t d0 = sdesc(smem_u32(smem));
      uint32_t s = 0, ph = 0, acc = 0, aph = 0;
      bool ok = true;
      for (int u = u0; u < U && ok; u += ustep) {
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait_phase(tempty_bar(acc), aph ^ 1u, abort_flag, p.err, kErrMmaTmem) ||
              !wait_phase(full_bar(s), ph, abort_flag, p.err, kErrMmaFull)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t da = d0 + (uint64_t)s * (kStageBytes >> 4);
          const uint64_t db = da + (kBoxBytes >> 4);
          const uint32_t d_tmem = tmem_base + acc * kBN;
#pragma unroll
          for (int j = 0; j < kBK / 32; ++j)
            mma_e4m3(d_tmem, da + 2 * j, db + 2 * j, idesc, j ? 1u : 0u);
          mma_commit(empty_bar(s));
          mma_commit(tfull_bar(acc));
          if (++s == (uint32_t)S) { s = 0; ph ^= 1u; }
          if (++acc == kAcc) { acc = 0; aph ^= 1u; }
        }
      }
      // every MMA this thread issued has completed before TMEM is freed
      mma_commit(done_bar);
      volatile int never = 0;
      wait_phase(done_bar, 0u, &never, p.err, kErrDone);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    // ---------------- epilogue ----------------
    const int q = warp & 3;                 // TMEM lane quarter this warp may access
    const int h = (warp - kEpiWarp0) >> 2;          // column half
    const int r = q * 32 + lane;            // token row of the tile
    uint32_t acc = 0, aph = 0, par = 0;
    bool ok = true;
    // The tile, this thread's row of it and its scales: those of a K block are loaded one
    // block ahead of its sums, a tile's first ones ahead of the output of the tile before
    // (65536 rows over 896 experts: 608 -> 565 us with that and no branch around the loads).
    int ft = 0, row = 0;
    bool active = false, row_ok = false;
    const float *xsp = nullptr, *wsp = nullptr;
    const long long up_scales = kSitu ? (long long)(p.ws_rows / 2) * p.nkb : 0;
    float nx = 0.0f, nw = 0.0f, nw2 = 0.0f;
    auto scales = [&](int kb) {      // (without a branch, behind which the loads would be waited for)
      nx = ld_ahead(xsp + kb);
      nw = ld_ahead(wsp + kb);
      if (kSitu) nw2 = ld_ahead(wsp + up_scales + kb);
    };
    auto move_to = [&](int u) {
      const Tile x = tile_of_warp(p, prefix, first, end, u, lane);
      ft = x.feat_tile;
      // scale block of this thread's columns (SituGLU: the gate's)
      int blk = kSitu ? ft : ft * kNH + (kNH == 2 ? h : 0);
      active = q * 32 < x.nvalid && blk < p.ws_rows;   // warp-uniform
      blk = min(blk, p.ws_rows - 1);
      row_ok = active && r < x.nvalid;
      row = (int)x.row0 + (row_ok ? r : 0);
      xsp = p.xs + (long long)row * p.nkb;
      wsp = p.ws + ((long long)x.group * p.ws_rows + blk) * p.nkb;
      scales(kb0);
    };
    if (u0 < U) move_to(u0);
    for (int u = u0; u < U; u += ustep) {
      f32x2 y[kCols / 2];
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) y[i] = 0ull;
      if (kForm == kFormPlain && p.add)     // (`row` exists for every thread)
        add_first<kCols>(y, p.add + (long long)row * p.feat, ft * kBN + h * kCols, p.feat, p.wide_add);
      auto release = [&]() {                      // the accumulator is free again
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed(tempty_bar(acc));
      };
      for (int kb = kb0; kb < kb1 && ok; ++kb) {
        const float fg = nx * nw, fu = nx * nw2;
        scales(min(kb + 1, kb1 - 1));
        // (one outcome for the warp, whose lanes meet again below)
        ok = __all_sync(0xFFFFFFFFu, wait_phase(tfull_bar(acc), aph, abort_flag, p.err, kErrEpilogue));
        if (!ok) break;
        tc_fence_after();
        if (active) {
          const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + acc * kBN;
          const f32x2 f = f2_splat(fg), f2 = f2_splat(fu);
          // A load waits for the MMA that the tensor core is at, whatever its width: two of 64
          // columns cost half of what four of 32 do.
#pragma unroll
          for (int i = 0; i < kCols / 64; ++i) {
            uint32_t v[64];
            tmem_ld64(tb + (kSitu ? (uint32_t)(i * 128 + h * 64) : (uint32_t)(h * kCols + i * 64)), v);
            tmem_wait_ld64(v);
            if (i == kCols / 64 - 1) release();   // ahead of the last sums
#pragma unroll
            for (int j = 0; j < 32; ++j)
              y[i * 32 + j] = f2_fma(f2_make(v[2 * j], v[2 * j + 1]), kSitu && i == 1 ? f2 : f,
                                     y[i * 32 + j]);
          }
        } else {
          release();
        }
        if (++acc == kAcc) { acc = 0; aph ^= 1u; }
      }
      const bool store = active, store_row = ok && row_ok;
      const int orow = row, oft = ft;
      if (u + ustep < U) {
        move_to(u + ustep);
        if (kForm == kFormPlain && p.add && row_ok)
          prefetch_addend<kCols>(p.add + (long long)row * p.feat, ft * kBN + h * kCols, p.feat);
      }
      // (a warp whose waits ran out still meets the other half's below)
      if constexpr (kSitu) {
        if (store) {
          // 64 gate columns (y[0..31]) and the up columns of the same features
          // (y[32..63]); the row's other 64 features are the warp of the other
          // half's.  Their joint maximum is the row's scale for these 128.
          uint32_t m = 0;
          auto situ = [&](auto linear) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              y[j] = situ2_pair_as<decltype(linear)::value>(y[j], y[32 + j], p.sp);
              m = max(m, max(abs_bits(f2_lo(y[j])), abs_bits(f2_hi(y[j]))));
            }
          };
          // (one branch a tile, so that the 32 chains of special functions interleave)
          if (p.sp.has_lbeta) situ(std::true_type{}); else situ(std::false_type{});
          uint32_t* ex = amax_ex + par * 256;
          ex[h * 128 + r] = m;
          asm volatile("bar.sync %0, 64;" ::"r"(1 + q) : "memory");
          m = max(m, ex[(h ^ 1) * 128 + r]);
          const BlockScale bs = block_scale(m);
          if (store_row) {
            const int d = p.feat / 2;
            uint8_t* o = p.act + (long long)orow * d + oft * 128 + h * 64;
#pragma unroll
            for (int j = 0; j < 32; j += 16) {     // 32 codes
              uint32_t w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const f32x2 a = y[j + 2 * i], b = y[j + 2 * i + 1];
                w[i] = pack_e4m3x4(__fmul_rn(f2_lo(a), bs.inv), __fmul_rn(f2_hi(a), bs.inv),
                                   __fmul_rn(f2_lo(b), bs.inv), __fmul_rn(f2_hi(b), bs.inv));
              }
              st_global32(o + 2 * j, w);
            }
            if (h == 0) p.act_s[(long long)orow * (d / 128) + oft] = bs.scale;
          }
          par ^= 1u;
        }
      } else if constexpr (kSplit) {
        // every MMA of this CTA has completed: the ring is free
        if (store_row) {
          float* o = reinterpret_cast<float*>(smem) + r * (kBN + kPartPad) + h * kCols;
#pragma unroll
          for (int j = 0; j < kCols / 2; j += 2)
            *reinterpret_cast<float4*>(o + 2 * j) =
                make_float4(f2_lo(y[j]), f2_hi(y[j]), f2_lo(y[j + 1]), f2_hi(y[j + 1]));
        }
      } else if (store_row) {
        const int col0 = oft * kBN + h * kCols;
        const long long at = (long long)orow * p.feat + col0;
#pragma unroll
        for (int j = 0; j < kCols / 2; j += 8) {   // 16 columns
          if (col0 + 2 * j >= p.feat) break;       // feat % 8 == 0
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(f2_lo(y[j + i]), f2_hi(y[j + i]));
          if (p.wide_store) {
            st_global32(p.out + at + 2 * j, w);
          } else {
            *reinterpret_cast<uint4*>(p.out + at + 2 * j) = make_uint4(w[0], w[1], w[2], w[3]);
            if (col0 + 2 * j + 8 < p.feat)
              *reinterpret_cast<uint4*>(p.out + at + 2 * j + 8) = make_uint4(w[4], w[5], w[6], w[7]);
          }
        }
      }
    }
  }

  if constexpr (kSplit) {
    __syncwarp();
    cluster_sync();
    const Tile x = tile_of(p, prefix, first, end, u0);
    const int col0 = x.feat_tile * kBN;
    const int cols = min(kBN, p.feat - col0);        // a multiple of 8
    const int n4 = x.nvalid * (cols / 4);
    const uint32_t part = smem_u32(smem);
    for (int i = rank * kThreads + threadIdx.x; i < n4; i += p.splits * kThreads) {
      const int row = i / (cols / 4), col = (i - row * (cols / 4)) * 4;
      const uint32_t at = part + (uint32_t)(row * (kBN + kPartPad) + col) * 4u;
      float4 v[kMaxSplits];
#pragma unroll
      for (int k = 0; k < kMaxSplits; ++k)
        if (k < p.splits) v[k] = ld_cluster4(at, k);
      float4 t = v[0];
#pragma unroll
      for (int k = 1; k < kMaxSplits; ++k)
        if (k < p.splits) { t.x += v[k].x; t.y += v[k].y; t.z += v[k].z; t.w += v[k].w; }
      const long long o = (x.row0 + row) * p.feat + col0 + col;
      if (p.add) {
        const uint2 a = __ldg(reinterpret_cast<const uint2*>(p.add + o));
        t.x += bf16_lo(a.x); t.y += bf16_hi(a.x); t.z += bf16_lo(a.y); t.w += bf16_hi(a.y);
      }
      *reinterpret_cast<uint2*>(p.out + o) = make_uint2(pack_bf16x2(t.x, t.y), pack_bf16x2(t.z, t.w));
    }
    cluster_sync();     // no CTA leaves while another still reads its partial tile
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512u)
                 : "memory");
  }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// byte matrix [rows, K] in boxes of [box_rows][128 bytes], 128-byte swizzle; bytes
// outside it read as zeros
bool make_map(CUtensorMap* m, const void* base, long long rows, int K, int box_rows) {
  const EncodeTiledFn enc = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)K};
  cuuint32_t box[2] = {(cuuint32_t)kBK, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kRingBytes = 192 * 1024;

template <int kNH, int kForm>
cudaError_t launch_form(const Fp8Gemm& g, int splits, cudaStream_t s) {
  constexpr bool kSitu = kForm == kFormSitu;
  constexpr int kBN = 128 * kNH;
  constexpr int kStage = (int)kBoxBytes * (1 + kNH);
  static_assert(128 * (kBN + kPartPad) * 4 <= kRingBytes / kStage * kStage, "a partial tile fits the ring");
  Fp8Params p{};
  p.feat = g.feat;
  p.nkb = fp8_blocks(g.K);
  p.groups = g.groups;
  p.nfeat = kSitu ? g.feat / 2 / 128 : ceil_div(g.feat, kBN);
  p.stages = kRingBytes / kStage;
  p.ws_rows = fp8_blocks(g.feat);
  p.rows = g.rows;
  p.offsets = g.offsets;
  p.xs = g.xs;
  p.ws = g.ws;
  p.add = g.add;
  p.out = g.out;
  p.act = g.act;
  p.act_s = g.act_s;
  p.splits = splits;
  p.min_rows = g.min_rows;
  p.wide_store = g.feat % 16 == 0 && (reinterpret_cast<uintptr_t>(g.out) & 31u) == 0;
  p.wide_add = g.feat % 16 == 0 && (reinterpret_cast<uintptr_t>(g.add) & 31u) == 0;
  p.err = device_error_word();
  p.sp = make_situ_params(g.beta > 0.0f ? g.beta : 1.0f, g.linear_beta);
  if (!p.err) return cudaErrorInvalidValue;
  CUtensorMap mx, mxs, mw;
  if (!make_map(&mx, g.X, g.rows, g.K, BM) || !make_map(&mxs, g.X, g.rows, g.K, kSmallTok) ||
      !make_map(&mw, g.W, (long long)g.groups * g.feat, g.K, 128))
    return cudaErrorInvalidValue;
  const size_t smem = 1024 + (size_t)p.stages * kStage + (2 * p.stages + 2 * (512 / kBN) + 1) * 8 +
                      8 + 512 * 4 + kThreads / 32 * 4 + (g.offsets ? (3 * g.groups + 1) * 4 : 4);
  auto* kern = fp8_gemm_kernel<kNH, kForm>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const long long tok = g.offsets ? (g.rows + BM - 1) / BM + (g.rows < g.groups ? g.rows : g.groups)
                                  : (g.rows + BM - 1) / BM;
  const long long units = tok * p.nfeat;
  if (kForm == kFormSplit)
    return launch_k_cluster(kern, dim3((unsigned)(units * splits)), dim3(kThreads), smem, s, splits, mx,
                            mxs, mw, p);
  const int grid = units < num_sms() ? (int)units : num_sms();
  return launch_k(kern, dim3(grid), dim3(kThreads), smem, s, mx, mxs, mw, p);
}

// Form of a dense product: the one with the least modelled time, in SM cycles.
//   pair          256 x 256 tiles on two SMs each (fp8_pair.cu)
//   wide / splits 128 x 256 or 128 x 128 tiles, their K blocks split over clusters
// A wave of tiles costs its K blocks (more with more token rows) and its output, a launch a
// fixed part, a split the cluster's start and the exchange of the partial tiles.  The
// constants were fitted to sweeps of all forms over T 24 .. 4096 at [N, K] = [1024, 1024],
// [2048, 7168], [7168, 2048], [7168, 4096] and [8192, 7168]: the chosen form is within 5 % of
// the best one at all 50 of them (T = 128, [2048, 7168]: split four ways 12.6 us, unsplit
// 24.4; T = 4096, [8192, 7168]: pair 188 us, wide 202, narrow 305).  Clusters of eight were never
// clearly the best: about 13 fit at once.
struct DenseForm {
  bool pair, wide;
  int splits;
};
DenseForm dense_form(long long T, int N, int nkb, int nsm) {
  constexpr double kLaunch = 5700, kSplit = 5000, kExchange = 1.0 / 15;
  const long long tok = (T + BM - 1) / BM;
  const double rows = T < BM ? (double)T : (double)BM;
  const auto waves = [](long long n, int slots) { return (double)((n + slots - 1) / slots); };
  DenseForm best{true, true, 1};
  double least = waves((T + 255) / 256 * ceil_div(N, 256), nsm / 2) * (nkb * 900.0 + 5700) + kLaunch;
  for (int wide = 0; wide < 2; ++wide) {
    const int bn = wide ? 256 : 128;
    const double block = (wide ? 700 : 350) + 2.3 * rows;
    const long long tiles = tok * ceil_div(N, bn);
    for (int c = 1; c <= kMaxSplits && c <= nkb; c *= 2) {
      // clusters of four that fit at once: 32 of 152 / 4
      const int slots = c == 1 ? nsm : c == 2 ? nsm / 2 : nsm * 32 / 152;
      const double cost = c == 1 ? waves(tiles, slots) * (nkb * block + (wide ? 3800 : 3300)) + kLaunch
                                 : waves(tiles, slots) * ((nkb + c - 1) / c * block + kLaunch + kSplit +
                                                          rows * bn * 4 * kExchange);
      if (cost < least) { least = cost; best = DenseForm{false, wide != 0, c}; }
    }
  }
  return best;
}

}  // namespace

cudaError_t launch_fp8_gemm(const Fp8Gemm& g, cudaStream_t s) {
  // 9 to 16 tokens cost a stream's unit as many bytes of tokens as of weights, from L2:
  // [16, 7168] x [2048, 7168] 7.0 us as a stream, 10.2 here, [16, 4096] x [7168, 4096] 11.9 and
  // 11.1, [16, 7168] x [8192, 7168] 22.4 and 15.7 (8 tokens 13.7 and 15.4)
  const long long weights = (long long)g.feat * g.K;
  if (!g.offsets &&
      (g.rows <= kStreamRows / 2 || (g.rows <= kStreamRows && weights <= 24ll << 20)))
    return launch_fp8_stream(g, s);
  if (g.act) return launch_form<2, kFormSitu>(g, 1, s);
  DenseForm f{false, g.feat > 128, 1};
  if (!g.offsets) f = dense_form(g.rows, g.feat, fp8_blocks(g.K), num_sms());
  if (f.pair) return launch_fp8_pair(g, s);
  if (f.splits > 1)
    return f.wide ? launch_form<2, kFormSplit>(g, f.splits, s)
                  : launch_form<1, kFormSplit>(g, f.splits, s);
  return f.wide ? launch_form<2, kFormPlain>(g, 1, s) : launch_form<1, kFormPlain>(g, 1, s);
}

cudaError_t launch_quantize_scatter_fp8(const uint16_t* Z, int T, int L, int k,
                                        const int32_t* row_of, uint8_t* codes, float* scales,
                                        cudaStream_t s) {
  return launch_k(quantize_scatter_kernel, dim3(T, ceil_div(L, kQuantThreads * 16)),
                  dim3(kQuantThreads), 0, s, Z, row_of, L, k, codes, scales);
}

cudaError_t launch_quantize_fp8(const uint16_t* x, uint8_t* codes, float* scales, long long rows,
                                int K, int block_rows, cudaStream_t s) {
  const uint32_t nkb = (uint32_t)fp8_blocks(K);
  if (block_rows == 1) {
    const uint32_t nblocks = (uint32_t)(rows * nkb);
    constexpr uint32_t per = kQuantThreads / 8;
    return launch_k(quantize_rows_kernel, dim3((nblocks + per - 1) / per), dim3(kQuantThreads), 0, s,
                    x, codes, scales, nblocks, nkb, K);
  }
  return launch_k(quantize_blocks_kernel, dim3((uint32_t)fp8_blocks(rows) * nkb),
                  dim3(kQuantThreads), 0, s, x, codes, scales, rows, nkb, K);
}

}  // namespace lmoe
