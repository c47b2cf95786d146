// bf16 products of rows grouped by expert and their gradients, on pairs of SMs:
//   forward   out[r] = W_e x[r]
//   backward  grad_x[r] = W_e^T grad_out[r],   grad_W_e = sum over r of grad_out[r] x[r]^T
// for the rows r of expert e, offsets[e] .. offsets[e+1] - 1; products summed in fp32 on the
// tensor cores and rounded once.
//
// One kernel in three modes.  The two CTAs of a cluster compute a tile of 256 x N (tcgen05
// cta_group::2); each brings in its own 128 rows of the M side and half of the N side, and the
// tensor cores of both read both halves.
//   forward   M: rows of W (K-major),     N: token rows (K-major),      summed over K
//   rows      M: columns of W (M-major),  N: token rows (K-major),      summed over W's rows
//   weights   M: columns of grad_out,     N: columns of x (both M/N-major),  summed over tokens
// With the weights on the M side a tile's cost follows the number of an expert's rows in steps
// of 32, where 128 or 256 rows on the M side would pay for all of them; the columns of other
// experts' rows behind the last are not stored.  The major-ness is a bit of the MMA's operand
// descriptors: nothing is transposed in memory.
//
// Where the token rows are the sum's index (weights), an expert's last block of 64 may have fewer rows,
// and those behind them up to the next 16, the next expert's, have to read as zeros.  (Both operands': 0
// times another expert's NaN is NaN.)  The copies bring them, too: boxes of 16, 4 and 1 rows make up the
// expert's own, boxes of 4 and 1 rows behind the last row of all, outside the tensor map, the zeros.  Zeros
// that threads write (a barrier of the CTA's own, a warp that clears the rows and passes the block on)
// have to be released to the other CTA's MMAs in cluster scope: fp32 331 us, bf16 271 at the case below.
// (Boxes of every power of two up to 16 or 32: 264 us and 212 there, but 896 experts 1412 and 758 for 1412
// and 660, and a small call 1 us more for the maps.)
//
//   warp 0      TMA producer of this CTA's halves; their bytes count on the leader's (rank 0's)
//               barrier
//   warp 1      allocates TMEM; in the leader one lane issues the MMAs of both CTAs, and its
//               commits arrive in both
//   warps 4..11 read a finished tile from TMEM (warp w: the 32 M rows of lane quarter w % 4, half of
//               the columns) and write it: token rows through shared memory in 256-byte pieces, gradients
//               of weights through shared memory and bulk tensor stores, an addend added on the way
// Two accumulators of 256 columns: a tile's output runs beside the next one's sums.
// Every wait is bounded; neither CTA leaves or frees its TMEM before both are done.
//
// Times (GB300), and what bounds them:
//   forward, rows 65536 over 896 experts, 1024 x 2048: 593 us, memory (4.2 GB, 7.0 TB/s); 128 rows over
//                 121 of them: 80 us (6.3 TB/s)
//   forward       [4096, 7168] x [8192, 7168], one expert: 254 us, tensor pipe (1.89 PFLOP/s)
//   forward       65536 rows over 128 experts, 1024 x 2048: 178 us with 512 rows each (1.55 PFLOP/s), 190
//                 with uneven ones: a tile of fewer than 256 rows brings in more bytes per MMA cycle
//   rows          65536 over 128 experts, 2048 x 512: 107 us (604 MB, 5.6 TB/s; 1.28 PFLOP/s) where the tiles
//                 are eight rounds of the 76 pairs, 117 to 118 where they are nine: both, and the rounds
//   weights       65536 rows over 128 experts, 1024 x 2048: fp32 269 us, with addend 438 (2.55 GB,
//                 5.8 TB/s), bf16 215; with 512 rows each 245, 435, 195: memory, and the latency of the rows against a ring of six stages
//                 (one stage fewer: 16 % more in fp32, 8 % in bf16)
// Taking tiles over from clusters that have not started (cluster launch control) was no faster than
// tile u on pair u mod pairs, L2 prefetches of the next tile's rows or addend were slower.
#include <cuda.h>

#include <mutex>

#include "grouped.cuh"
#include "tc_ptx.cuh"

namespace lmoe {
namespace {

enum : int { kForward = 0, kRows = 1, kWeights = 2 };          // modes
enum : int { kErrProducer = 1, kErrMmaFull = 2, kErrMmaTmem = 3, kErrEpilogue = 4,
             kErrDrain = 5, kErrDone = 6 };                     // device error word codes

constexpr int kEpiWarp0 = 4, kEpiWarps = 8;
constexpr int kThreads = (kEpiWarp0 + kEpiWarps) * 32;
constexpr int kHalf = 128;                          // M rows of one CTA
constexpr int kTile = 2 * kHalf;
constexpr int kBK = 64;                             // a K block: 128 bytes
constexpr uint32_t kChunk = kBK * 128;              // 64 M or N columns of a block, K rows of 128 bytes
constexpr uint32_t kABytes = kHalf * kBK * 2;
constexpr int kAcc = 2;                             // TMEM accumulators of 256 columns
// weights: rows that the tensor cores add up before registers take over, whose additions round.  The
// tensor cores' truncate: of a step of 16 terms each is cut to 2^-25 of the largest magnitude's power of
// two, their sum to 2^-23 (seen with one term of 1 and others below it).  256 rows are off by 2.3e-7 of
// their norm (normal ones; 3.1e-7, all of them low, for positive ones), 512 rows by 4.7e-7 (7.1e-7), 65536
// rows in such sums by 3.7e-7 and 5.0e-7.  A read of TMEM every 2048 cycles of MMAs hides behind them but for
// the registers that the addend takes: 65536 rows, 128 experts, 1024 x 2048, 256 / 512 rows: fp32 269 / 268
// us, bf16 215 / 215, with addend 469 / 438.
template <int kOut>
constexpr int kFlushRows = kOut == 2 ? 512 : 256;
constexpr int kMaxStages = 8;
constexpr int kPartBox = 32;                        // token rows of a partial box
constexpr int kMaxGroups = 1024;
// shared memory of the epilogue: a box of 32 tokens x 128 bf16 features for each column half, or for
// each warp one of 32 rows x 128 bytes of a gradient of weights
constexpr uint32_t kRowBox = 32 * 256, kWeightBox = 32 * 128;
__host__ __device__ constexpr uint32_t out_bytes(int mode) {
  return mode == kWeights ? kEpiWarps * kWeightBox : 2 * kRowBox;
}

struct Params {
  int E, mdim, depth, ncols;     // M side's extent; terms of a sum and (weights) N side's extent
  int mtiles, ntiles;            // tiles of a group, ntiles: weights only
  int nt;                        // most token rows of a tile
  int stages;
  uint32_t stage_bytes;
  long long R;
  const int32_t* offsets;
  uint16_t* out;                 // forward, rows
  const float* add;              // weights
  int* err;
};

// A bounded wait: each further try suspends the thread for about a microsecond at most,
// 2^21 of them (about two seconds) end it.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                           int* err, int code) {
  if (mbar_try_wait(bar, parity)) return true;
  for (int n = 0; n < (1 << 21); ++n) {
    if (mbar_try_wait_ns(bar, parity, 1000u)) return true;
    if (*abort_flag) return false;
  }
  atomicCAS(err, 0, code);
  *abort_flag = 1;
  return false;
}

// kind::f16, bf16 operands, fp32 sums, M = 256
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Operand descriptors, both with the 128-byte swizzle.  K-major: rows of 64 K elements, groups of
// eight rows 1024 bytes apart.  M/N-major: a row is one K index of 64 M or N elements, groups of
// eight K 1024 bytes apart, the next 64 elements kChunk further.
template <bool kMajorK>
__device__ __forceinline__ uint64_t sdesc(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(kMajorK ? 1 : kChunk >> 4) << 16 |
         (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// 16 K further: 32 bytes in a row, or 16 rows
template <bool kMajorK>
constexpr uint64_t kStep = (kMajorK ? 32 : 16 * 128) >> 4;

template <int kMode>
__device__ __forceinline__ uint32_t idesc(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((kMode == kForward ? 0u : 1u) << 15) |
         ((kMode == kWeights ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(kTile >> 4) << 24);
}

// forward, rows: token tiles before each expert [E + 1], its first row and the one behind its
// last [E], in shared memory.
struct Groups {
  int* prefix;
  int2* rows;
};

// One tile of the walk.
struct Tile {
  int group, m0;      // first M row
  int row0;           // token rows: the first and how many (weights: the group's)
  int rows;
  int n0, n;          // N side: first column (weights), the MMA's N
};

__device__ __forceinline__ int2 group_rows(const Params& p, int e) {
  const int R = (int)p.R;
  const int a = min(max(__ldg(p.offsets + e), 0), R);
  return make_int2(a, min(max(__ldg(p.offsets + e + 1), a), R));
}

// forward, rows: tiles of an expert's token rows, the M tile changing fastest.  weights: an
// expert's M x N tiles.
template <int kMode>
__device__ __forceinline__ Tile tile_of(const Params& p, const Groups& t, int u) {
  Tile x;
  if constexpr (kMode == kWeights) {
    const int per = p.mtiles * p.ntiles;
    x.group = u / per;
    const int rem = u - x.group * per, m = rem / p.ntiles;
    x.m0 = m * kTile;
    x.n0 = (rem - m * p.ntiles) * kTile;
    x.n = p.ncols - x.n0 > kHalf ? kTile : kHalf;
    const int2 r = group_rows(p, x.group);
    x.row0 = r.x;
    x.rows = r.y - r.x;
  } else {
    const int i = u / p.mtiles;
    x.m0 = (u - i * p.mtiles) * kTile;
    int lo = 0, hi = p.E - 1;      // the last group whose prefix is <= i
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (t.prefix[mid] <= i) lo = mid; else hi = mid - 1;
    }
    x.group = lo;
    // an expert's rows in tiles of about the same size: a rest of a few rows would read all
    // weights for them (none is empty: the rows are more than nt times one tile less)
    const int2 r = t.rows[lo];
    const int tiles = t.prefix[lo + 1] - t.prefix[lo];
    const int each = ((r.y - r.x + tiles - 1) / tiles + 31) & ~31;
    x.row0 = r.x + (i - t.prefix[lo]) * each;
    x.rows = min(each, r.y - x.row0);
    x.n0 = 0;
    x.n = (x.rows + 31) & ~31;
  }
  return x;
}

// The table of the groups, by all threads of the CTA.
__device__ void build_groups(const Params& p, const Groups& t, int* warp_sum) {
  constexpr int kPer = (kMaxGroups + kThreads - 1) / kThreads;
  const int g0 = threadIdx.x * kPer;
  int tiles[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    tiles[i] = 0;
    if (g0 + i < p.E) {
      const int2 r = group_rows(p, g0 + i);
      t.rows[g0 + i] = r;
      tiles[i] = (r.y - r.x + p.nt - 1) / p.nt;
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
    if (g0 + i <= p.E) t.prefix[g0 + i] = run;
    run += tiles[i];
  }
}

// The four epilogue warps of a column half meet.
__device__ __forceinline__ void half_sync(int h) {
  asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + h) : "memory");
}
// ... and agree whether all of them are to go on.
__device__ __forceinline__ bool half_all(int h, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "barrier.cta.red.and.pred q, %1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(1 + h), "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}

// forward, rows: 32 token columns of the CTA's 128 features into rows of out, by the four warps of a
// half.  A lane has one feature of all tokens: neighbours swap halves, so that each holds two
// features of every second token, and the box [32 tokens][128 features] in shared memory gives 256
// bytes of a token's row to 16 lanes (the warps' own 64 bytes a row took 1.6 times as long).  Every
// second row of the box has its 64-byte halves swapped, so that the pairs meet no bank twice.
__device__ __forceinline__ void store_rows(const Params& p, uint8_t* box, const uint32_t (&v)[32],
                                           int row0, int valid, int f0, int q, int h, int lane) {
  half_sync(h);                                  // the box has been read
  uint8_t* to = box + (lane & 1) * 256 + ((q ^ (lane & 1)) * 64 + (lane >> 1) * 4);
#pragma unroll
  for (int j = 0; j < 32; j += 2) {
    const uint32_t own = pack_bf16x2(__uint_as_float(v[j]), __uint_as_float(v[j + 1]));
    const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, own, 1);
    // even lane: row j, features f, f + 1 = own low, other low; odd: row j + 1, other high, own high
    const uint32_t two = lane & 1 ? __byte_perm(other, own, 0x7632) : __byte_perm(own, other, 0x5410);
    *reinterpret_cast<uint32_t*>(to + j * 256) = two;
  }
  half_sync(h);
  const int c = lane & 15, f = f0 + c * 8;       // (mdim % 8 == 0)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + q * 2 + (lane >> 4);
    const uint4 w = *reinterpret_cast<const uint4*>(box + r * 256 + ((c ^ ((r & 1) << 2)) * 16));
    if (r < valid && f < p.mdim)
      *reinterpret_cast<uint4*>(p.out + (long long)(row0 + r) * p.mdim + f) = w;
  }
}

// weights: the addend of a box at row m, column col: 128 bytes of a row by eight lanes, four rows a load
__device__ __forceinline__ void load_addend(const Params& p, const Tile& x, int m, int col, int lane,
                                            uint4 (&add)[8]) {
  const int r = m + (lane >> 3), c = col + (lane & 7) * 4;       // (ncols % 8 == 0)
  const float* at = p.add + ((long long)x.group * p.mdim + r) * p.ncols + c;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    add[i] = make_uint4(0, 0, 0, 0);
    if (r + i * 4 < p.mdim && c < p.ncols)
      asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(add[i].x), "=r"(add[i].y), "=r"(add[i].z), "=r"(add[i].w)
                   : "l"(at + (long long)i * 4 * p.ncols));
  }
}

// part: boxes of fewer rows.  forward, rows: kPartBox of b; weights: 16, 4 and 1 of a and of b
template <int kMode>
struct Maps {
  CUtensorMap a, b, o, part[kMode == kWeights ? 6 : 1];
};

// kOut (weights): 0 fp32, 1 bf16, 2 fp32 with an addend
template <int kMode, int kOut>
__global__ void __launch_bounds__(kThreads, 1)
grouped_kernel(const __grid_constant__ Maps<kMode> maps, const Params p) {
  constexpr bool kAK = kMode == kForward, kBK_ = kMode != kWeights;   // K-major operands
  constexpr int kFlush = kFlushRows<kOut>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* boxes = smem + (size_t)p.stages * p.stage_bytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(boxes + out_bytes(kMode));
  constexpr int kFull = 0, kEmpty = kMaxStages, kTfull = 2 * kMaxStages, kTempty = kTfull + kAcc,
                kDone = kTempty + kAcc, kBars = kDone + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* warp_sum = reinterpret_cast<int*>(tmem_holder + 2);
  const Groups groups{warp_sum + kThreads / 32 + 2 * p.E, reinterpret_cast<int2*>(warp_sum + kThreads / 32)};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bar0 = smem_u32(bars);
  auto bar_at = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  const uint32_t rank = cluster_rank();

  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(bar_at(kFull + i), 1);
      mbar_init(bar_at(kEmpty + i), 1);
    }
    for (int i = 0; i < kAcc; ++i) {
      mbar_init(bar_at(kTfull + i), 1);
      mbar_init(bar_at(kTempty + i), 2 * kEpiWarps);             // (the leader's: both CTAs' epilogues)
    }
    mbar_init(bar_at(kDone), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_holder)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  int U;
  if constexpr (kMode == kWeights) {
    U = p.E * p.mtiles * p.ntiles;
  } else {
    build_groups(p, groups, warp_sum);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();      // both CTAs' barriers are there before any copy or commit reaches them
  tc_fence_after();
  // (offsets that do not ascend may count rows more than once: the walk ends somewhere)
  if constexpr (kMode != kWeights) U = (int)min((long long)groups.prefix[p.E] * p.mtiles, 1ll << 30);
  const uint32_t tmem_base = *tmem_holder;
  const int u0 = (int)(blockIdx.x >> 1), ustep = (int)(gridDim.x >> 1);
  const int nkb_rows = (p.depth + kBK - 1) / kBK;

  // weights: the launch's 168 registers a thread, split anew: 168 * 384 = 40 * 128 + 232 * 256
  if (warp < kEpiWarp0) {
    if constexpr (kMode == kWeights) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0) {
      // ---------------- TMA producer ----------------
      // (the warp runs as one and a lane issues, as in the MMA warp)
      int s = 0;
      uint32_t ph = 0, it = 0;
      bool ok = true;
      for (int u = u0; u < U && ok; u += ustep) {
        const Tile x = tile_of<kMode>(p, groups, u);
        const int m = x.m0 + (int)rank * kHalf, half = x.n >> 1;
        const int nkb = kMode == kWeights ? (x.rows + kBK - 1) / kBK : nkb_rows;
        // token rows: one box of all, or as many partial ones as this CTA's half takes
        const bool whole = x.n == p.nt;
        const int nbox = whole ? 1 : (half + kPartBox - 1) / kPartBox;
        const int brows = whole ? p.nt >> 1 : kPartBox;
        const int tok = x.row0 + (int)rank * half;
        const int nchunk = x.n >> 7;                   // (weights: 64 columns each)
        const int n0 = x.n0 + (int)rank * half;
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          ok = __all_sync(0xFFFFFFFFu, wait_phase(bar_at(kEmpty + s), ph ^ 1u, abort_flag, p.err, kErrProducer));
          if (!ok) break;
          const uint32_t at = smem_u32(smem) + (uint32_t)s * p.stage_bytes, bt = at + kABytes;
          const int k = kb * kBK;
          const int left = x.rows - k;                 // (weights)
          const bool part = kMode == kWeights && left < kBK;
          const int filled = part ? (left + 15) & ~15 : kBK;
          if (elect_one()) {
            const uint32_t bar = cluster_addr(bar_at(kFull + s), 0);
            if (rank == 0) {
              const uint32_t bytes = kMode == kWeights ? (uint32_t)((2 + nchunk) * filled) * 128u
                                                       : kABytes + (uint32_t)(nbox * brows) * 128u;
              mbar_arrive_expect_tx(bar_at(kFull + s), 2 * bytes);
            }
            if constexpr (kMode == kForward) {
              tma_load_pair_3d(&maps.a, at, bar, k, m, x.group);
            } else if constexpr (kMode == kRows) {
              tma_load_pair_3d(&maps.a, at, bar, m, k, x.group);
              tma_load_pair_3d(&maps.a, at + kChunk, bar, m + 64, k, x.group);
            }
            if constexpr (kMode != kWeights) {
              if (whole) {
                tma_load_pair(&maps.b, bt, bar, k, tok);
              } else {
                for (int i = 0; i < nbox; ++i)
                  tma_load_pair(&maps.part[0], bt + (uint32_t)(i * brows) * 128u, bar, k, tok + i * brows);
              }
            } else {
              // a box of both operands: to row r of the block
              auto box = [&](const CUtensorMap* a, const CUtensorMap* b, int r, int row) {
                tma_load_pair(a, at + r * 128u, bar, m, row);
                tma_load_pair(a, at + kChunk + r * 128u, bar, m + 64, row);
                tma_load_pair(b, bt + r * 128u, bar, n0, row);
                if (nchunk > 1) tma_load_pair(b, bt + kChunk + r * 128u, bar, n0 + 64, row);
              };
              const int row0 = x.row0 + k, beyond = (int)p.R;
              if (!part) {
                box(&maps.a, &maps.b, 0, row0);
              } else {
                int r = 0;
                for (; r + 16 <= left; r += 16) box(&maps.part[0], &maps.part[1], r, row0 + r);
                for (; r + 4 <= left; r += 4) box(&maps.part[2], &maps.part[3], r, row0 + r);
                for (; r < left; ++r) box(&maps.part[4], &maps.part[5], r, row0 + r);
                for (; r & 3; ++r) box(&maps.part[4], &maps.part[5], r, beyond);
                for (; r < filled; r += 4) box(&maps.part[2], &maps.part[3], r, beyond);
              }
            }
          }
          __syncwarp();
          if (++s == p.stages) { s = 0; ph ^= 1u; }
        }
      }
      // the leader: every copy of the pair has landed before the CTAs exit
      if (rank == 0)
        for (uint32_t j = it > (uint32_t)p.stages ? it - p.stages : 0u; j < it; ++j) {
          volatile int never = 0;
          if (!wait_phase(bar_at(kFull + (int)(j % p.stages)), (j / p.stages) & 1u, &never, p.err, kErrDrain))
            break;
        }
    } else if (warp == 1) {
      if (rank == 0) {
        // ---------------- MMA issuer of the pair ----------------
        // The warp runs the loop as one and a lane of it issues: an MMA's operands go through
        // registers of the warp, which a branch of one lane fills at about 130 cycles an MMA.
        const uint64_t a0 = sdesc<kAK>(smem_u32(smem)), b0 = sdesc<kBK_>(smem_u32(smem) + kABytes);
        int s = 0;
        uint32_t ph = 0, acc = 0, aph = 0;
        bool ok = true;
        for (int u = u0; u < U && ok; u += ustep) {
          const Tile x = tile_of<kMode>(p, groups, u);
          const int depth = kMode == kWeights ? x.rows : p.depth;
          if (depth == 0) continue;                    // (an expert without rows: the epilogue writes zeros)
          const uint32_t id = idesc<kMode>(x.n);
          for (int k = 0; k < depth; k += kBK) {
            const bool fresh = kMode == kWeights ? k % kFlush == 0 : k == 0;     // a new accumulator
            if (fresh) {
              ok = __all_sync(0xFFFFFFFFu, wait_phase(bar_at(kTempty + (int)acc), aph ^ 1u, abort_flag,
                                                      p.err, kErrMmaTmem));
              if (!ok) break;
            }
            ok = __all_sync(0xFFFFFFFFu, wait_phase(bar_at(kFull + s), ph, abort_flag, p.err, kErrMmaFull));
            if (!ok) break;
            tc_fence_after();
            const uint64_t da = a0 + (uint64_t)s * (p.stage_bytes >> 4), db = b0 + (uint64_t)s * (p.stage_bytes >> 4);
            const uint32_t d = tmem_base + acc * kTile;
            const bool last = k + kBK >= depth || (kMode == kWeights && (k + kBK) % kFlush == 0);
            if (elect_one()) {
#pragma unroll
              for (int j = 0; j < kBK / 16; ++j)
                // (weights: not past the zeros; the others' blocks are whole or filled up with zeros)
                if (kMode != kWeights || k + 16 * j < depth)
                  mma_pair(d, da + j * kStep<kAK>, db + j * kStep<kBK_>, id, j ? 1u : (uint32_t)!fresh);
              commit_both(bar_at(kEmpty + s));
              if (last) commit_both(bar_at(kTfull + (int)acc));
            }
            __syncwarp();
            if (++s == p.stages) { s = 0; ph ^= 1u; }
            if (last && ++acc == kAcc) { acc = 0; aph ^= 1u; }
          }
          if (!ok) break;
        }
        // every MMA the lane issued has completed before TMEM is freed
        if (elect_one())
          asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                           bar_at(kDone))
                       : "memory");
        __syncwarp();
        volatile int never = 0;
        wait_phase(bar_at(kDone), 0u, &never, p.err, kErrDone);
      }
    }
  } else {
    if constexpr (kMode == kWeights) asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    // ---------------- epilogue ----------------
    const int q = warp & 3;                      // TMEM lane quarter this warp may access
    const int h = (warp - kEpiWarp0) >> 2;
    const uint32_t tempty = cluster_addr(bar_at(kTempty), 0);
    const uint32_t tmem = tmem_base + ((uint32_t)(q * 32) << 16);
    uint32_t acc = 0, aph = 0;
    bool ok = true;
    // (a wait's outcome is one for the warp, whose lanes meet again below)
    auto wait_full = [&] {
      ok = __all_sync(0xFFFFFFFFu, wait_phase(bar_at(kTfull + (int)acc), aph, abort_flag, p.err, kErrEpilogue));
      if constexpr (kMode != kWeights) ok = half_all(h, ok);     // (they meet again in store_rows)
      tc_fence_after();
      return ok;
    };
    auto give_back = [&] {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(tempty + 8u * acc);
    };
    if constexpr (kMode != kWeights) {
      uint8_t* box = boxes + h * kRowBox;
      for (int u = u0; u < U && ok; u += ustep) {
        const Tile x = tile_of<kMode>(p, groups, u);
        const int f0 = x.m0 + (int)rank * kHalf;
        if (!wait_full()) break;
        // the next columns are on their way while these are written; behind the last the
        // accumulator goes back
        const uint32_t at = tmem + acc * kTile;
        uint32_t va[32], vb[32];
        int c = h * 32;
        if (c < x.rows) tmem_ld32(at + c, va);
        else give_back();
        for (; c < x.rows; c += 128) {
          tmem_wait_ld32(va);
          if (c + 64 < x.rows) tmem_ld32(at + c + 64, vb);
          else give_back();
          store_rows(p, box, va, x.row0 + c, x.rows - c, f0, q, h, lane);
          if (c + 64 >= x.rows) break;
          tmem_wait_ld32(vb);
          if (c + 128 < x.rows) tmem_ld32(at + c + 128, va);
          else give_back();
          store_rows(p, box, vb, x.row0 + c + 64, x.rows - c - 64, f0, q, h, lane);
        }
        if (++acc == kAcc) { acc = 0; aph ^= 1u; }
      }
    } else {
      constexpr int kCols = kOut == 1 ? 64 : 32;                 // columns of a box, one box a warp
      uint8_t* box = boxes + (warp - kEpiWarp0) * kWeightBox;
      uint4 add[8];
      if constexpr (kOut == 2)
        if (u0 < U) {
          const Tile x = tile_of<kMode>(p, groups, u0);
          load_addend(p, x, x.m0 + (int)rank * kHalf + q * 32, x.n0 + h * (x.n >> 1), lane, add);
        }
      for (int u = u0; u < U && ok; u += ustep) {
        const Tile x = tile_of<kMode>(p, groups, u);
        const int m = x.m0 + (int)rank * kHalf + q * 32;         // first M row of the warp
        const int width = x.n >> 1, c0 = x.n0 + h * width;       // its columns
        f32x2 y[kHalf / 2];
#pragma unroll
        for (int j = 0; j < kHalf / 2; ++j) y[j] = 0ull;
        for (int r = 0; r < x.rows; r += kFlush) {
          if (!wait_full()) break;
          constexpr int kLoad = kOut == 2 ? 32 : 64;             // (the addend takes registers, too)
#pragma unroll
          for (int i = 0; i < kHalf; i += kLoad) {
            if (i >= width) break;
            uint32_t v[kLoad];
            if constexpr (kLoad == 64) {
              tmem_ld64(tmem + acc * kTile + h * width + i, v);
              tmem_wait_ld64(v);
            } else {
              tmem_ld32(tmem + acc * kTile + h * width + i, v);
              tmem_wait_ld32(v);
            }
            if (i + kLoad == width) give_back();
#pragma unroll
            for (int j = 0; j < kLoad / 2; ++j)
              y[i / 2 + j] = f2_add(y[i / 2 + j], f2_make(v[2 * j], v[2 * j + 1]));
          }
          if (++acc == kAcc) { acc = 0; aph ^= 1u; }
        }
        if (!ok) break;
#pragma unroll
        for (int b = 0; b < kHalf / kCols; ++b) {
          if (b * kCols >= width) break;
          const int col = c0 + b * kCols;
          if (lane == 0) bulk_wait_read();                       // the box's last store has read it
          __syncwarp();
          if constexpr (kOut == 2) {
            // the addend, 128 bytes of a row by eight lanes, then the next box's on its way
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4*>(box + (i * 4 + (lane >> 3)) * 128 +
                                        (((lane ^ (i * 4 + (lane >> 3))) & 7) << 4)) = add[i];
            __syncwarp();
            if ((b + 1) * kCols < width) load_addend(p, x, m, col + kCols, lane, add);
            else if (u + ustep < U) {
              const Tile t = tile_of<kMode>(p, groups, u + ustep);
              load_addend(p, t, t.m0 + (int)rank * kHalf + q * 32, t.n0 + h * (t.n >> 1), lane, add);
            }
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint4* at = reinterpret_cast<uint4*>(box + lane * 128 + ((j ^ (lane & 7)) << 4));
            if constexpr (kOut == 1) {
              const f32x2* v = y + b * 32 + 4 * j;
              *at = make_uint4(pack_bf16x2(f2_lo(v[0]), f2_hi(v[0])), pack_bf16x2(f2_lo(v[1]), f2_hi(v[1])),
                               pack_bf16x2(f2_lo(v[2]), f2_hi(v[2])), pack_bf16x2(f2_lo(v[3]), f2_hi(v[3])));
            } else {
              f32x2 v0 = y[b * 16 + 2 * j], v1 = y[b * 16 + 2 * j + 1];
              if constexpr (kOut == 2) {
                const uint4 a = *at;
                v0 = f2_add(v0, f2_make(a.x, a.y));
                v1 = f2_add(v1, f2_make(a.z, a.w));
              }
              *at = make_uint4((uint32_t)v0, (uint32_t)(v0 >> 32), (uint32_t)v1, (uint32_t)(v1 >> 32));
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (m < p.mdim && col < p.ncols) tma_store_3d(&maps.o, smem_u32(box), col, m, x.group);
            bulk_commit();
          }
        }
      }
    }
    if (kMode == kWeights && lane == 0) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();      // the pair's MMAs and commits are done with both CTAs
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512u)
                 : "memory");
  }
  cluster_sync();
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// [groups, rows, cols], or (groups = 0) [rows, cols], in boxes of box_rows rows of 128 bytes, 128-byte
// swizzle; elements outside read as zeros and are not written
bool make_map(CUtensorMap* m, const void* base, bool fp32, long long groups, long long rows, int cols,
              int box_rows) {
  const EncodeTiledFn enc = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
  if (!enc) return false;
  const cuuint64_t size = fp32 ? 4 : 2;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)groups};
  cuuint64_t strides[2] = {(cuuint64_t)cols * size, (cuuint64_t)cols * size * (cuuint64_t)rows};
  cuuint32_t box[3] = {(cuuint32_t)(128 / size), (cuuint32_t)box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
             groups ? 3 : 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr size_t kMaxSmem = 227 * 1024;

// shared memory of a launch but for its stages
constexpr size_t other_smem(int mode, int E) {
  return 1024 + out_bytes(mode) +
         (2 * kMaxStages + 2 * kAcc + 1) * 8 + 8 + (kThreads / 32) * 4 +
         (mode == kWeights ? 0 : (size_t)(3 * E + 1) * 4) + 16;
}

// Pairs that fit on the current device at once (pairs share a GPC), 0 on failure.
template <int kMode, int kOut>
int pairs_resident() {
  static int cache[64] = {};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (cache[dev]) return cache[dev];
  auto* kern = grouped_kernel<kMode, kOut>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem) != cudaSuccess)
    return 0;
  // (the register split of the weights' kernels waits for ever in a launch with fewer)
  cudaFuncAttributes fa;
  if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess ||
      (kMode == kWeights && fa.numRegs * kThreads < 40 * kEpiWarp0 * 32 + 232 * kEpiWarps * 32))
    return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * num_sms());
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kMaxSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) return 0;
  return cache[dev] = n;
}

template <int kMode, int kOut>
cudaError_t launch(const Maps<kMode>& m, Params& p, long long units, cudaStream_t s) {
  const int pairs = pairs_resident<kMode, kOut>();
  if (pairs < 1) return cudaErrorInvalidConfiguration;
  p.err = device_error_word();
  if (!p.err) return cudaErrorInvalidValue;
  const size_t other = other_smem(kMode, p.E);
  p.stages = (int)((kMaxSmem - other) / p.stage_bytes);
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  return launch_k_cluster(grouped_kernel<kMode, kOut>, dim3(2 * (unsigned)(units < pairs ? units : pairs)),
                          dim3(kThreads), other + (size_t)p.stages * p.stage_bytes, s, 2, m, p);
}

// Whether few rows stream through registers (grouped_stream.cu), by what both forms take in
// microseconds if every row has an expert of its own (the offsets are on the device).  That form:
// its CTAs, then the weights at 4.4 TB/s.  Here: the launch and a unit's K blocks one after another,
// or the weights at 6.2 TB/s.  Measured, stream / here, rows of different experts:
//   forward 1024 x 2048:  1 row 4.8 / 12.2, 8 rows 8.6 / 12.5, 16 rows 16.2 / 16.0
//   forward 2048 x 512:   1 row 2.8 / 7.2,  8 rows 5.8 / 7.6,  16 rows 11.7 / 10.3
//   rows    1024 x 2048:  1 row 5.3 / 9.2,  4 rows 5.6 / 9.4,  8 rows 10.8 / 9.7
//   rows    2048 x 512:   1 row 5.6 / 12.1, 16 rows 10.1 / 12.5, 32 rows 19.2 / 16.2
//   forward 256 x 128:    1 row 2.0 / 5.0,  128 rows of 16 experts 4.1 / 5.1, 256 rows 5.8 / 5.2
bool streams(const GroupedLinear& g, bool backward) {
  const long long ctas = grouped_stream_ctas(g, backward);
  if (ctas > 4096) return false;
  const double bytes = 2.0 * (double)(g.R < g.E ? g.R : g.E) * g.N * g.K;
  const double few = 2.2 + 0.0009 * (double)ctas + bytes / 4.4e6;
  const double latency = 5.3 + 0.0035 * (backward ? g.N : g.K), stream = bytes / 6.2e6;
  return few < (latency > stream ? latency : stream);
}

}  // namespace

cudaError_t launch_grouped_linear(const GroupedLinear& g, bool backward, cudaStream_t s) {
  if (streams(g, backward)) return launch_grouped_stream(g, backward, s);
  Params p{};
  p.E = g.E;
  p.mdim = backward ? g.K : g.N;
  p.depth = backward ? g.N : g.K;
  p.mtiles = ceil_div(p.mdim, kTile);
  // Most token rows of a tile: with few rows an expert, smaller token boxes leave room for eight stages
  // of weights, not six (896 experts of 1024 x 2048, 128 / 256 rows: 16384 rows 560 / 575 us, 65536 rows
  // 604 / 619; 128 experts of 2048 x 512: 8192 rows 52 / 54, 32768 rows 102 / 78.  32 and 64 were behind
  // one of the two everywhere.)
  p.nt = g.R <= 96ll * g.E ? 128 : 256;
  p.stage_bytes = kABytes + (uint32_t)p.nt * 64;
  p.R = g.R;
  p.offsets = g.offsets;
  p.out = g.rows_out;
  CUtensorMap a, b, part;
  if (!make_map(&a, g.w, false, g.E, g.N, g.K, backward ? kBK : kHalf) ||
      !make_map(&b, g.rows_in, false, 0, g.R, p.depth, p.nt / 2) ||
      !make_map(&part, g.rows_in, false, 0, g.R, p.depth, kPartBox))
    return cudaErrorInvalidValue;
  // token tiles: one a started nt rows and expert at most
  const long long units = (g.R / p.nt + (g.R < g.E ? g.R : g.E)) * p.mtiles;
  return backward ? launch<kRows, 0>({a, b, a, {part}}, p, units, s)
                  : launch<kForward, 0>({a, b, a, {part}}, p, units, s);
}

cudaError_t launch_grouped_weight_grad(const GroupedWeightGrad& g, cudaStream_t s) {
  Params p{};
  p.E = g.E;
  p.mdim = g.N;
  p.ncols = g.K;
  p.mtiles = ceil_div(g.N, kTile);
  p.ntiles = ceil_div(g.K, kTile);
  p.stage_bytes = 2 * kABytes;
  p.R = g.R;
  p.offsets = g.offsets;
  p.add = g.add;
  Maps<kWeights> m;
  const bool fp32 = g.dw != nullptr;
  bool ok = make_map(&m.a, g.dy, false, 0, g.R, g.N, kBK) && make_map(&m.b, g.x, false, 0, g.R, g.K, kBK) &&
            make_map(&m.o, fp32 ? (const void*)g.dw : g.dw_bf16, fp32, g.E, g.N, g.K, 32);
  for (int i = 0; ok && i < 3; ++i)
    ok = make_map(&m.part[2 * i], g.dy, false, 0, g.R, g.N, 16 >> 2 * i) &&
         make_map(&m.part[2 * i + 1], g.x, false, 0, g.R, g.K, 16 >> 2 * i);
  if (!ok) return cudaErrorInvalidValue;
  const long long units = (long long)p.E * p.mtiles * p.ntiles;
  if (!fp32) return launch<kWeights, 1>(m, p, units, s);
  return p.add ? launch<kWeights, 2>(m, p, units, s) : launch<kWeights, 0>(m, p, units, s);
}

}  // namespace lmoe
