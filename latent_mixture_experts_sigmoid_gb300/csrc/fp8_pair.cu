// Block-scaled e4m3 products on pairs of SMs (fp8.cu has the formula and the form
// for one SM).
//
// A tile of 128 x 256 on one SM moves 48 KB of operands through its shared memory per
// K block of 512 tensor cycles, once in from L2 and once out to the tensor core.  Here the
// two CTAs of a cluster compute one 256 x 256 tile (tcgen05 cta_group::2, M = 256, N = 256):
// each brings in its own 128 token rows and 128 of the weight rows, 32 KB a block, and the
// tensor cores of both read both halves.
//
// Bound by the epilogue: a K block must leave TMEM and be scaled before the accumulator takes
// the next but one (about 930 cycles a block; sixteen epilogue warps of half the columns each
// took longer, two accumulators of N = 128 per half too).  [4096, 7168] x [8192, 7168]: 188 us,
// 2.56 PFLOP/s, tensor pipe 55 % busy; the one-SM form takes 202.
//
//   warp 0      TMA producer of this CTA's halves; their bytes count on the leader's
//               (rank 0's) barrier;
//   warp 1      allocates TMEM; in the leader one thread issues the MMAs of both CTAs,
//               and its commits arrive in both;
//   warp 2      brings the token rows' scales into shared memory, K block by K block;
//   warps 4..11 read the finished K block of this CTA's 128 rows from TMEM, scale and add
//               it in registers, and write the tile (warp w: the 32 rows of lane quarter
//               w % 4, half (w - 4) / 4 of the columns).
// Every wait is bounded; neither CTA leaves or frees its TMEM before both are done.
#include <cuda.h>

#include <mutex>

#include "fp8.cuh"
#include "fp8_epilogue.cuh"
#include "tc_ptx.cuh"

namespace lmoe {
namespace {

constexpr int kEpiWarp0 = 4, kEpiWarps = 8;
constexpr int kThreads = (kEpiWarp0 + kEpiWarps) * 32;
constexpr int kHalf = 128;                         // token and weight rows of one CTA
constexpr int kTile = 2 * kHalf;
constexpr int kBK = 128;
constexpr uint32_t kBoxBytes = kHalf * kBK;
constexpr uint32_t kStageBytes = 2 * kBoxBytes;    // of one CTA
constexpr int kStages = 6;
constexpr int kAcc = 2;                            // TMEM accumulators of 256 columns
constexpr int kScaleBlocks = 16, kScaleBuffers = 2, kScaleStride = kHalf + 4;
constexpr int kBand = 8;                           // feature tiles of a band of the walk
enum : int { kErrProducer = 1, kErrMmaFull = 2, kErrMmaTmem = 3, kErrEpilogue = 4,
             kErrDrain = 5, kErrDone = 6 };        // device error word codes

struct PairParams {
  int T, feat, nkb, nfeat, ntok, ws_rows;
  int wide_store, wide_add;    // rows of out / of add start on 32 bytes
  const float* xs;
  const float* ws;
  const uint16_t* add;
  uint16_t* out;
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

__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// K-major operand, 128-byte rows with the 128-byte swizzle, 8-row groups 1024 bytes apart
__device__ __forceinline__ uint64_t sdesc(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// kind::f8f6f4: fp32 accumulator, e4m3 A and B, both K-major, M = N = 256
constexpr uint32_t kIdesc = (1u << 4) | ((uint32_t)(kTile >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);

// Tile u of the walk: bands of kBand feature tiles, inside a band the feature tile
// changing fastest, so that the tiles under way share their operands in L2.
__device__ __forceinline__ int2 tile_of(const PairParams& p, int u) {
  const int band = min(u / (p.ntok * kBand), (p.nfeat - 1) / kBand);
  const int rem = u - band * p.ntok * kBand;
  const int width = min(kBand, p.nfeat - band * kBand);
  const int t = rem / width;
  return make_int2(t, band * kBand + rem - t * width);
}

// kAdd: with an addend (an instance of its own: the branch cost the other 2 %)
template <bool kAdd>
__global__ void __launch_bounds__(kThreads, 1)
fp8_pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                const PairParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  float* tok_scale = reinterpret_cast<float*>(smem + kStages * kStageBytes);   // [buffer][K block][row]
  uint64_t* bars = reinterpret_cast<uint64_t*>(tok_scale + kScaleBuffers * kScaleBlocks * kScaleStride);
  constexpr int kFull = 0, kEmpty = kStages, kTfull = 2 * kStages, kTempty = kTfull + kAcc,
                kDone = kTempty + kAcc, kSfull = kDone + 1, kSempty = kSfull + kScaleBuffers,
                kBars = kSempty + kScaleBuffers;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bar0 = smem_u32(bars);
  auto bar_at = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  const uint32_t rank = cluster_rank();

  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar_at(kFull + i), 1);
      mbar_init(bar_at(kEmpty + i), 1);
    }
    for (int i = 0; i < kAcc; ++i) {
      mbar_init(bar_at(kTfull + i), 1);
      mbar_init(bar_at(kTempty + i), 2 * kEpiWarps);    // (the leader's: both CTAs' epilogues)
    }
    mbar_init(bar_at(kDone), 1);
    for (int i = 0; i < kScaleBuffers; ++i) {
      mbar_init(bar_at(kSfull + i), 32);
      mbar_init(bar_at(kSempty + i), kEpiWarps);
    }
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
  tc_fence_before();
  __syncthreads();
  cluster_sync();      // both CTAs' barriers are there before any copy or commit reaches them
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const int U = p.ntok * p.nfeat;
  const int u0 = (int)(blockIdx.x >> 1), ustep = (int)(gridDim.x >> 1);

  // the launch's 168 registers a thread, split anew: 168 * 384 = 40 * 128 + 232 * 256
  // (216 an epilogue thread: 195 us for [4096, 7168] x [8192, 7168], 232: 187)
  if (warp < kEpiWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0 && lane == 0) {
      // ---------------- TMA producer ----------------
      int s = 0;
      uint32_t ph = 0, it = 0;
      bool ok = true;
      for (int u = u0; u < U && ok; u += ustep) {
        const int2 x = tile_of(p, u);
        const int row = x.x * kTile + (int)rank * kHalf, w = x.y * kTile + (int)rank * kHalf;
        for (int kb = 0; kb < p.nkb; ++kb, ++it) {
          if (!wait_phase(bar_at(kEmpty + s), ph ^ 1u, abort_flag, p.err, kErrProducer)) { ok = false; break; }
          if (rank == 0) mbar_arrive_expect_tx(bar_at(kFull + s), 2 * kStageBytes);
          const uint32_t bar = cluster_addr(bar_at(kFull + s), 0);
          const uint32_t at = smem_u32(smem) + (uint32_t)s * kStageBytes;
          // (rows past the last read as zeros)
          tma_load_pair(&tmX, at, bar, kb * kBK, row);
          tma_load_pair(&tmW, at + kBoxBytes, bar, kb * kBK, w);
          if (++s == kStages) { s = 0; ph ^= 1u; }
        }
      }
      // the leader: every copy of the pair has landed before the CTAs exit
      if (rank == 0)
        for (uint32_t j = it > kStages ? it - kStages : 0u; j < it; ++j) {
          volatile int never = 0;
          if (!wait_phase(bar_at(kFull + (int)(j % kStages)), (j / kStages) & 1u, &never, p.err, kErrDrain))
            break;
        }
    } else if (warp == 1 && lane == 0 && rank == 0) {
      // ---------------- MMA issuer of the pair ----------------
      const uint64_t d0 = sdesc(smem_u32(smem));
      int s = 0;
      uint32_t ph = 0, acc = 0, aph = 0;
      bool ok = true;
      for (int u = u0; u < U && ok; u += ustep) {
        for (int kb = 0; kb < p.nkb; ++kb) {
          if (!wait_phase(bar_at(kTempty + (int)acc), aph ^ 1u, abort_flag, p.err, kErrMmaTmem) ||
              !wait_phase(bar_at(kFull + s), ph, abort_flag, p.err, kErrMmaFull)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t da = d0 + (uint64_t)s * (kStageBytes >> 4);
          const uint64_t db = da + (kBoxBytes >> 4);
#pragma unroll
          for (int j = 0; j < kBK / 32; ++j)
            mma_pair(tmem_base + acc * kTile, da + 2 * j, db + 2 * j, kIdesc, j ? 1u : 0u);
          commit_both(bar_at(kEmpty + s));
          commit_both(bar_at(kTfull + (int)acc));
          if (++s == kStages) { s = 0; ph ^= 1u; }
          if (++acc == kAcc) { acc = 0; aph ^= 1u; }
        }
      }
      // every MMA this thread issued has completed before TMEM is freed
      asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                       bar_at(kDone))
                   : "memory");
      volatile int never = 0;
      wait_phase(bar_at(kDone), 0u, &never, p.err, kErrDone);
    } else if (warp == 2) {
      // ---------------- token scales ----------------
      int buf = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int u = u0; u < U && ok; u += ustep) {
        const int row0 = tile_of(p, u).x * kTile + (int)rank * kHalf;
        const int rows = min(kHalf, p.T - row0);
        const float* src = p.xs + (long long)row0 * p.nkb;
        for (int kb = 0; kb < p.nkb; kb += kScaleBlocks) {
          ok = __all_sync(0xFFFFFFFFu, wait_phase(bar_at(kSempty + buf), ph ^ 1u, abort_flag, p.err, kErrProducer));
          if (!ok) break;
          // a lane: one of the K blocks of every fourth row (eight lanes: a row's sector)
#pragma unroll
          for (int k8 = 0; k8 < kScaleBlocks; k8 += 8) {
            const int k = kb + k8 + (lane & 7);
            if (k < p.nkb) {
              uint32_t dst =
                  smem_u32(tok_scale + (buf * kScaleBlocks + k8 + (lane & 7)) * kScaleStride + (lane >> 3));
              for (int r = lane >> 3; r < rows; r += 4, dst += 16u)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst),
                             "l"(src + (long long)r * p.nkb + k)
                             : "memory");
            }
          }
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar_at(kSfull + buf))
                       : "memory");
          if (++buf == kScaleBuffers) { buf = 0; ph ^= 1u; }
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    // ---------------- epilogue ----------------
    const int q = warp & 3;                      // TMEM lane quarter this warp may access
    const int h = (warp - kEpiWarp0) >> 2;       // column half: one block of weight scales
    const int r = q * 32 + lane;                 // token row of this CTA's half
    const uint32_t tempty = cluster_addr(bar_at(kTempty), 0);
    const uint32_t tmem = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(h * kHalf);
    uint32_t acc = 0, aph = 0, sph = 0;
    int sbuf = 0;
    bool ok = true;
    for (int u = u0; u < U && ok; u += ustep) {
      const int2 x = tile_of(p, u);
      const int row0 = x.x * kTile + (int)rank * kHalf;
      const int blk = min(x.y * 2 + h, p.ws_rows - 1);
      const float* wsp = p.ws + (long long)blk * p.nkb;
      f32x2 y[kHalf / 2];
#pragma unroll
      for (int i = 0; i < kHalf / 2; ++i) y[i] = 0ull;
      if constexpr (kAdd) {
        add_first<kHalf>(y, p.add + (long long)min(row0 + r, p.T - 1) * p.feat,
                         x.y * kTile + h * kHalf, p.feat, p.wide_add);
        if (u + ustep < U) {
          const int2 n = tile_of(p, u + ustep);
          const int row = n.x * kTile + (int)rank * kHalf + r;
          if (row < p.T)
            prefetch_addend<kHalf>(p.add + (long long)row * p.feat, n.y * kTile + h * kHalf, p.feat);
        }
      }
      float nw = __ldg(wsp);                     // a K block's scale is loaded one block ahead
      for (int kb0 = 0; kb0 < p.nkb && ok; kb0 += kScaleBlocks) {
        // (a wait's outcome is one for the warp, whose lanes meet again below)
        ok = __all_sync(0xFFFFFFFFu, wait_phase(bar_at(kSfull + sbuf), sph, abort_flag, p.err, kErrEpilogue));
        if (!ok) break;
        const float* sp = tok_scale + sbuf * kScaleBlocks * kScaleStride + r;
        const int kb1 = min(kb0 + kScaleBlocks, p.nkb);
        for (int kb = kb0; kb < kb1; ++kb, sp += kScaleStride) {
          const f32x2 f = f2_splat(*sp * nw);
          nw = __ldg(wsp + min(kb + 1, p.nkb - 1));
          ok = __all_sync(0xFFFFFFFFu, wait_phase(bar_at(kTfull + (int)acc), aph, abort_flag, p.err, kErrEpilogue));
          if (!ok) break;
          tc_fence_after();
          // A load waits for the MMA that the tensor core is at, whatever its width: two of 64
          // columns cost half of what four of 32 do.
#pragma unroll
          for (int i = 0; i < kHalf / 64; ++i) {
            uint32_t v[64];
            tmem_ld64(tmem + acc * kTile + i * 64, v);
            tmem_wait_ld64(v);
            if (i == kHalf / 64 - 1) {           // the accumulator is free ahead of the last sums
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_cluster(tempty + 8u * acc);
            }
#pragma unroll
            for (int j = 0; j < 32; ++j)
              y[i * 32 + j] = f2_fma(f2_make(v[2 * j], v[2 * j + 1]), f, y[i * 32 + j]);
          }
          if (++acc == kAcc) { acc = 0; aph ^= 1u; }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_at(kSempty + sbuf));
        if (++sbuf == kScaleBuffers) { sbuf = 0; sph ^= 1u; }
      }
      if (!ok) break;
      const int row = row0 + r, col0 = x.y * kTile + h * kHalf;
      const int ncol = row < p.T ? min(kHalf, p.feat - col0) : 0;    // a multiple of 8
      const long long at = (long long)row * p.feat + col0;
#pragma unroll
      for (int j = 0; j < kHalf / 2; j += 8) {   // 16 columns: 32 bytes
        if (2 * j >= ncol) break;
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(f2_lo(y[j + i]), f2_hi(y[j + i]));
        if (p.wide_store) {
          st_global32(p.out + at + 2 * j, w);
        } else {
          *reinterpret_cast<uint4*>(p.out + at + 2 * j) = make_uint4(w[0], w[1], w[2], w[3]);
          if (2 * j + 8 < ncol)
            *reinterpret_cast<uint4*>(p.out + at + 2 * j + 8) = make_uint4(w[4], w[5], w[6], w[7]);
        }
      }
      __syncwarp();
    }
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

// byte matrix [rows, K] in boxes of [128][128 bytes], 128-byte swizzle; bytes outside it
// read as zeros
bool make_map(CUtensorMap* m, const void* base, long long rows, int K) {
  const EncodeTiledFn enc = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)K};
  cuuint32_t box[2] = {(cuuint32_t)kBK, (cuuint32_t)kHalf};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr size_t kSmem = 1024 + kStages * kStageBytes +
                         kScaleBuffers * kScaleBlocks * kScaleStride * sizeof(float) +
                         (2 * kStages + 2 * kAcc + 1 + 2 * kScaleBuffers) * 8 + 8;

// Pairs that fit on the current device at once (pairs share a GPC), 0 on failure.
template <bool kAdd>
int pairs_resident() {
  static int cache[64] = {};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (cache[dev]) return cache[dev];
  auto* kern = fp8_pair_kernel<kAdd>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem) != cudaSuccess)
    return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * num_sms());
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
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

template <bool kAdd>
cudaError_t launch_pair(const CUtensorMap& mx, const CUtensorMap& mw, const PairParams& p, cudaStream_t s) {
  const int pairs = pairs_resident<kAdd>();
  if (pairs < 1) return cudaErrorInvalidConfiguration;
  const long long units = (long long)p.ntok * p.nfeat;
  return launch_k_cluster(fp8_pair_kernel<kAdd>, dim3(2 * (unsigned)(units < pairs ? units : pairs)),
                          dim3(kThreads), kSmem, s, 2, mx, mw, p);
}

}  // namespace

cudaError_t launch_fp8_pair(const Fp8Gemm& g, cudaStream_t s) {
  PairParams p{};
  p.T = (int)g.rows;
  p.feat = g.feat;
  p.nkb = fp8_blocks(g.K);
  p.nfeat = ceil_div(g.feat, kTile);
  p.ntok = ceil_div(g.rows, kTile);
  p.ws_rows = fp8_blocks(g.feat);
  p.wide_store = g.feat % 16 == 0 && (reinterpret_cast<uintptr_t>(g.out) & 31u) == 0;
  p.wide_add = g.feat % 16 == 0 && (reinterpret_cast<uintptr_t>(g.add) & 31u) == 0;
  p.xs = g.xs;
  p.ws = g.ws;
  p.add = g.add;
  p.out = g.out;
  p.err = device_error_word();
  CUtensorMap mx, mw;
  if (!p.err || !make_map(&mx, g.X, g.rows, g.K) || !make_map(&mw, g.W, g.feat, g.K))
    return cudaErrorInvalidValue;
  return g.add ? launch_pair<true>(mx, mw, p, s) : launch_pair<false>(mx, mw, p, s);
}

}  // namespace lmoe
