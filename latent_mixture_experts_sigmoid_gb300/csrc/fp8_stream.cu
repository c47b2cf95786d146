// Block-scaled e4m3 products for a few token rows (fp8.cu has the formula and the
// tensor-core kernel for many).
//
// With up to 16 tokens a product is the streaming of its weights: 2 T flops a byte.  The
// 128 x 128 tiles of the other kernel are too coarse for that (a product of 2048 weight
// rows has 16 of them for 152 SMs) and a K block passes through TMEM and four barriers
// there.  Here a persistent CTA on each SM takes units of kRows weight rows and up to
// 8 NT tokens.  Its warps form groups, each with units of its own, so that one group's
// epilogue and the latencies before its products fall into the others' streaming:
//   a producer warp  keeps the group's ring of stages filled by TMA, across unit
//                boundaries: 128 K columns of the unit's weight rows and of its tokens
//                (about 160 KB are under way per SM);
//   kGroupWarps consumer warps take the K blocks in turn, multiply them with
//                warp-level MMAs (m16n8k32, weights on M, tokens on N) and add them with
//                their scales in registers; the group sums its warps' parts through
//                shared memory in warp order and applies the epilogue.
// A K block's columns go to the MMAs' k indexes in the order in which 16-byte reads
// bring them (lane c of a row's four has bytes 16 c .. 16 c + 15 of each half): the
// same for both operands, so it drops out of the sum.
//
// Bound by the weights' bytes once there are enough of them: 128 rows over 96 of 896 experts
// (the mean of four batches), latent 2048, inter 512, both products 55.5 us (303 MB, 5.5 TB/s;
// 45 us at the copy bandwidth, the rest is mostly the two launches' ends and first loads).  A
// dense product of a few microseconds is its launch, one memory latency and its bytes:
// [1, 7168] x [2048, 7168] 5.5 us, 5.0 with its weights in L2 (14.7 MB, 2.2 us at full rate), 9.5
// on the tensor-core kernel with its K split four ways; [8, 7168] x [8192, 7168] 13.7 us
// (58.8 MB, 4.3 TB/s), 15.4 there.
#include <cuda.h>

#include "fp8.cuh"
#include "fp8_quant.cuh"
#include "tc_ptx.cuh"

namespace lmoe {
namespace {

enum : int {
  kDense = 0,     // out = bf16(x W^T + add)
  kGateUp = 1,    // experts' first product: act = SituGLU(x W13^T), fp32
  kSecond = 2     // experts' second product: out = bf16(q(act) W2^T)
};

struct StreamParams {
  const float* xs;           // [rows, nkb] (not kSecond)
  const float* act;          // kSecond: fp32 [rows, K]
  const float* ws;           // [groups, ws_rows, nkb]
  const uint16_t* add;
  uint16_t* out;             // [rows, feat]
  float* act_out;            // kGateUp: fp32 [rows, feat / 2]
  const int32_t* offsets;    // grouped: [groups + 1]
  int rows, feat, K, nkb, ws_rows, groups, stages;
  int max_rows;              // experts of more rows are another kernel's
  int beside;                // kGateUp: see Fp8Gemm
  int* err;
  SituParams sp;
};

constexpr int kConsumers = 16;                 // consumer warps of a CTA, in kGroups groups
constexpr int kProducers = 4;                  // producer warps, likewise
constexpr int kMaxExperts = 1024;
constexpr long long kWaitCycles = 1ll << 32;   // ~2 s at 2 GHz
enum : int { kErrProducer = 1, kErrConsumer = 4, kErrDrain = 5 };   // device error word codes

__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag,
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

__device__ __forceinline__ void mma_k32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16-byte chunk `chunk` of row `row` of a box of 128-byte rows with the 128-byte swizzle
__device__ __forceinline__ uint4 ld_chunk(const uint8_t* box, int row, int chunk) {
  return *reinterpret_cast<const uint4*>(box + row * 128 + ((chunk ^ (row & 7)) << 4));
}

// The experts that have rows (up to max_rows), in expert order (clamped to the rows there are).
struct ExpertList {
  uint16_t* id;
  int* first;
  int* count;
};
template <int kThreads>
__device__ int build_list(const StreamParams& p, const ExpertList& l, int* warp_sum) {
  constexpr int kPer = (kMaxExperts + kThreads - 1) / kThreads;
  const int g0 = threadIdx.x * kPer, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int a[kPer], n[kPer], has = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    n[i] = 0;
    if (g0 + i < p.groups) {
      a[i] = min(max(__ldg(p.offsets + g0 + i), 0), p.rows);
      n[i] = min(max(__ldg(p.offsets + g0 + i + 1), a[i]), p.rows) - a[i];
      if (n[i] > p.max_rows) n[i] = 0;
    }
    has += n[i] > 0;
  }
  int incl = has;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int at = incl - has, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) at += warp_sum[w];
    total += warp_sum[w];
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (n[i] > 0) {
      l.id[at] = (uint16_t)(g0 + i);
      l.first[at] = a[i];
      l.count[at++] = n[i];
    }
  return total;
}

// One unit's pass over the weights: kRows weight rows, up to 8 NT tokens.
struct Item {
  int e;        // expert
  int f0;       // first feature
  int row0;     // first token row
  int nt;       // tokens
};

// A group's items in order: units from `u` on, `step` apart; feature blocks change
// fastest, so that CTAs side by side share their tokens; an expert with more than
// 8 NT tokens has its weights passed over again (from L2) for each further 8 NT.
template <int kTok, int kMode>
struct Walk {
  int u, step, units, nfb, t0 = 0;
  int feats;    // output features of a unit
  const StreamParams& p;
  const ExpertList& l;
  __device__ __forceinline__ Walk(const StreamParams& p, const ExpertList& l, int u, int step,
                                  int units, int nfb, int feats)
      : u(u), step(step), units(units), nfb(nfb), feats(feats), p(p), l(l) {}
  __device__ __forceinline__ bool done() const { return u >= units; }
  __device__ __forceinline__ Item item() const {
    const int i = u / nfb;
    Item x;
    x.f0 = (u - i * nfb) * feats;
    if (kMode == kDense) {
      x.e = 0;
      x.row0 = i * kTok;
      x.nt = min(kTok, p.rows - x.row0);
    } else {
      x.e = l.id[i];
      x.row0 = l.first[i] + t0;
      x.nt = min(kTok, l.count[i] - t0);
    }
    return x;
  }
  __device__ __forceinline__ void next() {
    if (kMode != kDense) {
      t0 += kTok;
      if (t0 < l.count[u / nfb]) return;
      t0 = 0;
    }
    u += step;
  }
};

// kRows: weight rows of a unit (kGateUp: half of them gate, half up rows).
// kKB: K blocks of a stage (over 1: K % 128 == 0).  A producer's thread takes about
// 470 cycles a stage (waits, copies), so the stages of one group, 3 KB a K block at 16
// rows, hold four blocks and have four producers.
template <int kRows, int NT, int kMode, int kGroups, int kKB>
__global__ void __launch_bounds__((kConsumers + kProducers) * 32, 1)
fp8_stream_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                  const StreamParams p) {
  constexpr int kThreads = (kConsumers + kProducers) * 32;
  constexpr int kGroupWarps = kConsumers / kGroups, kGroupProducers = kProducers / kGroups;
  constexpr int MT = kRows / 16;
  constexpr int kTok = 8 * NT;
  constexpr uint32_t kWBytes = kRows * 128, kXBytes = kMode == kSecond ? 0 : kTok * 128;
  constexpr uint32_t kStage = kKB * (kWBytes + kXBytes);   // the blocks' weight boxes, then the tokens'
  constexpr int kPartStride = kRows + 4;         // floats of a token's partial sums
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t S = (uint32_t)p.stages;        // of a group's ring: a multiple of kGroupWarps
  float* part = reinterpret_cast<float*>(smem + (size_t)kGroups * S * kStage);   // [group][warp][kTok][stride]
  uint64_t* bars = reinterpret_cast<uint64_t*>(part + kGroups * kGroupWarps * kTok * kPartStride);
  int* warp_sum = reinterpret_cast<int*>(bars + 2 * kGroups * S);
  volatile int* abort_flag = warp_sum + kThreads / 32;
  ExpertList list;
  list.first = warp_sum + kThreads / 32 + 1;
  list.count = list.first + kMaxExperts;
  list.id = reinterpret_cast<uint16_t*>(list.count + kMaxExperts);

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cw = warp - kProducers;             // the first warps are the producers
  const int group = cw < 0 ? warp / kGroupProducers : cw / kGroupWarps;
  const uint32_t bar0 = smem_u32(bars + 2 * group * S);
  auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (S + s); };
  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < 2 * kGroups * S; ++s) mbar_init(smem_u32(bars + s), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  // The first product triggers the second only after its own wait, so by then
  // everything before the first is complete: the second reads its weights, their
  // scales and the offsets, none of which the first writes, ahead of its wait.
  if (kMode == kDense || (kMode == kGateUp && !p.beside)) pdl_wait();
  pdl_trigger();
  const int feats = kMode == kGateUp ? kRows / 2 : kRows;
  const int nfb = kMode == kDense ? (p.feat - 1) / kRows + 1 : p.feat / kRows;
  int units = nfb;
  if (kMode == kDense) units *= (p.rows + kTok - 1) / kTok;
  else units *= build_list<kThreads>(p, list, warp_sum);
  __syncthreads();
  // groups of different SMs before groups of the same: an SM more or less has a unit more
  Walk<kTok, kMode> walk(p, list, group * (int)gridDim.x + (int)blockIdx.x, kGroups * (int)gridDim.x,
                         units, nfb, feats);
  uint8_t* ring = smem + (size_t)group * S * kStage;

  if (cw < 0) {
    if (lane == 0) {
      // ---------------- TMA producer ----------------
      // a group's producers take its stages in turn
      const uint32_t turn = (uint32_t)(warp % kGroupProducers);
      uint32_t it = 0;
      bool ok = true;
      for (; !walk.done() && ok; walk.next()) {
        const Item x = walk.item();
        const int w0 = x.e * p.feat + x.f0;
        for (int kb = 0; kb < p.nkb; kb += kKB, ++it) {
          if (it % kGroupProducers != turn) continue;
          const uint32_t s = it % S;
          if (!wait_phase(empty_bar(s), (it / S & 1u) ^ 1u, abort_flag, p.err, kErrProducer)) {
            ok = false;
            break;
          }
          const uint32_t bar = full_bar(s), at = smem_u32(ring) + s * kStage;
          mbar_arrive_expect_tx(bar, kStage);
          // blocks past the last read as zeros
          const int k0 = kKB > 1 ? 0 : kb * 128, kz = kKB > 1 ? kb : 0;
          tma_load_3d(&tmW, at, bar, k0, w0, kz);
          if (kMode != kDense)
            tma_load_3d(&tmW, at + kWBytes / 2, bar, k0,
                        w0 + (kMode == kGateUp ? p.feat / 2 : kRows / 2), kz);
          if (kMode != kSecond) tma_load_3d(&tmX, at + kKB * kWBytes, bar, k0, x.row0, kz);
        }
      }
      // every copy this thread issued has landed before the CTA exits
      for (uint32_t j = it > S ? it - S : 0u; j < it; ++j) {
        volatile int never = 0;
        if (j % kGroupProducers == turn &&
            !wait_phase(full_bar(j % S), (j / S) & 1u, &never, p.err, kErrDrain))
          break;
      }
    }
  } else {
    // ---------------- consumers ----------------
    const int kw = cw % kGroupWarps;
    const int g = lane >> 2, c = lane & 3;
    float* gpart = part + group * kGroupWarps * kTok * kPartStride;
    if (kMode == kSecond) pdl_wait();
    bool ok = true;
    // Stage number of the item's first.  Stages go to the warps in turn, and
    // the ring is a multiple of their number: a slot is always the same warp's, which
    // so meets all of its phases (a barrier tells a phase from the next only).
    const int nst = (p.nkb + kKB - 1) / kKB;
    uint32_t base = 0;
    for (; !walk.done(); walk.next(), base += (uint32_t)nst) {
      const int st0 = (int)((kw - base) % kGroupWarps);
      const Item x = walk.item();
      const float* wsp = p.ws + ((long long)x.e * p.ws_rows + x.f0 / kFp8Block) * p.nkb;
      const float* wsp2 = wsp + (long long)(p.ws_rows / 2) * p.nkb;      // kGateUp: the up rows'
      const float* xsp = p.xs + (long long)x.row0 * p.nkb;
      const float* act = p.act + (long long)x.row0 * p.K;
      float y[MT][NT][4] = {};
      // a stage's scales, loaded a turn ahead
      float nw[kKB] = {}, nw2[kKB] = {}, nx[kKB][NT][2] = {};
      auto scales = [&](int st) {
#pragma unroll
        for (int i = 0; i < kKB; ++i) {
          const int kb = st * kKB + i;
          if (kb >= p.nkb) continue;
          nw[i] = __ldg(wsp + kb);
          if (kMode == kGateUp) nw2[i] = __ldg(wsp2 + kb);
          if (kMode != kSecond) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const int tok = t * 8 + c * 2 + j;
                nx[i][t][j] = tok < x.nt ? __ldg(xsp + tok * p.nkb + kb) : 0.0f;
              }
          }
        }
      };
      scales(st0);
      for (int st = st0; st < nst; st += kGroupWarps) {
        const uint32_t it = base + (uint32_t)st, s = it % S;
        float fw[kKB], fw2[kKB], fx[kKB][NT][2];
#pragma unroll
        for (int i = 0; i < kKB; ++i) {
          fw[i] = nw[i];
          fw2[i] = nw2[i];
#pragma unroll
          for (int t = 0; t < NT; ++t) { fx[i][t][0] = nx[i][t][0]; fx[i][t][1] = nx[i][t][1]; }
        }
        scales(st + kGroupWarps);
        const uint8_t* wbox = ring + (size_t)s * kStage;
        uint4 b[NT][2];
        if (kMode == kSecond) {
          const int kb = st;
          // a token's 128 activations of the block, 32 in each lane of its four
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            float4 v[8];
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              if (t * 8 + g < x.nt)
                v[j] = __ldcg(reinterpret_cast<const float4*>(
                    act + (t * 8 + g) * p.K + kb * 128 + (j >> 2) * 64 + c * 16 + (j & 3) * 4));
              m = max(m, max(max(abs_bits(v[j].x), abs_bits(v[j].y)),
                             max(abs_bits(v[j].z), abs_bits(v[j].w))));
            }
            m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
            m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
            const BlockScale bs = block_scale(m);
            uint32_t q[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
              q[j] = pack_e4m3x4(__fmul_rn(v[j].x, bs.inv), __fmul_rn(v[j].y, bs.inv),
                                 __fmul_rn(v[j].z, bs.inv), __fmul_rn(v[j].w, bs.inv));
            b[t][0] = make_uint4(q[0], q[1], q[2], q[3]);
            b[t][1] = make_uint4(q[4], q[5], q[6], q[7]);
            // the scale of token 2 c + j is in the lanes of row 2 c + j
#pragma unroll
            for (int j = 0; j < 2; ++j) fx[0][t][j] = __shfl_sync(0xFFFFFFFFu, bs.scale, (c * 2 + j) * 4);
          }
        }
        if (ok) ok = wait_phase(full_bar(s), (it / S) & 1u, abort_flag, p.err, kErrConsumer);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) continue;                      // (the group's barriers below are still met)
#pragma unroll
        for (int i = 0; i < kKB; ++i) {
          if (kKB > 1 && st * kKB + i >= p.nkb) break;
          const uint8_t* xbox = wbox + kKB * kWBytes + i * kXBytes;
          if (kMode != kSecond) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              b[t][0] = ld_chunk(xbox, t * 8 + g, c);
              b[t][1] = ld_chunk(xbox, t * 8 + g, 4 + c);
            }
          }
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            uint4 r0[2], r1[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              r0[h] = ld_chunk(wbox + i * kWBytes, m * 16 + g, h * 4 + c);
              r1[h] = ld_chunk(wbox + i * kWBytes, m * 16 + 8 + g, h * 4 + c);
            }
            const float f = kMode == kGateUp && m >= MT / 2 ? fw2[i] : fw[i];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                mma_k32(sum, r0[h].x, r1[h].x, r0[h].y, r1[h].y, b[t][h].x, b[t][h].y);
                mma_k32(sum, r0[h].z, r1[h].z, r0[h].w, r1[h].w, b[t][h].z, b[t][h].w);
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) y[m][t][j] = fmaf(sum[j], fx[i][t][j & 1] * f, y[m][t][j]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty_bar(s));
      }
      // the group's sum and the epilogue
      float* mine = gpart + kw * kTok * kPartStride;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mine[(t * 8 + c * 2 + (j & 1)) * kPartStride + m * 16 + (j >> 1) * 8 + g] = y[m][t][j];
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kGroupWarps * 32) : "memory");
      auto sum = [&](int t, int f) {
        float v = gpart[t * kPartStride + f];
#pragma unroll
        for (int k = 1; k < kGroupWarps; ++k) v += gpart[(k * kTok + t) * kPartStride + f];
        return v;
      };
      for (int o = kw * 32 + lane; o < feats * x.nt; o += kGroupWarps * 32) {
        const int t = o / feats, f = o - t * feats;
        const long long row = x.row0 + t;
        if (kMode == kGateUp) {
          const f32x2 v = situ2_pair(f2_splat(sum(t, f)), f2_splat(sum(t, kRows / 2 + f)), p.sp);
          p.act_out[row * (p.feat / 2) + x.f0 + f] = f2_lo(v);
        } else if (kMode == kSecond || x.f0 + f < p.feat) {
          const long long at = row * p.feat + x.f0 + f;
          float v = sum(t, f);
          if (p.add) v += __uint_as_float((uint32_t)p.add[at] << 16);
          p.out[at] = to_bf16(v);
        }
      }
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kGroupWarps * 32) : "memory");   // the parts are free again
    }
    if (kMode == kGateUp && p.beside) pdl_wait();
  }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// byte matrix [rows, K] in boxes of [blocks][box_rows][128 bytes], 128-byte swizzle;
// bytes outside it read as zeros.  Over one block: columns as [K / 128][128].
bool make_map(CUtensorMap* m, const void* base, long long rows, int K, int box_rows, int blocks) {
  const EncodeTiledFn enc = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
  if (!enc) return false;
  const bool split = blocks > 1;
  cuuint64_t dims[3] = {(cuuint64_t)(split ? 128 : K), (cuuint64_t)rows,
                        (cuuint64_t)(split ? K / 128 : 1)};
  cuuint64_t strides[2] = {(cuuint64_t)K, (cuuint64_t)(split ? 128 : (cuuint64_t)K * rows)};
  cuuint32_t box[3] = {128, (cuuint32_t)box_rows, (cuuint32_t)blocks};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kRingBytes = 192 * 1024;
constexpr int kMaxStages = 64;

template <int kRows, int NT, int kMode, int kGroups, int kKB>
cudaError_t launch_stream(const Fp8Gemm& g, cudaStream_t s) {
  constexpr int kTok = 8 * NT;
  constexpr int kStage = kKB * (kRows * 128 + (kMode == kSecond ? 0 : kTok * 128));
  constexpr int kPart = kConsumers * kTok * (kRows + 4) * (int)sizeof(float);
  StreamParams p{};
  p.xs = g.xs;
  p.act = g.act_in;
  p.ws = g.ws;
  p.add = g.add;
  p.out = g.out;
  p.act_out = g.act_f32;
  p.offsets = g.offsets;
  p.rows = (int)g.rows;
  p.feat = g.feat;
  p.K = g.K;
  p.nkb = fp8_blocks(g.K);
  p.ws_rows = fp8_blocks(g.feat);
  p.groups = g.groups;
  p.max_rows = g.max_rows > 0 ? g.max_rows : 0x7FFFFFFF;
  p.beside = g.beside;
  constexpr int kFit = (kRingBytes + 16 * 1024 - kPart) / kStage;
  constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
  constexpr int kGroupWarps = kConsumers / kGroups;
  p.stages = kStages / kGroups / kGroupWarps * kGroupWarps;
  static_assert(kStages >= kConsumers, "a stage a warp at the least");
  p.err = device_error_word();
  p.sp = make_situ_params(g.beta > 0.0f ? g.beta : 1.0f, g.linear_beta);
  if (!p.err) return cudaErrorInvalidValue;
  CUtensorMap mw, mx;
  if (!make_map(&mw, g.W, (long long)g.groups * g.feat, g.K, kMode == kDense ? kRows : kRows / 2,
                kKB))
    return cudaErrorInvalidValue;
  mx = mw;
  if (kMode != kSecond && !make_map(&mx, g.X, g.rows, g.K, kTok, kKB)) return cudaErrorInvalidValue;
  const size_t smem = 1024 + (size_t)kGroups * p.stages * kStage +
                      kPart + kGroups * p.stages * 16 + (kConsumers + kProducers + 1) * 4 +
                      (kMode == kDense ? 0 : kMaxExperts * (4 + 4 + 2));
  auto* kern = fp8_stream_kernel<kRows, NT, kMode, kGroups, kKB>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  // units: feature blocks of the experts that may have rows, or of the token blocks
  const long long blocks = ceil_div(g.feat, kRows);
  const long long units = blocks * (kMode == kDense ? (g.rows + kTok - 1) / kTok
                                                    : g.rows < g.groups ? g.rows : g.groups);
  const int grid = units < num_sms() ? (int)units : num_sms();
  return launch_k(kern, dim3(grid), dim3((kConsumers + kProducers) * 32), smem, s, mw,
                  mx, p);
}

}  // namespace

cudaError_t launch_fp8_stream(const Fp8Gemm& g, cudaStream_t s) {
  if (g.act_f32) return launch_stream<64, 1, kGateUp, 4, 1>(g, s);
  if (g.act_in) return launch_stream<64, 1, kSecond, 4, 1>(g, s);
  if (g.K % kFp8Block)
    return g.rows <= 8 ? launch_stream<16, 1, kDense, 1, 1>(g, s) : launch_stream<16, 2, kDense, 1, 1>(g, s);
  // as many groups as leave each a ring of about one unit: long rows need the whole
  // ring for one unit, short ones would leave most warps without a stage
  const int nkb = g.K / kFp8Block;
  if (g.rows <= 8) {
    if (nkb <= 16) return launch_stream<16, 1, kDense, 4, 4>(g, s);
    if (nkb <= 32) return launch_stream<16, 1, kDense, 2, 4>(g, s);
    // units of 32 rows read the tokens half as often; not where their coarser waves cost
    // more ([8, 7168] x [8192, 7168]: 13.6 against 15.0 us; 7168 rows: 2 waves against 3 halves)
    if (ceil_div(ceil_div(g.feat, 32), num_sms()) * 2 <= ceil_div(ceil_div(g.feat, 16), num_sms()))
      return launch_stream<32, 1, kDense, 1, 2>(g, s);
    return launch_stream<16, 1, kDense, 1, 4>(g, s);
  }
  if (nkb <= 8) return launch_stream<16, 2, kDense, 4, 2>(g, s);
  if (nkb <= 16) return launch_stream<16, 2, kDense, 2, 2>(g, s);
  return launch_stream<16, 2, kDense, 1, 2>(g, s);
}

}  // namespace lmoe
