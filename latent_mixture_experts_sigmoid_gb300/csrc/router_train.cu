// Training of the sigmoid router: the balance loss with its per-expert counts,
// and the gradient of the router logits.
//
//   s[t,e] = sigmoid(l[t,e]),  Z[t] = sum_e s[t,e],  q = s / Z
//   c[b,e] = how often the valid tokens of sequence b chose e,  n_b = valid tokens
//   f[b,e] = E / (k n_b) c[b,e],   P[b,e] = 1/n_b sum_t q[t,e]
//   loss   = alpha/S sum_b sum_e f[b,e] P[b,e]
//          = alpha/S sum_b 1/n_b sum_t (sum_e f[b,e] s[t,e]) / Z[t]
// The second form needs no [S, E] column sums: once the counts are there, one
// pass over the logits gives each token's term.  Its gradient (counts are
// constants of the selection):
//   dloss/dl[t,e] = alpha/(S n_b) (f[b,e] - (sum f s)/Z) q[t,e] (1 - s[t,e])
// and that of the routing weights w_j = rsf p_j, p_j = s_j / sum of the chosen s:
//   dl[t,i] = rsf (g_i - sum_j g_j p_j) p_i (1 - s_i)     (renormalised)
//   dl[t,i] = rsf g_i s_i (1 - s_i)                       (not)
//
// The logits are read once (a token's row lives in its warp's registers, the
// next tokens' are on their way meanwhile) and the gradient is written once; a
// sequence's counts stay in registers from token to token.  Every sum has a
// fixed order, so results repeat to the bit (the counts are sums of integers).
//
// 16384 tokens, 896 experts, 16 choices, 4 sequences: loss 19.4 us (60 MB, 8.8 us at full
// rate), of which the counts, which the token pass must have first, take about 5; gradient
// 24.3 us (120 MB, 4.9 TB/s).  What bounds the token kernels is not the bandwidth but the
// latencies of a row on its warp, 16 warps an SM (gradient: 685 instructions a token, 1.95
// of 4 a cycle; 24 warps with fewer registers each were slower).
// 256 tokens of 64 experts: loss 5 us, gradient 2.9 us, launches and one chain of latencies.
#include "lmoe_internal.cuh"
#include "router_train.cuh"
#include "tc_ptx.cuh"

namespace lmoe {
namespace {

constexpr int kWarps = 8;                 // warps of a CTA of the token kernels
constexpr int kCountThreads = 512;
constexpr int kMaxE = 1024;
constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr float kLog2e = 1.4426950408889634f;
// Below this sum of sigmoids every logit is under -27: there sigmoid(l) is
// exp(l) to 2^-39, and shares are taken from exp(l - max l), which cannot underflow.
constexpr float kTinySum = 9.094947017729282e-13f;   // 2^-40

// {s, 1 - s} of a logit.  With e = exp(-|l|) the smaller of the two is e / (1 + e), the larger
// 1 / (1 + e): neither is the difference of the other from 1, which a rounded s near 1 would
// leave nothing of (1 - s at l = 12: 1 % off, from l = 17 on 0).
__device__ __forceinline__ float2 sigmoid_f(float l) {
  const float e = ex2_fast(-kLog2e * fabsf(l)), r = rcp_fast(1.0f + e), u = e * r;
  return l > 0.0f ? make_float2(r, u) : make_float2(u, r);
}

// min(x, 127), NaN staying NaN (as it would not in fminf)
__device__ __forceinline__ float most_127(float x) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(127.0f));
  return y;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

// ---------------------------------------------------------------------------
// Counts: one kernel zeroes them, the next spreads the tokens evenly over its
// CTAs, each with a histogram in shared memory for the sequence at hand that it
// adds to the global counts (integers: the order does not matter).
//
// Both trigger their dependents after their own wait, so a CTA of a later kernel
// of the call exists only once all work before the call is complete: it may read
// the call's inputs before its own wait, which is for what the call itself writes.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256)
zero_kernel(int32_t* __restrict__ counts, long long n, int32_t* __restrict__ tokens, int S,
            unsigned* __restrict__ ticket) {
  pdl_wait();
  pdl_trigger();
  const long long i0 = (long long)blockIdx.x * 256 + threadIdx.x, step = (long long)gridDim.x * 256;
  for (long long i = i0; i < n; i += step) counts[i] = 0;
  for (long long i = i0; i < S; i += step) tokens[i] = 0;
  if (i0 == 0) *ticket = 0;
}

__device__ __forceinline__ int2 sequence_range(const RouterBatch& b, int s) {
  if (!b.seq) return make_int2(0, b.T);
  const int a = min(max(__ldg(b.seq + s), 0), b.T);
  return make_int2(a, min(max(__ldg(b.seq + s + 1), a), b.T));
}

// End of a run of up to n tokens from `first` <= T on.  T may be 2^31 - 1, so here and below
// the distance to the end is what is compared: a token number past the end could wrap.
__device__ __forceinline__ int run_end(int first, int n, int T) { return first + min(n, T - first); }

// The last sequence that begins at or before token t (0 where none does).
__device__ __forceinline__ int sequence_of(const RouterBatch& b, int t) {
  if (!b.seq) return 0;
  int lo = 0, hi = b.S - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(b.seq + mid) <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kCountThreads)
count_kernel(const RouterBatch b, int per_cta, int32_t* __restrict__ counts,
             int32_t* __restrict__ tokens) {
  __shared__ int hist[kMaxE + 1];      // [E]: the slice's valid tokens
  pdl_trigger();                       // (the kernel before has waited: see above)
  for (int e = threadIdx.x; e <= b.E; e += kCountThreads) hist[e] = 0;
  __syncthreads();
  bool waited = false;
  const int first = (int)min((long long)blockIdx.x * per_cta, (long long)b.T);
  const int last = run_end(first, per_cta, b.T);
  // the slice's choices and masks on their way while the sequence is looked up
  for (long long i = (long long)first * b.k + threadIdx.x * 32; i < (long long)last * b.k; i += kCountThreads * 32)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(b.ids + i));
  if (b.mask && (int)threadIdx.x * 128 < last - first)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(b.mask + first + threadIdx.x * 128));
  for (int t0 = first; t0 < last;) {
    const int s = sequence_of(b, t0);
    const int2 r = sequence_range(b, s);
    if (t0 < r.x) { t0 = min(r.x, last); continue; }   // before the first sequence
    if (t0 >= r.y) break;                              // behind the last
    const int t1 = min(r.y, last);
    const long long i1 = (long long)t1 * b.k;
    constexpr int kUnroll = 4;
    for (long long i = (long long)t0 * b.k + threadIdx.x; i < i1; i += kCountThreads * kUnroll) {
      int id[kUnroll];
      bool keep[kUnroll];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const long long at = i + j * kCountThreads;
        id[j] = -1;
        keep[j] = true;
        if (at < i1) {
          id[j] = __ldg(b.ids + at);
          if (b.mask) keep[j] = __ldg(b.mask + (unsigned)at / (unsigned)b.k) != 0;
        }
      }
#pragma unroll
      for (int j = 0; j < kUnroll; ++j)
        if (keep[j] && (unsigned)id[j] < (unsigned)b.E) atomicAdd(&hist[id[j]], 1);
    }
    if (b.mask) {
      for (int i = threadIdx.x; i < t1 - t0; i += kCountThreads)
        if (__ldg(b.mask + t0 + i)) atomicAdd(&hist[b.E], 1);
    } else if (threadIdx.x == 0) {
      hist[b.E] = t1 - t0;
    }
    __syncthreads();
    if (!waited) pdl_wait();           // the counts are zero
    waited = true;
    for (int e = threadIdx.x; e <= b.E; e += kCountThreads) {
      const int n = hist[e];
      hist[e] = 0;
      if (n) atomicAdd(e < b.E ? counts + (long long)s * b.E + e : tokens + s, n);
    }
    __syncthreads();
    t0 = t1;
  }
  if (!waited) pdl_wait();
}

// ---------------------------------------------------------------------------
// The token kernels: a warp takes a run of consecutive tokens.  A lane holds
// 4 kNI experts of the row: kVec (E % 4 == 0): four consecutive ones per 16-byte
// load, otherwise one per load.
// ---------------------------------------------------------------------------
template <int kNI, bool kVec>
__device__ __forceinline__ int expert_of(int i, int j, int lane) {
  return kVec ? (i * 32 + lane) * 4 + j : (i * 4 + j) * 32 + lane;
}

// A warp's ring of logit rows in shared memory, filled by asynchronous copies.
// Every lane copies and reads its own experts only, so that its own copies'
// completion is all there is to wait for.  kSlots rows are on their way per warp:
// 16 warps an SM and a latency of about 1.5 us need two rows each at full
// bandwidth (16384 x 896: two slots 24.3 us for the gradient, three 24.8, four 25.6; with a
// row ahead in registers instead 37).
constexpr int kSlots = 2;

template <int kNI, bool kVec>
struct RowRing {
  float* slots;            // this lane's part of slot 0: [kNI][4] at a stride of 32 lanes
  __device__ __forceinline__ RowRing(float* smem, int warp, int lane)
      : slots(smem + (size_t)warp * kSlots * kNI * 128 + lane * 4) {}

  __device__ __forceinline__ void fetch(int slot, const float* row, int E, int lane) {
    const uint32_t dst = smem_u32(slots + slot * kNI * 128);
#pragma unroll
    for (int i = 0; i < kNI; ++i) {
      if (kVec) {
        const int e = expert_of<kNI, kVec>(i, 0, lane);
        if (e < E)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + i * 512), "l"(row + e)
                       : "memory");
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = expert_of<kNI, kVec>(i, j, lane);
          if (e < E)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst + i * 512 + j * 4),
                         "l"(row + e)
                         : "memory");
        }
      }
    }
  }
  static __device__ __forceinline__ void commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // the oldest of the kSlots groups has landed
  static __device__ __forceinline__ void wait_oldest() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 1) : "memory");
  }
  __device__ __forceinline__ float4 own(int slot, int i) const {
    return *reinterpret_cast<const float4*>(slots + (slot * kNI + i) * 128);
  }
  __device__ __forceinline__ void clear(int slot) {
#pragma unroll
    for (int i = 0; i < kNI; ++i)
      *reinterpret_cast<float4*>(slots + (slot * kNI + i) * 128) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  // where expert e's element of a slot is (any lane's)
  __device__ __forceinline__ float* place(int slot, int e, int lane) {
    const int at = kVec ? e : (e & ~127) + (e & 31) * 4 + ((e >> 5) & 3);
    return slots - lane * 4 + slot * kNI * 128 + at;
  }
  // the row as pairs; places past the last expert (in the last 128 only) read as -infinity
  __device__ __forceinline__ void read(f32x2 (&v)[kNI][2], int slot, int E, int lane) const {
#pragma unroll
    for (int i = 0; i < kNI; ++i) {
      float4 a = own(slot, i);
      if (i == kNI - 1) {
        if (expert_of<kNI, kVec>(i, 0, lane) >= E) a.x = -INFINITY;
        if (expert_of<kNI, kVec>(i, 1, lane) >= E) a.y = -INFINITY;
        if (expert_of<kNI, kVec>(i, 2, lane) >= E) a.z = -INFINITY;
        if (expert_of<kNI, kVec>(i, 3, lane) >= E) a.w = -INFINITY;
      }
      v[i][0] = f2_make(__float_as_uint(a.x), __float_as_uint(a.y));
      v[i][1] = f2_make(__float_as_uint(a.z), __float_as_uint(a.w));
    }
  }
};

// Walk of a warp's tokens, in ascending order, through the sequences: `c` holds the
// counts of the current one, `unit` E / (k n) and `part` 1 / (S n) (0 without valid
// tokens), bit i of `keep` whether token `base` + i counts as far as the mask goes
// (one load for 32 tokens: a load a token would be a latency a token).
template <int kNI, bool kVec>
struct SequenceWalk {
  int s = 0, begin = 0, end = 0, base = 0;
  unsigned keep = 0;
  bool fresh = true;       // the counts of sequence s are not loaded yet
  float unit = 0.0f, part = 0.0f;
  f32x2 c[kNI][2];

  // The place of the warp's first token; reads the call's inputs only.
  __device__ __forceinline__ void start(const RouterBatch& b, int t, int lane) {
    find(b, t);
    masks(b, t, lane);
  }
  __device__ __forceinline__ void find(const RouterBatch& b, int t) {
    s = sequence_of(b, t);
    const int2 r = sequence_range(b, s);
    begin = r.x;
    end = r.y;
    fresh = true;
  }
  __device__ __forceinline__ void masks(const RouterBatch& b, int t, int lane) {
    base = t;
    keep = b.mask ? __ballot_sync(kFull, lane < b.T - t && __ldg(b.mask + t + lane) != 0) : kFull;
  }

  // Moves to token t; whether it counts.  (kShared: counts and tokens are in shared memory.)
  template <bool kShared = false>
  __device__ __forceinline__ bool at(const RouterBatch& b, const int32_t* counts,
                                     const int32_t* tokens, int t, int lane) {
    if (t >= end && s + 1 < b.S) find(b, t);
    if (t - base >= 32) masks(b, t, lane);
    if (t < begin || t >= end || !(keep >> (t - base) & 1u)) return false;
    if (fresh) load<kShared>(b, counts, tokens, lane);
    return true;
  }
  template <bool kShared>
  __device__ __forceinline__ void load(const RouterBatch& b, const int32_t* counts,
                                       const int32_t* tokens, int lane) {
    fresh = false;
    const int32_t* row = counts + (long long)s * b.E;
#pragma unroll
    for (int i = 0; i < kNI; ++i) {
      int4 n = make_int4(0, 0, 0, 0);
      if (kVec) {
        if (expert_of<kNI, kVec>(i, 0, lane) < b.E)
          n = kShared ? *reinterpret_cast<const int4*>(row + expert_of<kNI, kVec>(i, 0, lane))
                      : __ldcg(reinterpret_cast<const int4*>(row + expert_of<kNI, kVec>(i, 0, lane)));
      } else {
        int x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = expert_of<kNI, kVec>(i, j, lane);
          x[j] = e >= b.E ? 0 : kShared ? row[e] : __ldcg(row + e);
        }
        n = make_int4(x[0], x[1], x[2], x[3]);
      }
      c[i][0] = f2_make(__float_as_uint((float)n.x), __float_as_uint((float)n.y));
      c[i][1] = f2_make(__float_as_uint((float)n.z), __float_as_uint((float)n.w));
    }
    const int n = kShared ? tokens[s] : __ldcg(tokens + s);
    unit = n > 0 ? (float)b.E / ((float)b.k * (float)n) : 0.0f;
    part = n > 0 ? 1.0f / ((float)b.S * (float)n) : 0.0f;
  }
};

// The row of a slot -> {Z, sum_e c s}.  kKeep: `s` becomes s (1 - s), otherwise s.  1 - s is
// e s with e = exp(-l), without a difference (see sigmoid_f); e ends at 2^127, where the
// reciprocal of 1 + e is 0 already, so that e s is 0 and not NaN.  Where Z would underflow, s is
// exp(l - max l) instead (see kTinySum) and 1 - s is 1.  Pairs of experts go through the
// packed fp32 operations: 4 instructions an expert, 6 with kKeep.
template <bool kKeep, int kNI, bool kVec>
__device__ __forceinline__ float2 row_sums(f32x2 (&s)[kNI][2], const f32x2 (&c)[kNI][2],
                                           const RowRing<kNI, kVec>& ring, int slot, int E, int lane) {
  ring.read(s, slot, E, lane);
  f32x2 z2 = 0ull, dot2 = 0ull;
#pragma unroll
  for (int i = 0; i < kNI; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      f32x2 x = f2_mul(s[i][j], f2_splat(-kLog2e));
      if (kKeep) x = LMOE_F2_APPLY(most_127, x);
      const f32x2 e = LMOE_F2_APPLY(ex2_fast, x);
      const f32x2 v = LMOE_F2_APPLY(rcp_fast, f2_add(e, f2_splat(1.0f)));
      z2 = f2_add(z2, v);
      dot2 = f2_fma(c[i][j], v, dot2);
      s[i][j] = kKeep ? f2_mul(f2_mul(e, v), v) : v;
    }
  float z = f2_lo(z2) + f2_hi(z2), dot = f2_lo(dot2) + f2_hi(dot2);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    z += __shfl_xor_sync(kFull, z, o);
    dot += __shfl_xor_sync(kFull, dot, o);
  }
  if (z < kTinySum) {
    ring.read(s, slot, E, lane);
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kNI; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) m = fmaxf(m, fmaxf(f2_lo(s[i][j]), f2_hi(s[i][j])));
    m = warp_max(m);
    z2 = dot2 = 0ull;
#pragma unroll
    for (int i = 0; i < kNI; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const f32x2 d = f2_add(s[i][j], f2_splat(-m));
        s[i][j] = m == -INFINITY ? 0ull : LMOE_F2_APPLY(ex2_fast, f2_mul(d, f2_splat(kLog2e)));
        z2 = f2_add(z2, s[i][j]);
        dot2 = f2_fma(c[i][j], s[i][j], dot2);
      }
    z = warp_sum(f2_lo(z2) + f2_hi(z2));
    dot = warp_sum(f2_lo(dot2) + f2_hi(dot2));
  }
  return make_float2(z, dot);
}

template <int kNI, bool kVec>
__global__ void __launch_bounds__(kWarps * 32, 2)
loss_kernel(const RouterBatch b, float alpha, const int32_t* __restrict__ counts,
            const int32_t* __restrict__ tokens, int per_warp, float* __restrict__ partial,
            unsigned* __restrict__ ticket, float* __restrict__ loss) {
  extern __shared__ __align__(16) float ring_smem[];
  __shared__ float sums[kWarps];
  __shared__ bool last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_trigger();
  const long long w = (long long)blockIdx.x * kWarps + warp;
  const int t0 = (int)min(w * per_warp, (long long)b.T), t1 = run_end(t0, per_warp, b.T);
  RowRing<kNI, kVec> ring(ring_smem, warp, lane);
  // the logits are complete (see the counts); the counts are not
  for (int i = 0; i < kSlots; ++i) {
    if (i < t1 - t0) ring.fetch(i, b.logits + (long long)(t0 + i) * b.E, b.E, lane);
    ring.commit();
  }
  SequenceWalk<kNI, kVec> q;
  if (t0 < t1) q.start(b, t0, lane);
  pdl_wait();
  // A warp's run may have hundreds of thousands of tokens (2^31 - 1 of them: 883012 on 152 SMs),
  // whose terms are about equal: in one fp32 sum each would lose the same part (50 million
  // tokens: 1.4e-4 of the loss).  `lost` holds what the last addition rounded off.
  float total = 0.0f, lost = 0.0f;
  auto add = [&](float term) {
    const float x = term - lost, sum = total + x;
    lost = (sum - total) - x;
    total = sum;
  };
  int slot = 0;
  for (int t = t0; t < t1; ++t) {
    f32x2 v[kNI][2];
    ring.wait_oldest();
    if (q.at(b, counts, tokens, t, lane)) {
      const float2 zd = row_sums<false, kNI, kVec>(v, q.c, ring, slot, b.E, lane);
      if (zd.x > 0.0f) add(q.part * (q.unit * zd.y / zd.x));
      else if (!(zd.x == 0.0f)) add(zd.x);          // NaN logits stay NaN
    }
    // refilled once its row is used
    if (t1 - t > kSlots) ring.fetch(slot, b.logits + (long long)(t + kSlots) * b.E, b.E, lane);
    ring.commit();
    slot = slot + 1 == kSlots ? 0 : slot + 1;
  }
  if (lane == 0) sums[warp] = total;
  __syncthreads();
  if (threadIdx.x == 0) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) v += sums[i];
    partial[blockIdx.x] = v;
    __threadfence();
    last = atomicAdd(ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  // the last CTA to finish adds the partial sums, in an order of their own
  __threadfence();
  float v = 0.0f;
  for (int i = threadIdx.x; i < (int)gridDim.x; i += kWarps * 32) v += __ldcg(partial + i);
  v = warp_sum(v);
  if (lane == 0) sums[warp] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) v += sums[i];
    *loss = alpha * v;
  }
}

// The whole of a small batch's loss in one cluster: counts per CTA, summed over the cluster
// through its shared memory, then the tokens' terms, then their sum.  Three launches one
// after the other cost such a batch more than its work ([tokens, experts] of four sequences,
// one launch and three: [16, 64] 4.1 and 7.1 us, [256, 64] 5.7 and 7.4, [256, 448] 8.1 and 8.2;
// [256, 896] 10.7 and 8.0, and of one sequence [512, 64] 6.6 and 5.3).
constexpr int kSmallCtas = 8;
constexpr int kSmallTokens = 4 * kSmallCtas * kWarps;    // at most four tokens a warp
constexpr int kSmallLogits = 1 << 17;                    // T * E at most
constexpr int kSmallCounts = 4096;                       // S * (E + 1) at most

__device__ __forceinline__ int ld_cluster(const int* p, uint32_t rank) {
  uint32_t a;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

template <int kNI, bool kVec>
__global__ void __launch_bounds__(kWarps * 32, 2)
small_loss_kernel(const RouterBatch b, float alpha, int32_t* __restrict__ counts,
                  int32_t* __restrict__ tokens, int per_warp, float* __restrict__ loss) {
  extern __shared__ __align__(16) float ring_smem[];
  __shared__ __align__(16) int hist[kSmallCounts];       // this CTA's counts [S, E], tokens [S]
  __shared__ __align__(16) int total[kSmallCounts];      // the cluster's
  __shared__ float sums[kWarps];
  __shared__ float part;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = (int)cluster_rank(), n = b.S * b.E;
  pdl_trigger();
  for (int i = threadIdx.x; i < n + b.S; i += kWarps * 32) hist[i] = 0;
  pdl_wait();
  const int w = rank * kWarps + warp;
  const int t0 = min(w * per_warp, b.T), t1 = min(t0 + per_warp, b.T);
  RowRing<kNI, kVec> ring(ring_smem, warp, lane);
  for (int i = 0; i < kSlots; ++i) {
    if (i < t1 - t0) ring.fetch(i, b.logits + (long long)(t0 + i) * b.E, b.E, lane);
    ring.commit();
  }
  SequenceWalk<kNI, kVec> q;
  if (t0 < t1) q.start(b, t0, lane);
  __syncthreads();
  // this warp's tokens, 32 choices at a time
  for (int i = t0 * b.k + lane; i < t1 * b.k; i += 32) {
    const int t = i / b.k, id = __ldg(b.ids + i);
    const int s = sequence_of(b, t);
    const int2 r = sequence_range(b, s);
    const bool counts_in = t >= r.x && t < r.y && (!b.mask || __ldg(b.mask + t) != 0);
    if (counts_in && (unsigned)id < (unsigned)b.E) atomicAdd(&hist[s * b.E + id], 1);
    if (counts_in && i == t * b.k) atomicAdd(&hist[n + s], 1);
  }
  cluster_sync();
  for (int i = threadIdx.x; i < n + b.S; i += kWarps * 32) {
    int v[kSmallCtas], c = 0;
#pragma unroll
    for (int k = 0; k < kSmallCtas; ++k) v[k] = ld_cluster(&hist[i], (uint32_t)k);
#pragma unroll
    for (int k = 0; k < kSmallCtas; ++k) c += v[k];
    total[i] = c;
    if (rank == 0) {
      if (i < n) counts[i] = c;
      else tokens[i - n] = c;
    }
  }
  __syncthreads();
  float sum = 0.0f;
  int slot = 0;
  for (int t = t0; t < t1; ++t) {
    f32x2 v[kNI][2];
    ring.wait_oldest();
    if (q.template at<true>(b, total, total + n, t, lane)) {
      const float2 zd = row_sums<false, kNI, kVec>(v, q.c, ring, slot, b.E, lane);
      if (zd.x > 0.0f) sum += q.part * (q.unit * zd.y / zd.x);
      else if (!(zd.x == 0.0f)) sum += zd.x;
    }
    if (t1 - t > kSlots) ring.fetch(slot, b.logits + (long long)(t + kSlots) * b.E, b.E, lane);
    ring.commit();
    slot = slot + 1 == kSlots ? 0 : slot + 1;
  }
  if (lane == 0) sums[warp] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) v += sums[i];
    part = v;
  }
  cluster_sync();
  if (rank == 0 && threadIdx.x == 0) {
    float v = 0.0f;
    for (int k = 0; k < kSmallCtas; ++k)
      v += __int_as_float(ld_cluster(reinterpret_cast<const int*>(&part), (uint32_t)k));
    *loss = alpha * v;
  }
  cluster_sync();   // no CTA leaves while another still reads its shared memory
}

struct BackwardArgs {
  const float* grad_w;     // [T, k] or NULL
  const float* grad_loss;  // [1] or NULL
  const int32_t* counts;
  const int32_t* tokens;
  float alpha, rsf;
  int renorm, per_warp;
  float* grad;
};

template <int kNI, bool kVec>
__global__ void __launch_bounds__(kWarps * 32, 2)
backward_kernel(const RouterBatch b, const BackwardArgs a) {
  extern __shared__ __align__(16) float ring_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_trigger();
  pdl_wait();
  const long long w = (long long)blockIdx.x * kWarps + warp;
  const int t0 = (int)min(w * a.per_warp, (long long)b.T), t1 = run_end(t0, a.per_warp, b.T);
  const float gl = a.grad_loss ? a.alpha * __ldg(a.grad_loss) : 0.0f;
  SequenceWalk<kNI, kVec> q;
  RowRing<kNI, kVec> ring(ring_smem, warp, lane);
  if (t0 < t1 && a.grad_loss) {
    q.start(b, t0, lane);
    for (int i = 0; i < kSlots; ++i) {
      if (i < t1 - t0) ring.fetch(i, b.logits + (long long)(t0 + i) * b.E, b.E, lane);
      ring.commit();
    }
  }
  // the j-th chosen expert of a token and its gradient are lane j's; they are loaded
  // a token ahead, as is the expert's logit where the row itself is not read
  auto choice = [&](int t, int ahead, int& id, float& g) {      // of token t + ahead
    id = -1;
    g = 0.0f;
    if (a.grad_w && t1 - t > ahead && lane < b.k) {
      id = __ldg(b.ids + (long long)(t + ahead) * b.k + lane);
      g = __ldg(a.grad_w + (long long)(t + ahead) * b.k + lane);
    }
  };
  auto logit = [&](int t, int ahead, int id) {                  // (no id behind the last token)
    return !a.grad_loss && (unsigned)id < (unsigned)b.E
               ? __ldg(b.logits + (long long)(t + ahead) * b.E + id)
               : -INFINITY;
  };
  int id1, id2;
  float g1, g2, l1;
  choice(t0, 0, id1, g1);
  choice(t0, 1, id2, g2);
  l1 = logit(t0, 0, id1);
  int slot = 0;
  for (int t = t0; t < t1; ++t) {
    const long long row = (long long)t * b.E;
    f32x2 v[kNI][2];
    int id = id1;
    float g = g1, l = l1;
    id1 = id2;
    g1 = g2;
    l1 = logit(t, 1, id1);
    choice(t, 2, id2, g2);
    if ((unsigned)id >= (unsigned)b.E) {       // no choice of this lane's, or a dropped one
      id = -1;
      g = 0.0f;
    }
    // 1. the balance loss's gradient: coef (c - mean) s (1 - s)
    float coef = 0.0f, mean = 0.0f;
    if (a.grad_loss) {
      ring.wait_oldest();
      __syncwarp();                            // the whole row has landed
      if (id >= 0) l = *ring.place(slot, id, lane);
      if (q.at(b, a.counts, a.tokens, t, lane)) {
        const float2 zd = row_sums<true, kNI, kVec>(v, q.c, ring, slot, b.E, lane);
        if (!(zd.x == 0.0f)) {
          coef = gl * q.part * q.unit / zd.x;
          mean = zd.y / zd.x;
        }
      }
    }
    // 2. the weights' gradient: lane j puts the j-th chosen expert's in its place
    // of the slot, whose row has been used
    if (a.grad_w) {
      const float2 sc = sigmoid_f(l);          // s, 1 - s
      const float s = sc.x;
      float d = a.rsf * g * s;
      if (a.renorm) {
        float p = s, z = warp_sum(s);
        if (z < kTinySum) {
          const float m = warp_max(l);
          p = m == -INFINITY ? 0.0f : ex2_fast(kLog2e * (l - m));
          z = warp_sum(p);
        }
        p = z == 0.0f ? 0.0f : p / z;
        d = a.rsf * (g - warp_sum(g * p)) * p;
      }
      __syncwarp();                            // every lane has its logit
      ring.clear(slot);
      __syncwarp();
      if (id >= 0) *ring.place(slot, id, lane) = d * sc.y;
      __syncwarp();
    }
    // coef (c - mean) s (1 - s)
    const f32x2 scale = f2_splat(coef), shift = f2_splat(-coef * mean);
#pragma unroll
    for (int i = 0; i < kNI; ++i) {
      f32x2 o[2] = {0ull, 0ull};
      if (a.grad_w) {
        const float4 x = ring.own(slot, i);
        o[0] = f2_make(__float_as_uint(x.x), __float_as_uint(x.y));
        o[1] = f2_make(__float_as_uint(x.z), __float_as_uint(x.w));
      }
      if (coef != 0.0f) {
#pragma unroll
        for (int j = 0; j < 2; ++j) o[j] = f2_fma(f2_fma(q.c[i][j], scale, shift), v[i][j], o[j]);
      }
      const float4 r = make_float4(f2_lo(o[0]), f2_hi(o[0]), f2_lo(o[1]), f2_hi(o[1]));
      if (kVec) {
        const int e = expert_of<kNI, kVec>(i, 0, lane);
        if (i < kNI - 1 || e < b.E) *reinterpret_cast<float4*>(a.grad + row + e) = r;
      } else {
        const float x[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = expert_of<kNI, kVec>(i, j, lane);
          if (i < kNI - 1 || e < b.E) a.grad[row + e] = x[j];
        }
      }
    }
    // the slot is refilled once all of the row's uses are over
    if (a.grad_loss) {
      if (t1 - t > kSlots) ring.fetch(slot, b.logits + row + (long long)kSlots * b.E, b.E, lane);
      ring.commit();
    }
    slot = slot + 1 == kSlots ? 0 : slot + 1;
  }
}

// Tokens a warp takes and CTAs of the token kernels: two CTAs an SM at the most.
constexpr int kCtasPerSm = 2;
struct TokenGrid {
  int per_warp, ctas;
};
TokenGrid token_grid(int T) {
  const long long warps = (long long)kCtasPerSm * num_sms() * kWarps;
  TokenGrid g;
  g.per_warp = (int)((T + warps - 1) / warps);
  g.ctas = ceil_div(ceil_div(T, g.per_warp), kWarps);
  return g;
}

// A token kernel with its warps' rings of kNI * 128 floats a slot.
template <typename... KArgs, typename... Args>
cudaError_t launch_ring(void (*kernel)(KArgs...), int ctas, int ni, int cluster, cudaStream_t s,
                        Args&&... args) {
  const size_t smem = (size_t)kWarps * kSlots * ni * 128 * sizeof(float);
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  if (cluster > 1)
    return launch_k_cluster(kernel, dim3(ctas), dim3(kWarps * 32), smem, s, cluster,
                            std::forward<Args>(args)...);
  return launch_k(kernel, dim3(ctas), dim3(kWarps * 32), smem, s, std::forward<Args>(args)...);
}

// kNI is ceil(E / 128) exactly: the kernels take all of a row's chunks but the last as full.
#define LMOE_BY_CHUNKS(NI, CALL, VEC)     \
  switch (NI) {                           \
    case 1: return CALL(1, VEC);          \
    case 2: return CALL(2, VEC);          \
    case 3: return CALL(3, VEC);          \
    case 4: return CALL(4, VEC);          \
    case 5: return CALL(5, VEC);          \
    case 6: return CALL(6, VEC);          \
    case 7: return CALL(7, VEC);          \
    case 8: return CALL(8, VEC);          \
    default: return cudaErrorInvalidValue; \
  }
#define LMOE_BY_EXPERTS(E, CALL)                        \
  do {                                                  \
    const int ni = ((E) + 127) / 128;                   \
    if ((E) % 4 == 0) LMOE_BY_CHUNKS(ni, CALL, true)    \
    LMOE_BY_CHUNKS(ni, CALL, false)                     \
  } while (0)

}  // namespace

// the ticket, then a partial sum per CTA of the loss kernel: room for the most CTAs of any T,
// so that the workspace of the largest batch serves smaller ones (their CTAs may be more)
size_t balance_workspace_bytes(int T) {
  const size_t n = 256 + (T > 0 ? (size_t)kCtasPerSm * num_sms() * 4 : 0);
  return (n + 255) & ~size_t(255);
}

namespace {
cudaError_t launch_small_loss(const RouterBatch& b, float alpha, float* loss, int32_t* counts,
                              int32_t* tokens, cudaStream_t s) {
  const int per_warp = ceil_div(b.T, kSmallCtas * kWarps);
#define LMOE_CALL(NI, VEC)                                                                      \
  launch_ring(small_loss_kernel<NI, VEC>, kSmallCtas, NI, kSmallCtas, s, b, alpha, counts, tokens, \
              per_warp, loss)
  LMOE_BY_EXPERTS(b.E, LMOE_CALL);
#undef LMOE_CALL
}
}  // namespace

cudaError_t launch_balance_loss(const RouterBatch& b, float alpha, float* loss, int32_t* counts,
                                int32_t* tokens, void* workspace, cudaStream_t s) {
  if (b.T <= kSmallTokens && (long long)b.T * b.E <= kSmallLogits &&
      (long long)b.S * (b.E + 1) <= kSmallCounts)
    return launch_small_loss(b, alpha, loss, counts, tokens, s);
  unsigned* ticket = static_cast<unsigned*>(workspace);
  float* partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + 256);
  const long long n = (long long)b.S * b.E;
  cudaError_t e = launch_k(zero_kernel, dim3((unsigned)(n < 256ll * 64 ? (n + 255) / 256 : 64)), dim3(256),
                           0, s, counts, n, tokens, b.S, ticket);
  if (e != cudaSuccess) return e;
  // a CTA an SM, but no fewer tokens each than fill its threads once
  const int least = ceil_div(kCountThreads, b.k);
  const int even = ceil_div(b.T, num_sms());
  const int per_cta = even > least ? even : least;
  e = launch_k(count_kernel, dim3(ceil_div(b.T, per_cta)), dim3(kCountThreads), 0, s, b, per_cta, counts,
               tokens);
  if (e != cudaSuccess) return e;
  const TokenGrid g = token_grid(b.T);
#define LMOE_CALL(NI, VEC)                                                                       \
  launch_ring(loss_kernel<NI, VEC>, g.ctas, NI, 1, s, b, alpha, (const int32_t*)counts,              \
              (const int32_t*)tokens, g.per_warp, partial, ticket, loss)
  LMOE_BY_EXPERTS(b.E, LMOE_CALL);
#undef LMOE_CALL
}

cudaError_t launch_router_backward(const RouterBatch& b, const float* grad_w, int renorm, float rsf,
                                   const float* grad_loss, const int32_t* counts,
                                   const int32_t* tokens, float alpha, float* grad,
                                   cudaStream_t s) {
  const TokenGrid g = token_grid(b.T);
  const BackwardArgs a{grad_w, grad_loss, counts, tokens, alpha, rsf, renorm, g.per_warp, grad};
#define LMOE_CALL(NI, VEC) \
  launch_ring(backward_kernel<NI, VEC>, g.ctas, NI, 1, s, b, a)
  LMOE_BY_EXPERTS(b.E, LMOE_CALL);
#undef LMOE_CALL
}

}  // namespace lmoe
