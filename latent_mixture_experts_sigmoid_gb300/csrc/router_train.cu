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
// All passes are bound by memory: the logits are read once (a token's row lives
// in its warp's registers, the next token's is on its way meanwhile) and the
// gradient is written once; a sequence's counts stay in registers from token to
// token.  Every sum has a fixed order, so results repeat to the bit (the counts
// are sums of integers).
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

__device__ __forceinline__ float sigmoid_f(float l) {
  return rcp_fast(1.0f + ex2_fast(-kLog2e * l));
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
// Counts: one cluster of CTAs a sequence, a slice of its tokens each, into a
// histogram in shared memory; then each CTA sums its share of the experts over
// the cluster's histograms.  No global atomics and nothing to zero first.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return n;
}
__device__ __forceinline__ int ld_cluster(const int* p, uint32_t rank) {
  uint32_t a;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ int2 sequence_range(const RouterBatch& b, int s) {
  if (!b.seq) return make_int2(0, b.T);
  const int a = min(max(__ldg(b.seq + s), 0), b.T);
  return make_int2(a, min(max(__ldg(b.seq + s + 1), a), b.T));
}

__global__ void __launch_bounds__(kCountThreads)
count_kernel(const RouterBatch b, int32_t* __restrict__ counts, int32_t* __restrict__ tokens,
             unsigned* __restrict__ ticket) {
  __shared__ int hist[kMaxE + 1];      // [E]: the slice's valid tokens
  const uint32_t rank = cluster_rank(), nr = cluster_size();
  const int s = blockIdx.x / nr;
  pdl_trigger();
  for (int e = threadIdx.x; e <= b.E; e += kCountThreads) hist[e] = 0;
  pdl_wait();
  __syncthreads();
  const int2 r = sequence_range(b, s);
  const int per = (int)(((long long)(r.y - r.x) + nr - 1) / nr);
  const int t0 = min(r.x + (int)rank * per, r.y), t1 = min(t0 + per, r.y);
  const long long i0 = (long long)t0 * b.k, i1 = (long long)t1 * b.k;
  constexpr int kUnroll = 8;
  for (long long i = i0 + threadIdx.x; i < i1; i += kCountThreads * kUnroll) {
    int id[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const long long at = i + j * kCountThreads;
      id[j] = -1;
      if (at < i1) {
        id[j] = __ldg(b.ids + at);
        if (b.mask && !__ldg(b.mask + (unsigned)at / (unsigned)b.k)) id[j] = -1;
      }
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j)
      if ((unsigned)id[j] < (unsigned)b.E) atomicAdd(&hist[id[j]], 1);
  }
  if (b.mask) {
    int n = 0;
    for (int t = t0 + threadIdx.x; t < t1; t += kCountThreads) n += __ldg(b.mask + t) != 0;
    n = __reduce_add_sync(kFull, n);
    if ((threadIdx.x & 31) == 0 && n) atomicAdd(&hist[b.E], n);
  } else if (threadIdx.x == 0) {
    hist[b.E] = t1 - t0;
  }
  cluster_sync();
  for (int e = (int)rank * kCountThreads + threadIdx.x; e <= b.E; e += (int)nr * kCountThreads) {
    int n = 0;
    for (uint32_t k = 0; k < nr; ++k) n += ld_cluster(&hist[e], k);
    if (e < b.E) counts[(long long)s * b.E + e] = n;
    else tokens[s] = n;
  }
  if (ticket && blockIdx.x == 0 && threadIdx.x == 0) *ticket = 0;
  cluster_sync();   // no CTA leaves while another still reads its histogram
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

template <int kNI, bool kVec>
__device__ __forceinline__ void load_row(float (&v)[kNI][4], const float* row, int E, int lane) {
#pragma unroll
  for (int i = 0; i < kNI; ++i) {
    if (kVec) {
      float4 a = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (expert_of<kNI, kVec>(i, 0, lane) < E)
        a = __ldcs(reinterpret_cast<const float4*>(row + expert_of<kNI, kVec>(i, 0, lane)));
      v[i][0] = a.x; v[i][1] = a.y; v[i][2] = a.z; v[i][3] = a.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = expert_of<kNI, kVec>(i, j, lane);
        v[i][j] = e < E ? __ldcs(row + e) : -INFINITY;
      }
    }
  }
}

// Walk of a warp's tokens through the sequences: `c` holds the counts of the
// current one, `unit` E / (k n) and `part` 1 / (S n) (0 without valid tokens).
template <int kNI, bool kVec>
struct SequenceWalk {
  int s = -1, begin = 0, end = 0;
  float unit = 0.0f, part = 0.0f;
  float c[kNI][4];

  // moves to the sequence of token t (tokens come in ascending order)
  __device__ __forceinline__ void at(const RouterBatch& b, const int32_t* counts,
                                     const int32_t* tokens, int t, int lane) {
    if (s >= 0 && t < end) return;
    if (!b.seq) {
      s = 0; begin = 0; end = b.T;
    } else {
      int lo = 0, hi = b.S - 1;       // the last sequence that begins at or before t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(b.seq + mid) <= t) lo = mid; else hi = mid - 1;
      }
      s = lo;
      const int2 r = sequence_range(b, s);
      begin = r.x;
      end = r.y;
    }
    const int n = __ldg(tokens + s);
    unit = n > 0 ? (float)b.E / ((float)b.k * (float)n) : 0.0f;
    part = n > 0 ? 1.0f / ((float)b.S * (float)n) : 0.0f;
    const int32_t* row = counts + (long long)s * b.E;
#pragma unroll
    for (int i = 0; i < kNI; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = expert_of<kNI, kVec>(i, j, lane);
        c[i][j] = e < b.E ? (float)__ldg(row + e) : 0.0f;
      }
  }
  // whether token t of the walk counts
  __device__ __forceinline__ bool valid(const RouterBatch& b, int t) const {
    return t >= begin && t < end && (!b.mask || __ldg(b.mask + t) != 0);
  }
};

// A row of logits -> sigmoids in place; returns {Z, sum_e c s}.  Where Z would
// underflow the row becomes exp(l - max l) instead (see kTinySum), `tiny` set.
template <int kNI, bool kVec>
__device__ __forceinline__ float2 row_sums(float (&v)[kNI][4], const float (&c)[kNI][4], bool* tiny) {
  float s[kNI][4];
  float z = 0.0f, dot = 0.0f;
#pragma unroll
  for (int i = 0; i < kNI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s[i][j] = sigmoid_f(v[i][j]);
      z += s[i][j];
      dot = fmaf(c[i][j], s[i][j], dot);
    }
  z = warp_sum(z);
  *tiny = z < kTinySum;
  if (*tiny) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kNI; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) m = fmaxf(m, v[i][j]);
    m = warp_max(m);
    z = dot = 0.0f;
#pragma unroll
    for (int i = 0; i < kNI; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = m == -INFINITY ? 0.0f : ex2_fast(kLog2e * (v[i][j] - m));
        z += s[i][j];
        dot = fmaf(c[i][j], s[i][j], dot);
      }
    z = warp_sum(z);
  }
  dot = warp_sum(dot);
#pragma unroll
  for (int i = 0; i < kNI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) v[i][j] = s[i][j];
  return make_float2(z, dot);
}

template <int kNI, bool kVec>
__global__ void __launch_bounds__(kWarps * 32, 2)
loss_kernel(const RouterBatch b, float alpha, const int32_t* __restrict__ counts,
            const int32_t* __restrict__ tokens, int per_warp, float* __restrict__ partial,
            unsigned* __restrict__ ticket, float* __restrict__ loss) {
  __shared__ float sums[kWarps];
  __shared__ bool last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_trigger();
  pdl_wait();
  const long long w = (long long)blockIdx.x * kWarps + warp;
  const int t0 = (int)min(w * per_warp, (long long)b.T), t1 = min(t0 + per_warp, b.T);
  SequenceWalk<kNI, kVec> q;
  float total = 0.0f;
  float next[kNI][4];
  if (t0 < t1) load_row<kNI, kVec>(next, b.logits + (long long)t0 * b.E, b.E, lane);
  for (int t = t0; t < t1; ++t) {
    float v[kNI][4];
#pragma unroll
    for (int i = 0; i < kNI; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][j] = next[i][j];
    if (t + 1 < t1) load_row<kNI, kVec>(next, b.logits + (long long)(t + 1) * b.E, b.E, lane);
    q.at(b, counts, tokens, t, lane);
    if (!q.valid(b, t)) continue;
    bool tiny;
    const float2 zd = row_sums<kNI, kVec>(v, q.c, &tiny);
    if (zd.x > 0.0f) total += q.part * (q.unit * zd.y / zd.x);
    else if (!(zd.x == 0.0f)) total += zd.x;      // NaN logits stay NaN
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
  // the weights' gradient of the token at hand, by expert (zero but at the chosen ones)
  __shared__ float add_all[kWarps][kNI * 128];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* add = add_all[warp];
  pdl_trigger();
  for (int e = lane; e < kNI * 128; e += 32) add[e] = 0.0f;
  __syncwarp();
  pdl_wait();
  const long long w = (long long)blockIdx.x * kWarps + warp;
  const int t0 = (int)min(w * a.per_warp, (long long)b.T), t1 = min(t0 + a.per_warp, b.T);
  const float gl = a.grad_loss ? a.alpha * __ldg(a.grad_loss) : 0.0f;
  SequenceWalk<kNI, kVec> q;
  float next[kNI][4];
  if (t0 < t1 && a.grad_loss) load_row<kNI, kVec>(next, b.logits + (long long)t0 * b.E, b.E, lane);
  for (int t = t0; t < t1; ++t) {
    const long long row = (long long)t * b.E;
    float v[kNI][4];
    // 1. the weights' gradient: lane j has the j-th chosen expert
    int id = -1;
    if (a.grad_w) {
      float l = -INFINITY, g = 0.0f;
      if (lane < b.k) {
        id = __ldg(b.ids + (long long)t * b.k + lane);
        if ((unsigned)id >= (unsigned)b.E) id = -1;      // a dropped choice
      }
      if (id >= 0) {
        l = __ldg(b.logits + row + id);
        g = __ldg(a.grad_w + (long long)t * b.k + lane);
      }
      const float s = sigmoid_f(l);
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
      if (id >= 0) add[id] = d * (1.0f - s);
      __syncwarp();
    }
    // 2. the balance loss's
    float coef = 0.0f, mean = 0.0f;
    bool tiny = false;
    if (a.grad_loss) {
#pragma unroll
      for (int i = 0; i < kNI; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j] = next[i][j];
      if (t + 1 < t1) load_row<kNI, kVec>(next, b.logits + row + b.E, b.E, lane);
      q.at(b, a.counts, a.tokens, t, lane);
      if (q.valid(b, t)) {
        const float2 zd = row_sums<kNI, kVec>(v, q.c, &tiny);
        if (!(zd.x == 0.0f)) {
          coef = gl * q.part * q.unit / zd.x;
          mean = zd.y / zd.x;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kNI; ++i) {
      float o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = expert_of<kNI, kVec>(i, j, lane);
        o[j] = a.grad_w ? add[e] : 0.0f;
        if (coef != 0.0f) {
          const float s = v[i][j];
          o[j] += coef * (q.c[i][j] - mean) * (tiny ? s : s * (1.0f - s));
        }
      }
      if (kVec) {
        const int e = expert_of<kNI, kVec>(i, 0, lane);
        if (e < b.E) *reinterpret_cast<float4*>(a.grad + row + e) = make_float4(o[0], o[1], o[2], o[3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = expert_of<kNI, kVec>(i, j, lane);
          if (e < b.E) a.grad[row + e] = o[j];
        }
      }
    }
    if (a.grad_w) {
      __syncwarp();
      if (id >= 0) add[id] = 0.0f;
      __syncwarp();
    }
  }
}

// Tokens a warp takes and CTAs of the token kernels: two CTAs an SM at the most.
struct TokenGrid {
  int per_warp, ctas;
};
TokenGrid token_grid(int T) {
  const long long warps = 2ll * num_sms() * kWarps;
  TokenGrid g;
  g.per_warp = (int)((T + warps - 1) / warps);
  g.ctas = ceil_div(ceil_div(T, g.per_warp), kWarps);
  return g;
}

#define LMOE_BY_EXPERTS(E, CALL)                                  \
  do {                                                            \
    const int ni = ((E) + 127) / 128;                             \
    if ((E) % 4 == 0) {                                           \
      switch (ni) {                                               \
        case 1: return CALL(1, true);                             \
        case 2: return CALL(2, true);                             \
        case 3: return CALL(3, true);                             \
        case 4: return CALL(4, true);                             \
        case 5: return CALL(5, true);                             \
        case 6: return CALL(6, true);                             \
        case 7: return CALL(7, true);                             \
        default: return CALL(8, true);                            \
      }                                                           \
    }                                                             \
    if (ni <= 1) return CALL(1, false);                           \
    if (ni <= 2) return CALL(2, false);                           \
    if (ni <= 4) return CALL(4, false);                           \
    return CALL(8, false);                                        \
  } while (0)

}  // namespace

// the ticket, then a partial sum per CTA of the loss kernel
size_t balance_workspace_bytes(int T) {
  const size_t n = 256 + (T > 0 ? (size_t)token_grid(T).ctas * 4 : 0);
  return (n + 255) & ~size_t(255);
}

cudaError_t launch_balance_loss(const RouterBatch& b, float alpha, float* loss, int32_t* counts,
                                int32_t* tokens, void* workspace, cudaStream_t s) {
  unsigned* ticket = static_cast<unsigned*>(workspace);
  float* partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + 256);
  // eight CTAs a sequence where it is long enough to feed them
  const int cluster = (long long)b.T * b.k > 4096ll * b.S ? 8 : 1;
  cudaError_t e = launch_k_cluster(count_kernel, dim3(b.S * cluster), dim3(kCountThreads), 0, s,
                                   cluster, b, counts, tokens, ticket);
  if (e != cudaSuccess) return e;
  const TokenGrid g = token_grid(b.T);
#define LMOE_CALL(NI, VEC)                                                                       \
  launch_k(loss_kernel<NI, VEC>, dim3(g.ctas), dim3(kWarps * 32), 0, s, b, alpha,                 \
           (const int32_t*)counts, (const int32_t*)tokens, g.per_warp, partial, ticket, loss)
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
  launch_k(backward_kernel<NI, VEC>, dim3(g.ctas), dim3(kWarps * 32), 0, s, b, a)
  LMOE_BY_EXPERTS(b.E, LMOE_CALL);
#undef LMOE_CALL
}

}  // namespace lmoe
