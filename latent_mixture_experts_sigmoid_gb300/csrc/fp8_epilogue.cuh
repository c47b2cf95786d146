// The addend of the e4m3 products' epilogues (fp8.cu, fp8_pair.cu).
//
// A thread's sums begin with its row's part of the addend: the loads run beside the first
// operands', where after the sums nothing would hide them.  A thread reads kCols columns of a
// row of its own, so that each load of a warp touches 32 lines, however wide: 32 bytes at a
// time where the addend's rows start on them.
#pragma once

#include "lmoe_internal.cuh"
#include "tc_ptx.cuh"

namespace lmoe {

// y: the columns from col0 on (feat % 8 == 0).  Past feat, where nothing is stored, they repeat
// the last ones: a load behind a branch of its own would be waited for before the next.
template <int kCols>
__device__ __forceinline__ void add_first(f32x2 (&y)[kCols / 2], const uint16_t* row, int col0, int feat,
                                          bool wide) {
  uint32_t w[kCols / 16][8];
  if (wide) {
#pragma unroll
    for (int i = 0; i < kCols / 16; ++i) ld_global32(row + min(col0 + 16 * i, feat - 16), w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kCols / 8; ++i) {
      const uint4 a = __ldg(reinterpret_cast<const uint4*>(row + min(col0 + 8 * i, feat - 8)));
      uint32_t* v = w[i / 2] + 4 * (i & 1);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    }
  }
#pragma unroll
  for (int i = 0; i < kCols / 2; ++i)
    y[i] = f2_make(w[i / 8][i & 7] << 16, w[i / 8][i & 7] & 0xFFFF0000u);
}

// the same columns of another tile's row on their way to L2
template <int kCols>
__device__ __forceinline__ void prefetch_addend(const uint16_t* row, int col0, int feat) {
#pragma unroll
  for (int i = 0; i < kCols; i += 64)
    if (col0 + i < feat) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + col0 + i));
}

}  // namespace lmoe
