// grouped.cuh -- device helpers of the products over experts' row segments: the
// numbering of row blocks and the way from an epilogue warp's registers to rows
// of bf16.
#pragma once

#include "activation.cuh"
#include "common.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace moe {

// Exclusive prefix over the experts of their counts of blocks of `per` rows, by
// one warp; blk[e] is the total.
__device__ __forceinline__ void prefix_blocks(const int* cnt, int* blk, int e, int per, int lane) {
  int carry = 0;
  for (int x0 = 0; x0 < e; x0 += 32) {
    const int x = x0 + lane;
    const int c = x < e ? cnt[x] : 0;
    const int blocks = c > 0 ? (c + per - 1) / per : 0;
    int v = blocks;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int w = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += w;
    }
    if (x < e) blk[x] = carry + v - blocks;
    carry += __shfl_sync(0xffffffffu, v, 31);
  }
  if (lane == 0) blk[e] = carry;
}

// The expert of block b: blk[x] <= b < blk[x + 1].
__device__ __forceinline__ int expert_of(int b, const int* blk, int e) {
  int lo = 0, hi = e;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (blk[mid] <= b) lo = mid; else hi = mid;
  }
  return lo;
}

constexpr int kRowStage = 32 * 64;  // a warp's staging tile: 32 rows x 32 bf16 columns

__device__ __forceinline__ void pack_bf16(const float (&f)[32], uint32_t (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
}

// 32 columns of this lane's row (16 words of bf16 pairs) to out[row * ld + col ..],
// rows below `rows`, columns below `cols` (a multiple of 8).  Through shared memory,
// 16-byte parts XOR-swizzled by the row, so that four lanes store 64 consecutive
// bytes of a row.
__device__ __forceinline__ void store_rows(uint8_t* stage, const uint32_t (&w)[16], __nv_bfloat16* out, long long ld,
                                           int rows, int cols, int lane) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    *reinterpret_cast<uint4*>(stage + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)) =
        make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
  __syncwarp();
  const int part = lane & 3;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 8 * i + (lane >> 2);
    if (row < rows && 8 * part < cols)
      *reinterpret_cast<uint4*>(out + row * ld + 8 * part) =
          *reinterpret_cast<const uint4*>(stage + row * 64 + ((part ^ ((row >> 1) & 3)) << 4));
  }
  __syncwarp();
}

}  // namespace moe
