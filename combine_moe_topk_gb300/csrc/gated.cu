// gated.cu -- gradients of a gated product's two projections, and what a shared
// expert's backward pass makes of them.
//
//   h = act(g) u,  [g | u] = z = x W^T + b
//   dg = dh u act'(g),  du = dh act(g),  dz = [dg | du];  db = sum_rows dz
//   dx = dz W,  dW = dz^T x   (the products of linear.cu over 2N columns)
//
// dz is rounded to bf16 for the tensor cores; db sums it before that.  Memory bound: 10
// bytes an element of h in bf16.
#include <math_constants.h>

#include "activation.cuh"
#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

typedef __nv_bfloat16 bf16;

struct DzArgs {
  const void* dh;
  const bf16* z;
  bf16* dz;       // [s][2N] (kTwo: and what its rounding left, s rows further on), or NULL: only the column sums
  float* part;    // [gridDim.y][2N] column sums, or NULL
  long long lddh, ldz;
  int s, N;
  const int32_t *offsets, *counts;  // kGrouped: rows that no expert owns are passed over
  int e;
};

__device__ __forceinline__ void load_f(const float* p, float (&f)[8]) {
  Vec<float>::to_float(ld_plain(reinterpret_cast<const uint4*>(p)), f);
  Vec<float>::to_float(ld_plain(reinterpret_cast<const uint4*>(p) + 1), f + 4);
}
__device__ __forceinline__ void load_f(const bf16* p, float (&f)[8]) {
  Vec<bf16>::to_float(ld_plain(reinterpret_cast<const uint4*>(p)), f);
}

__device__ __forceinline__ void store_dz(bf16* at, long long further, bool two, float (&d)[8]) {
  *reinterpret_cast<uint4*>(at) = Vec<bf16>::from_float(d);
  if (!two) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    d[j] -= __bfloat162float(__float2bfloat16_rn(d[j]));
    if (!(fabsf(d[j]) < CUDART_INF_F)) d[j] = 0.f;  // of an infinity or a NaN
  }
  *reinterpret_cast<uint4*>(at + further) = Vec<bf16>::from_float(d);
}

// A warp walks rows of 256 columns of h, eight a lane; a block's eight warps add
// their column sums up through shared memory, each block one partial row.
template <typename T, int kAct, bool kTwo, bool kGrouped>
__global__ void __launch_bounds__(256, 4) gated_dz_kernel(const DzArgs p) {
  __shared__ float acc[kGrouped ? 1 : 8][2][256 + 8];
  __shared__ SegmentStage seg[1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = blockIdx.x * 256 + lane * 8;
  float sum[2][8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sum[0][j] = sum[1][j] = 0.f;
  grid_dependency_wait();
  bool gaps = false;
  if constexpr (kGrouped) {
    stage_segments_async(seg[0], p.offsets, p.counts, p.e);
    segments_wait();
    bool gap = false;
    for (int x = threadIdx.x; x < p.e; x += blockDim.x) gap |= seg[0].offsets[x] + seg[0].counts[x] != seg[0].offsets[x + 1];
    gaps = __syncthreads_or(gap);
  }
  const long long step = (long long)gridDim.y * 8;
  if (col < p.N) {
    for (long long row = (long long)blockIdx.y * 8 + warp; row < p.s; row += step) {
      if constexpr (kGrouped) {
        if (gaps ? !row_is_owned(row, seg[0].offsets, seg[0].counts, p.e) : row >= seg[0].offsets[p.e]) continue;
      }
      float dh[8], g[8], u[8];
      load_f(static_cast<const T*>(p.dh) + row * p.lddh + col, dh);
      load_f(p.z + row * p.ldz + col, g);
      load_f(p.z + row * p.ldz + p.N + col, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float a, s;
        act_and_slope(g[j], kAct, a, s);
        g[j] = __fmul_rn(__fmul_rn(dh[j], u[j]), s);
        u[j] = __fmul_rn(dh[j], a);
        if constexpr (!kGrouped) {
          sum[0][j] += g[j];
          sum[1][j] += u[j];
        }
      }
      if (p.dz) {
        bf16* at = p.dz + row * 2 * p.N + col;
        const long long further = (long long)p.s * 2 * p.N;
        store_dz(at, further, kTwo, g);
        store_dz(at + p.N, further, kTwo, u);
      }
    }
  }
  grid_dependents_launch();
  if constexpr (!kGrouped) {
    if (!p.part) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      acc[warp][0][lane * 8 + j] = sum[0][j];
      acc[warp][1][lane * 8 + j] = sum[1][j];
    }
    __syncthreads();
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c < p.N) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) v += acc[w][q][threadIdx.x];
        p.part[(size_t)blockIdx.y * 2 * p.N + q * p.N + c] = v;
      }
    }
  }
}

size_t up(size_t v) { return (v + 255) / 256 * 256; }

int dz_rows(int s, int N) {  // blocks along the rows: enough to fill the machine, at least 32 rows each
  const int cols = (N + 255) / 256;
  int rows = (4 * 152 + cols - 1) / cols;
  const int most = (s + 31) / 32;
  if (rows > most) rows = most;
  return rows < 1 ? 1 : rows;
}

template <typename T, bool kTwo, bool kGrouped>
cudaError_t run_dz(const DzArgs& p, int act, int rows, cudaStream_t st) {
  const dim3 grid((unsigned)((p.N + 255) / 256), (unsigned)rows);
  auto kern = gated_dz_kernel<T, MOE_ACT_NONE, kTwo, kGrouped>;
  switch (act) {
    case MOE_ACT_RELU: kern = gated_dz_kernel<T, MOE_ACT_RELU, kTwo, kGrouped>; break;
    case MOE_ACT_GELU: kern = gated_dz_kernel<T, MOE_ACT_GELU, kTwo, kGrouped>; break;
    case MOE_ACT_GELU_TANH: kern = gated_dz_kernel<T, MOE_ACT_GELU_TANH, kTwo, kGrouped>; break;
    case MOE_ACT_SILU: kern = gated_dz_kernel<T, MOE_ACT_SILU, kTwo, kGrouped>; break;
    default: break;
  }
  return launch_chained(kern, grid, dim3(256), 0, st, p);
}

struct BwdPlan {
  size_t dz, part, total;
};
BwdPlan plan_bwd(int s, int N, int copies, bool db) {
  BwdPlan q;
  size_t at = 0;
  q.dz = at, at += up((size_t)s * 2 * N * 2 * copies);
  q.part = at, at += db ? up((size_t)dz_rows(s, N) * 2 * N * 4) : 0;
  q.total = at;
  return q;
}

int copies_of(bool products, bool f32_results) { return products ? f32_results ? 2 : 1 : 0; }

}  // namespace

size_t gated_bwd_workspace(int s, int N, bool products, bool f32_results, bool db) {
  return plan_bwd(s, N, copies_of(products, f32_results), db).total;
}

cudaError_t launch_gated_bwd(const GatedBwdArgs& a, const DeviceInfo& di, cudaStream_t st) {
  const int copies = copies_of(a.dx || a.dW, (a.dx && a.dx_f32) || (a.dW && a.dw_f32));
  const BwdPlan q = plan_bwd(a.s, a.N, copies, a.db != nullptr);
  char* ws = static_cast<char*>(a.workspace);
  DzArgs p = {};
  p.dh = a.dh;
  p.z = static_cast<const bf16*>(a.z);
  p.dz = copies ? reinterpret_cast<bf16*>(ws + q.dz) : nullptr;
  p.part = a.db ? reinterpret_cast<float*>(ws + q.part) : nullptr;
  p.lddh = a.lddh;
  p.ldz = a.ldz;
  p.s = a.s;
  p.N = a.N;
  const int rows = dz_rows(a.s, a.N);
  cudaError_t err;
  if (a.dh_f32) err = copies == 2 ? run_dz<float, true, false>(p, a.act, rows, st) : run_dz<float, false, false>(p, a.act, rows, st);
  else err = copies == 2 ? run_dz<bf16, true, false>(p, a.act, rows, st) : run_dz<bf16, false, false>(p, a.act, rows, st);
  if (err != cudaSuccess) return err;
  if (a.db) {
    err = launch_sum_parts(p.part, rows, 0, 2 * a.N, 2 * a.N, a.db, nullptr, st);
    if (err != cudaSuccess) return err;
  }
  if (!copies) return cudaSuccess;
  return launch_products_bwd({p.dz, a.x, a.W, a.dx, a.dW, a.status, 2LL * a.N, a.ldx, a.ldw, a.s, a.K, 2 * a.N, a.dx_f32,
                              a.dw_f32, copies == 2}, di, st);
}

cudaError_t launch_grouped_dz(const int32_t* offsets, const int32_t* counts, int e, int rows, int N, int act, const void* dH,
                              const void* Z, void* dz, const DeviceInfo&, cudaStream_t st) {
  DzArgs p = {};
  p.dh = dH;
  p.z = static_cast<const bf16*>(Z);
  p.dz = static_cast<bf16*>(dz);
  p.lddh = N;
  p.ldz = 2LL * N;
  p.s = rows;
  p.N = N;
  p.offsets = offsets;
  p.counts = counts;
  p.e = e;
  return run_dz<bf16, false, true>(p, act, dz_rows(rows, N), st);
}

}  // namespace moe
