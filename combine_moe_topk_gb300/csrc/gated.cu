// gated.cu -- the gated product of few rows (decoded tokens), and the gradients
// of its two projections with what a shared expert's backward pass makes of them.
//
//   h = act(g) u,  [g | u] = z = x W^T + b
//   dg = dh u act'(g),  du = dh act(g),  dz = [dg | du];  db = sum_rows dz
//   dx = dz W,  dW = dz^T x   (the products of linear.cu over 2N columns)
//
// dz is rounded to bf16 for the tensor cores (for bf16 results: their error over 64 bits
// grows from 0.0017, their own rounding, to 0.0023 of their norm); db sums it before that.
// In two bf16 terms, as for fp32 results, its products take twice the time and more:
// 6001 x 4096 x 4096, gelu_tanh, biases 486 us with bf16 results, 976 with an fp32 dW, 1416
// with dx in fp32 too.  Memory bound: 10
// bytes an element of h in bf16 (6001 x 4096, gelu_tanh with column sums 38.0 us, 6.5
// TB/s; 131072 skewed rows x 512, silu, 96 us, 7.0 TB/s).
#include <math_constants.h>

#include "common.cuh"
#include "grouped.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace moe {

namespace {

typedef __nv_bfloat16 bf16;

// ---- few rows -------------------------------------------------------------------

// Bound by reading W once.  The rows come in blocks of at most 16: one block of a
// shared expert's s <= 16 rows, or those of every expert that a route chose.  All
// blocks' columns of h, one block's after another's, are cut into as many equal
// shares as there are SMs, so that each SM streams the same amount of W whatever
// the routing.  W goes through a deep ring in shared memory (a stage: 8 rows x 2048
// of the contracted axis, a bulk copy a row; 190 KB an SM in flight), 8 rows of the
// gate and the same 8 of the factor in turn; the rows of x take the same way, a
// stage or two in front of each chunk's W.
//   warp 8          producer: lane r copies row r of a stage
//   warps 0..7      every eighth 32 of the contracted axis, by warp-level MMA (16
//                   rows of x times 8 of W: idle rows cost nothing, the tensor
//                   cores wait for memory)
// As in the dense product of few rows, lane c of a row's four feeds its 8
// consecutive elements to two MMAs as their k pairs, and the accumulator, which
// drops the bits below its last place, is emptied into an fp32 sum after every
// chunk.  The warps' sums are added in order through shared memory every 16 columns.
// One row, 4096 x 4096: 12.7 us (by tiles 24.4), x 14336: 35.4 us, 6.6 TB/s; 8 tokens
// through 64 experts of 2048 x 1408, six each, 34 of them chosen: 63.9 us (by tiles
// 75.0), 6.1 TB/s.
// A wait that runs out sets the status and everyone runs on without waiting, so
// that the barriers stay matched.
constexpr int kFewK = 2048;                    // of the contracted axis a stage
constexpr int kFewRow = kFewK * 2 + 64;        // row pitch: 64 bytes more, free of bank conflicts
constexpr int kFewStage = 8 * kFewRow;
constexpr int kFewStages = 6;
constexpr int kFewTiles = 2;                   // 8 columns of h each, between two joins
constexpr int kFewCols = 8 * kFewTiles;
constexpr int kFewSmem = kFewStages * kFewStage;
constexpr int kAhead = 64 * 1024;              // of a shared expert's W, fetched to L2 in advance
constexpr int kMaxE = 256;

// To L2; p and bytes are multiples of 16.
__device__ __forceinline__ void prefetch_bulk(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

struct FewArgs {
  const bf16* x;     // [s][ldx]: one block's rows, the dispatched rows, or (inv_row) the token rows
  const bf16* W;     // [e][2][N][ldw]
  long long ldx, ldw;
  int s, K, N, e;
  const int32_t *offsets, *counts, *inv_row;  // NULL: one block of s rows
  int tokens;        // rows of x with inv_row
  const void* bias;  // [2N] or NULL
  int bias_f32, act;
  bf16 *h, *z;       // [..][N], [..][2N] or NULL
  int32_t* status;
  long long timeout_ns;
};

__device__ __forceinline__ float bias_at(const FewArgs& p, int i) {
  return p.bias_f32 ? ld_plain(static_cast<const float*>(p.bias) + i)
                    : __bfloat162float(ld_plain(static_cast<const bf16*>(p.bias) + i));
}

// kExperts: blocks of the experts' segments; else one block of p.s rows, known
// without a look at memory.
template <bool kExperts>
__global__ void __launch_bounds__(288, 1) few_gated_kernel(const __grid_constant__ FewArgs p) {
  constexpr int kBlocks = kFewK / 32 / 8;  // 32-wide blocks of a stage and warp
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ __align__(8) uint64_t full[kFewStages], empty[kFewStages];
  __shared__ float red[8][16][2 * kFewCols + 1];
  __shared__ int s_cnt[kExperts ? kMaxE : 1], s_off[kExperts ? kMaxE : 1], s_blk[kExperts ? kMaxE + 1 : 1];
  __shared__ int s_err;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    s_err = 0;
    for (int i = 0; i < kFewStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 8);
    }
    fence_barrier_init();
  }
  __syncthreads();
  if (!kExperts && warp == 8) {
    // While the kernel before still runs, the first of this SM's rows of W travel to
    // L2 (a prefetch reads nothing: should they be written meanwhile, the copies below
    // find what was written).  64 KB an SM: one row, 4096 x 4096, 13.9 -> 12.7 us (128 KB
    // 12.8, 256 KB 13.3); the tiles' kernel gained nothing by the same.
    const int c0 = (int)((long long)p.N * blockIdx.x / gridDim.x), c1 = (int)((long long)p.N * (blockIdx.x + 1) / gridDim.x);
    const int bytes = min(p.K * 2, 16384), n = min(c1 - c0, kAhead / (2 * bytes));
    for (int i = lane; i < 2 * n; i += 32)
      prefetch_bulk(p.W + ((long long)(i & 1) * p.N + c0 + (i >> 1)) * p.ldw, (uint32_t)bytes);
  }
  grid_dependency_wait();
  if constexpr (kExperts) {
    for (int x = threadIdx.x; x < p.e; x += blockDim.x) {
      s_cnt[x] = ld_plain(p.counts + x);
      s_off[x] = ld_plain(p.offsets + x);
    }
    __syncthreads();
    if (warp == 0) prefix_blocks(s_cnt, s_blk, p.e, 16, lane);
    __syncthreads();
  }
  const long long all = kExperts ? (long long)s_blk[p.e] * p.N : p.N;
  const long long f0 = all * blockIdx.x / gridDim.x, f1 = all * (blockIdx.x + 1) / gridDim.x;
  const int chunks = (p.K + kFewK - 1) / kFewK;
  int stage = 0;
  uint32_t phase = 0;
  bool ok = true;
  auto advance = [&]() {
    if (++stage == kFewStages) {
      stage = 0;
      phase ^= 1u;
    }
  };
  // a group of up to kFewCols columns [c0, c0 + cols) of block b: expert x, rows [row, row + rows)
  struct Group {
    int x, rows, c0, cols;
    long long row;
  };
  auto group_of = [&](long long f) {
    Group g;
    const int b = kExperts ? (int)(f / p.N) : 0;
    g.c0 = (int)(f - (long long)b * p.N);
    g.cols = (int)min((long long)min(kFewCols, p.N - g.c0), f1 - f);
    if constexpr (kExperts) {
      g.x = expert_of(b, s_blk, p.e);
      const int first = 16 * (b - s_blk[g.x]);
      g.rows = min(16, s_cnt[g.x] - first);
      g.row = (long long)s_off[g.x] + first;
    } else {
      g.x = 0;
      g.rows = p.s;
      g.row = 0;
    }
    return g;
  };
  if (warp == 8) {
    auto put = [&](const bf16* mine, int rows, int kc) {  // mine: this lane's row
      ok = ok && __all_sync(0xffffffffu, mbar_wait_limited(&empty[stage], phase ^ 1u, p.timeout_ns));
      if (ok) {
        if (lane == 0) mbar_arrive_expect_tx(&full[stage], (uint32_t)(rows * kc * 2));
        __syncwarp();
        if (lane < rows) bulk_g2s(ring + stage * kFewStage + lane * kFewRow, mine, (uint32_t)kc * 2, &full[stage]);
      }
      advance();
    };
    long long known = -1;
    const bf16* row[2] = {nullptr, nullptr};  // this lane's rows of x: lane and 8 + lane of the block
    for (long long f = f0; f < f1;) {
      const Group g = group_of(f);
      if (g.row != known) {
        known = g.row;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (8 * q + lane >= g.rows || lane >= 8) continue;
          long long r = g.row + 8 * q + lane;
          if (kExperts && p.inv_row) {
            const int t = ld_plain(p.inv_row + r);
            r = (unsigned)t < (unsigned)p.tokens ? t : 0;
          }
          row[q] = p.x + r * p.ldx;
        }
      }
      const bf16* w = p.W + ((long long)2 * g.x * p.N + g.c0 + lane) * p.ldw;
      for (int ch = 0; ch < chunks; ++ch) {
        const int k0 = ch * kFewK, kc = min(kFewK, p.K - k0);
        put(row[0] + k0, min(8, g.rows), kc);
        if (g.rows > 8) put(row[1] + k0, g.rows - 8, kc);
        for (int t = 0; t < g.cols; t += 8) {
          const int n = min(8, g.cols - t);
          put(w + t * p.ldw + k0, n, kc);
          put(w + (t + (long long)p.N) * p.ldw + k0, n, kc);
        }
      }
      f += g.cols;
    }
    // the last copies are waited for by the consumers, which have read all stages
  } else {
    const int gr = lane >> 2, c = lane & 3;
    auto wait_full = [&]() {
      ok = ok && __all_sync(0xffffffffu, mbar_wait_limited(&full[stage], phase, p.timeout_ns));
    };
    auto release = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);
      advance();
    };
    // this lane's 16 bytes of block i of its warp: zeros past the row's end
    auto frag = [&](int i, int kc) {
      const int k = (warp + 8 * i) * 32 + c * 8;
      return k < kc ? *reinterpret_cast<const uint4*>(ring + stage * kFewStage + gr * kFewRow + k * 2) : make_uint4(0, 0, 0, 0);
    };
    for (long long f = f0; f < f1;) {
      const Group g = group_of(f);
      float sum[2 * kFewTiles][4];
#pragma unroll
      for (int t = 0; t < 2 * kFewTiles; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[t][j] = 0.f;
      for (int ch = 0; ch < chunks; ++ch) {
        const int kc = min(kFewK, p.K - ch * kFewK);
        uint4 xa[kBlocks], xb[kBlocks];
        wait_full();
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) xa[i] = frag(i, kc);
        release();
        if (g.rows > 8) {
          wait_full();
#pragma unroll
          for (int i = 0; i < kBlocks; ++i) xb[i] = frag(i, kc);
          release();
        } else {
#pragma unroll
          for (int i = 0; i < kBlocks; ++i) xb[i] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int t = 0; t < 2 * kFewTiles; ++t) {  // gate and factor of 8 columns in turn
          if (8 * (t >> 1) < g.cols) {
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
            wait_full();
#pragma unroll
            for (int i = 0; i < kBlocks; ++i) {
              const uint4 w = frag(i, kc);
              const uint32_t a0[4] = {xa[i].x, xb[i].x, xa[i].y, xb[i].y}, a1[4] = {xa[i].z, xb[i].z, xa[i].w, xb[i].w};
              mma16816(acc, a0, w.x, w.y);
              mma16816(acc, a1, w.z, w.w);
            }
            release();
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[t][j] += acc[j];
          }
        }
      }
#pragma unroll
      for (int t = 0; t < 2 * kFewTiles; ++t) {
        const int at = (t & 1) * kFewCols + 8 * (t >> 1) + 2 * c;
        red[warp][gr][at] = sum[t][0];
        red[warp][gr][at + 1] = sum[t][1];
        red[warp][gr + 8][at] = sum[t][2];
        red[warp][gr + 8][at + 1] = sum[t][3];
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      const int r = threadIdx.x / kFewCols, j = threadIdx.x % kFewCols;  // 16 rows x 16 columns: one value a thread
      if (r < g.rows && j < g.cols) {
        float v[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          v[q] = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) v[q] += red[k][r][q * kFewCols + j];
          if (p.bias) v[q] += bias_at(p, q * p.N + g.c0 + j);
          if (p.z) p.z[(g.row + r) * 2 * p.N + q * p.N + g.c0 + j] = __float2bfloat16_rn(v[q]);
        }
        activate<1>(v, p.act);
        p.h[(g.row + r) * p.N + g.c0 + j] = __float2bfloat16_rn(v[0] * v[1]);
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");  // the sums are rewritten
      f += g.cols;
    }
  }
  if (!ok && lane == 0) atomicOr(&s_err, 1);
  grid_dependents_launch();
  __syncthreads();
  if (s_err) {  // let copies in flight land before shared memory goes
    const uint64_t until = globaltimer_ns() + 200000;
    while (globaltimer_ns() < until) {
    }
    if (threadIdx.x == 0) raise_status(p.status, MOE_DEV_TIMEOUT);
  }
}

template <bool kExperts>
cudaError_t run_few(const FewArgs& p, long long most, const DeviceInfo& di, cudaStream_t st) {
  static OncePerDevice once;
  cudaError_t err = once.run([] {
    return cudaFuncSetAttribute(few_gated_kernel<kExperts>, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem);
  });
  if (err != cudaSuccess) return err;
  return launch_chained(few_gated_kernel<kExperts>, dim3((unsigned)(most < di.sms ? most : di.sms)), dim3(288), kFewSmem, st, p);
}

// ---- dz and the biases' gradients -------------------------------------------------

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
// their column sums up through shared memory, each block one partial row.  Four
// blocks an SM hide the loads (five 52 us at 6001 x 4096, six 58, with the next row's
// loads under way in three 63, in two 39).
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

cudaError_t launch_few_gated(const GatedArgs& a, const DeviceInfo& di, cudaStream_t st) {
  FewArgs p = {};
  p.x = static_cast<const bf16*>(a.x);
  p.W = static_cast<const bf16*>(a.W);
  p.ldx = a.ldx;
  p.ldw = a.ldw;
  p.s = a.s;
  p.K = a.K;
  p.N = a.N;
  p.e = 1;
  p.bias = a.bias;
  p.bias_f32 = a.bias_f32;
  p.act = a.act;
  p.h = static_cast<bf16*>(a.h);
  p.z = static_cast<bf16*>(a.z);
  p.status = a.status;
  p.timeout_ns = kWaitNs;
  return run_few<false>(p, a.N, di, st);
}

cudaError_t launch_few_grouped(const int32_t* offsets, const int32_t* counts, const int32_t* inv_row, int e, int rows, int s,
                               int K, int N, int act, const void* x, const void* W, void* H, void* Z, int32_t* status,
                               const DeviceInfo& di, cudaStream_t st) {
  FewArgs p = {};
  p.x = static_cast<const bf16*>(x);
  p.W = static_cast<const bf16*>(W);
  p.ldx = p.ldw = K;
  p.s = rows;
  p.K = K;
  p.N = N;
  p.e = e;
  p.offsets = offsets;
  p.counts = counts;
  p.inv_row = inv_row;
  p.tokens = s;
  p.act = act;
  p.h = static_cast<bf16*>(H);
  p.z = static_cast<bf16*>(Z);
  p.status = status;
  p.timeout_ns = kWaitNs;
  return run_few<true>(p, (long long)rows * N, di, st);
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
                              a.dw_f32, copies == 2, true}, di, st);
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
