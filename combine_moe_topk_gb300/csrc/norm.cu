// norm.cu -- the layer norm in front of the MoE block, forward and backward.
//
//   mu = mean(x), r = 1/sqrt(mean((x - mu)^2) + eps), xh = (x - mu) r
//   y  = xh w + b
//   g  = dy w;  dx = r (g - mean(g) - xh mean(g xh)) [+ dres]
//   dw = sum_rows dy xh;  db = sum_rows dy
//
// About ten flops an element: both directions are bound by device memory,
// so each row is read once and stays in registers between its reductions.
// A group of G warps owns a row; thread t of the group holds chunks t,
// t + 32G, ... of C elements (C = one 16-byte vector, or one element where
// the width or a stride is not a multiple of 16 bytes).  The variance is
// taken around the mean (a second reduction over the registers), not as
// E[x^2] - mu^2, which cancels on rows with a large common offset.
// All statistics and sums are fp32; each output is rounded once.
#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

// ---- elements --------------------------------------------------------------

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// C consecutive elements in their memory form: one 16-byte vector, or one element.
template <typename T, int C>
struct Chunk {
  uint4 v;
  __device__ __forceinline__ void load(const T* p) { v = ld_stream(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float* f) const { Vec<T>::to_float(v, f); }
  __device__ __forceinline__ static void store(T* p, const float* f) {
    st_stream(reinterpret_cast<uint4*>(p), Vec<T>::from_float(f));
  }
};
template <typename T>
struct Chunk<T, 1> {
  T v;
  __device__ __forceinline__ void load(const T* p) { v = __ldg(p); }
  __device__ __forceinline__ void get(float* f) const { f[0] = to_f<T>(v); }
  __device__ __forceinline__ static void store(T* p, const float* f) { *p = from_f<T>(f[0]); }
};

// C weights starting at column c (fp32 or bf16 memory, 16-byte aligned when C > 1).
template <int C>
__device__ __forceinline__ void load_weights(const void* w, int is_f32, long long c, float* f) {
  if (C == 1) {
    f[0] = is_f32 ? __ldg(static_cast<const float*>(w) + c)
                  : __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(w) + c));
  } else if (is_f32) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(w) + c);
#pragma unroll
    for (int q = 0; q < C / 4; ++q) Vec<float>::to_float(__ldg(p + q), f + 4 * q);
  } else if (C == 8) {
    Vec<__nv_bfloat16>::to_float(__ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w) + c)), f);
  } else {  // four bf16 beside fp32 rows
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(w) + c));
    f[0] = __uint_as_float(u.x << 16);
    f[1] = __uint_as_float(u.x & 0xffff0000u);
    f[2] = __uint_as_float(u.y << 16);
    f[3] = __uint_as_float(u.y & 0xffff0000u);
  }
}

// ---- sums over a group of G warps --------------------------------------------

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

__device__ __forceinline__ void group_barrier(int group, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
}

// Sum of (a, b) over the group's threads, the same value in all of them;
// `slot`: the group's G words of shared memory for this reduction.
__device__ __forceinline__ float2 group_sum2(float a, float b, float2* slot, int G, int gw, int group) {
  a = warp_sum(a);
  b = warp_sum(b);
  if (G == 1) return make_float2(a, b);
  if ((threadIdx.x & 31) == 0) slot[gw] = make_float2(a, b);
  group_barrier(group, 32 * G);
  float2 v = (threadIdx.x & 31) < G ? slot[threadIdx.x & 31] : make_float2(0.f, 0.f);
  return make_float2(warp_sum(v.x), warp_sum(v.y));
}

constexpr int kMaxWarps = 32;

struct NormFwd {
  const void* x;
  const void* w;
  const void* b;
  void* y;
  float* mean;
  float* rstd;
  long long ldx;
  int s, m, w_f32, b_f32;
  float eps;
};

template <typename T, int C, int E>
__global__ void __launch_bounds__(32 * kMaxWarps) layernorm_kernel(const NormFwd p, const int G) {
  __shared__ float2 slots[2][kMaxWarps];
  const int warp = threadIdx.x >> 5, group = warp / G, gw = warp - group * G;
  const int groups = (blockDim.x >> 5) / G;
  const long long row = (long long)blockIdx.x * groups + group;
  if (row >= p.s) return;  // the whole group together
  grid_dependency_wait();
  const int t = threadIdx.x - group * 32 * G, span = 32 * G;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  Chunk<T, C> raw[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int c = (t + i * span) * C;
    if (c < p.m) raw[i].load(x + c);
  }
  float f[E][C], sum = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    if ((t + i * span) * C < p.m) {
      raw[i].get(f[i]);
#pragma unroll
      for (int j = 0; j < C; ++j) sum += f[i][j];
    }
  }
  const float inv_m = 1.f / (float)p.m;
  const float mu = group_sum2(sum, 0.f, slots[0] + group * G, G, gw, group).x * inv_m;
  float sq = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    if ((t + i * span) * C < p.m) {
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const float d = f[i][j] - mu;
        sq = fmaf(d, d, sq);
      }
    }
  }
  const float var = group_sum2(sq, 0.f, slots[1] + group * G, G, gw, group).x * inv_m;
  const float r = 1.f / sqrtf(var + p.eps);
  T* y = static_cast<T*>(p.y) + row * p.m;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int c = (t + i * span) * C;
    if (c < p.m) {
      float o[C], wv[C];
#pragma unroll
      for (int j = 0; j < C; ++j) o[j] = (f[i][j] - mu) * r;
      if (p.w) {
        load_weights<C>(p.w, p.w_f32, c, wv);
#pragma unroll
        for (int j = 0; j < C; ++j) o[j] *= wv[j];
      }
      if (p.b) {
        load_weights<C>(p.b, p.b_f32, c, wv);
#pragma unroll
        for (int j = 0; j < C; ++j) o[j] += wv[j];
      }
      Chunk<T, C>::store(y + c, o);
    }
  }
  if (t == 0) {
    if (p.mean) p.mean[row] = mu;
    if (p.rstd) p.rstd[row] = r;
  }
  grid_dependents_launch();
}

// Rows too long for the registers of a block: three passes over the row,
// the later ones mostly from L2.  One block per row, any width.
template <typename T>
__global__ void __launch_bounds__(512) layernorm_wide_kernel(const NormFwd p) {
  __shared__ float2 slots[2][16];
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const int gw = threadIdx.x >> 5;
  float sum = 0.f;
  for (int c = threadIdx.x; c < p.m; c += blockDim.x) sum += to_f<T>(__ldg(x + c));
  const float inv_m = 1.f / (float)p.m;
  const float mu = group_sum2(sum, 0.f, slots[0], 16, gw, 0).x * inv_m;
  float sq = 0.f;
  for (int c = threadIdx.x; c < p.m; c += blockDim.x) {
    const float d = to_f<T>(__ldg(x + c)) - mu;
    sq = fmaf(d, d, sq);
  }
  const float r = 1.f / sqrtf(group_sum2(sq, 0.f, slots[1], 16, gw, 0).x * inv_m + p.eps);
  T* y = static_cast<T*>(p.y) + row * p.m;
  for (int c = threadIdx.x; c < p.m; c += blockDim.x) {
    float o = (to_f<T>(__ldg(x + c)) - mu) * r, v[1];
    if (p.w) {
      load_weights<1>(p.w, p.w_f32, c, v);
      o *= v[0];
    }
    if (p.b) {
      load_weights<1>(p.b, p.b_f32, c, v);
      o += v[0];
    }
    y[c] = from_f<T>(o);
  }
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[row] = mu;
    if (p.rstd) p.rstd[row] = r;
  }
}

// ---- backward ------------------------------------------------------------------

struct NormBwd {
  const void* dy;
  const void* x;
  const void* w;
  const void* dres;
  const float* mean;
  const float* rstd;
  void* dx;
  float* part;  // [2][parts][m] partial dw and db, or NULL when neither is wanted
  long long lddy, ldx, lddres;
  int s, m, w_f32, parts;
};

// Each group walks rows gid, gid + groups_total, ...; a thread owns the same
// columns of all of them, so dw and db accumulate in its registers without
// atomics.  The next row's loads are issued before this row's reduction.  At
// the end a block's groups add up through shared memory, one after another,
// and the block writes one partial row; sum_parts_kernel adds those in a
// fixed order, so the gradients are the same on every run.
template <typename T, int C, int E>
__global__ void __launch_bounds__(512) layernorm_bwd_kernel(const NormBwd p, const int G) {
  extern __shared__ float acc_smem[];  // groups > 1: [2][m]
  __shared__ float2 slots[2][16];
  const int warp = threadIdx.x >> 5, group = warp / G, gw = warp - group * G;
  const int groups = (blockDim.x >> 5) / G;
  const int t = threadIdx.x - group * 32 * G, span = 32 * G;
  const long long stride = (long long)gridDim.x * groups;
  grid_dependency_wait();
  float wv[E][C], dw[E][C], db[E][C];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int c = (t + i * span) * C;
#pragma unroll
    for (int j = 0; j < C; ++j) dw[i][j] = db[i][j] = 0.f, wv[i][j] = 1.f;
    if (p.w && c < p.m) load_weights<C>(p.w, p.w_f32, c, wv[i]);
  }
  const float inv_m = 1.f / (float)p.m;
  const T* dy = static_cast<const T*>(p.dy);
  const T* x = static_cast<const T*>(p.x);
  long long row = (long long)blockIdx.x * groups + group;
  Chunk<T, C> rx[E], rd[E];
  float mu = 0.f, r = 0.f;
  if (row < p.s) {
    mu = __ldg(p.mean + row);
    r = __ldg(p.rstd + row);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = (t + i * span) * C;
      if (c < p.m) {
        rx[i].load(x + row * p.ldx + c);
        rd[i].load(dy + row * p.lddy + c);
      }
    }
  }
  for (int it = 0; row < p.s; row += stride, ++it) {
    float xh[E][C], g[E][C], s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = (t + i * span) * C;
      if (c < p.m) {
        rx[i].get(xh[i]);
        rd[i].get(g[i]);
#pragma unroll
        for (int j = 0; j < C; ++j) {
          xh[i][j] = (xh[i][j] - mu) * r;
          dw[i][j] = fmaf(g[i][j], xh[i][j], dw[i][j]);
          db[i][j] += g[i][j];
          g[i][j] *= wv[i][j];
          s1 += g[i][j];
          s2 = fmaf(g[i][j], xh[i][j], s2);
        }
      }
    }
    const long long next = row + stride;
    const float r_now = r;
    if (next < p.s) {
      mu = __ldg(p.mean + next);
      r = __ldg(p.rstd + next);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int c = (t + i * span) * C;
        if (c < p.m) {
          rx[i].load(x + next * p.ldx + c);
          rd[i].load(dy + next * p.lddy + c);
        }
      }
    }
    const float2 sums = group_sum2(s1, s2, slots[it & 1] + group * G, G, gw, group);
    const float c1 = sums.x * inv_m, c2 = sums.y * inv_m;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = (t + i * span) * C;
      if (c < p.m) {
        float o[C];
#pragma unroll
        for (int j = 0; j < C; ++j) o[j] = r_now * (g[i][j] - c1 - xh[i][j] * c2);
        if (p.dres) {
          Chunk<T, C> q;
          float add[C];
          q.load(static_cast<const T*>(p.dres) + row * p.lddres + c);
          q.get(add);
#pragma unroll
          for (int j = 0; j < C; ++j) o[j] += add[j];
        }
        Chunk<T, C>::store(static_cast<T*>(p.dx) + row * p.m + c, o);
      }
    }
  }
  grid_dependents_launch();
  if (!p.part) return;
  for (int q = 0; q < groups; ++q) {
    const bool last = q == groups - 1;
    if (group == q) {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int c = (t + i * span) * C;
        if (c < p.m) {
#pragma unroll
          for (int j = 0; j < C; ++j) {
            float a = dw[i][j], b = db[i][j];
            if (q > 0) {
              a += acc_smem[c + j];
              b += acc_smem[p.m + c + j];
            }
            if (last) {
              p.part[(size_t)blockIdx.x * p.m + c + j] = a;
              p.part[((size_t)p.parts + blockIdx.x) * p.m + c + j] = b;
            } else {
              acc_smem[c + j] = a;
              acc_smem[p.m + c + j] = b;
            }
          }
        }
      }
    }
    if (!last) __syncthreads();
  }
}

// Rows too long for the registers: one block per row, the row read twice (the
// second time mostly from L2), the column sums in the block's partial row,
// each column always updated by the same thread.
template <typename T>
__global__ void __launch_bounds__(512) layernorm_bwd_wide_kernel(const NormBwd p) {
  __shared__ float2 slots[2][16];
  const int gw = threadIdx.x >> 5;
  const float inv_m = 1.f / (float)p.m;
  float* pw = p.part ? p.part + (size_t)blockIdx.x * p.m : nullptr;
  float* pb = p.part ? p.part + ((size_t)p.parts + blockIdx.x) * p.m : nullptr;
  int it = 0;
  for (long long row = blockIdx.x; row < p.s; row += gridDim.x, ++it) {
    const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const float mu = __ldg(p.mean + row), r = __ldg(p.rstd + row);
    float s1 = 0.f, s2 = 0.f;
    for (int c = threadIdx.x; c < p.m; c += blockDim.x) {
      float wv[1] = {1.f};
      if (p.w) load_weights<1>(p.w, p.w_f32, c, wv);
      const float d = to_f<T>(__ldg(dy + c)), xh = (to_f<T>(__ldg(x + c)) - mu) * r, g = d * wv[0];
      s1 += g;
      s2 = fmaf(g, xh, s2);
      if (pw) {
        pw[c] = it ? fmaf(d, xh, pw[c]) : d * xh;
        pb[c] = it ? pb[c] + d : d;
      }
    }
    const float2 sums = group_sum2(s1, s2, slots[it & 1], 16, gw, 0);
    const float c1 = sums.x * inv_m, c2 = sums.y * inv_m;
    for (int c = threadIdx.x; c < p.m; c += blockDim.x) {
      float wv[1] = {1.f};
      if (p.w) load_weights<1>(p.w, p.w_f32, c, wv);
      const float g = to_f<T>(__ldg(dy + c)) * wv[0], xh = (to_f<T>(__ldg(x + c)) - mu) * r;
      float o = r * (g - c1 - xh * c2);
      if (p.dres) o += to_f<T>(__ldg(static_cast<const T*>(p.dres) + row * p.lddres + c));
      static_cast<T*>(p.dx)[row * p.m + c] = from_f<T>(o);
    }
  }
}

// out[c] = sum over parts of part[q][c], for the two halves (blockIdx.y):
// 32 columns a block, 16 threads a column, a fixed tree over them.
__global__ void __launch_bounds__(512) sum_parts_kernel(const float* part, int parts, int stride_parts, int m,
                                                        float* out0, float* out1) {
  __shared__ float acc[16][33];
  float* out = blockIdx.y ? out1 : out0;
  const int col = blockIdx.x * 32 + threadIdx.x;
  const float* src = part + (size_t)blockIdx.y * stride_parts * m;
  float v = 0.f;
  grid_dependency_wait();
  if (col < m) {
#pragma unroll 4
    for (int q = threadIdx.y; q < parts; q += 16) v += src[(size_t)q * m + col];
  }
  acc[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  grid_dependents_launch();
  if (threadIdx.y == 0 && col < m && out) {
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < 16; ++q) sum += acc[q][threadIdx.x];
    out[col] = sum;
  }
}

int chunks_per_group(int chunks, int G) { return (chunks + 32 * G - 1) / (32 * G); }

template <typename T, int C, int E>
cudaError_t run_fwd(const NormFwd& p, int G, cudaStream_t st) {
  const int warps = G < 4 ? 4 : G, rows = warps / G;
  return launch_chained(layernorm_kernel<T, C, E>, dim3((unsigned)((p.s + rows - 1) / rows)), dim3(32 * warps), 0, st, p, G);
}

template <typename T, int C>
cudaError_t fwd_for(const NormFwd& p, cudaStream_t st) {
  constexpr int kPer = C == 1 ? 16 : 16 / C;  // elements a thread: 16 while a block's threads last, then 32
  const int chunks = (p.m + C - 1) / C;
  int G = 1;
  while (G < kMaxWarps && chunks_per_group(chunks, G) > kPer) G *= 2;
  const int need = chunks_per_group(chunks, G);
  if (need * C <= 4) return run_fwd<T, C, (C == 8 ? 1 : 4 / C)>(p, G, st);
  if (need * C <= 8) return run_fwd<T, C, 8 / C>(p, G, st);
  if (need * C <= 16) return run_fwd<T, C, 16 / C>(p, G, st);
  if (need * C <= 32) return run_fwd<T, C, 32 / C>(p, G, st);
  layernorm_wide_kernel<T><<<(unsigned)p.s, 512, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int C, int E>
cudaError_t run_bwd(NormBwd p, int G, int grid, cudaStream_t st) {
  const int warps = G < 8 ? 8 : G, groups = warps / G;
  const size_t smem = groups > 1 && p.part ? 2 * sizeof(float) * (size_t)p.m : 0;
  return launch_chained(layernorm_bwd_kernel<T, C, E>, dim3((unsigned)grid), dim3(32 * warps), smem, st, p, G);
}

template <typename T, int C>
cudaError_t bwd_for(const NormBwd& p, int* grid, const DeviceInfo& di, cudaStream_t st) {
  const int chunks = (p.m + C - 1) / C;
  int G = 1;
  while (G < 16 && chunks_per_group(chunks, G) * C > 16) G *= 2;
  const int need = chunks_per_group(chunks, G) * C;
  const int groups = G < 8 ? 8 / G : 1;
  long long blocks = ((long long)p.s + groups - 1) / groups;
  if (need > 16) blocks = p.s;
  const long long most = need > 16 ? di.sms : 2LL * di.sms;
  *grid = (int)(blocks < most ? blocks : most);
  if (*grid > p.parts) *grid = p.parts;
  if (need <= 4) return run_bwd<T, C, (C == 8 ? 1 : 4 / C)>(p, G, *grid, st);
  if (need <= 8) return run_bwd<T, C, 8 / C>(p, G, *grid, st);
  if (need <= 16) return run_bwd<T, C, 16 / C>(p, G, *grid, st);
  layernorm_bwd_wide_kernel<T><<<(unsigned)*grid, 512, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_sum_parts(const float* part, int parts, int stride_parts, int m, float* out0, float* out1,
                             cudaStream_t st) {
  return launch_chained(sum_parts_kernel, dim3((unsigned)((m + 31) / 32), out1 ? 2 : 1), dim3(32, 16), 0, st, part, parts,
                        stride_parts, m, out0, out1);
}

cudaError_t launch_layernorm(const void* x, long long ldx, int s, int m, int dtype, const void* w, int w_dtype,
                             const void* b, int b_dtype, float eps, void* y, float* mean, float* rstd,
                             cudaStream_t st) {
  NormFwd p = {x, w, b, y, mean, rstd, ldx, s, m, w_dtype == 0, b_dtype == 0, eps};
  const int vec = dtype == 0 ? 4 : 8;
  const bool whole = m % vec == 0 && ldx % vec == 0;
  if (dtype == 0) return whole ? fwd_for<float, 4>(p, st) : fwd_for<float, 1>(p, st);
  return whole ? fwd_for<__nv_bfloat16, 8>(p, st) : fwd_for<__nv_bfloat16, 1>(p, st);
}

cudaError_t launch_layernorm_bwd(const void* dy, long long lddy, const void* x, long long ldx, const void* dres,
                                 long long lddres, int s, int m, int dtype, const void* w, int w_dtype,
                                 const float* mean, const float* rstd, void* dx, float* dw, float* db, float* part,
                                 const DeviceInfo& di, cudaStream_t st) {
  const bool sums = dw || db;
  NormBwd p = {dy, x, w, dres, mean, rstd, dx, sums ? part : nullptr, lddy, ldx, lddres, s, m, w_dtype == 0, layernorm_bwd_parts(s)};
  const int vec = dtype == 0 ? 4 : 8;
  const bool whole = m % vec == 0 && ldx % vec == 0 && lddy % vec == 0 && (!dres || lddres % vec == 0);
  int grid = 0;
  if (s > 0) {
    cudaError_t err;
    if (dtype == 0) err = whole ? bwd_for<float, 4>(p, &grid, di, st) : bwd_for<float, 1>(p, &grid, di, st);
    else err = whole ? bwd_for<__nv_bfloat16, 8>(p, &grid, di, st) : bwd_for<__nv_bfloat16, 1>(p, &grid, di, st);
    if (err != cudaSuccess) return err;
  }
  return sums ? launch_sum_parts(part, grid, p.parts, m, dw, db, st) : cudaSuccess;
}

}  // namespace moe
