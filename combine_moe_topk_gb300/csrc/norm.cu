// norm.cu -- the layer norm in front of the MoE block, forward and backward.
//
//   mu = mean(x), r = 1/sqrt(mean((x - mu)^2) + eps), xh = (x - mu) r
//   y  = xh w + b
//   g  = dy w;  dx = r (g - mean(g) - xh mean(g xh)) [+ dres]
//   dw = sum_rows dy xh;  db = sum_rows dy
//
// About ten flops an element: both directions are bound by device memory, so
// each row is read once.  A group of G warps owns a row at a time and walks
// over rows; its thread t holds chunks t, t + 32G, ... of C elements, E of
// them.  Rows come through a ring of stages in shared memory, filled by
// cp.async: a thread copies and reads only its own chunks, so the ring needs
// no barrier, and the loads of the next rows are in flight while one is
// worked on.  A chunk is a 16-byte vector; where the width or a stride is not
// of 16 bytes, one fp32 element, or two bf16 elements, which may straddle two
// words (each thread then copies both).  The variance is taken around the
// mean (a second reduction over the registers), not as E[x^2] - mu^2, which
// cancels on rows with a large common offset.  All statistics and sums are
// fp32; each output is rounded once.
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

// cp.async of 16 or 4 bytes to shared memory, of which n are read (the rest: zeros).
template <int kBytes>
__device__ __forceinline__ void async_copy(uint32_t dst, const void* src, int n) {
  if (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest n groups of this thread have landed.
__device__ __forceinline__ void async_wait(int n) {
  if (n >= 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (n == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Columns c .. c+C-1 of a row of m: their copy into a slot of shared memory
// (zeros where the row or the columns are not there), their values from it,
// and the store of C results.
template <typename T, int C>
struct Chunk {  // one 16-byte vector; C divides m
  static constexpr int kSlot = 16;
  __device__ __forceinline__ static void fetch(uint32_t slot, const T* row, int c, int m, bool there) {
    there = there && c < m;
    async_copy<16>(slot, there ? row + c : row, there ? 16 : 0);
  }
  __device__ __forceinline__ static void get(const uint8_t* slot, const T*, float* f) {
    Vec<T>::to_float(*reinterpret_cast<const uint4*>(slot), f);
  }
  __device__ __forceinline__ static void store(T* row, int c, int, const float* f) {
    st_stream(reinterpret_cast<uint4*>(row + c), Vec<T>::from_float(f));
  }
};
template <>
struct Chunk<float, 1> {
  static constexpr int kSlot = 4;
  __device__ __forceinline__ static void fetch(uint32_t slot, const float* row, int c, int m, bool there) {
    there = there && c < m;
    async_copy<4>(slot, there ? row + c : row, there ? 4 : 0);
  }
  __device__ __forceinline__ static void get(const uint8_t* slot, const float*, float* f) {
    f[0] = *reinterpret_cast<const float*>(slot);
  }
  __device__ __forceinline__ static void store(float* row, int c, int, const float* f) { row[c] = f[0]; }
};
template <>
struct Chunk<__nv_bfloat16, 2> {  // c even; a row may start in the middle of a word; m may be odd
  static constexpr int kSlot = 8;
  // bytes of the first word before column 0 (0 or 2)
  __device__ __forceinline__ static int skew(const __nv_bfloat16* row) { return (int)(reinterpret_cast<uintptr_t>(row) & 2); }
  __device__ __forceinline__ static void fetch(uint32_t slot, const __nv_bfloat16* row, int c, int m, bool there) {
    there = there && c < m;
    const int off = skew(row), end = !there ? 0 : off + (c + 1 < m ? 4 : 2);
    const uint8_t* word = reinterpret_cast<const uint8_t*>(there ? row + c : row) - off;
    async_copy<4>(slot, word, end < 4 ? end : 4);  // nothing past the row's last element is read
    async_copy<4>(slot + 4, end > 4 ? word + 4 : word, end > 4 ? 2 : 0);
  }
  __device__ __forceinline__ static void get(const uint8_t* slot, const __nv_bfloat16* row, float* f) {
    const uint2 w = *reinterpret_cast<const uint2*>(slot);
    const uint32_t v = skew(row) ? __funnelshift_r(w.x, w.y, 16) : w.x;
    f[0] = __uint_as_float(v << 16);
    f[1] = __uint_as_float(v & 0xffff0000u);
  }
  __device__ __forceinline__ static void store(__nv_bfloat16* row, int c, int m, const float* f) {
    if (c + 1 < m && !skew(row)) {
      *reinterpret_cast<__nv_bfloat162*>(row + c) = __floats2bfloat162_rn(f[0], f[1]);
    } else {
      row[c] = __float2bfloat16_rn(f[0]);
      if (c + 1 < m) row[c + 1] = __float2bfloat16_rn(f[1]);
    }
  }
};

// C weights starting at column c (fp32 or bf16 memory, 16-byte aligned when C > 2).
template <int C>
__device__ __forceinline__ void load_weights(const void* w, int is_f32, int c, int m, float* f) {
  if (C <= 2) {
#pragma unroll
    for (int j = 0; j < C; ++j) {
      f[j] = 0.f;
      if (c + j < m)
        f[j] = is_f32 ? ld_plain(static_cast<const float*>(w) + c + j)
                      : __bfloat162float(ld_plain(static_cast<const __nv_bfloat16*>(w) + c + j));
    }
  } else if (is_f32) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(w) + c);
#pragma unroll
    for (int q = 0; q < C / 4; ++q) Vec<float>::to_float(ld_plain(p + q), f + 4 * q);
  } else if (C == 8) {
    Vec<__nv_bfloat16>::to_float(ld_plain(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w) + c)), f);
  } else {  // four bf16 beside fp32 rows
    const uint2 u = ld_plain(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(w) + c));
    f[0] = __uint_as_float(u.x << 16);
    f[1] = __uint_as_float(u.x & 0xffff0000u);
    f[2] = __uint_as_float(u.y << 16);
    f[3] = __uint_as_float(u.y & 0xffff0000u);
  }
}

// Two fp32 operations an instruction.
__device__ __forceinline__ uint64_t bits(float2 v) { return *reinterpret_cast<uint64_t*>(&v); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// ---- sums over a group of G warps --------------------------------------------

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// The group's barrier: named 1 + group, so that groups do not wait for one another.
__device__ __forceinline__ void group_barrier(int group, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
}

// Sums of R pairs over the group's threads, the same values in all of them;
// slots[.][at ..]: the group's words of shared memory for this reduction.
template <int G, int R>
__device__ __forceinline__ void group_sums(float2 (&v)[R], float2 (*slots)[32], int at, int gw, int group) {
#pragma unroll
  for (int u = 0; u < R; ++u) v[u] = make_float2(warp_sum(v[u].x), warp_sum(v[u].y));
  if (G == 1) return;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int u = 0; u < R; ++u)
    if (lane == 0) slots[u][at + gw] = v[u];
  group_barrier(group, 32 * G);
#pragma unroll
  for (int u = 0; u < R; ++u) {
    v[u] = slots[u][at + (lane & (G - 1))];
#pragma unroll
    for (int d = G / 2; d > 0; d >>= 1) {
      v[u].x += __shfl_xor_sync(0xffffffffu, v[u].x, d);
      v[u].y += __shfl_xor_sync(0xffffffffu, v[u].y, d);
    }
  }
}
template <int G>
__device__ __forceinline__ float group_sum(float a, float2* slot, int gw, int group) {
  a = warp_sum(a);
  if (G == 1) return a;
  const int lane = threadIdx.x & 31;
  if (lane == 0) slot[gw].x = a;
  group_barrier(group, 32 * G);
  float v = slot[lane & (G - 1)].x;
#pragma unroll
  for (int d = G / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// Ring stages: as many of `most` as fit beside the SM's other blocks.
constexpr size_t kRingBytes = 216 * 1024;
int ring_depth(size_t stage, int per_sm, int most) {
  int depth = most;
  while (depth > 1 && depth * stage > kRingBytes / per_sm) --depth;
  return depth;
}

constexpr int threads_of(int G) { return 32 * (G < 8 ? 8 : G); }  // a block: one group, or several small ones

// Blocks a SM of the forward kernel, which hold its registers down: four of
// 256 threads with wide chunks (16384 x 4096 bf16: 57 us with three, 42 with
// four), three with narrow ones, which would spill more with four (2791 x 2815
// fp32: 17 against 26 us).
constexpr int fwd_blocks(int C, int G) { return G == 32 ? 1 : (C > 2 ? 1024 : 768) / threads_of(G); }

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

// Weights and biases stay in registers (with 32 warps a group they are read
// again for every row, from L1).
template <typename T, int C, int E, int G>
__global__ void __launch_bounds__(threads_of(G), fwd_blocks(C, G)) layernorm_kernel(const NormFwd p, const int depth) {
  typedef Chunk<T, C> Ch;
  constexpr int kThreads = threads_of(G), groups = kThreads / (32 * G), span = 32 * G, kPairs = E * C / 2;
  constexpr int kStage = E * kThreads * Ch::kSlot;
  constexpr bool kKeepW = G < 32;
  extern __shared__ __align__(16) uint8_t ring[];  // [depth][E][threads] slots
  __shared__ float2 slots[2][32];
  const int group = threadIdx.x / span, t = threadIdx.x - group * span, gw = t >> 5;
  const long long stride = (long long)gridDim.x * groups;
  const T* x = static_cast<const T*>(p.x);
  const float inv_m = 1.f / (float)p.m;
  grid_dependency_wait();
  auto slot_of = [&](int stage, int i) { return ring + stage * kStage + (i * kThreads + threadIdx.x) * Ch::kSlot; };
  auto fetch = [&](long long r, int stage) {
    if (r < p.s) {
      const T* row = x + r * p.ldx;
#pragma unroll
      for (int i = 0; i < E; ++i) Ch::fetch(smem_addr(slot_of(stage, i)), row, (t + i * span) * C, p.m, true);
    }
    async_commit();
  };
  long long row = (long long)blockIdx.x * groups + group;
  for (int d = 0; d < depth - 1; ++d) fetch(row + d * stride, d);
  union Row {
    float f[E * C];
    float2 p2[kPairs];
  };
  [[maybe_unused]] Row w, b;
  auto load_wb = [&](const void* src, int is_f32, float none, Row& to) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = (t + i * span) * C;
#pragma unroll
      for (int j = 0; j < C; ++j) to.f[i * C + j] = none;
      if (src && c < p.m) load_weights<C>(src, is_f32, c, p.m, to.f + i * C);
    }
  };
  if constexpr (kKeepW) {
    load_wb(p.w, p.w_f32, 1.f, w);
    load_wb(p.b, p.b_f32, 0.f, b);
  }
  int stage = 0;
  for (; row < p.s; row += stride) {
    // the copies replace what the last iteration has read
    fetch(row + (depth - 1) * stride, stage == 0 ? depth - 1 : stage - 1);
    async_wait(depth - 1);
    Row v;
    float2 acc = both(0.f);
#pragma unroll
    for (int i = 0; i < E; ++i) Ch::get(slot_of(stage, i), x + row * p.ldx, v.f + i * C);
#pragma unroll
    for (int q = 0; q < kPairs; ++q) acc = add2(acc, v.p2[q]);
    const float mu = group_sum<G>(acc.x + acc.y, slots[0] + group * G, gw, group) * inv_m;
    acc = both(0.f);
#pragma unroll
    for (int q = 0; q < kPairs; ++q) v.p2[q] = add2(v.p2[q], both(-mu));
#pragma unroll
    for (int i = 0; i < E; ++i)  // columns past the row: no deviation
#pragma unroll
      for (int j = 0; j < C; ++j)
        if ((t + i * span) * C + (C == 2 ? j : 0) >= p.m) v.f[i * C + j] = 0.f;
#pragma unroll
    for (int q = 0; q < kPairs; ++q) acc = fma2(v.p2[q], v.p2[q], acc);
    const float var = group_sum<G>(acc.x + acc.y, slots[1] + group * G, gw, group) * inv_m;
    const float r = 1.f / sqrtf(var + p.eps);
    T* y = static_cast<T*>(p.y) + row * p.m;
    if constexpr (kKeepW) {
#pragma unroll
      for (int q = 0; q < kPairs; ++q) v.p2[q] = fma2(mul2(v.p2[q], both(r)), w.p2[q], b.p2[q]);
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = (t + i * span) * C;
      if (c < p.m) {
        if constexpr (!kKeepW) {
          float a[C];
#pragma unroll
          for (int j = 0; j < C; ++j) v.f[i * C + j] *= r;
          if (p.w) {
            load_weights<C>(p.w, p.w_f32, c, p.m, a);
#pragma unroll
            for (int j = 0; j < C; ++j) v.f[i * C + j] *= a[j];
          }
          if (p.b) {
            load_weights<C>(p.b, p.b_f32, c, p.m, a);
#pragma unroll
            for (int j = 0; j < C; ++j) v.f[i * C + j] += a[j];
          }
        }
        Ch::store(y, c, p.m, v.f + i * C);
      }
    }
    if (t == 0) {
      if (p.mean) p.mean[row] = mu;
      if (p.rstd) p.rstd[row] = r;
    }
    if (++stage == depth) stage = 0;
  }
  async_wait(0);
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
  for (int c = threadIdx.x; c < p.m; c += blockDim.x) sum += to_f<T>(ld_plain(x + c));
  const float inv_m = 1.f / (float)p.m;
  const float mu = group_sum<16>(sum, slots[0], gw, 0) * inv_m;
  float sq = 0.f;
  for (int c = threadIdx.x; c < p.m; c += blockDim.x) {
    const float d = to_f<T>(ld_plain(x + c)) - mu;
    sq = fmaf(d, d, sq);
  }
  const float r = 1.f / sqrtf(group_sum<16>(sq, slots[1], gw, 0) * inv_m + p.eps);
  T* y = static_cast<T*>(p.y) + row * p.m;
  for (int c = threadIdx.x; c < p.m; c += blockDim.x) {
    float o = (to_f<T>(ld_plain(x + c)) - mu) * r, v[1];
    if (p.w) {
      load_weights<1>(p.w, p.w_f32, c, p.m, v);
      o *= v[0];
    }
    if (p.b) {
      load_weights<1>(p.b, p.b_f32, c, p.m, v);
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

// A thread owns the same columns of all its group's rows, so dw and db
// accumulate in its registers without atomics.  Both passes over a row read
// it from the ring, which leaves the registers to the sums; with 32 warps a
// group the weights too are read again for each pass, from L1.  (Rows through
// registers, one row ahead, kept too little in flight: 143 us for 16384 x 4096
// bf16 with dres, now 90.)  With a ring of one stage nothing is fetched ahead; the
// other blocks of the SM, if any, fill the gap.  At the end a block's groups
// add up through shared memory, one after another, and the block writes one
// partial row; sum_parts_kernel adds those in a fixed order, so the gradients
// are the same on every run.
constexpr int bwd_blocks(int G) { return G < 16 ? 2 : 1; }  // a SM

// Rows a group works on at once: two, one barrier for both, where two stages
// of them fit in shared memory.
template <typename T, int C, int E, int G>
constexpr int rows_at_once() {
  return (size_t)2 * 2 * 2 * E * threads_of(G) * Chunk<T, C>::kSlot <= kRingBytes / bwd_blocks(G) ? 2 : 1;
}

template <typename T, int C, int E, int G>
__global__ void __launch_bounds__(threads_of(G), bwd_blocks(G)) layernorm_bwd_kernel(const NormBwd p, const int depth,
                                                                                      const int tensors) {
  typedef Chunk<T, C> Ch;
  constexpr int kThreads = threads_of(G), groups = kThreads / (32 * G), span = 32 * G;
  // values are worked on in pairs: one chunk a step, or two single-element chunks
  constexpr int kPer = C == 1 ? 2 : 1, kSteps = E / kPer, kHalf = kPer * C / 2;
  constexpr int kTensor = E * kThreads * Ch::kSlot, R = rows_at_once<T, C, E, G>();
  constexpr bool kKeepW = G < 32;
  extern __shared__ __align__(16) uint8_t ring[];  // [depth][R][dy, x, (dres)][E][threads] slots; later [2][m] fp32 sums
  __shared__ float2 slots[2][R][32];
  const int group = threadIdx.x / span, t = threadIdx.x - group * span, gw = t >> 5;
  const long long stride = (long long)gridDim.x * groups * R;
  const int row_bytes = tensors * kTensor;
  union Vals {
    float f[2 * kHalf];
    float2 p2[kHalf];
  };
  grid_dependency_wait();
  Vals wv[kKeepW ? kSteps : 1], dw[kSteps], db[kSteps];
  auto load_w = [&](Vals& to, int step) {
#pragma unroll
    for (int j = 0; j < 2 * kHalf; ++j) to.f[j] = 1.f;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int c = (t + (step * kPer + u) * span) * C;
      if (p.w && c < p.m) load_weights<C>(p.w, p.w_f32, c, p.m, to.f + u * C);
    }
  };
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
#pragma unroll
    for (int j = 0; j < kHalf; ++j) dw[i].p2[j] = db[i].p2[j] = both(0.f);
    if (kKeepW) load_w(wv[kKeepW ? i : 0], i);
  }
  const float inv_m = 1.f / (float)p.m;
  const T* dy = static_cast<const T*>(p.dy);
  const T* x = static_cast<const T*>(p.x);
  const T* dres = static_cast<const T*>(p.dres);
  auto slot_of = [&](int stage, int u, int q, int i) {
    return ring + (stage * R + u) * row_bytes + q * kTensor + (i * kThreads + threadIdx.x) * Ch::kSlot;
  };
  auto fetch = [&](long long r0, int stage) {
    if (r0 < p.s) {
#pragma unroll
      for (int u = 0; u < R; ++u) {
        const bool there = r0 + u < p.s;
        const long long r = there ? r0 + u : r0;
        const T *dy_row = dy + r * p.lddy, *x_row = x + r * p.ldx, *res_row = dres + r * p.lddres;
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const int c = (t + i * span) * C;
          Ch::fetch(smem_addr(slot_of(stage, u, 0, i)), dy_row, c, p.m, there);
          Ch::fetch(smem_addr(slot_of(stage, u, 1, i)), x_row, c, p.m, there);
          if (tensors == 3) Ch::fetch(smem_addr(slot_of(stage, u, 2, i)), res_row, c, p.m, there);
        }
      }
    }
    async_commit();
  };
  auto get = [&](Vals& to, int stage, int u, int q, const T* row, int step) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) Ch::get(slot_of(stage, u, q, step * kPer + k), row, to.f + k * C);
  };
  long long row = ((long long)blockIdx.x * groups + group) * R;
  for (int d = 0; d < depth - 1; ++d) fetch(row + d * stride, d);
  float mu[R], rs[R];
  auto load_stats = [&](long long r0) {
#pragma unroll
    for (int u = 0; u < R; ++u) {
      const long long r = r0 + u < p.s ? r0 + u : r0;
      if (r < p.s) {
        mu[u] = ld_plain(p.mean + r);
        rs[u] = ld_plain(p.rstd + r);
      }
    }
  };
  load_stats(row);
  int stage = 0;
  for (int it = 0; row < p.s; row += stride, ++it) {
    if (depth == 1) fetch(row, 0);
    async_wait(depth == 1 ? 0 : depth - 2);
    float mu_now[R], r_now[R];
    float2 s1[R], s2[R];
#pragma unroll
    for (int u = 0; u < R; ++u) {
      mu_now[u] = mu[u];
      r_now[u] = rs[u];
      s1[u] = s2[u] = both(0.f);
      // where there is no column, or no second row, dy is 0, and so is all that follows from it
      const T *dy_row = dy + (row + u) * p.lddy, *x_row = x + (row + u) * p.ldx;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        Vals d, xv;
        get(d, stage, u, 0, dy_row, i);
        get(xv, stage, u, 1, x_row, i);
        if (!kKeepW) load_w(wv[0], i);
#pragma unroll
        for (int j = 0; j < kHalf; ++j) {
          const float2 xh = mul2(add2(xv.p2[j], both(-mu_now[u])), both(r_now[u]));
          dw[i].p2[j] = fma2(d.p2[j], xh, dw[i].p2[j]);
          db[i].p2[j] = add2(db[i].p2[j], d.p2[j]);
          const float2 g = mul2(d.p2[j], wv[kKeepW ? i : 0].p2[j]);
          s1[u] = add2(s1[u], g);
          s2[u] = fma2(g, xh, s2[u]);
        }
      }
    }
    load_stats(row + stride);
    if (depth > 1) fetch(row + (depth - 1) * stride, stage == 0 ? depth - 1 : stage - 1);
    float2 sums[R];
#pragma unroll
    for (int u = 0; u < R; ++u) sums[u] = make_float2(s1[u].x + s1[u].y, s2[u].x + s2[u].y);
    group_sums<G, R>(sums, slots[it & 1], group * G, gw, group);
#pragma unroll
    for (int u = 0; u < R; ++u) {
      if (u > 0 && row + u >= p.s) break;
      const float c1 = -r_now[u] * (sums[u].x * inv_m), c2 = -r_now[u] * r_now[u] * (sums[u].y * inv_m);
      const T *dy_row = dy + (row + u) * p.lddy, *x_row = x + (row + u) * p.ldx, *res_row = dres + (row + u) * p.lddres;
      T* dx_row = static_cast<T*>(p.dx) + (row + u) * p.m;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        Vals g, xv, add;
        get(g, stage, u, 0, dy_row, i);
        get(xv, stage, u, 1, x_row, i);
        if (!kKeepW) load_w(wv[0], i);
        if (p.dres) {
          if (tensors == 3) {
            get(add, stage, u, 2, res_row, i);
          } else {
#pragma unroll
            for (int j = 0; j < 2 * kHalf; ++j) {
              const int c = (t + (i * kPer + j / C) * span) * C + j % C;
              add.f[j] = c < p.m ? to_f<T>(ld_plain(res_row + c)) : 0.f;
            }
          }
        }
#pragma unroll
        for (int j = 0; j < kHalf; ++j) {
          // r (g - c1 - xh c2), the deviation x - mu kept as one term
          float2 o = fma2(mul2(g.p2[j], wv[kKeepW ? i : 0].p2[j]), both(r_now[u]), both(c1));
          o = fma2(add2(xv.p2[j], both(-mu_now[u])), both(c2), o);
          g.p2[j] = p.dres ? add2(o, add.p2[j]) : o;
        }
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const int c = (t + (i * kPer + k) * span) * C;
          if (c < p.m) Ch::store(dx_row, c, p.m, g.f + k * C);
        }
      }
    }
    if (++stage == depth) stage = 0;
  }
  async_wait(0);
  grid_dependents_launch();
  if (!p.part) return;
  float* acc_smem = reinterpret_cast<float*>(ring);
  if (groups > 1) __syncthreads();  // every group is done with the ring
  for (int q = 0; q < groups; ++q) {
    const bool last = q == groups - 1;
    if (group == q) {
      float* out_w = p.part + (size_t)blockIdx.x * p.m;
      float* out_b = out_w + (size_t)p.parts * p.m;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const int c = (t + (i * kPer + k) * span) * C;
          if (c >= p.m) continue;
          float *a = dw[i].f + k * C, *b = db[i].f + k * C;
#pragma unroll
          for (int j = 0; j < C; ++j) {
            if (C == 2 && c + j >= p.m) continue;
            if (q > 0) {
              a[j] += acc_smem[c + j];
              b[j] += acc_smem[p.m + c + j];
            }
            if (!last) {
              acc_smem[c + j] = a[j];
              acc_smem[p.m + c + j] = b[j];
            } else if (C <= 2) {
              out_w[c + j] = a[j];
              out_b[c + j] = b[j];
            }
          }
          if (C > 2 && last) {
#pragma unroll
            for (int h = 0; h < C / 4; ++h) {
              *reinterpret_cast<uint4*>(out_w + c + 4 * h) = Vec<float>::from_float(a + 4 * h);
              *reinterpret_cast<uint4*>(out_b + c + 4 * h) = Vec<float>::from_float(b + 4 * h);
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
  __shared__ float2 slots[2][1][32];
  const int gw = threadIdx.x >> 5;
  const float inv_m = 1.f / (float)p.m;
  float* pw = p.part ? p.part + (size_t)blockIdx.x * p.m : nullptr;
  float* pb = p.part ? p.part + ((size_t)p.parts + blockIdx.x) * p.m : nullptr;
  int it = 0;
  for (long long row = blockIdx.x; row < p.s; row += gridDim.x, ++it) {
    const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const float mu = ld_plain(p.mean + row), r = ld_plain(p.rstd + row);
    float s1 = 0.f, s2 = 0.f;
    for (int c = threadIdx.x; c < p.m; c += blockDim.x) {
      float wv[1] = {1.f};
      if (p.w) load_weights<1>(p.w, p.w_f32, c, p.m, wv);
      const float d = to_f<T>(ld_plain(dy + c)), xh = (to_f<T>(ld_plain(x + c)) - mu) * r, g = d * wv[0];
      s1 += g;
      s2 = fmaf(g, xh, s2);
      if (pw) {
        pw[c] = it ? fmaf(d, xh, pw[c]) : d * xh;
        pb[c] = it ? pb[c] + d : d;
      }
    }
    float2 sums[1] = {make_float2(s1, s2)};
    group_sums<16, 1>(sums, slots[it & 1], 0, gw, 0);
    const float c1 = sums[0].x * inv_m, c2 = sums[0].y * inv_m;
    for (int c = threadIdx.x; c < p.m; c += blockDim.x) {
      float wv[1] = {1.f};
      if (p.w) load_weights<1>(p.w, p.w_f32, c, p.m, wv);
      const float g = to_f<T>(ld_plain(dy + c)) * wv[0], xh = (to_f<T>(ld_plain(x + c)) - mu) * r;
      float o = r * (g - c1 - xh * c2);
      if (p.dres) o += to_f<T>(ld_plain(static_cast<const T*>(p.dres) + row * p.lddres + c));
      static_cast<T*>(p.dx)[row * p.m + c] = from_f<T>(o);
    }
  }
}

// out[c] = sum over parts of part[q][c], for the two halves (blockIdx.y):
// 32 columns a block, 32 threads a column, each with its loads (ten for 304
// parts) in flight together, a fixed order over all.
__global__ void __launch_bounds__(1024) sum_parts_kernel(const float* part, int parts, int stride_parts, int m,
                                                         float* out0, float* out1) {
  __shared__ float acc[32][33];
  float* out = blockIdx.y ? out1 : out0;
  const int col = blockIdx.x * 32 + threadIdx.x;
  const float* src = part + (size_t)blockIdx.y * stride_parts * m;
  float v = 0.f;
  grid_dependency_wait();
  if (col < m) {
    for (int q0 = threadIdx.y; q0 < parts; q0 += 320) {
      float t[10];
#pragma unroll
      for (int i = 0; i < 10; ++i) t[i] = q0 + 32 * i < parts ? ld_plain(src + (size_t)(q0 + 32 * i) * m + col) : 0.f;
#pragma unroll
      for (int i = 0; i < 10; ++i) v += t[i];
    }
  }
  acc[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  grid_dependents_launch();
  const float sum = warp_sum(acc[threadIdx.x][threadIdx.y]);  // a warp for each column
  if (threadIdx.x == 0 && blockIdx.x * 32 + threadIdx.y < m && out) out[blockIdx.x * 32 + threadIdx.y] = sum;
}


int chunks_per_group(int chunks, int G) { return (chunks + 32 * G - 1) / (32 * G); }

template <typename T, int C, int E, int G>
cudaError_t run_fwd(const NormFwd& p, const DeviceInfo& di, cudaStream_t st) {
  constexpr int kThreads = threads_of(G), groups = kThreads / (32 * G), per_sm = fwd_blocks(C, G);
  constexpr size_t kStage = (size_t)E * kThreads * Chunk<T, C>::kSlot;
  static OncePerDevice once;
  cudaError_t err = once.run([] {
    return cudaFuncSetAttribute(layernorm_kernel<T, C, E, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRingBytes);
  });
  if (err != cudaSuccess) return err;
  const long long blocks = ((long long)p.s + groups - 1) / groups, most = (long long)per_sm * di.sms;
  const int grid = (int)(blocks < most ? blocks : most);
  // one row a group: nothing to fetch ahead; a third stage gained nothing over two
  const int depth = blocks <= most ? 1 : ring_depth(kStage, per_sm, 2);
  return launch_chained(layernorm_kernel<T, C, E, G>, dim3((unsigned)grid), dim3(kThreads), depth * kStage, st, p, depth);
}

template <typename T, int C>
cudaError_t fwd_for(const NormFwd& p, const DeviceInfo& di, cudaStream_t st) {
  // 16 elements a thread in the fewest warps; one warp may have fewer, 32 warps 32
  const int chunks = (p.m + C - 1) / C;
  int G = 1;
  while (G < 32 && chunks_per_group(chunks, G) * C > 16) G *= 2;
  const int need = chunks_per_group(chunks, G) * C;
  switch (G) {
    case 1: return need <= 8 ? run_fwd<T, C, 8 / C, 1>(p, di, st) : run_fwd<T, C, 16 / C, 1>(p, di, st);
    case 2: return run_fwd<T, C, 16 / C, 2>(p, di, st);
    case 4: return run_fwd<T, C, 16 / C, 4>(p, di, st);
    case 8: return run_fwd<T, C, 16 / C, 8>(p, di, st);
    case 16: return run_fwd<T, C, 16 / C, 16>(p, di, st);
    default: break;
  }
  if (need <= 16) return run_fwd<T, C, 16 / C, 32>(p, di, st);
  if (need <= 32) return run_fwd<T, C, 32 / C, 32>(p, di, st);
  layernorm_wide_kernel<T><<<(unsigned)p.s, 512, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int C, int E, int G>
cudaError_t run_bwd(const NormBwd& p, int* grid, const DeviceInfo& di, cudaStream_t st) {
  constexpr int kThreads = threads_of(G), groups = kThreads / (32 * G), per_sm = bwd_blocks(G), R = rows_at_once<T, C, E, G>();
  constexpr size_t kTensor = (size_t)R * E * kThreads * Chunk<T, C>::kSlot;
  static OncePerDevice once;
  cudaError_t err = once.run([] {
    return cudaFuncSetAttribute(layernorm_bwd_kernel<T, C, E, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRingBytes);
  });
  if (err != cudaSuccess) return err;
  // dres goes through the ring too, unless that leaves a single stage
  int tensors = p.dres && ring_depth(3 * kTensor, per_sm, 3) > 1 ? 3 : 2;
  const int depth = ring_depth(tensors * kTensor, per_sm, R == 2 || G == 32 ? 2 : 3);
  size_t smem = depth * tensors * kTensor;
  if (groups > 1 && smem < 2 * sizeof(float) * (size_t)p.m) smem = 2 * sizeof(float) * (size_t)p.m;
  const long long blocks = ((long long)p.s + groups * R - 1) / (groups * R), most = (long long)per_sm * di.sms;
  *grid = (int)(blocks < most ? blocks : most);
  if (*grid > p.parts) *grid = p.parts;
  return launch_chained(layernorm_bwd_kernel<T, C, E, G>, dim3((unsigned)*grid), dim3(kThreads), smem, st, p, depth, tensors);
}

template <typename T, int C>
cudaError_t bwd_for(const NormBwd& p, int* grid, const DeviceInfo& di, cudaStream_t st) {
  // as the forward pass, but at most 16 elements a thread: it holds their sums too
  const int chunks = (p.m + C - 1) / C;
  int G = 1;
  while (G < 32 && chunks_per_group(chunks, G) * C > 16) G *= 2;
  const int need = chunks_per_group(chunks, G) * C;
  if (need > 16) {
    *grid = p.s < di.sms ? p.s : di.sms;
    layernorm_bwd_wide_kernel<T><<<(unsigned)*grid, 512, 0, st>>>(p);
    return cudaGetLastError();
  }
  switch (G) {
    case 1: return need <= 8 ? run_bwd<T, C, 8 / C, 1>(p, grid, di, st) : run_bwd<T, C, 16 / C, 1>(p, grid, di, st);
    case 2: return run_bwd<T, C, 16 / C, 2>(p, grid, di, st);
    case 4: return run_bwd<T, C, 16 / C, 4>(p, grid, di, st);
    case 8: return run_bwd<T, C, 16 / C, 8>(p, grid, di, st);
    case 16: return run_bwd<T, C, 16 / C, 16>(p, grid, di, st);
    default: return run_bwd<T, C, 16 / C, 32>(p, grid, di, st);
  }
}

}  // namespace

cudaError_t launch_sum_parts(const float* part, int parts, int stride_parts, int m, float* out0, float* out1,
                             cudaStream_t st) {
  return launch_chained(sum_parts_kernel, dim3((unsigned)((m + 31) / 32), out1 ? 2 : 1), dim3(32, 32), 0, st, part, parts,
                        stride_parts, m, out0, out1);
}

cudaError_t launch_layernorm(const void* x, long long ldx, int s, int m, int dtype, const void* w, int w_dtype,
                             const void* b, int b_dtype, float eps, void* y, float* mean, float* rstd,
                             const DeviceInfo& di, cudaStream_t st) {
  NormFwd p = {x, w, b, y, mean, rstd, ldx, s, m, w_dtype == 0, b_dtype == 0, eps};
  const int vec = dtype == 0 ? 4 : 8;
  const bool whole = m % vec == 0 && ldx % vec == 0;
  if (dtype == 0) return whole ? fwd_for<float, 4>(p, di, st) : fwd_for<float, 1>(p, di, st);
  return whole ? fwd_for<__nv_bfloat16, 8>(p, di, st) : fwd_for<__nv_bfloat16, 2>(p, di, st);
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
    else err = whole ? bwd_for<__nv_bfloat16, 8>(p, &grid, di, st) : bwd_for<__nv_bfloat16, 2>(p, &grid, di, st);
    if (err != cudaSuccess) return err;
  }
  return sums ? launch_sum_parts(part, grid, p.parts, m, dw, db, st) : cudaSuccess;
}

}  // namespace moe
