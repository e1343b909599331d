// norm.cu -- the layer norm in front of the MoE block, forward and backward.
//
//   mu = mean(x), r = 1/sqrt(mean((x - mu)^2) + eps), xh = (x - mu) r
//   y  = xh w + b
//   g  = dy w;  dx = r (g - mean(g) - xh mean(g xh)) [+ dres]
//   dw = sum_rows dy xh;  db = sum_rows dy
//
// About ten flops an element: both directions are bound by device memory, so
// each row is read once.  A group of G warps owns a row at a time and walks
// over rows; its thread t holds chunks t, t + 32G, ... of 16 bytes, E of them.
// Rows come through a ring of stages in shared memory, filled by cp.async, the
// next rows on their way while one is worked on.
// Where all rows start on 16 bytes a thread copies and reads only its own
// chunks, and the ring needs no barrier.  Otherwise (kShift: an odd width, a
// strided view) a stage holds the aligned 16-byte pieces that cover the row, and
// a barrier stands between their copies and the reads.  Then it depends on the type:
//   bf16  a chunk is cut out of two pieces by the row's own offset, and results
//         go back through shared memory the same way, another barrier
//         (2791 x 2815 forward 13.6 us, backward 26.5; two elements at a time,
//         copied 4 bytes a lane without barriers, 20.5 and 40.0).
//   fp32  a chunk is two single elements, read and stored 4 bytes a lane, without
//         bank conflicts and coalesced (forward 12.8 us, backward 25.6; copied 4
//         bytes a lane too 15.1 and 29.8, cut out of pieces 17.2 and 38.6).
// Measured, 16384 x 4096 bf16: forward 42.5 us (6.3 TB/s), backward with the
// residual branch's gradient 84.2 us (6.4 TB/s), of which the weight gradients
// are 5; one row of 4096 2.6 us.
// The variance is taken around the mean (a second reduction over the
// registers), not as E[x^2] - mu^2, which cancels on rows with a large common
// offset.  All statistics and sums are fp32; each output is rounded once.
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

// cp.async of 16 bytes to shared memory, of which n are read (the rest: zeros).
__device__ __forceinline__ void async_copy(uint32_t dst, const void* src, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest n groups of this thread have landed.
__device__ __forceinline__ void async_wait(int n) {
  if (n >= 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (n == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Bytes that a row starts past a 16-byte boundary.
__device__ __forceinline__ int skew(const void* row) { return (int)(reinterpret_cast<uintptr_t>(row) & 15); }

// The 16 bytes that start `off` (0..15, even) bytes into the 32 bytes a, b.
__device__ __forceinline__ uint4 cut(const uint4& a, const uint4& b, int off) {
  const int sh = (off & 2) * 8;
  switch (off >> 2) {  // the same for the whole row
    case 0:
      return make_uint4(__funnelshift_r(a.x, a.y, sh), __funnelshift_r(a.y, a.z, sh), __funnelshift_r(a.z, a.w, sh),
                        __funnelshift_r(a.w, b.x, sh));
    case 1:
      return make_uint4(__funnelshift_r(a.y, a.z, sh), __funnelshift_r(a.z, a.w, sh), __funnelshift_r(a.w, b.x, sh),
                        __funnelshift_r(b.x, b.y, sh));
    case 2:
      return make_uint4(__funnelshift_r(a.z, a.w, sh), __funnelshift_r(a.w, b.x, sh), __funnelshift_r(b.x, b.y, sh),
                        __funnelshift_r(b.y, b.z, sh));
    default:
      return make_uint4(__funnelshift_r(a.w, b.x, sh), __funnelshift_r(b.x, b.y, sh), __funnelshift_r(b.y, b.z, sh),
                        __funnelshift_r(b.z, b.w, sh));
  }
}

// C weights starting at column c (fp32 or bf16 memory on 16 bytes); past m: 0.
template <int C>
__device__ __forceinline__ void load_weights(const void* w, int is_f32, int c, int m, float* f) {
  if (C == 1 || c + C > m) {
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

template <int G>
__device__ __forceinline__ void group_sync(int group) {
  if (G == 1) __syncwarp();
  else group_barrier(group, 32 * G);
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

constexpr int threads_of(int G) { return 32 * (G < 8 ? 8 : G); }  // a block: one group, or several small ones

// Copies the 16 bytes `at` bytes into the aligned pieces that cover a row (zeros
// past its end, or all where `there` is false).
template <typename T>
__device__ __forceinline__ void fetch_piece(uint8_t* img, const T* row, int at, int m, bool there) {
  const int off = skew(row), n = there ? min(16, max(0, off + m * (int)sizeof(T) - at)) : 0;
  const uint8_t* start = reinterpret_cast<const uint8_t*>(row) - off;
  async_copy(smem_addr(img + at), n > 0 ? start + at : start, n);
}

// How a group's threads share a row: chunks of C values, their places in
// shared memory (kSlots pieces of 16 bytes a row and group) and in the row.
template <typename T, int E, int G, bool kShift>
struct Form {
  static constexpr int C = 16 / (int)sizeof(T), kChunks = E;
  static constexpr int kThreads = threads_of(G), kGroups = kThreads / (32 * G), kSpan = 32 * G;
  static constexpr bool kCut = kShift;  // a chunk is not one piece: one piece more than chunks, read by other threads
  static constexpr bool kPut = kShift;  // results go through shared memory
  static constexpr int kSlots = E * kSpan + (kCut ? 1 : 0);
  static constexpr int kRow = kGroups * kSlots * 16;                   // bytes of one row of each group
  static constexpr int kOut = kPut ? kGroups * (kSlots + 1) * 16 : 0;  // and of its results

  // Column of value j of this thread's chunk i.
  __device__ __forceinline__ static int col(int t, int i, int j) { return (t + i * kSpan) * C + j; }
  static constexpr int kPieces = E + (kCut ? 1 : 0);
  // Copies of piece i < kPieces of a row (zeros where `there` is false or the row ends).
  __device__ __forceinline__ static void fetch(uint8_t* img, const T* row, int t, int i, int m, bool there) {
    if constexpr (kCut) {
      if (i < E || t == 0) fetch_piece(img, row, (i * kSpan + t) * 16, m, there);
    } else {
      const bool in = there && col(t, i, 0) < m;
      async_copy(smem_addr(img + (i * kSpan + t) * 16), in ? row + col(t, i, 0) : row, in ? 16 : 0);
    }
  }
  // Chunk i of this thread, as floats.
  __device__ __forceinline__ static void get(const uint8_t* img, int off, int t, int i, float* f) {
    const uint4* v = reinterpret_cast<const uint4*>(img) + i * kSpan + t;
    if constexpr (kCut) Vec<T>::to_float(cut(v[0], v[1], off), f);
    else Vec<T>::to_float(v[0], f);
  }
  __device__ __forceinline__ static void store(T* row, int t, int i, int, const float* f) {
    st_stream(reinterpret_cast<uint4*>(row + col(t, i, 0)), Vec<T>::from_float(f));
  }
  __device__ __forceinline__ static void weights(const void* w, int is_f32, int t, int i, int m, float* f) {
    load_weights<C>(w, is_f32, col(t, i, 0), m, f);
  }
  // Sums of chunk i to a partial row (of whole 16-byte pieces).
  __device__ __forceinline__ static void partial(float* row, int t, int i, int, const float* f) {
#pragma unroll
    for (int h = 0; h < C / 4; ++h)
      *reinterpret_cast<uint4*>(row + col(t, i, 4 * h)) = Vec<float>::from_float(f + 4 * h);
  }
  // kPut: chunk i of the results into the group's output pieces (one piece of
  // room before them), and, after a barrier, those to the row.
  __device__ __forceinline__ static void put(uint8_t* img, int t, int i, const float* f) {
    reinterpret_cast<uint4*>(img)[i * kSpan + t + 1] = Vec<T>::from_float(f);
  }
  __device__ __forceinline__ static void write(const uint8_t* img, T* row, int t, int m) {
    const int off = skew(row), bytes = m * (int)sizeof(T), n = (off + bytes + 15) / 16;
    const uint4* v = reinterpret_cast<const uint4*>(img);
    for (int q = t; q < n; q += kSpan) {
      const int lo = 16 * q - off;  // the piece's place in the row
      const uint4 u = off ? cut(v[q], v[q + 1], 16 - off) : v[q + 1];
      uint8_t* to = reinterpret_cast<uint8_t*>(row) + lo;
      if (lo >= 0 && lo + 16 <= bytes) {
        st_stream(reinterpret_cast<uint4*>(to), u);
      } else {
        float f[C];
        Vec<T>::to_float(u, f);
#pragma unroll
        for (int j = 0; j < C; ++j) {
          const int pos = lo + j * (int)sizeof(T);
          if (pos >= 0 && pos < bytes) *reinterpret_cast<T*>(to + j * sizeof(T)) = from_f<T>(f[j]);
        }
      }
    }
  }
};

// fp32 rows off 16 bytes: a chunk is two single elements, in columns
// t + (2 i + j) kSpan (four at once would spill registers).
template <int E, int G>
struct Form<float, E, G, true> {
  static constexpr int C = 2, kChunks = 2 * E;
  static constexpr int kThreads = threads_of(G), kGroups = kThreads / (32 * G), kSpan = 32 * G;
  static constexpr bool kCut = true, kPut = false;
  static constexpr int kSlots = E * kSpan + 1, kRow = kGroups * kSlots * 16, kOut = 0;

  __device__ __forceinline__ static int col(int t, int i, int j) { return t + (2 * i + j) * kSpan; }
  static constexpr int kPieces = E + 1;
  __device__ __forceinline__ static void fetch(uint8_t* img, const float* row, int t, int i, int m, bool there) {
    if (i < E || t == 0) fetch_piece(img, row, (i * kSpan + t) * 16, m, there);
  }
  __device__ __forceinline__ static void get(const uint8_t* img, int off, int t, int i, float* f) {
#pragma unroll
    for (int j = 0; j < C; ++j) f[j] = reinterpret_cast<const float*>(img + off)[col(t, i, j)];
  }
  __device__ __forceinline__ static void store(float* row, int t, int i, int m, const float* f) {
#pragma unroll
    for (int j = 0; j < C; ++j)
      if (col(t, i, j) < m) row[col(t, i, j)] = f[j];
  }
  __device__ __forceinline__ static void weights(const void* w, int is_f32, int t, int i, int m, float* f) {
#pragma unroll
    for (int j = 0; j < C; ++j) load_weights<1>(w, is_f32, col(t, i, j), m, f + j);
  }
  __device__ __forceinline__ static void partial(float* row, int t, int i, int m, const float* f) { store(row, t, i, m, f); }
  __device__ __forceinline__ static void put(uint8_t*, int, int, const float*) {}
  __device__ __forceinline__ static void write(const uint8_t*, float*, int, int) {}
};

// Ring stages: as many of `most` as fit beside the SM's other blocks.
constexpr size_t kRingBytes = 216 * 1024;
int ring_depth(size_t stage, size_t beside, int per_sm, int most) {
  int depth = most;
  while (depth > 1 && depth * stage + beside > kRingBytes / per_sm) --depth;
  return depth;
}

// Blocks a SM of the forward kernel, four of 256 threads, which hold its
// registers down (16384 x 4096 bf16: 57 us with three, 42 with four).
constexpr int fwd_blocks(int G) { return G == 32 ? 1 : 1024 / threads_of(G); }

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
template <typename T, int E, int G, bool kShift>
__global__ void __launch_bounds__(threads_of(G), fwd_blocks(G)) layernorm_kernel(const NormFwd p, const int depth) {
  typedef Form<T, E, G, kShift> F;
  constexpr int C = F::C, kChunks = F::kChunks, groups = F::kGroups, span = F::kSpan, kPairs = kChunks * C / 2;
  constexpr bool kKeepW = G < 32;
  extern __shared__ __align__(16) uint8_t ring[];  // [depth] rows, then the results' pieces
  __shared__ float2 slots[2][32];
  const int group = threadIdx.x / span, t = threadIdx.x - group * span, gw = t >> 5;
  const long long stride = (long long)gridDim.x * groups;
  const T* x = static_cast<const T*>(p.x);
  const float inv_m = 1.f / (float)p.m;
  grid_dependency_wait();
  auto image = [&](int stage) { return ring + stage * F::kRow + group * F::kSlots * 16; };
  uint8_t* out = ring + depth * F::kRow + group * (F::kSlots + 1) * 16;
  auto fetch = [&](long long r, int stage) {
    if (r < p.s) {
#pragma unroll
      for (int i = 0; i < F::kPieces; ++i) F::fetch(image(stage), x + r * p.ldx, t, i, p.m, true);
    }
    async_commit();
  };
  long long row = (long long)blockIdx.x * groups + group;
  for (int d = 0; d < depth - 1; ++d) fetch(row + d * stride, d);
  union Row {
    float f[kChunks * C];
    float2 p2[kPairs];
  };
  [[maybe_unused]] Row w, b;
  auto load_wb = [&](const void* src, int is_f32, float none, Row& to) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
#pragma unroll
      for (int j = 0; j < C; ++j) to.f[i * C + j] = none;
      if (src && F::col(t, i, 0) < p.m) F::weights(src, is_f32, t, i, p.m, to.f + i * C);
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
    if (F::kCut) group_sync<G>(group);  // the others' pieces too
    Row v;
    float2 acc = both(0.f);
    const int off = F::kCut ? skew(x + row * p.ldx) : 0;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) F::get(image(stage), off, t, i, v.f + i * C);
#pragma unroll
    for (int q = 0; q < kPairs; ++q) acc = add2(acc, v.p2[q]);
    const float mu = group_sum<G>(acc.x + acc.y, slots[0] + group * G, gw, group) * inv_m;
    acc = both(0.f);
#pragma unroll
    for (int q = 0; q < kPairs; ++q) v.p2[q] = add2(v.p2[q], both(-mu));
#pragma unroll
    for (int i = 0; i < kChunks; ++i)  // columns past the row: no deviation
#pragma unroll
      for (int j = 0; j < C; ++j)
        if (F::col(t, i, kShift ? j : 0) >= p.m) v.f[i * C + j] = 0.f;
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
    for (int i = 0; i < kChunks; ++i) {
      if (F::col(t, i, 0) < p.m) {
        if constexpr (!kKeepW) {
          float a[C];
#pragma unroll
          for (int j = 0; j < C; ++j) v.f[i * C + j] *= r;
          if (p.w) {
            F::weights(p.w, p.w_f32, t, i, p.m, a);
#pragma unroll
            for (int j = 0; j < C; ++j) v.f[i * C + j] *= a[j];
          }
          if (p.b) {
            F::weights(p.b, p.b_f32, t, i, p.m, a);
#pragma unroll
            for (int j = 0; j < C; ++j) v.f[i * C + j] += a[j];
          }
        }
        if constexpr (F::kPut) F::put(out, t, i, v.f + i * C);
        else F::store(y, t, i, p.m, v.f + i * C);
      }
    }
    if constexpr (F::kPut) {  // the barriers of the next row come before the next put
      group_sync<G>(group);
      F::write(out, y, t, p.m);
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
  int s, m, w_f32, parts, mp;  // mp: floats of a partial row, m up to a multiple of 8
};

// A thread owns the same columns of all its group's rows, so dw and db
// accumulate in its registers without atomics.  Both passes over a row read
// it from the ring, which leaves the registers to the sums; with 32 warps a
// group the weights too are read again for each pass, from L1.  (Rows through
// registers, one row ahead, kept too little in flight: 143 us for 16384 x 4096
// bf16 with dres, now 84.)  With a ring of one stage nothing is fetched ahead; the
// other blocks of the SM, if any, fill the gap.  At the end a block's groups
// add up through shared memory, one after another, and the block writes one
// partial row; sum_parts_kernel adds those in a fixed order, so the gradients
// are the same on every run.
constexpr int bwd_blocks(int G) { return G < 16 ? 2 : 1; }  // a SM

// Rows a group works on at once: two, one barrier for both, where two stages
// of them fit in shared memory.
template <typename T, int E, int G, bool kShift>
constexpr int rows_at_once() {
  typedef Form<T, E, G, kShift> F;
  return (size_t)2 * 2 * 2 * F::kRow + 2 * F::kOut <= kRingBytes / bwd_blocks(G) ? 2 : 1;
}

template <typename T, int E, int G, bool kShift>
__global__ void __launch_bounds__(threads_of(G), bwd_blocks(G)) layernorm_bwd_kernel(const NormBwd p, const int depth,
                                                                                     const int tensors) {
  typedef Form<T, E, G, kShift> F;
  constexpr int C = F::C, kChunks = F::kChunks, groups = F::kGroups, span = F::kSpan, kHalf = C / 2;
  constexpr int R = rows_at_once<T, E, G, kShift>();
  constexpr bool kKeepW = G < 32;
  extern __shared__ __align__(16) uint8_t ring[];  // [depth][R][dy, x, (dres)] rows, the results' pieces; later [2][m] sums
  __shared__ float2 slots[2][R][32];
  const int group = threadIdx.x / span, t = threadIdx.x - group * span, gw = t >> 5;
  const long long stride = (long long)gridDim.x * groups * R;
  union Vals {
    float f[C];
    float2 p2[kHalf];
  };
  grid_dependency_wait();
  Vals wv[kKeepW ? kChunks : 1], dw[kChunks], db[kChunks];
  auto load_w = [&](Vals& to, int i) {
#pragma unroll
    for (int j = 0; j < C; ++j) to.f[j] = 1.f;
    if (p.w && F::col(t, i, 0) < p.m) F::weights(p.w, p.w_f32, t, i, p.m, to.f);
  };
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
#pragma unroll
    for (int j = 0; j < kHalf; ++j) dw[i].p2[j] = db[i].p2[j] = both(0.f);
    if (kKeepW) load_w(wv[kKeepW ? i : 0], i);
  }
  const float inv_m = 1.f / (float)p.m;
  const T* dy = static_cast<const T*>(p.dy);
  const T* x = static_cast<const T*>(p.x);
  const T* dres = static_cast<const T*>(p.dres);
  const int row_bytes = tensors * F::kRow;
  auto image = [&](int stage, int u, int q) {
    return ring + (stage * R + u) * row_bytes + q * F::kRow + group * F::kSlots * 16;
  };
  uint8_t* out = ring + depth * R * tensors * F::kRow + group * (F::kSlots + 1) * 16;  // and F::kOut on, the second row's
  auto fetch = [&](long long r0, int stage) {
    if (r0 < p.s) {
#pragma unroll
      for (int u = 0; u < R; ++u) {
        const bool there = r0 + u < p.s;
        const long long r = there ? r0 + u : r0;
        const T *dy_row = dy + r * p.lddy, *x_row = x + r * p.ldx, *res_row = dres + r * p.lddres;
#pragma unroll
        for (int i = 0; i < F::kPieces; ++i) {
          F::fetch(image(stage, u, 0), dy_row, t, i, p.m, there);
          F::fetch(image(stage, u, 1), x_row, t, i, p.m, there);
          if (tensors == 3) F::fetch(image(stage, u, 2), res_row, t, i, p.m, there);
        }
      }
    }
    async_commit();
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
    if (depth == 1) {
      if (F::kCut) group_sync<G>(group);  // the last row has been read by all
      fetch(row, 0);
    }
    async_wait(depth == 1 ? 0 : depth - 2);
    if (F::kCut) group_sync<G>(group);  // the others' pieces too
    float mu_now[R], r_now[R];
    float2 s1[R], s2[R];
#pragma unroll
    for (int u = 0; u < R; ++u) {
      mu_now[u] = mu[u];
      r_now[u] = rs[u];
      s1[u] = s2[u] = both(0.f);
      // where there is no column, or no second row, dy is 0, and so is all that follows from it
      const int dy_off = F::kCut ? skew(dy + (row + u) * p.lddy) : 0, x_off = F::kCut ? skew(x + (row + u) * p.ldx) : 0;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        Vals d, xv;
        F::get(image(stage, u, 0), dy_off, t, i, d.f);
        F::get(image(stage, u, 1), x_off, t, i, xv.f);
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
      const T* res_row = dres + (row + u) * p.lddres;
      const int dy_off = F::kCut ? skew(dy + (row + u) * p.lddy) : 0, x_off = F::kCut ? skew(x + (row + u) * p.ldx) : 0;
      const int res_off = F::kCut ? skew(res_row) : 0;
      T* dx_row = static_cast<T*>(p.dx) + (row + u) * p.m;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        Vals g, xv, add;
        F::get(image(stage, u, 0), dy_off, t, i, g.f);
        F::get(image(stage, u, 1), x_off, t, i, xv.f);
        if (!kKeepW) load_w(wv[0], i);
        if (p.dres) {
          if (tensors == 3) {
            F::get(image(stage, u, 2), res_off, t, i, add.f);
          } else {
#pragma unroll
            for (int j = 0; j < C; ++j) add.f[j] = F::col(t, i, j) < p.m ? to_f<T>(ld_plain(res_row + F::col(t, i, j))) : 0.f;
          }
        }
#pragma unroll
        for (int j = 0; j < kHalf; ++j) {
          // r (g - c1 - xh c2), the deviation x - mu kept as one term
          float2 o = fma2(mul2(g.p2[j], wv[kKeepW ? i : 0].p2[j]), both(r_now[u]), both(c1));
          o = fma2(add2(xv.p2[j], both(-mu_now[u])), both(c2), o);
          g.p2[j] = p.dres ? add2(o, add.p2[j]) : o;
        }
        if (F::col(t, i, 0) < p.m) {
          if constexpr (F::kPut) F::put(out + u * F::kOut, t, i, g.f);
          else F::store(dx_row, t, i, p.m, g.f);
        }
      }
    }
    if constexpr (F::kPut) {  // the barriers of the next rows come before the next put
      group_sync<G>(group);
#pragma unroll
      for (int u = 0; u < R; ++u)
        if (row + u < p.s) F::write(out + u * F::kOut, static_cast<T*>(p.dx) + (row + u) * p.m, t, p.m);
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
      float* out_w = p.part + (size_t)blockIdx.x * p.mp;
      float* out_b = out_w + (size_t)p.parts * p.mp;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        if (F::col(t, i, 0) >= p.m) continue;
        float *a = dw[i].f, *b = db[i].f;
#pragma unroll
        for (int j = 0; j < C; ++j) {
          const int c = F::col(t, i, j);
          if (kShift && c >= p.m) continue;
          if (q > 0) {
            a[j] += acc_smem[c];
            b[j] += acc_smem[p.m + c];
          }
          if (!last) {
            acc_smem[c] = a[j];
            acc_smem[p.m + c] = b[j];
          }
        }
        if (last) {
          F::partial(out_w, t, i, p.m, a);
          F::partial(out_b, t, i, p.m, b);
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
  float* pw = p.part ? p.part + (size_t)blockIdx.x * p.mp : nullptr;
  float* pb = p.part ? p.part + ((size_t)p.parts + blockIdx.x) * p.mp : nullptr;
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
__global__ void __launch_bounds__(1024) sum_parts_kernel(const float* part, int parts, int stride_parts, int m, int mp,
                                                         float* out0, float* out1) {
  __shared__ float acc[32][33];
  float* out = blockIdx.y ? out1 : out0;
  const int col = blockIdx.x * 32 + threadIdx.x;
  const float* src = part + (size_t)blockIdx.y * stride_parts * mp;
  float v = 0.f;
  grid_dependency_wait();
  if (col < m) {
    for (int q0 = threadIdx.y; q0 < parts; q0 += 320) {
      float t[10];
#pragma unroll
      for (int i = 0; i < 10; ++i) t[i] = q0 + 32 * i < parts ? ld_plain(src + (size_t)(q0 + 32 * i) * mp + col) : 0.f;
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

template <typename T, int E, int G, bool kShift>
cudaError_t run_fwd(const NormFwd& p, const DeviceInfo& di, cudaStream_t st) {
  typedef Form<T, E, G, kShift> F;
  constexpr int per_sm = fwd_blocks(G);
  static OncePerDevice once;
  cudaError_t err = once.run([] {
    return cudaFuncSetAttribute(layernorm_kernel<T, E, G, kShift>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRingBytes);
  });
  if (err != cudaSuccess) return err;
  const long long blocks = ((long long)p.s + F::kGroups - 1) / F::kGroups, most = (long long)per_sm * di.sms;
  const int grid = (int)(blocks < most ? blocks : most);
  // one row a group: nothing to fetch ahead; a third stage gained nothing over two
  const int depth = blocks <= most ? 1 : ring_depth(F::kRow, F::kOut, per_sm, 2);
  return launch_chained(layernorm_kernel<T, E, G, kShift>, dim3((unsigned)grid), dim3(F::kThreads), depth * F::kRow + F::kOut,
                        st, p, depth);
}

template <typename T, bool kShift>
cudaError_t fwd_for(const NormFwd& p, const DeviceInfo& di, cudaStream_t st) {
  // 16 elements a thread in the fewest warps; one warp may have fewer, 32 warps 32
  constexpr int C = 16 / (int)sizeof(T);
  const int chunks = (p.m + C - 1) / C;
  int G = 1;
  while (G < 32 && chunks_per_group(chunks, G) * C > 16) G *= 2;
  const int need = chunks_per_group(chunks, G) * C;
  switch (G) {
    case 1: return need <= 8 ? run_fwd<T, 8 / C, 1, kShift>(p, di, st) : run_fwd<T, 16 / C, 1, kShift>(p, di, st);
    case 2: return run_fwd<T, 16 / C, 2, kShift>(p, di, st);
    case 4: return run_fwd<T, 16 / C, 4, kShift>(p, di, st);
    case 8: return run_fwd<T, 16 / C, 8, kShift>(p, di, st);
    case 16: return run_fwd<T, 16 / C, 16, kShift>(p, di, st);
    default: break;
  }
  if (need <= 16) return run_fwd<T, 16 / C, 32, kShift>(p, di, st);
  if (need <= 32) return run_fwd<T, 32 / C, 32, kShift>(p, di, st);
  layernorm_wide_kernel<T><<<(unsigned)p.s, 512, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int E, int G, bool kShift>
cudaError_t run_bwd(const NormBwd& p, int* grid, const DeviceInfo& di, cudaStream_t st) {
  typedef Form<T, E, G, kShift> F;
  constexpr int per_sm = bwd_blocks(G), R = rows_at_once<T, E, G, kShift>();
  constexpr size_t kRows = (size_t)R * F::kRow, kOut = (size_t)R * F::kOut;
  static OncePerDevice once;
  cudaError_t err = once.run([] {
    return cudaFuncSetAttribute(layernorm_bwd_kernel<T, E, G, kShift>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)kRingBytes);
  });
  if (err != cudaSuccess) return err;
  // dres goes through the ring too, unless that leaves a single stage
  const int tensors = p.dres && ring_depth(3 * kRows, kOut, per_sm, 3) > 1 ? 3 : 2;
  const int depth = ring_depth(tensors * kRows, kOut, per_sm, R == 2 || G == 32 ? 2 : 3);
  size_t smem = depth * tensors * kRows + kOut;
  if (F::kGroups > 1 && smem < 2 * sizeof(float) * (size_t)p.m) smem = 2 * sizeof(float) * (size_t)p.m;
  const long long blocks = ((long long)p.s + F::kGroups * R - 1) / (F::kGroups * R), most = (long long)per_sm * di.sms;
  *grid = (int)(blocks < most ? blocks : most);
  if (*grid > p.parts) *grid = p.parts;
  return launch_chained(layernorm_bwd_kernel<T, E, G, kShift>, dim3((unsigned)*grid), dim3(F::kThreads), smem, st, p, depth,
                        tensors);
}

template <typename T, bool kShift>
cudaError_t bwd_for(const NormBwd& p, int* grid, const DeviceInfo& di, cudaStream_t st) {
  // as the forward pass, but at most 16 elements a thread: it holds their sums too
  constexpr int C = 16 / (int)sizeof(T);
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
    case 1: return need <= 8 ? run_bwd<T, 8 / C, 1, kShift>(p, grid, di, st) : run_bwd<T, 16 / C, 1, kShift>(p, grid, di, st);
    case 2: return run_bwd<T, 16 / C, 2, kShift>(p, grid, di, st);
    case 4: return run_bwd<T, 16 / C, 4, kShift>(p, grid, di, st);
    case 8: return run_bwd<T, 16 / C, 8, kShift>(p, grid, di, st);
    case 16: return run_bwd<T, 16 / C, 16, kShift>(p, grid, di, st);
    default: return run_bwd<T, 16 / C, 32, kShift>(p, grid, di, st);
  }
}

}  // namespace

cudaError_t launch_sum_parts(const float* part, int parts, int stride_parts, int m, int mp, float* out0, float* out1,
                             cudaStream_t st) {
  return launch_chained(sum_parts_kernel, dim3((unsigned)((m + 31) / 32), out1 ? 2 : 1), dim3(32, 32), 0, st, part, parts,
                        stride_parts, m, mp, out0, out1);
}

cudaError_t launch_layernorm(const void* x, long long ldx, int s, int m, int dtype, const void* w, int w_dtype,
                             const void* b, int b_dtype, float eps, void* y, float* mean, float* rstd,
                             const DeviceInfo& di, cudaStream_t st) {
  NormFwd p = {x, w, b, y, mean, rstd, ldx, s, m, w_dtype == 0, b_dtype == 0, eps};
  const int vec = dtype == 0 ? 4 : 8;
  const bool whole = m % vec == 0 && ldx % vec == 0;
  if (dtype == 0) return whole ? fwd_for<float, false>(p, di, st) : fwd_for<float, true>(p, di, st);
  return whole ? fwd_for<__nv_bfloat16, false>(p, di, st) : fwd_for<__nv_bfloat16, true>(p, di, st);
}

cudaError_t launch_layernorm_bwd(const void* dy, long long lddy, const void* x, long long ldx, const void* dres,
                                 long long lddres, int s, int m, int dtype, const void* w, int w_dtype,
                                 const float* mean, const float* rstd, void* dx, float* dw, float* db, float* part,
                                 const DeviceInfo& di, cudaStream_t st) {
  const bool sums = dw || db;
  NormBwd p = {dy, x, w, dres, mean, rstd, dx, sums ? part : nullptr, lddy, ldx, lddres, s, m, w_dtype == 0, layernorm_bwd_parts(s), (m + 7) / 8 * 8};
  const int vec = dtype == 0 ? 4 : 8;
  const bool whole = m % vec == 0 && ldx % vec == 0 && lddy % vec == 0 && (!dres || lddres % vec == 0);
  int grid = 0;
  if (s > 0) {
    cudaError_t err;
    if (dtype == 0) err = whole ? bwd_for<float, false>(p, &grid, di, st) : bwd_for<float, true>(p, &grid, di, st);
    else err = whole ? bwd_for<__nv_bfloat16, false>(p, &grid, di, st) : bwd_for<__nv_bfloat16, true>(p, &grid, di, st);
    if (err != cudaSuccess) return err;
  }
  return sums ? launch_sum_parts(part, grid, p.parts, m, p.mp, dw, db, st) : cudaSuccess;
}

}  // namespace moe
