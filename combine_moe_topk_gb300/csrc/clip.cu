// clip.cu -- the global 2-norm of a list of gradients, and clipping to it.
//
//   norm = sqrt(sum over tensors and elements of g^2)
//   g'   = g min(1, max_norm / (norm + 1e-6))
//
// Bound by memory: every gradient is read once for the norm and, where it is
// clipped, read again and written.  The tensors travel in the kernels'
// parameters (up to 1024 a launch), so a call copies no table to the device and
// can be captured.  Each is cut into chunks of 32 KB; a block takes every
// gridDim-th of all chunks (with a contiguous range for each block the norm of
// 1.2 G bf16 took 559 us, 1183 with the clipping), and the second pass goes
// backwards, so that what the first read last is still in L2.  1.2 G bf16, to other
// tensors: 1077 us, against 1066 for three passes at the copy's rate; 301 odd pieces
// of 110 MB together 63 us.  Where a tensor and its place in `out` lie differently on
// 16 bytes, elements are stored one by one: 200 M bf16 190 us, 634 so; fp32 374 and 389.
// Eight 16-byte pieces a thread in two blocks an SM: four
// in four took 1111 us, eight in four 1441.
//
// The squares of a thread's 64 (32) elements of a chunk are added in fp32, half of
// them at a time, the chunks' sums in two fp32 terms (the second what the first's
// additions rounded off; 64-bit additions are slow on this GPU), everything beyond
// a thread in 64 bits.  Beside them runs the largest magnitude: where a block's is
// so large or so small that squares leave fp32's range, the block goes over its
// chunks again with the values scaled by a power of two.  Blocks write one 64-bit
// sum each, joined in a fixed order: the same bits on every run.
#include <math_constants.h>

#include "common.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace moe {

namespace {

typedef __nv_bfloat16 bf16;

constexpr int kThreads = 256;
constexpr int kUnroll = 8;                             // 16-byte pieces a thread of a chunk
constexpr int kChunkBytes = kThreads * kUnroll * 16;   // 32 KB
constexpr int kPerSm = 2;                              // blocks: 64 KB of loads in flight an SM
constexpr int kMaxBlocks = kPerSm * 152;
constexpr int kLarge = 1024, kSmall = 64;              // tensors a launch
constexpr float kEps = 1e-6f;
// Largest magnitude whose squares a thread adds unscaled.  A block has at most 2^30 / 304
// of a list's chunks, under 2^22, and a thread 64 elements of each: 2^28 squares of 2^96.
constexpr float kTop = 281474976710656.f;               // 2^48
constexpr float kLow = 8.8817841970012523e-16f;         // 2^-50: below it squares would lose bits

// chunk c of tensor i: first[i] <= c < first[i + 1] (the last ends at `chunks`).
template <int C>
struct Table {
  int count, chunks;
  const void* p[C];
  void* q[C];        // where the clipped values go
  long long n[C];    // elements
  int first[C];
  uint8_t f32[C];
};
static_assert(sizeof(Table<kLarge>) + 128 <= 32764, "a launch's parameters");

template <typename T>
__device__ __forceinline__ float one(const T* p);
template <>
__device__ __forceinline__ float one(const float* p) { return ld_plain(p); }
template <>
__device__ __forceinline__ float one(const bf16* p) { return __bfloat162float(ld_plain(p)); }

// Elements before the first 16-byte boundary, at most n.
template <typename T>
__device__ __forceinline__ int head_of(const T* p, long long n) {
  const int h = (int)(((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T));
  return n < h ? (int)n : h;
}

// Chunk c (of its tensor) of n elements at p: whole 16-byte pieces past the head; the
// first chunk takes the head too, and the last what follows the last piece.
struct Span {
  long long first;   // element
  int pieces, lead, trail;  // trail elements follow the pieces
};
template <typename T>
__device__ __forceinline__ Span span_of(const T* p, long long n, int c) {
  constexpr int kElems = 16 / sizeof(T), kChunk = kChunkBytes / sizeof(T);
  const int head = head_of(p, n);
  Span s;
  s.lead = c == 0 ? head : 0;
  s.first = head + (long long)c * kChunk;
  const long long left = n - s.first;
  s.pieces = left >= kChunk ? kThreads * kUnroll : (int)(left / kElems);
  s.trail = left < kChunk ? (int)(left - (long long)s.pieces * kElems) : 0;
  return s;
}

// The tensor of chunk c; i: that of the chunk before, which it may be too.
template <int C>
__device__ __forceinline__ int tensor_of(const Table<C>& t, int c, int i) {
  if (t.first[i] <= c && c < (i + 1 < t.count ? t.first[i + 1] : t.chunks)) return i;
  int lo = 0, hi = t.count;  // empty tensors have no chunk: the last that starts at c or before has it
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.first[mid] <= c) lo = mid; else hi = mid;
  }
  return lo;
}

// meanwhile: done between the loads and their use (the search for the next chunk's
// tensor, whose parameters come one after another from far away: 301 tensors of 110
// MB, norm and clipping, 67.4 -> 64.8 us).
template <typename T, bool kScaled, typename F>
__device__ __forceinline__ float squares(const T* p, long long n, int c, float scale, float& top, F meanwhile) {
  constexpr int kElems = 16 / sizeof(T);
  const Span s = span_of(p, n, c);
  const uint4* at = reinterpret_cast<const uint4*>(p + s.first);
  uint4 v[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int k = threadIdx.x + i * kThreads;
    v[i] = k < s.pieces ? ld_stream(at + k) : make_uint4(0, 0, 0, 0);
  }
  meanwhile();
  float half[2] = {0.f, 0.f};
  auto add = [&](float f, int i) {
    if (kScaled) f *= scale;
    half[i & 1] = fmaf(f, f, half[i & 1]);
    top = fmaxf(top, fabsf(f));
  };
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    float f[kElems];
    Vec<T>::to_float(v[i], f);
#pragma unroll
    for (int j = 0; j < kElems; ++j) add(f[j], i);
  }
  if ((int)threadIdx.x < s.lead) add(one(p + threadIdx.x), 0);
  if ((int)threadIdx.x < s.trail) add(one(p + s.first + (long long)s.pieces * kElems + threadIdx.x), 1);
  return half[0] + half[1];
}

// The block's chunks: this thread's sum of squares (of scaled values) and largest magnitude.
template <int C, bool kScaled>
__device__ __forceinline__ double sum_range(const Table<C>& t, float scale, float& top) {
  float sum = 0.f, low = 0.f;
  int i = t.chunks ? tensor_of(t, blockIdx.x, 0) : 0, then = i;
  for (int c = blockIdx.x; c < t.chunks; c += gridDim.x, i = then) {
    auto next = [&]() {
      if (c + (int)gridDim.x < t.chunks) then = tensor_of(t, c + (int)gridDim.x, i);
    };
    const int k = c - t.first[i];
    const float v = t.f32[i] ? squares<float, kScaled>(static_cast<const float*>(t.p[i]), t.n[i], k, scale, top, next)
                             : squares<bf16, kScaled>(static_cast<const bf16*>(t.p[i]), t.n[i], k, scale, top, next);
    const float s = sum + v, b = s - sum;
    low += (sum - (s - b)) + (v - b);
    sum = s;
  }
  // past fp32's range, or of a NaN: what was rounded off is none
  return sum < CUDART_INF_F ? (double)sum + (double)low : (double)sum;
}

__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) v += red[w];
  return v;
}

__device__ __forceinline__ float block_max(float v, float* red) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) v = fmaxf(v, red[w]);
  return v;
}

// This block's sum of squares, in every thread.
template <int C>
__device__ __forceinline__ double sum_block(const Table<C>& t, double* red) {
  float top = 0.f;
  double sum = sum_range<C, false>(t, 1.f, top);
  top = block_max(top, reinterpret_cast<float*>(red));
  if (top < CUDART_INF_F && (top > kTop || (top > 0.f && top < kLow))) {
    const int e = ilogbf(top);
    const int by = e < -100 ? 100 : -e;  // e goes down to -149, 2^149 is out of range
    float unused = 0.f;
    sum = ldexp(sum_range<C, true>(t, ldexpf(1.f, by), unused), -2 * by);
  }
  return block_sum(sum, red);
}

template <int C>
__global__ void __launch_bounds__(kThreads, kPerSm) grad_norm_kernel(const __grid_constant__ Table<C> t, double* part) {
  __shared__ double red[kThreads / 32];
  grid_dependency_wait();
  const double sum = sum_block(t, red);
  grid_dependents_launch();
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// All blocks' sums, by every thread of a block.
__device__ __forceinline__ double join(const double* part, int parts, double* red) {
  double v = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) v += ld_plain(part + i);
  return block_sum(v, red);
}

__device__ __forceinline__ float norm_of(double total) { return (float)sqrt(total); }  // an infinity past fp32's range

__device__ __forceinline__ void report(double total, float* norm, int32_t* status) {
  const float n = norm_of(total);
  *norm = n;
  if (!(n < CUDART_INF_F)) raise_status(status, MOE_DEV_NONFINITE);
}

__global__ void __launch_bounds__(kThreads) grad_norm_join_kernel(const double* part, int parts, float* norm, int32_t* status) {
  __shared__ double red[kThreads / 32];
  grid_dependency_wait();
  const double total = join(part, parts, red);
  grid_dependents_launch();
  if (threadIdx.x == 0) report(total, norm, status);
}

template <typename T>
__device__ __forceinline__ T rounded(float v);
template <>
__device__ __forceinline__ float rounded<float>(float v) { return v; }
template <>
__device__ __forceinline__ bf16 rounded<bf16>(float v) { return __float2bfloat16_rn(v); }

// Loads and stores that give way in L2 first: the second pass is done with what it
// reads and writes, while what the first pass read and the second has not come to
// yet should stay.
__device__ __forceinline__ uint64_t policy_first() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint4 ld_first(const uint4* p, uint64_t policy) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.u32 {%0,%1,%2,%3}, [%4], %5;"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p), "l"(policy));
  return v;
}
__device__ __forceinline__ void st_first(uint4* p, const uint4& v, uint64_t policy) {
  asm volatile("st.global.L2::cache_hint.v4.u32 [%0], {%1,%2,%3,%4}, %5;" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w),
               "l"(policy)
               : "memory");
}

// The chunk times coef; its bits where it is not to be scaled (a NaN's too).
template <typename T, typename F>
__device__ __forceinline__ void scale_chunk(const T* p, T* q, long long n, int c, bool scales, float coef, F meanwhile) {
  constexpr int kElems = 16 / sizeof(T);
  const Span s = span_of(p, n, c);
  const uint4* at = reinterpret_cast<const uint4*>(p + s.first);
  const uint64_t policy = policy_first();
  uint4 v[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int k = threadIdx.x + i * kThreads;
    if (k < s.pieces) v[i] = ld_first(at + k, policy);
  }
  meanwhile();
  const bool whole = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15) == 0;
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int k = threadIdx.x + i * kThreads;
    if (k >= s.pieces) continue;
    if (scales) {
      float f[kElems];
      Vec<T>::to_float(v[i], f);
#pragma unroll
      for (int j = 0; j < kElems; ++j) f[j] *= coef;
      v[i] = Vec<T>::from_float(f);
    }
    if (whole) {
      st_first(reinterpret_cast<uint4*>(q + s.first) + k, v[i], policy);
    } else {
      T* to = q + s.first + (long long)k * kElems;
      __align__(16) T e[kElems];
      *reinterpret_cast<uint4*>(e) = v[i];
#pragma unroll
      for (int j = 0; j < kElems; ++j) to[j] = e[j];
    }
  }
  auto single = [&](long long k) { q[k] = scales ? rounded<T>(one(p + k) * coef) : ld_plain(p + k); };
  if ((int)threadIdx.x < s.lead) single(threadIdx.x);
  if ((int)threadIdx.x < s.trail) single(s.first + (long long)s.pieces * kElems + threadIdx.x);
}

// This block's chunks, from the last to the first, clipped to max_norm; n is the norm
// as the caller sees it, so that a norm that was given and one that was just computed
// lead to the same bits.
template <int C>
__device__ __forceinline__ void clip_range(const Table<C>& t, float n, float max_norm) {
  // a norm that is not finite says nothing: the gradients stay as they are
  const bool scales = n < CUDART_INF_F && (double)max_norm < (double)n + (double)kEps;
  const float coef = scales ? (float)((double)max_norm / ((double)n + (double)kEps)) : 1.f;
  const int last = t.chunks - 1 - (int)blockIdx.x;
  int i = last >= 0 ? tensor_of(t, last, 0) : 0, then = i;
  for (int c = last; c >= 0; c -= (int)gridDim.x, i = then) {
    auto next = [&]() {
      if (c >= (int)gridDim.x) then = tensor_of(t, c - (int)gridDim.x, i);
    };
    const int k = c - t.first[i];
    if (!scales && t.p[i] == t.q[i]) next();
    else if (t.f32[i]) scale_chunk(static_cast<const float*>(t.p[i]), static_cast<float*>(t.q[i]), t.n[i], k, scales, coef, next);
    else scale_chunk(static_cast<const bf16*>(t.p[i]), static_cast<bf16*>(t.q[i]), t.n[i], k, scales, coef, next);
  }
}

// part: the norm kernels' sums, joined here by every block (a few microseconds
// less than another launch); or NULL, then *norm is given.
template <int C>
__global__ void __launch_bounds__(kThreads, kPerSm)
    grad_clip_kernel(const __grid_constant__ Table<C> t, const double* part, int parts, float* norm, float max_norm, int writes,
                     int32_t* status) {
  __shared__ double red[kThreads / 32];
  grid_dependency_wait();
  float n;
  if (part) {
    const double total = join(part, parts, red);
    if (writes && blockIdx.x == 0 && threadIdx.x == 0) report(total, norm, status);
    n = norm_of(total);
  } else {
    n = ld_plain(norm);
  }
  grid_dependents_launch();
  clip_range(t, n, max_norm);
}

// A short list: one cluster of up to 8 blocks takes the norm and clips, the blocks'
// sums by way of distributed shared memory, so that one launch does.  Up to 16 chunks:
// in two kernels / this way 8 take 8.1 / 6.8 us on the device, 16 8.8 / 8.6, 32 9.1 /
// 12.3; a call from Python 15 / 10.3 us.
constexpr int kClusterChunks = 16;

template <int C>
__global__ void __launch_bounds__(kThreads) grad_small_kernel(const __grid_constant__ Table<C> t, float* norm, float max_norm,
                                                              int clips, int32_t* status) {
  __shared__ double red[kThreads / 32];
  __shared__ double own;
  grid_dependency_wait();
  const double sum = sum_block(t, red);
  if (threadIdx.x == 0) own = sum;
  cluster_sync_all();
  double total = 0.0;
  for (unsigned r = 0; r < gridDim.x; ++r) {
    double v;
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(mapa_shared(smem_addr(&own), r)));
    total += v;
  }
  cluster_arrive();
  if (blockIdx.x == 0 && threadIdx.x == 0) report(total, norm, status);
  grid_dependents_launch();
  if (clips) clip_range(t, norm_of(total), max_norm);
  cluster_wait();  // nobody reads this block's sum any more
}

// ---- host ----------------------------------------------------------------------

int chunks_of(const GradTensor& g) {
  const int size = g.f32 ? 4 : 2;
  const long long head = ((16 - (reinterpret_cast<uintptr_t>(g.p) & 15)) & 15) / size, per = kChunkBytes / size;
  if (g.n <= 0) return 0;
  const long long body = g.n > head ? g.n - head : 0;
  return (int)(body <= per ? 1 : (body + per - 1) / per);
}

template <int C>
Table<C> table_of(const GradTensor* g, const GradTensor* out, int count) {
  Table<C> t;
  t.count = count;
  int at = 0;
  for (int i = 0; i < count; ++i) {
    t.p[i] = g[i].p;
    t.q[i] = out ? out[i].p : g[i].p;
    t.n[i] = g[i].n;
    t.f32[i] = (uint8_t)g[i].f32;
    t.first[i] = at;
    at += chunks_of(g[i]);
  }
  t.chunks = at;
  return t;
}

int blocks_of(int chunks) { return chunks < 1 ? 1 : chunks < kMaxBlocks ? chunks : kMaxBlocks; }

template <int C>
cudaError_t run_norm(const GradTensor* g, int count, double* part, int* blocks, cudaStream_t st) {
  const Table<C> t = table_of<C>(g, nullptr, count);
  *blocks = blocks_of(t.chunks);
  return launch_chained(grad_norm_kernel<C>, dim3((unsigned)*blocks), dim3(kThreads), 0, st, t, part);
}

template <int C>
cudaError_t run_clip(const GradTensor* g, const GradTensor* out, int count, const double* part, int parts, float* norm,
                     float max_norm, int writes, int32_t* status, cudaStream_t st) {
  const Table<C> t = table_of<C>(g, out, count);
  return launch_chained(grad_clip_kernel<C>, dim3((unsigned)blocks_of(t.chunks)), dim3(kThreads), 0, st, t, part, parts, norm,
                        max_norm, writes, status);
}

// The batches' sums behind one another; the number of them in *parts.
cudaError_t all_norms(const GradTensor* g, int count, double* part, int* parts, cudaStream_t st) {
  *parts = 0;
  for (int at = 0; at < count || at == 0; at += kLarge) {
    const int n = count - at < kLarge ? count - at : kLarge;
    int blocks = 0;
    cudaError_t err = n <= kSmall ? run_norm<kSmall>(g + at, n, part + *parts, &blocks, st)
                                  : run_norm<kLarge>(g + at, n, part + *parts, &blocks, st);
    if (err != cudaSuccess) return err;
    *parts += blocks;
  }
  return cudaSuccess;
}

cudaError_t run_small(const GradTensor* g, const GradTensor* out, int count, float* norm, float max_norm, int clips,
                      int32_t* status, cudaStream_t st) {
  const Table<kSmall> t = table_of<kSmall>(g, out, count);
  unsigned blocks = 1;
  while (blocks < 8 && (int)blocks < t.chunks) blocks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = blocks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, grad_small_kernel<kSmall>, t, norm, max_norm, clips, status);
}

bool is_small(const GradTensor* g, int count) {
  if (count > kSmall) return false;
  int chunks = 0;
  for (int i = 0; i < count && chunks <= kClusterChunks; ++i) {
    if (g[i].n > kClusterChunks * (long long)kChunkBytes) return false;
    chunks += chunks_of(g[i]);
  }
  return chunks <= kClusterChunks;
}

}  // namespace

long long grad_chunks(const GradTensor& g) { return g.n / (kChunkBytes / 4) + 2; }

size_t grad_norm_workspace(int count) {
  const size_t batches = count < 1 ? 1 : ((size_t)count + kLarge - 1) / kLarge;
  return batches * kMaxBlocks * sizeof(double);
}

cudaError_t launch_grad_norm(const GradTensor* g, int count, float* norm, void* workspace, int32_t* status, cudaStream_t st) {
  if (is_small(g, count)) return run_small(g, nullptr, count, norm, 0.f, 0, status, st);
  double* part = static_cast<double*>(workspace);
  int parts = 0;
  cudaError_t err = all_norms(g, count, part, &parts, st);
  if (err != cudaSuccess) return err;
  return launch_chained(grad_norm_join_kernel, dim3(1), dim3(kThreads), 0, st, part, parts, norm, status);
}

cudaError_t launch_grad_clip(const GradTensor* g, const GradTensor* out, int count, float* norm, float max_norm, void* workspace,
                             int32_t* status, cudaStream_t st) {
  if (workspace && is_small(g, count)) return run_small(g, out, count, norm, max_norm, 1, status, st);
  double* part = static_cast<double*>(workspace);
  int parts = 0;
  if (part) {
    cudaError_t err = all_norms(g, count, part, &parts, st);
    if (err != cudaSuccess) return err;
  }
  // from the last batch to the first, as the chunks within each; the first of these launches writes the norm
  for (int at = count > 0 ? (count - 1) / kLarge * kLarge : 0, first = 1; at >= 0; at -= kLarge, first = 0) {
    const int n = count - at < kLarge ? count - at : kLarge;
    const GradTensor* o = out ? out + at : nullptr;
    cudaError_t err = n <= kSmall ? run_clip<kSmall>(g + at, o, n, part, parts, norm, max_norm, first, status, st)
                                  : run_clip<kLarge>(g + at, o, n, part, parts, norm, max_norm, first, status, st);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

}  // namespace moe
