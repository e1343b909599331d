// linear.cu -- dense products beside the token path (the router's projection,
// a shared expert): a product with bias, activation and residual in its
// epilogue, and its backward pass.
//
//   z = x W^T + b;  y = act(z) + residual
//   dz = dy act'(z);  db = sum_rows dz;  dx = dz W;  dW = dz^T x
//
// Three matrix products of one form, D[m,n] = sum_k A[m,k] B[n,k], which
// differ in which axis of each operand is contiguous in memory:
//   y   A = x  [m][k]          B = W [n][k]
//   dx  A = dz [m][k]          B = W [k][n] (contracts over W's rows)
//   dW  A = dz [k][m]          B = x [k][n] (contracts over the tokens)
// The tensor cores read either order from shared memory, so no operand is
// transposed in memory: TMA writes 64-element rows of 128 bytes with the
// 128-byte swizzle, and the matrix descriptors say which axis those rows run
// along.  Accumulation is fp32 in TMEM.
//
// gemm_kernel: persistent; work units are output tiles (times parts of the
// contracted axis), each CTA or pair of CTAs taking every gridDim-th:
//   warp 0 lane 0   TMA producer of a shared-memory ring
//   warp 1 lane 0   MMA issuer (of the pair's first CTA)
//   warp 2          TMEM allocation
//   warps 4..11     epilogue, two warps for each quarter of the TMEM lanes,
//                   from one of two accumulators while the other fills
// Bound by the tensor cores where both sides are long (8192 x 4096 x 16384 558 us,
// 1.97 PFLOP/s; 8192 x 4096 x 4096 147, backward dx 148, dW 165 us), by what an SM
// takes in where one is short (16384 x 4096 x 128 28.5 us), by the weights' bytes
// and the launch where rows are few (64 x 4096 x 4096 11.9 us).
// Every mbarrier wait is bounded on the global timer, each from its own start, so
// that a long product does not run into the limit; a time-out records
// MOE_DEV_TIMEOUT and the roles wind down to the TMEM release.
#include <math_constants.h>

#include "common.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace moe {

namespace {

typedef __nv_bfloat16 bf16;

// ---- activations -------------------------------------------------------------

constexpr float kInvSqrt2Pi = 0.39894228040143268f;  // 1 / sqrt(2 pi)
constexpr float kTanhA = 0.79788456080286536f;       // sqrt(2 / pi)
constexpr float kTanhB = 0.044715f;

// 1 / (1 + exp(-v)); exp overflows to inf and the quotient to 0.
__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

// One value, or two in one instruction.
template <typename T>
__device__ __forceinline__ T all_of(float v);
template <>
__device__ __forceinline__ float all_of<float>(float v) { return v; }
template <>
__device__ __forceinline__ float2 all_of<float2>(float v) { return both(v); }
template <typename F>
__device__ __forceinline__ float each(float v, F f) { return f(v); }
template <typename F>
__device__ __forceinline__ float2 each(float2 v, F f) { return make_float2(f(v.x), f(v.y)); }

// Phi(z) = (1 + erf(z / sqrt 2)) / 2 and e = exp(-z^2 / 2), of one value or two.  For
// x >= 0, Phi(-x) = e R(x) with R smooth and falling like 1 / x: a polynomial of
// degree 8 in t = 1 / (1 + 0.305 x), without a constant, fitted for the least
// largest relative error on [0, 14] (1.6 units of 2^-24; 6.4 with fp32's
// roundings, to which the exponential adds about 2 z^2).  So the tail keeps its
// relative precision, where 1 + erf cancels, and one exponential serves gelu's
// slope too.  (With erff and expf the backward pass' kernel was bound by
// instructions.)
template <typename T>
__device__ __forceinline__ T normal_cdf(T z, T& e) {
  auto k = [](float v) { return all_of<T>(v); };
  const T x = each(z, [](float v) { return fabsf(v); });
  const T t = each(fma2(k(0.305f), x, k(1.f)), [](float v) { return __fdividef(1.f, v); });
  e = each(mul2(mul2(x, x), k(-0.72134752044448170f)), exp2_approx);  // 2^(-x^2 / 2 log2 e)
  T q = fma2(k(0.03669917955994606f), t, k(-0.1529882699251175f));
  q = fma2(q, t, k(0.18571682274341583f));
  q = fma2(q, t, k(-0.03797676041722298f));
  q = fma2(q, t, k(0.12102164328098297f));
  q = fma2(q, t, k(0.10342087596654892f));
  q = fma2(q, t, k(0.12246681749820709f));
  q = fma2(q, t, k(0.12163973599672318f));
  q = mul2(q, mul2(t, e));
  if constexpr (sizeof(T) == 8) return make_float2(z.x < 0.f ? q.x : 1.f - q.x, z.y < 0.f ? q.y : 1.f - q.y);
  else return z < 0.f ? q : 1.f - q;
}

__device__ __forceinline__ float activated(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z > 0.f ? z : (z != z ? z : 0.f);  // NaN stays
    case MOE_ACT_GELU_TANH: return z * sigmoid(2.f * kTanhA * (z + kTanhB * z * z * z));  // (1 + tanh(u)) / 2 = sigmoid(2u)
    case MOE_ACT_SILU: return z * sigmoid(z);
    default: return z;
  }
}

template <int N>
__device__ __forceinline__ void activate(float* f, int act) {
  switch (act) {  // uniform over the grid; one loop for each, so that the code that runs is short
    case MOE_ACT_RELU:
#pragma unroll
      for (int j = 0; j < N; ++j) f[j] = activated(f[j], MOE_ACT_RELU);
      break;
    case MOE_ACT_GELU:
      if constexpr (N == 1) {
        float e;
        f[0] *= normal_cdf(f[0], e);
      } else {
        // two values an instruction: 16384 x 128 x 4096, bound by this, 136 -> 113 us
#pragma unroll
        for (int j = 0; j < N; j += 2) {
          float2 e;
          const float2 cdf = normal_cdf(make_float2(f[j], f[j + 1]), e);
          f[j] *= cdf.x;
          f[j + 1] *= cdf.y;
        }
      }
      break;
    case MOE_ACT_GELU_TANH:
#pragma unroll
      for (int j = 0; j < N; ++j) f[j] = activated(f[j], MOE_ACT_GELU_TANH);
      break;
    case MOE_ACT_SILU:
#pragma unroll
      for (int j = 0; j < N; ++j) f[j] = activated(f[j], MOE_ACT_SILU);
      break;
    default: break;
  }
}

__device__ __forceinline__ float slope(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z > 0.f ? 1.f : 0.f;
    case MOE_ACT_GELU: {
      float e;
      const float cdf = normal_cdf(z, e);
      return fmaf(z * kInvSqrt2Pi, e, cdf);
    }
    case MOE_ACT_GELU_TANH: {
      // s + z s' with s = sigmoid(2u); past 16 the slope is 0 or 1 in fp32, and z's
      // square there would overflow beside s (1 - s) = 0
      z = fabsf(z) > 16.f ? copysignf(16.f, z) : z;
      const float s = sigmoid(2.f * kTanhA * (z + kTanhB * z * z * z));
      return fmaf(z * s * (1.f - s), 2.f * kTanhA * (1.f + 3.f * kTanhB * z * z), s);
    }
    case MOE_ACT_SILU: {
      const float s = sigmoid(z);
      return s * (1.f + z * (1.f - s));
    }
    default: return 1.f;
  }
}

// ---- epilogue ------------------------------------------------------------------

struct Epi {
  void* out;
  bf16* z;          // the value before the activation, or NULL
  const void* bias;
  const void* res;
  long long ldres;
  int act, out_f32, bias_f32, res_f32;
  int narrow;       // stores of 64-byte rows
  int wide;         // N and the residual's stride are multiples of 8: rows of 16-byte pieces
};

__device__ __forceinline__ float load_any(const void* p, int is_f32, long long i) {
  return is_f32 ? ld_plain(static_cast<const float*>(p) + i) : __bfloat162float(ld_plain(static_cast<const bf16*>(p) + i));
}

// Eight consecutive values of fp32 or bf16 memory, 16-byte aligned.
__device__ __forceinline__ void load8(const void* p, int is_f32, long long i, float* f) {
  if (is_f32) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
    Vec<float>::to_float(ld_plain(q), f);
    Vec<float>::to_float(ld_plain(q + 1), f + 4);
  } else {
    Vec<bf16>::to_float(ld_plain(reinterpret_cast<const uint4*>(static_cast<const bf16*>(p) + i)), f);
  }
}

// Four, aligned to their size (`whole`), or one by one, those from `n` on as n - 1.
__device__ __forceinline__ void load4(const void* p, int is_f32, long long i, bool whole, int n, float* f) {
  if (!whole) {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = load_any(p, is_f32, i + min(j, n - 1));
  } else if (is_f32) {
    Vec<float>::to_float(ld_plain(reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i)), f);
  } else {
    const uint2 u = ld_plain(reinterpret_cast<const uint2*>(static_cast<const bf16*>(p) + i));
    f[0] = __uint_as_float(u.x << 16);
    f[1] = __uint_as_float(u.x & 0xffff0000u);
    f[2] = __uint_as_float(u.y << 16);
    f[3] = __uint_as_float(u.y & 0xffff0000u);
  }
}

__device__ __forceinline__ void store4(void* p, int is_f32, long long i, bool whole, int n, const float* f) {
  if (!whole) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j >= n) continue;
      if (is_f32) static_cast<float*>(p)[i + j] = f[j];
      else static_cast<bf16*>(p)[i + j] = __float2bfloat16_rn(f[j]);
    }
  } else if (is_f32) {
    *reinterpret_cast<uint4*>(static_cast<float*>(p) + i) = Vec<float>::from_float(f);
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
    *reinterpret_cast<uint2*>(static_cast<bf16*>(p) + i) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
}

// Bias, activation and residual of one value.
__device__ __forceinline__ void finish1(const Epi& e, long long row, int col, int N, float f) {
  const long long at = row * N + col;
  if (e.bias) f += load_any(e.bias, e.bias_f32, col);
  if (e.z) e.z[at] = __float2bfloat16_rn(f);
  activate<1>(&f, e.act);
  if (e.res) f += load_any(e.res, e.res_f32, row * e.ldres + col);
  if (e.out_f32) static_cast<float*>(e.out)[at] = f;
  else static_cast<bf16*>(e.out)[at] = __float2bfloat16_rn(f);
}

// ---- the product ----------------------------------------------------------------

struct GemmArgs {
  int M, N, K;
  int tiles_m, tiles_n, splits, per_split, kblocks;  // K blocks of 128
  int pass, lower;  // kTwice: K blocks of one pass over B, rows from A's first terms to its second
  Epi epi;
  int32_t* status;
  long long timeout_ns;  // of a single wait
};

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kEpiBytes = kEpiWarps * 32 * 128;  // a warp: 32 rows x 32 fp32 columns
constexpr int kKB = 2;                           // 64-wide K blocks per ring stage
constexpr int kSubA = 128 * 128;                 // 16 KB: 128 rows x 64 of A

// Per variant: CG CTAs (1 or 2) make a tile of 128 CG x BN.
template <int CG, int BN>
struct Shape {
  static constexpr int kRowsB = BN / CG;               // rows of B held by one CTA
  static constexpr int kSubB = kRowsB * 128;
  static constexpr int kStage = kKB * (kSubA + kSubB);
  static constexpr int kStages = (192 * 1024) / kStage;  // 3 at 64 KB a stage, 4 at 48 KB
  static constexpr int kSmem = kStages * kStage + kEpiBytes + 1024;
  static constexpr int kTmemCols = 2 * BN;
  static constexpr int kPartRow = BN * 4 + 16;  // pitch of a split tile's fp32 rows, over the ring
  static_assert(128 * kPartRow <= kStages * kStage, "a part fits in the ring");
};

// Matrix descriptor of a tile in shared memory, 128-byte swizzle, base on 1024
// bytes.  Rows of 128 bytes along the contracted axis: groups of 8 rows 1024
// bytes apart.  Rows along the other axis (kMN): 8 steps of the contracted axis
// are 1024 bytes, the next 64 elements of the other axis 8192 bytes on.
template <bool kMN>
__device__ __forceinline__ uint64_t tile_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3ffffu) >> 4);
  d |= (uint64_t)(kMN ? 8192 >> 4 : 1) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
// Descriptor step of one MMA (16 of the contracted axis), in 16-byte units.
template <bool kMN>
constexpr uint64_t kstep() { return kMN ? 2048 >> 4 : 32 >> 4; }

template <int CG, int BN, bool AT, bool BT>
__device__ __forceinline__ uint32_t instr_desc() {
  uint32_t d = 0;
  d |= 1u << 4;                             // fp32 accumulator
  d |= 1u << 7;                             // A bf16
  d |= 1u << 10;                            // B bf16
  d |= (AT ? 1u : 0u) << 15;                // A's rows run along m
  d |= (BT ? 1u : 0u) << 16;                // B's rows run along n
  d |= (uint32_t)(BN >> 3) << 17;
  d |= (uint32_t)((128 * CG) >> 4) << 24;
  return d;
}

__device__ __forceinline__ void tma_load_2d(void* sdst, const CUtensorMap* map, int x, int y, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_addr(sdst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(mbar)
      : "memory");
}

template <int CG>
__device__ __forceinline__ void load_tile(void* sdst, const CUtensorMap* map, int x, int y, uint32_t mbar) {
  if constexpr (CG == 2) tma_load_2d_pair(sdst, map, x, y, mbar);
  else tma_load_2d(sdst, map, x, y, mbar);
}

template <int CG>
__device__ __forceinline__ void mma(uint32_t dt, uint64_t ad, uint64_t bd, uint32_t idesc, int accumulate) {
  if constexpr (CG == 2) {
    mma_bf16_pair(dt, ad, bd, idesc, accumulate);
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(dt),
        "l"(ad), "l"(bd), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}

template <int CG>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (CG == 2) {
    mma_commit_pair(bar);
  } else {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
  }
}

// 32 rows x 32 columns starting at (r0, n0), lane = row, v its columns.  The
// usual way out (bulk): bias, activation and residual in that layout, then
// the rounded rows into the warp's staging tile, which a TMA store writes,
// clipped at the tensor's edge.  The tile is one piece of 32 rows x 128 bytes
// (64 bf16 columns, filled in two halves, or 32 fp32), or, where z is stored
// beside y or a warp's columns are only 32, two pieces of 64 bytes a row used
// in turn; 16-byte parts XOR-swizzled by the row (128-byte and 64-byte
// swizzle), free of bank conflicts.  Against 16-byte stores by lanes this takes
// a quarter of the instructions: dx of 16384 x 4096 from 128 columns, a product
// that is little but its output, 75.7 -> 47 us (44 without the stores, 28
// without the epilogue: what is left is the tile's hand-over between load,
// product and epilogue; 38.9 since a gradient's product is compiled without the
// rest of the epilogue).  Rows of 128 bytes instead of 64 matter to the large
// products (8192 x 4096 x 16384: 566 -> 545 us).
struct Bulk {
  uint8_t* stage;  // this warp's 4 KB
  int piece;
};

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(smem_addr(src))
               : "memory");
}

__device__ __forceinline__ void store_piece(const CUtensorMap* map, const void* src, int x, int y, int lane) {
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(map, src, x, y);
    bulk_commit();
  }
}

// 16 words of each lane's row, 64-byte pieces, columns starting at x.
__device__ __forceinline__ void put_narrow(Bulk& b, const CUtensorMap* map, const uint32_t* w, int x, int y, int lane) {
  uint8_t* dst = b.stage + b.piece * 2048;
  if (lane == 0) bulk_wait_read<1>();  // the store before last, from this piece
  __syncwarp();
#pragma unroll
  for (int q = 0; q < 4; ++q)
    *reinterpret_cast<uint4*>(dst + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)) =
        make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
  store_piece(map, dst, x, y, lane);
  b.piece ^= 1;
}

// 16 words as half `half` of a 128-byte piece whose columns start at x; the
// piece leaves with its second half, or at once where `last`.
__device__ __forceinline__ void put_half(Bulk& b, const CUtensorMap* map, const uint32_t* w, int half, bool last, int x,
                                         int y, int lane) {
  if (half == 0) {
    if (lane == 0) bulk_wait_read<0>();
    __syncwarp();
  }
#pragma unroll
  for (int q = 0; q < 4; ++q)
    *reinterpret_cast<uint4*>(b.stage + lane * 128 + (((4 * half + q) ^ (lane & 7)) << 4)) =
        make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
  if (half == 1 || last) store_piece(map, b.stage, x, y, lane);
}

__device__ __forceinline__ void pack_bf16(const float (&f)[32], uint32_t (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
}

// 32 consecutive values of fp32 or bf16 memory, of which the first n (a
// multiple of 8, at least 8) exist; in the others' places the last eight come
// again.  All loads first and none behind a condition, so that they travel
// together, then the sum.
struct Raw32 {
  uint4 v[8];
};

__device__ __forceinline__ void load32(Raw32& r, const void* p, int is_f32, long long at, int n) {
  if (is_f32) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at);
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i] = ld_plain(q + min(i, n / 4 - 1));
  } else {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const bf16*>(p) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) r.v[i] = ld_plain(q + min(i, n / 8 - 1));
  }
}

__device__ __forceinline__ void add32(const Raw32& r, int is_f32, float (&f)[32]) {
  float t[32];
  if (is_f32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) Vec<float>::to_float(r.v[i], t + 4 * i);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) Vec<bf16>::to_float(r.v[i], t + 8 * i);
  }
#pragma unroll
  for (int j = 0; j < 32; ++j) f[j] += t[j];
}

// The residual of this lane's row, loaded before the accumulator is waited for.
__device__ __forceinline__ void load_residual(const Epi& e, Raw32& r, int row, int n0, int M, int N) {
  if (e.res && n0 < N) load32(r, e.res, e.res_f32, (long long)min(row, M - 1) * e.ldres + n0, N - n0);
}

// c: which of the warp's 32-column blocks this is; kPair: they come in pairs.
template <bool kPair>
__device__ __forceinline__ void finish_bulk(const Epi& e, Bulk& b, const CUtensorMap* tmY, const CUtensorMap* tmZ,
                                            const uint32_t (&v)[32], const Raw32& res, int c, int r0, int n0, int M,
                                            int N, int lane) {
  if (r0 >= M || n0 >= N) return;  // the whole warp
  float f[32];
#pragma unroll
  for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(v[j]);
  if (e.bias) {
    Raw32 bias;
    load32(bias, e.bias, e.bias_f32, n0, N - n0);
    add32(bias, e.bias_f32, f);
  }
  uint32_t w[16];
  if (e.z) {
    pack_bf16(f, w);
    put_narrow(b, tmZ, w, n0, r0, lane);
  }
  if (e.act != MOE_ACT_NONE) activate<32>(f, e.act);
  if (e.res) add32(res, e.res_f32, f);
  if (e.out_f32) {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(f);
    if (e.narrow) {
      put_narrow(b, tmY, u, n0, r0, lane);
      if (n0 + 16 < N) put_narrow(b, tmY, u + 16, n0 + 16, r0, lane);
    } else {
      put_half(b, tmY, u, 0, false, n0, r0, lane);
      put_half(b, tmY, u + 16, 1, true, n0, r0, lane);
    }
  } else {
    pack_bf16(f, w);
    if (!kPair || e.narrow) put_narrow(b, tmY, w, n0, r0, lane);
    else put_half(b, tmY, w, c & 1, n0 + 32 >= N, n0 - 32 * (c & 1), r0, lane);
  }
}

// The same where rows are not of 16 bytes, so that TMA cannot write them: a
// block goes as fp32 through the staging tile (16-byte pieces XOR-swizzled by
// the row), then each lane takes a column and walks down the rows, eight at a
// time (a step).  The residual is loaded two steps ahead, over the blocks'
// borders: with one step, and a fresh start in each block, the epilogue
// waited for memory in most of them (2791 x 2816 x 2815, gelu_tanh and residual:
// 51.9 -> 48.8 us; 130 x 1000 x 5001 17.8 -> 16.0).
struct Ahead {
  uint32_t v[2][8];  // steps s and s + 1
};

// Step s = 4 c + (rows / 8) of the tile half that starts at (r0, n0): the raw
// residual of this lane's column.  Past the last row or column: the last one
// again, unused, so that the loads are unconditional (behind a condition each
// waited for the one before it).
__device__ __forceinline__ void load_step(const Epi& e, uint32_t (&to)[8], int s, int r0, int n0, int M, int N, int lane) {
  const int row = min(r0 + 8 * (s & 3), M - 1), col = min(n0 + 32 * (s >> 2) + lane, N - 1);
  const long long at = row * e.ldres + col;
  if (e.res_f32) {
    const uint32_t* p = static_cast<const uint32_t*>(e.res) + at;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      to[i] = ld_plain(p);
      p += row + i + 1 < M ? e.ldres : 0;
    }
  } else {
    const unsigned short* p = static_cast<const unsigned short*>(e.res) + at;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      to[i] = ld_plain(p);
      p += row + i + 1 < M ? e.ldres : 0;
    }
  }
}

// Before the first block of a tile half.
__device__ __forceinline__ void start_ragged(const Epi& e, Ahead& a, int r0, int n0, int M, int N, int lane) {
  if (!e.res || n0 >= N) return;
  load_step(e, a.v[0], 0, r0, n0, M, N, lane);
  load_step(e, a.v[1], 1, r0, n0, M, N, lane);
}

// Block c of `blocks` of the tile half.
__device__ __forceinline__ void finish_ragged(const Epi& e, uint8_t* stage, const uint32_t (&v)[32], Ahead& a, int c,
                                              int blocks, int r0, int n0, int M, int N, int lane) {
  if (r0 >= M || n0 + 32 * c >= N) return;  // the whole warp
#pragma unroll
  for (int q = 0; q < 8; ++q)
    *reinterpret_cast<uint4*>(stage + lane * 128 + ((q ^ (lane & 7)) << 4)) =
        make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
  __syncwarp();
  const int col = n0 + 32 * c + lane, rows = min(32, M - r0);
  const bool in = col < N;
  const float bias = e.bias ? load_any(e.bias, e.bias_f32, min(col, N - 1)) : 0.f;
  long long at = (long long)r0 * N + col;
  // all four steps, so that every block moves `a` on alike; a rolled loop:
  // unrolled, a fifth of the warps' time went to fetching instructions
#pragma unroll 1
  for (int q = 0; q < 32; q += 8) {
    uint32_t next[8];
    const int s = 4 * c + q / 8 + 2;
    if (e.res && s < 4 * blocks && n0 + 32 * (s >> 2) < N) load_step(e, next, s, r0, n0, M, N, lane);
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)  // q is a multiple of 8: row q + i is swizzled by i
      f[i] = bias + *reinterpret_cast<const float*>(stage + (q + i) * 128 + ((((lane >> 2) ^ i) << 4) | ((lane & 3) << 2)));
    if (e.z) {
      bf16* z = e.z + at;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (in && q + i < rows) *z = __float2bfloat16_rn(f[i]);
        z += N;
      }
    }
    if (e.act != MOE_ACT_NONE) activate<8>(f, e.act);
    if (e.res) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f[i] += __uint_as_float(e.res_f32 ? a.v[0][i] : a.v[0][i] << 16);
        a.v[0][i] = a.v[1][i];
        a.v[1][i] = next[i];
      }
    }
    if (e.out_f32) {
      float* out = static_cast<float*>(e.out) + at;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (in && q + i < rows) *out = f[i];
        out += N;
      }
    } else {
      bf16* out = static_cast<bf16*>(e.out) + at;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (in && q + i < rows) *out = __float2bfloat16_rn(f[i]);
        out += N;
      }
    }
    at += 8LL * N;
  }
  __syncwarp();
}

struct Unit {
  int m0, n0, kb0, kb1;
};

// Units run over tiles in bands of 8 rows of tiles (the m index fastest), so
// that the tiles in flight share operands in L2.
template <int CG, int BN>
__device__ __forceinline__ Unit unit_of(int u, int split, const GemmArgs& p) {
  constexpr int kBand = 8;
  Unit t;
  const int band = u / (kBand * p.tiles_n);
  const int rows = min(kBand, p.tiles_m - band * kBand);
  const int r = u - band * kBand * p.tiles_n;
  const int n = r / rows;
  t.m0 = (band * kBand + r - n * rows) * 128 * CG;
  t.n0 = n * BN;
  t.kb0 = split * p.per_split;
  t.kb1 = min(p.kblocks, t.kb0 + p.per_split);
  return t;
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// The cache lines of the residual that this lane's row of a tile will need.
__device__ __forceinline__ void prefetch_residual(const Epi& e, int row, int n0, int cols, int M, int N) {
  if (!e.res || row >= M) return;
  const int size = e.res_f32 ? 4 : 2, n = min(cols, N - n0);
  const char* at = static_cast<const char*>(e.res) + ((long long)row * e.ldres + n0) * size;
  for (int b = 0; b < n * size; b += 128) prefetch_l2(at + b);
}

__device__ __forceinline__ uint4 ld_cluster(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

// The rows of a split tile that each of its S CTAs finishes: an equal share of
// those that exist.
__device__ __forceinline__ int rows_of_share(int m0, int M, int S) { return (min(128, M - m0) + S - 1) / S; }

// This CTA's share of a split tile.  A warp reads 512 consecutive bytes of one
// part at a time; each CTA starts with its own part and goes round, so that the
// CTAs of a cluster do not all read one SM's memory at once (a row's parts are
// added in an order that only its place fixes).  Everything that is read
// travels at once, bias and residual before the cluster's barrier.  64 x 4096 x
// 4096, four parts: 14.3 -> 11.9 us (in 32-byte pieces, one part at a time, the
// join had taken 7 of 23 thousand cycles).  Ends with this CTA's arrival at the
// barrier after which the parts may go.
template <int S, int BN>
__device__ __forceinline__ void join_parts(const GemmArgs& p, const Epi& e, const Unit& t, int split, const uint8_t* parts) {
  constexpr int kGroups = BN / 4, kRounds = (128 / S * kGroups + kThreads - 1) / kThreads;
  const int per = rows_of_share(t.m0, p.M, S), end = min(min(128, p.M - t.m0), (split + 1) * per);
  float bias[kRounds][4], res[kRounds][4], f[kRounds][4];
  bool there[kRounds];
  auto row_of = [&](int j) { return split * per + (int)(threadIdx.x + j * kThreads) / kGroups; };
  auto col_of = [&](int j) { return (int)(threadIdx.x + j * kThreads) % kGroups * 4; };
#pragma unroll
  for (int j = 0; j < kRounds; ++j) {
    const int row = row_of(j), col = t.n0 + col_of(j);
    there[j] = row < end && col < p.N;
    if (there[j] && e.bias) load4(e.bias, e.bias_f32, col, e.wide, p.N - col, bias[j]);
    if (there[j] && e.res) load4(e.res, e.res_f32, (t.m0 + row) * e.ldres + col, e.wide, p.N - col, res[j]);
  }
  cluster_sync_all();  // every part is in its CTA's shared memory
  uint4 v[kRounds][S];
#pragma unroll
  for (int j = 0; j < kRounds; ++j) {
    const uint8_t* own = parts + min(row_of(j), 127) * Shape<1, BN>::kPartRow + col_of(j) * 4;
    if (there[j]) {
      v[j][0] = *reinterpret_cast<const uint4*>(own);
#pragma unroll
      for (int s = 1; s < S; ++s) v[j][s] = ld_cluster(mapa_shared(smem_addr(own), (split + s) & (S - 1)));
    }
  }
#pragma unroll
  for (int j = 0; j < kRounds; ++j) {
    Vec<float>::to_float(v[j][0], f[j]);
#pragma unroll
    for (int s = 1; s < S; ++s) {
      float g[4];
      Vec<float>::to_float(v[j][s], g);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[j][i] += g[i];
    }
  }
  cluster_arrive();
#pragma unroll
  for (int j = 0; j < kRounds; ++j) {
    if (!there[j]) continue;
    const int col = t.n0 + col_of(j), n = p.N - col;
    const long long at = (long long)(t.m0 + row_of(j)) * p.N + col;
    if (e.bias) {
#pragma unroll
      for (int i = 0; i < 4; ++i) f[j][i] += bias[j][i];
    }
    if (e.z) store4(e.z, 0, at, e.wide, n, f[j]);
    activate<4>(f[j], e.act);
    if (e.res) {
#pragma unroll
      for (int i = 0; i < 4; ++i) f[j][i] += res[j][i];
    }
    store4(e.out, e.out_f32, at, e.wide, n, f[j]);
  }
}

// kExact (fp32 outputs, and sums of more than kLongSum terms): the tensor cores'
// accumulator drops the bits below its last place at every step (measured:
// 4.4e-6 of the result over 4096 terms, against 6e-7 for fp32 additions), so a
// product hands its sum over every kExactBlocks K blocks, and the epilogue adds
// these up in registers.  Where all terms have one sign, n of them come out up to
// n / 16 units of 2^-24 short: at kLongSum 2^-10, a quarter of what rounding to bf16
// may take, so a bf16 output keeps the one accumulator up to there (4096 x 4096 from
// 2^19 terms takes 20.3 ms this way; that way 13.1, and up to 2e-3 short).
constexpr int kExactBlocks = 4;
constexpr int kLongSum = 1 << 18;

// kSplit (CG = 1): where tiles are too few to fill the machine, a cluster of
// 2, 4 or 8 CTAs shares one, each with its part of the contracted axis.  They
// leave their fp32 sums in their shared memory, and each finishes an equal
// share of the tile's rows (join_parts).  Partial products in global memory and
// a second kernel to add them took 13 to 16 us at 64 x 4096 x 4096 (11.9 this
// way), another launch and a workspace.
//
// kTwice (gradients in fp32): A is a sum of two bf16 terms, the second `lower` rows
// below the first, so the contracted axis is gone through twice.  Tiles that
// reach past the first term's end read into the second: rows of D that are not
// stored, or terms that meet B's zeros.  (As a second product with the first
// one's result for its residual: 16384 x 4096 x 128, dx and dW, 309 us; this way 114.)
template <int CG, int BN, bool AT, bool BT, bool kExact, bool kSplit, bool kTwice>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmZ,
                const __grid_constant__ GemmArgs p) {
  typedef Shape<CG, BN> S;
  constexpr int kStages = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kStages], empty[kStages], tfull[2], tempty[2], drain;
  __shared__ uint32_t tmem_base;
  __shared__ int s_err;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;
  static_assert(!kSplit || CG == 1, "a split tile belongs to single CTAs");
  const int split = kSplit ? (int)cluster_ctarank() : 0;
  uint8_t* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);

  if (threadIdx.x == 0) {
    s_err = 0;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmA)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmB)) : "memory");
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], CG * kEpiWarps);
    }
    mbar_init(&drain, 1);
    fence_barrier_init();
  }
  __syncthreads();
  if (warp == 2) {
    if constexpr (CG == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_base)),
                   "r"(S::kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_base)),
                   "r"(S::kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  grid_dependency_wait();  // all set-up is done: from here on memory of earlier kernels is read
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync_all();  // both CTAs' barriers exist before any remote signal
  tc_fence_after();
  const uint32_t tbase = tmem_base;

  // a gradient's product (BT) has nothing in its epilogue but the store
  Epi plain = {};
  if constexpr (BT) {
    plain.out = p.epi.out;
    plain.act = MOE_ACT_NONE;
    plain.out_f32 = p.epi.out_f32;
    plain.narrow = p.epi.narrow;
    plain.wide = p.epi.wide;
  }
  const Epi& epi = BT ? plain : p.epi;

  const int units = p.tiles_m * p.tiles_n;
  const int share = kSplit ? p.splits : CG;  // CTAs of a worker
  const int worker = blockIdx.x / share, workers = gridDim.x / share;

  if (warp == 0 && lane == 0) {
    // ---- TMA producer ------------------------------------------------------
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = worker; u < units && ok; u += workers) {
      const Unit t = unit_of<CG, BN>(u, split, p);
      const int m0 = t.m0 + 128 * (int)rank, n0 = t.n0 + S::kRowsB * (int)rank;
      for (int kb = t.kb0; kb < t.kb1; ++kb) {
        if (!mbar_wait_limited(&empty[stage], phase ^ 1u, p.timeout_ns)) {
          ok = false;
          break;
        }
        uint8_t* sa = smem + stage * S::kStage;
        const bool second = kTwice && kb >= p.pass;
        const int lower = second ? p.lower : 0, kb_in = second ? kb - p.pass : kb;
        const uint32_t fb = CG == 2 ? mapa_shared(smem_addr(&full[stage]), 0) : smem_addr(&full[stage]);
        if (rank == 0) mbar_arrive_expect_tx(&full[stage], CG * S::kStage);
#pragma unroll
        for (int q = 0; q < kKB; ++q) {
          const int k = (kb_in * kKB + q) * 64;
          if constexpr (AT) {
#pragma unroll
            for (int g = 0; g < 2; ++g) load_tile<CG>(sa + q * kSubA + g * 8192, &tmA, m0 + 64 * g, k + lower, fb);
          } else {
            load_tile<CG>(sa + q * kSubA, &tmA, k, m0 + lower, fb);
          }
          uint8_t* sb = sa + kKB * kSubA + q * S::kSubB;
          if constexpr (BT) {
#pragma unroll
            for (int g = 0; g < S::kRowsB / 64; ++g) load_tile<CG>(sb + g * 8192, &tmB, n0 + 64 * g, k, fb);
          } else {
            load_tile<CG>(sb, &tmB, k, n0, fb);
          }
        }
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // every stage's last fill consumed: nothing still arrives at this CTA's
    // barriers or shared memory when it leaves
    for (int i = 0; i < kStages && ok; ++i) {
      if (!mbar_wait_limited(&empty[stage], phase ^ 1u, p.timeout_ns)) ok = false;
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (!ok) atomicOr(&s_err, 1);
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // ---- MMA issuer ----------------------------------------------------------
    const uint32_t idesc = instr_desc<CG, BN, AT, BT>();
    int stage = 0, acc = 0;
    uint32_t phase = 0, tphase[2] = {0u, 0u};
    bool ok = true;
    for (int u = worker; u < units && ok; u += workers) {
      const Unit t = unit_of<CG, BN>(u, split, p);
      for (int kb0 = t.kb0; kb0 < t.kb1 && ok;) {
        const int kb1 = kExact ? min(t.kb1, kb0 + kExactBlocks) : t.kb1;
        if (!mbar_wait_cluster_limited(&tempty[acc], tphase[acc] ^ 1u, p.timeout_ns)) {
          ok = false;
          break;
        }
        tphase[acc] ^= 1u;
        tc_fence_after();
        const uint32_t dt = tbase + (uint32_t)(acc * BN);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait_cluster_limited(&full[stage], phase, p.timeout_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_addr(smem + stage * S::kStage);
#pragma unroll
          for (int q = 0; q < kKB; ++q) {
            const uint64_t ad = tile_desc<AT>(sa + q * kSubA);
            const uint64_t bd = tile_desc<BT>(sa + kKB * kSubA + q * S::kSubB);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma<CG>(dt, ad + kk * kstep<AT>(), bd + kk * kstep<BT>(), idesc, (kb > kb0) | (q | kk) != 0);
          }
          commit<CG>(&empty[stage]);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        commit<CG>(&tfull[acc]);
        acc ^= 1;
        kb0 = kb1;
      }
    }
    if (!ok) {
      // a wait ran out: let the MMAs issued so far finish reading shared
      // memory before the CTAs leave (one more commit, to this CTA only)
      if constexpr (CG == 2) mma_commit_pair(&drain, 0x1);
      else commit<CG>(&drain);
      mbar_wait_limited(&drain, 0, p.timeout_ns);
      atomicOr(&s_err, 1);
    }
  } else if (warp >= 4) {
    // ---- epilogue --------------------------------------------------------------
    const int ew = warp & 3, half = (warp - 4) >> 2;
    uint8_t* stage_buf = smem + kStages * S::kStage + (warp - 4) * 32 * 128;
    const uint32_t te[2] = {CG == 2 ? mapa_shared(smem_addr(&tempty[0]), 0) : smem_addr(&tempty[0]),
                            CG == 2 ? mapa_shared(smem_addr(&tempty[1]), 0) : smem_addr(&tempty[1])};
    constexpr int kChunks = BN / 64;  // of 32 columns, this warp's half of the tile
    int acc = 0;
    uint32_t tphase[2] = {0u, 0u};
    bool ok = true;
    Bulk bulk = {stage_buf, 0};
    // this warp's reads of the accumulator are done: the next product may have it
    auto release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 1 || rank == 0) mbar_arrive(&tempty[acc]);
        else mbar_arrive_cluster(te[acc]);
      }
    };
    for (int u = worker; u < units && ok; u += workers) {
      const Unit t = unit_of<CG, BN>(u, split, p);
      const int r0 = t.m0 + 128 * (int)rank + 32 * ew, n0 = t.n0 + half * (BN / 2);
      if constexpr (kSplit) {  // for the rows that this CTA will finish
        const int rows = rows_of_share(t.m0, p.M, p.splits), i = threadIdx.x - 128;
        if (i < rows) prefetch_residual(epi, t.m0 + split * rows + i, t.n0, BN, p.M, p.N);
      } else {
        prefetch_residual(epi, r0 + lane, n0, BN / 2, p.M, p.N);
      }
      Ahead ahead;
      auto start = [&]() {
        if (!kSplit && !epi.wide) start_ragged(epi, ahead, r0, n0, p.M, p.N, lane);
      };
      // a block of 32 columns on its way out, or into this CTA's part of a split tile
      auto emit = [&](const uint32_t (&v)[32], const Raw32& res, int c) {
        if constexpr (kSplit) {
          uint8_t* row = smem + (32 * ew + lane) * S::kPartRow + (half * (BN / 2) + 32 * c) * 4;
#pragma unroll
          for (int q = 0; q < 8; ++q)
            reinterpret_cast<uint4*>(row)[q] = make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        } else if (epi.wide) {
          finish_bulk<BN >= 128>(epi, bulk, &tmY, &tmZ, v, res, c, r0, n0 + 32 * c, p.M, p.N, lane);
        } else {
          finish_ragged(epi, stage_buf, v, ahead, c, kChunks, r0, n0, p.M, p.N, lane);
        }
      };
      auto residual = [&](Raw32& res, int c) {
        if (!kSplit && epi.wide) load_residual(epi, res, r0 + lane, n0 + 32 * c, p.M, p.N);
      };
      auto lanes_of = [&]() { return tbase + ((uint32_t)(32 * ew) << 16) + (uint32_t)(acc * BN + half * (BN / 2)); };
      if constexpr (kExact) {
        uint32_t sum[kChunks][32];
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
          for (int j = 0; j < 32; ++j) sum[c][j] = 0u;
        for (int kb = t.kb0; kb < t.kb1; kb += kExactBlocks) {
          if (!__all_sync(0xffffffffu, mbar_wait_limited(&tfull[acc], tphase[acc], p.timeout_ns))) {
            ok = false;
            break;
          }
          tphase[acc] ^= 1u;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            uint32_t v[32];
            tmem_ld32(lanes_of() + (uint32_t)(32 * c), v);
#pragma unroll
            for (int j = 0; j < 32; ++j) sum[c][j] = __float_as_uint(__uint_as_float(sum[c][j]) + __uint_as_float(v[j]));
          }
          release();
          acc ^= 1;
        }
        if (!ok) break;
        start();
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          Raw32 res;
          residual(res, c);
          emit(sum[c], res, c);
        }
      } else {
        start();
        if (!__all_sync(0xffffffffu, mbar_wait_limited(&tfull[acc], tphase[acc], p.timeout_ns))) {
          ok = false;
          break;
        }
        tphase[acc] ^= 1u;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < kChunks; ++c) {
          Raw32 res;
          residual(res, c);
          uint32_t v[32];
          tmem_ld32(lanes_of() + (uint32_t)(32 * c), v);
          if (c == kChunks - 1) release();
          emit(v, res, c);
        }
        acc ^= 1;
      }
    }
    if (lane == 0) bulk_wait_all();  // the stores have read the staging tile and are written
    if (!ok) atomicOr(&s_err, 1);
  }

  grid_dependents_launch();
  tc_fence_before();
  __syncthreads();
  if (s_err) {  // let copies in flight land before shared memory goes
    const uint64_t until = globaltimer_ns() + 200000;
    while (globaltimer_ns() < until) {
    }
  }
  if constexpr (kSplit) {
    const Unit t = unit_of<CG, BN>(worker, split, p);
    switch (p.splits) {
      case 2: join_parts<2, BN>(p, epi, t, split, smem); break;
      case 4: join_parts<4, BN>(p, epi, t, split, smem); break;
      default: join_parts<8, BN>(p, epi, t, split, smem); break;
    }
    cluster_wait();  // nobody reads this CTA's part any more
  }
  if constexpr (CG == 2) cluster_sync_all();
  tc_fence_after();
  if (warp == 2) {
    if constexpr (CG == 2)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(S::kTmemCols) : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(S::kTmemCols) : "memory");
  }
  if (threadIdx.x == 0 && s_err) raise_status(p.status, MOE_DEV_TIMEOUT);
}

// ---- few rows -------------------------------------------------------------------

constexpr int kFewRows = 16;

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

struct FewArgs {
  const bf16* x;
  const bf16* W;
  long long ldx, ldw;
  int s, K, N;
  Epi epi;
  int32_t* status;
  long long timeout_ns;
};

// Up to 16 rows of x (decoded tokens): bound by reading W once.  One block an
// SM takes N / gridDim consecutive columns of y, so every SM reads the same
// share of W to within a row.  W comes through a deep ring in shared memory (a
// stage: 8 rows x 2048 of the contracted axis, a bulk copy a row), which keeps
// up to 190 KB an SM in flight from the first microsecond on; loads into
// registers, 128 bytes a thread, had reached 2.9 TB/s at 4096 x 4096 (11.6 us; this
// way 8.8, and 23.8 us, 5.6 TB/s, at 16384 x 4096).  The rows
// of x take the same way, a stage or two before the chunk's W.
//   warp 8          producer: lane r copies row r of a stage
//   warps 0..7      every eighth 32 of the contracted axis, by warp-level MMA
//                   (16 rows of x times 8 rows of W: 8 of 16 rows idle when
//                   s <= 8, but the tensor cores wait for memory anyway)
// The order of the terms is free, so lane c of a row's four feeds its 8
// consecutive elements to two MMAs as their k pairs, the same for x and W.  The
// accumulator, which drops the bits below its last place as that of the tiles
// does, is emptied into an fp32 sum after every chunk: 256 terms of a warp.  The
// warps' sums are added in order through shared memory every 32 columns.
// A wait that runs out sets the status and everyone runs on without waiting,
// so that the barriers stay matched.
constexpr int kFewK = 2048;                    // of the contracted axis a stage
constexpr int kFewRow = kFewK * 2 + 64;        // row pitch: 64 bytes more, free of bank conflicts
constexpr int kFewStage = 8 * kFewRow;
constexpr int kFewStages = 6;
constexpr int kFewTiles = 4;                   // 8 columns each, between two joins
constexpr int kFewSmem = kFewStages * kFewStage;

template <bool kHigh>  // rows 8..15 exist
__global__ void __launch_bounds__(288, 1) few_rows_kernel(const __grid_constant__ FewArgs p) {
  constexpr int kBlocks = kFewK / 32 / 8;  // 32-wide blocks of a stage and warp
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ __align__(8) uint64_t full[kFewStages], empty[kFewStages];
  __shared__ float red[8][kHigh ? 16 : 8][8 * kFewTiles + 1];
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
  grid_dependency_wait();
  const int f0 = (int)((long long)p.N * blockIdx.x / gridDim.x), f1 = (int)((long long)p.N * (blockIdx.x + 1) / gridDim.x);
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
  if (warp == 8) {
    auto put = [&](const bf16* base, long long ld, int rows, int kc) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait_limited(&empty[stage], phase ^ 1u, p.timeout_ns));
      if (ok) {
        if (lane == 0) mbar_arrive_expect_tx(&full[stage], (uint32_t)(rows * kc * 2));
        __syncwarp();
        if (lane < rows) bulk_g2s(ring + stage * kFewStage + lane * kFewRow, base + lane * ld, (uint32_t)kc * 2, &full[stage]);
      }
      advance();
    };
    for (int g0 = f0; g0 < f1; g0 += 8 * kFewTiles) {
      for (int ch = 0; ch < chunks; ++ch) {
        const int k0 = ch * kFewK, kc = min(kFewK, p.K - k0);
        put(p.x + k0, p.ldx, min(8, p.s), kc);
        if (kHigh) put(p.x + 8 * p.ldx + k0, p.ldx, p.s - 8, kc);
        for (int t = g0; t < min(f1, g0 + 8 * kFewTiles); t += 8) put(p.W + (long long)t * p.ldw + k0, p.ldw, min(8, f1 - t), kc);
      }
    }
    // the last copies are waited for by the consumers, which have read all stages
  } else {
    const int g = lane >> 2, c = lane & 3;
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
      return k < kc ? *reinterpret_cast<const uint4*>(ring + stage * kFewStage + g * kFewRow + k * 2) : make_uint4(0, 0, 0, 0);
    };
    for (int g0 = f0; g0 < f1; g0 += 8 * kFewTiles) {
      float sum[kFewTiles][4];
#pragma unroll
      for (int t = 0; t < kFewTiles; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[t][j] = 0.f;
      for (int ch = 0; ch < chunks; ++ch) {
        const int kc = min(kFewK, p.K - ch * kFewK);
        uint4 xa[kBlocks], xb[kBlocks];
        wait_full();
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) xa[i] = frag(i, kc);
        release();
        if (kHigh) {
          wait_full();
#pragma unroll
          for (int i = 0; i < kBlocks; ++i) xb[i] = frag(i, kc);
          release();
        } else {
#pragma unroll
          for (int i = 0; i < kBlocks; ++i) xb[i] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int t = 0; t < kFewTiles; ++t) {
          if (g0 + 8 * t < f1) {
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
      for (int t = 0; t < kFewTiles; ++t) {
        red[warp][g][8 * t + 2 * c] = sum[t][0];
        red[warp][g][8 * t + 2 * c + 1] = sum[t][1];
        if constexpr (kHigh) {
          red[warp][g + 8][8 * t + 2 * c] = sum[t][2];
          red[warp][g + 8][8 * t + 2 * c + 1] = sum[t][3];
        }
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      const int cols = min(8 * kFewTiles, f1 - g0);
      for (int o = threadIdx.x; o < p.s * 8 * kFewTiles; o += 256) {
        const int row = o / (8 * kFewTiles), j = o - row * 8 * kFewTiles;
        if (j < cols) {
          float f = 0.f;
#pragma unroll
          for (int q = 0; q < 8; ++q) f += red[q][row][j];
          finish1(p.epi, row, g0 + j, p.N, f);
        }
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");  // the sums are rewritten
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

// ---- dz and the bias' gradient --------------------------------------------------

struct SlopeArgs {
  const void* dy;
  const bf16* z;
  bf16* dz;        // [s][lddz], or NULL: only the column sums
  float* part;     // [gridDim.y][N] column sums, or NULL
  long long lddy, ldz, lddz;
  int s, N;
};

// dz = dy act'(z) and its column sums: a warp walks rows of 32 W columns (W a
// lane: 16 bytes of bf16, or one element where rows are not of 16 bytes), a
// block's eight warps add up through shared memory, each block one partial
// row.  Six blocks an SM hide the loads and the slope's chain better than rows
// unrolled in fewer (8192 x 4096 silu, sums alone: four rows in two blocks 46.6 us,
// two in four 35.6, one in six 27.4; gelu at 8192 x 8192 81.6, with its slope two
// values an instruction 95.7, though 70 against 75 where L2 holds the data).  dz is
// rounded to bf16 for the tensor cores; the sums are taken before that.  For an
// fp32 result what the rounding left is stored too (kTwo), and the product
// goes over both: dz to 2^-16.  A bf16 result is rounded as coarsely as dz.  (kTwo as an
// argument of the kernel instead: gelu at 8192 x 8192 94 us.)
template <int W, bool kF32, int kAct, bool kTwo>
__global__ void __launch_bounds__(256, 6) slope_kernel(const SlopeArgs p) {
  __shared__ float acc[8][32 * W + 8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = blockIdx.x * 32 * W + lane * W;
  float sum[W];
#pragma unroll
  for (int j = 0; j < W; ++j) sum[j] = 0.f;
  const long long step = (long long)gridDim.y * 8;
  grid_dependency_wait();
  const int width = (int)p.lddz;  // dz's padding columns, up to 7, get zeros
  if (col < (p.dz ? width : p.N)) {
    const bool in = col < p.N;
    for (long long row = (long long)blockIdx.y * 8 + warp; row < p.s; row += step) {
      float d[W], z[W];
#pragma unroll
      for (int j = 0; j < W; ++j) d[j] = z[j] = 0.f;
      if (in) {
        if (W == 8) {
          load8(p.dy, kF32, row * p.lddy + col, d);
          if (kAct != MOE_ACT_NONE) load8(p.z, 0, row * p.ldz + col, z);
        } else {
          d[0] = load_any(p.dy, kF32, row * p.lddy + col);
          if (kAct != MOE_ACT_NONE) z[0] = load_any(p.z, 0, row * p.ldz + col);
        }
      }
#pragma unroll
      for (int j = 0; j < W; ++j) {
        // rounded here, whether or not dz is stored: db has the same bits either way
        if (kAct != MOE_ACT_NONE) d[j] = __fmul_rn(d[j], slope(z[j], kAct));
        sum[j] += d[j];
      }
      if (p.dz) {
        bf16* at = p.dz + row * p.lddz + col;
        if (W == 8) *reinterpret_cast<uint4*>(at) = Vec<bf16>::from_float(d);
        else *at = __float2bfloat16_rn(d[0]);
        if (kTwo) {  // and what the rounding left, [s][lddz] further on
#pragma unroll
          for (int j = 0; j < W; ++j) {
            d[j] -= __bfloat162float(__float2bfloat16_rn(d[j]));
            if (!(fabsf(d[j]) < CUDART_INF_F)) d[j] = 0.f;  // of an infinity or a NaN
          }
          at += (long long)p.s * p.lddz;
          if (W == 8) *reinterpret_cast<uint4*>(at) = Vec<bf16>::from_float(d);
          else *at = __float2bfloat16_rn(d[0]);
        }
      }
    }
  }
  grid_dependents_launch();
  if (!p.part) return;
#pragma unroll
  for (int j = 0; j < W; ++j) acc[warp][lane * W + j] = sum[j];
  __syncthreads();
  const int c = blockIdx.x * 32 * W + threadIdx.x;
  if (threadIdx.x < 32 * W && c < p.N) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += acc[w][threadIdx.x];
    p.part[(size_t)blockIdx.y * p.N + c] = v;
  }
}

// ---- host ------------------------------------------------------------------------

// Output [outer][inner] of 4- or 2-byte elements as the epilogue stores it:
// boxes of 32 rows x 64 or 128 bytes, swizzled.
bool make_out_map(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer, bool f32, bool narrow) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {inner * (f32 ? 4 : 2)};
  cuuint32_t box[2] = {(narrow ? 64u : 128u) / (f32 ? 4u : 2u), 32u};
  cuuint32_t estride[2] = {1, 1};
  return fn(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims,
            strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE, narrow ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 2-D bf16 [outer][inner], rows ld elements apart, 128-byte swizzle.
bool make_map(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer, uint64_t ld, uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {ld * 2};
  cuuint32_t box[2] = {64, box_rows};
  cuuint32_t estride[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estride,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One product's plan.  kind: index into the three tile shapes.
struct Plan {
  int kind, tiles_m, tiles_n, splits, per_split, kblocks;
};
constexpr int kKinds = 3;
constexpr int kKindCG[kKinds] = {2, 1, 1};
constexpr int kKindBN[kKinds] = {256, 128, 64};
constexpr int kPlanSms = 152;  // plans are made for a whole GB300

// The shape and split of least estimated time, in units of a K block of the
// widest tile (0.65 us).  Measured: a K block of a 128 x 128 tile takes 0.70 of
// that and of 128 x 64 0.66 (both wait for shared memory, so the wide tile wins
// wherever it fills the machine: 9728 x 4096 x 4096 172.8, 243.3, 457.1 us);
// a launch's fixed part is 6.9, 5.9 and 4.7 us, a split's join about 2 us.  So
// 512 x 4096 x 4096 goes to 128 x 128 (22 us against 30 and 34), 64 rows of it to
// four parts of 128 x 128 (11.8; two 14.8, unsplit 20.2, wide 26.7), 1024^3 to
// 128 x 64 (7.8 against 12.8 and 9.9), 64 x 1024 x 1024 to four parts of that (5.8;
// unsplit 6.9).
Plan plan_gemm(int M, int N, int K, int passes, bool exact) {
  const double cost[kKinds] = {1.0, 0.70, 0.66}, base[kKinds] = {9.0, 8.0, 6.0};
  // clusters of 2, 4 and 8 CTAs that run at once (sixteen of eight did not: 2048 x
  // 4096 x 128 18.6 us, in four parts 10.2)
  const int clusters[4] = {0, 72, 34, 8};
  Plan best = {};
  double best_t = 0;
  const int kblocks = (K + 127) / 128 * passes;
  for (int k = exact ? 1 : 0; k < kKinds; ++k) {  // exact: its running sums need registers, so not the widest
    Plan q;
    q.kind = k;
    q.kblocks = kblocks;
    q.tiles_m = (M + 128 * kKindCG[k] - 1) / (128 * kKindCG[k]);
    q.tiles_n = (N + kKindBN[k] - 1) / kKindBN[k];
    const long long tiles = (long long)q.tiles_m * q.tiles_n;
    const int workers = kPlanSms / kKindCG[k];
    for (int sh = 0; sh < 4; ++sh) {
      const int S = 1 << sh;
      // a split part keeps at least two K blocks (256 terms)
      if (S > 1 && (kKindCG[k] == 2 || tiles > clusters[sh] || kblocks < 2 * S)) break;
      q.per_split = (kblocks + S - 1) / S;
      if ((S - 1) * q.per_split >= kblocks) continue;  // the last part would be empty
      q.splits = S;
      const long long waves = S > 1 ? 1 : (tiles + workers - 1) / workers;
      const double t = (double)waves * (q.per_split * cost[k] + 1.0) + base[k] + (S > 1 ? 3.0 : 0.0);
      if (best.kblocks == 0 || t < best_t) {
        best = q;
        best_t = t;
      }
    }
  }
  return best;
}

template <int CG, int BN, bool AT, bool BT, bool kExact, bool kSplit, bool kTwice>
cudaError_t run_one(const CUtensorMap (&maps)[4], const GemmArgs& p, const DeviceInfo& di, cudaStream_t st) {
  typedef Shape<CG, BN> S;
  static OncePerDevice once;
  cudaError_t err = once.run([] {
    return cudaFuncSetAttribute(gemm_kernel<CG, BN, AT, BT, kExact, kSplit, kTwice>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  });
  if (err != cudaSuccess) return err;
  const long long units = (long long)p.tiles_m * p.tiles_n;
  long long workers = di.sms / CG;
  if (kSplit || units < workers) workers = units;
  const unsigned cluster = kSplit ? (unsigned)p.splits : CG;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)workers * cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, gemm_kernel<CG, BN, AT, BT, kExact, kSplit, kTwice>, maps[0], maps[1], maps[2], maps[3], p);
}

template <int CG, int BN, bool AT, bool BT, bool kExact, bool kTwice = false>
cudaError_t run_gemm(const CUtensorMap (&maps)[4], const GemmArgs& p, const DeviceInfo& di, cudaStream_t st) {
  if constexpr (CG == 1) {
    if (p.splits > 1) return run_one<CG, BN, AT, BT, kExact, true, kTwice>(maps, p, di, st);
  }
  return run_one<CG, BN, AT, BT, kExact, false, kTwice>(maps, p, di, st);
}

// D [M,N] = A B^T with A [M][K] (AT: [K][M]) and B [N][K] (BT: [K][N]).  twice: A is
// the sum of two such matrices, one behind the other (BT and fp32 results only).
template <bool AT, bool BT>
cudaError_t product(const void* A, long long lda, const void* B, long long ldb, int M, int N, int K, bool twice, Epi epi,
                    int32_t* status, const DeviceInfo& di, cudaStream_t st) {
  const bool exact = epi.out_f32 || K > kLongSum;
  const int passes = twice ? 2 : 1, rows = AT ? K : M;
  const Plan q = plan_gemm(M, N, K, passes, exact);
  CUtensorMap maps[4] = {};
  const int box_b = BT ? 64 : kKindBN[q.kind] / kKindCG[q.kind];
  if (!make_map(&maps[0], A, AT ? M : K, (uint64_t)rows * passes, lda, AT ? 64 : 128) ||
      !(BT ? make_map(&maps[1], B, N, K, ldb, box_b) : make_map(&maps[1], B, K, N, ldb, box_b)))
    return cudaErrorInvalidValue;
  epi.wide = N % 8 == 0 && (!epi.res || epi.ldres % 8 == 0);
  epi.narrow = epi.z || (!epi.out_f32 && kKindBN[q.kind] < 128);
  if (q.splits == 1 && epi.wide &&
      (!make_out_map(&maps[2], epi.out, N, M, epi.out_f32, epi.narrow) ||
       (epi.z && !make_out_map(&maps[3], epi.z, N, M, false, true))))
    return cudaErrorInvalidValue;
  // the longest wait is the epilogue's, for a tile's whole contraction: 0.65 us a K block when all is well
  const long long limit = kWaitNs + 20000LL * q.per_split;
  GemmArgs p = {M, N, K, q.tiles_m, q.tiles_n, q.splits, q.per_split, q.kblocks,
                q.kblocks / passes, rows, epi, status, limit};
  if constexpr (BT) {
    if (twice)
      return q.kind == 1 ? run_gemm<1, 128, AT, BT, true, true>(maps, p, di, st) : run_gemm<1, 64, AT, BT, true, true>(maps, p, di, st);
  }
  if (exact)
    return q.kind == 1 ? run_gemm<1, 128, AT, BT, true>(maps, p, di, st) : run_gemm<1, 64, AT, BT, true>(maps, p, di, st);
  switch (q.kind) {
    case 0: return run_gemm<2, 256, AT, BT, false>(maps, p, di, st);
    case 1: return run_gemm<1, 128, AT, BT, false>(maps, p, di, st);
    default: return run_gemm<1, 64, AT, BT, false>(maps, p, di, st);
  }
}

template <bool kHigh>
cudaError_t few_rows(const LinearArgs& a, const Epi& e, const DeviceInfo& di, cudaStream_t st) {
  static OncePerDevice once;
  cudaError_t err = once.run([] {
    return cudaFuncSetAttribute(few_rows_kernel<kHigh>, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem);
  });
  if (err != cudaSuccess) return err;
  FewArgs p = {static_cast<const bf16*>(a.x), static_cast<const bf16*>(a.W), a.ldx, a.ldw, a.s, a.K, a.N, e, a.status,
               kWaitNs};
  return launch_chained(few_rows_kernel<kHigh>, dim3((unsigned)(a.N < di.sms ? a.N : di.sms)), dim3(288), kFewSmem, st, p);
}

size_t up(size_t v) { return (v + 255) / 256 * 256; }

int slope_rows(int s, int N) {  // blocks along the rows: enough to fill the machine, at least 32 rows each
  const int cols = (N + (N % 8 == 0 ? 255 : 31)) / (N % 8 == 0 ? 256 : 32);
  int rows = (6 * kPlanSms + cols - 1) / cols;
  const int most = (s + 31) / 32;
  if (rows > most) rows = most;
  return rows < 1 ? 1 : rows;
}

// dz, where it is not dy itself (once, or with what its rounding left), and the
// partial sums of db.
struct BwdPlan {
  size_t dz, part, total;
};
BwdPlan plan_bwd(int s, int N, int dz, bool db) {
  BwdPlan q;
  size_t at = 0;
  q.dz = at, at += up((size_t)s * ((N + 7) / 8 * 8) * 2 * dz);
  q.part = at, at += db ? up((size_t)slope_rows(s, N) * N * 4) : 0;
  q.total = at;
  return q;
}

// Copies of dz: none where a bf16 dy with whole 16-byte rows, without an
// activation, is dz itself; two where dz is rounded and a result is fp32.
int copies_of_dz(bool products, bool f32_results, int act, bool dy_f32, long long lddy) {
  const bool rounded = act != MOE_ACT_NONE || dy_f32;
  if (!products || (!rounded && lddy % 8 == 0)) return 0;
  return rounded && f32_results ? 2 : 1;
}

}  // namespace

size_t linear_bwd_workspace(int s, int N) { return plan_bwd(s, N, 2, true).total; }

size_t linear_bwd_workspace(int s, int N, int act, bool dy_f32, long long lddy, bool products, bool f32_results, bool db) {
  return plan_bwd(s, N, copies_of_dz(products, f32_results, act, dy_f32, lddy), db).total;
}

namespace {

template <int W, bool kF32, bool kTwo>
cudaError_t run_slope(const SlopeArgs& p, int act, int rows, cudaStream_t st) {
  const dim3 grid((unsigned)((p.lddz + 32 * W - 1) / (32 * W)), (unsigned)rows);
  auto kern = slope_kernel<W, kF32, MOE_ACT_NONE, kTwo>;
  switch (act) {
    case MOE_ACT_RELU: kern = slope_kernel<W, kF32, MOE_ACT_RELU, kTwo>; break;
    case MOE_ACT_GELU: kern = slope_kernel<W, kF32, MOE_ACT_GELU, kTwo>; break;
    case MOE_ACT_GELU_TANH: kern = slope_kernel<W, kF32, MOE_ACT_GELU_TANH, kTwo>; break;
    case MOE_ACT_SILU: kern = slope_kernel<W, kF32, MOE_ACT_SILU, kTwo>; break;
    default: break;
  }
  return launch_chained(kern, grid, dim3(256), 0, st, p);
}

template <int W, bool kF32>
cudaError_t run_slope(const SlopeArgs& p, int act, int rows, bool two, cudaStream_t st) {
  return two ? run_slope<W, kF32, true>(p, act, rows, st) : run_slope<W, kF32, false>(p, act, rows, st);
}

}  // namespace

cudaError_t launch_linear(const LinearArgs& a, const DeviceInfo& di, cudaStream_t st) {
  Epi e = {};
  e.out = a.y;
  e.z = static_cast<bf16*>(a.z);
  e.bias = a.bias;
  e.res = a.res;
  e.ldres = a.ldres;
  e.act = a.act;
  e.out_f32 = a.out_f32;
  e.bias_f32 = a.bias_f32;
  e.res_f32 = a.res_f32;
  if (a.s <= kFewRows) return a.s > 8 ? few_rows<true>(a, e, di, st) : few_rows<false>(a, e, di, st);
  return product<false, false>(a.x, a.ldx, a.W, a.ldw, a.s, a.N, a.K, false, e, a.status, di, st);
}

cudaError_t launch_linear_bwd(const LinearBwdArgs& a, const DeviceInfo& di, cudaStream_t st) {
  const bool f32_dx = a.dx && a.dx_f32, f32_dw = a.dW && a.dw_f32;
  const int own = copies_of_dz(a.dx || a.dW, f32_dx || f32_dw, a.act, a.dy_f32, a.lddy);
  const BwdPlan q = plan_bwd(a.s, a.N, own, a.db != nullptr);
  char* ws = static_cast<char*>(a.workspace);
  const int lddz = (a.N + 7) / 8 * 8;
  if (own || a.db) {
    SlopeArgs p = {};
    p.dy = a.dy;
    p.z = a.act != MOE_ACT_NONE ? static_cast<const bf16*>(a.z) : nullptr;  // unused without an activation
    p.dz = own ? reinterpret_cast<bf16*>(ws + q.dz) : nullptr;
    p.part = a.db ? reinterpret_cast<float*>(ws + q.part) : nullptr;
    p.lddy = a.lddy;
    p.ldz = a.ldz;
    p.lddz = lddz;
    p.s = a.s;
    p.N = a.N;
    const int rows = slope_rows(a.s, a.N);
    const bool wide = a.N % 8 == 0 && a.lddy % 8 == 0 && (!p.z || a.ldz % 8 == 0);
    cudaError_t err;
    if (wide) err = a.dy_f32 ? run_slope<8, true>(p, a.act, rows, own == 2, st) : run_slope<8, false>(p, a.act, rows, own == 2, st);
    else err = a.dy_f32 ? run_slope<1, true>(p, a.act, rows, own == 2, st) : run_slope<1, false>(p, a.act, rows, own == 2, st);
    if (err != cudaSuccess) return err;
    if (a.db) {
      err = launch_sum_parts(p.part, rows, 0, a.N, a.N, a.db, nullptr, st);
      if (err != cudaSuccess) return err;
    }
  }
  const void* dz = own ? ws + q.dz : a.dy;
  const long long ld = own ? lddz : a.lddy;
  if (a.dx) {
    Epi e = {};
    e.out = a.dx;
    e.out_f32 = a.dx_f32;
    cudaError_t err = product<false, true>(dz, ld, a.W, a.ldw, a.s, a.K, a.N, own == 2 && f32_dx, e, a.status, di, st);
    if (err != cudaSuccess) return err;
  }
  if (a.dW) {
    Epi e = {};
    e.out = a.dW;
    e.out_f32 = a.dw_f32;
    cudaError_t err = product<true, true>(dz, ld, a.x, a.ldx, a.N, a.K, a.s, own == 2 && f32_dw, e, a.status, di, st);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

}  // namespace moe
