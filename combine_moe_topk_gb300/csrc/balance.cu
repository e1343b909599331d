// balance.cu -- the router's balance loss with its per-expert counts, the z
// loss from the same pass over the logits, and their gradient.
//
// The tokens are cut into B packed sequences by seq_offsets (one sequence of
// all tokens without them).  With T_b the valid tokens of sequence b, n_bj its
// routes to expert j, p = softmax(logits), P_bj = (1/T_b) sum_t p_tj, and B'
// the sequences with T_b > 0:
//   L = (1/B') sum_b e sum_j n_bj / (k T_b) P_bj,   Z = (1/T) sum_t lse_t^2
//   dl_tj = dL/B' p_tj (c_bj - sum_i c_bi p_ti) + dZ 2 lse_t p_tj / T,
//   c_bj = e n_bj / (k T_b^2)    (the counts are not differentiable)
// Both directions read each logit once and are bound by device memory; the
// forward pass keeps lse (one fp32 a token), so the backward pass needs no
// maximum: it takes a row's sum and its dot product with c in one reduction.
//
// L lanes share a row (the smallest power of two that covers it with one
// vector a lane), so a warp works on 32/L rows at once and few experts do
// not leave lanes idle.  A block owns a run of consecutive tokens; the part of
// a sequence inside a block (a piece) is summed in registers, then over the
// block through shared memory, and written to slot (block + sequence), which
// no other piece has.  join_kernel adds each sequence's pieces in block order:
// no floating-point atomics, so the results are the same on every run.
//
// Measured, 256 experts, 131072 tokens, top 8: forward 32.5 us (one sequence) and
// 36.2 (37 of them; 37.8 with padding), of which the join's latency is 7 and the blocks'
// uneven ends 4, the bytes alone 20.7; backward with a gradient added 66 us, its
// bytes 60.  8192 x 8: 6.7 and 2.6 us.
#include <float.h>
#include <math_constants.h>

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kBlock = 512;
constexpr int kWarps = kBlock / 32;
constexpr int kMaxExperts = 256;

// A piece's sums, [slots][...] in the workspace.
struct Pieces {
  float* psum;    // [slots][e]
  int* count;     // [slots][e]
  float* zsum;    // [slots]
  int* tokens;    // [slots]
};

// Row groups whose loads a warp keeps in flight: 16 values a lane.
constexpr int unroll_of(int V, int NI) { return V * NI >= 8 ? 2 : 4; }

struct BalanceFwd {
  const float* logits;
  const int32_t* idx;
  const uint8_t* valid;
  const int32_t* offsets;
  int s, e, k, B, chunk;
  float* lse;
  Pieces pc;
  unsigned* ticket;
  int32_t* status;
};

// First sequence that ends after token t (B when none does).
__device__ __forceinline__ int sequence_of(const int32_t* offsets, int B, int t) {
  int lo = 0, hi = B;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ld_plain(offsets + mid + 1) <= t) lo = mid + 1; else hi = mid;
  }
  return lo;
}

// Bounds of sequence b inside [lo, hi); empty (x >= y) where they do not meet.
__device__ __forceinline__ int2 piece_of(const int32_t* offsets, int s, int b, int lo, int hi) {
  if (!offsets) return make_int2(lo, hi);
  const int o0 = ld_plain(offsets + b), o1 = ld_plain(offsets + b + 1);
  return make_int2(o0 > lo ? o0 : lo, o1 < hi ? o1 : hi);
}

// One row's columns held by this lane: V consecutive at V * (lane + L * i).
template <int V>
__device__ __forceinline__ void load_cols(const float* p, float* f) {
  if (V == 4) {
    const uint4 v = ld_stream(reinterpret_cast<const uint4*>(p));
    Vec<float>::to_float(v, f);
  } else {
    f[0] = ld_plain(p);
  }
}

// The same by plain loads: `add` may be the buffer that is written.
template <int V>
__device__ __forceinline__ void load_add(const float* p, float* f) {
  if (V == 4) Vec<float>::to_float(*reinterpret_cast<const uint4*>(p), f);
  else f[0] = *p;
}

constexpr float kLog2e = 1.4426950408889634f;

template <int L>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// f = exp(f - base) of a lane's n values, and their sum; two values an
// instruction.  Subtracted before it is scaled, so that the largest term of a
// softmax is 1 whatever the logits' size (2^(f log2 e - base log2 e) in one fma
// keeps the rounding of base log2 e in the exponent: at 1e10 that is hundreds).
template <int n>
__device__ __forceinline__ float exponentials(float* f, float base) {
  if (n == 1) return f[0] = exp2_approx((f[0] - base) * kLog2e);
  float2 sum = both(0.f);
#pragma unroll
  for (int j = 0; j + 1 < n; j += 2) {
    float2 v = mul2(add2(make_float2(f[j], f[j + 1]), both(-base)), both(kLog2e));
    v = make_float2(exp2_approx(v.x), exp2_approx(v.y));
    sum = add2(sum, v);
    f[j] = v.x;
    f[j + 1] = v.y;
  }
  return sum.x + sum.y;
}

template <int V, int L, int NI>
__global__ void __launch_bounds__(kBlock, 2) balance_kernel(const BalanceFwd p) {
  constexpr int kRows = 32 / L;  // rows of a warp at once
  constexpr int U = unroll_of(V, NI);
  __shared__ int s_count[kMaxExperts];
  __shared__ float s_p[kWarps][V * L * NI];
  __shared__ float s_z[kWarps];
  __shared__ int s_t[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / L, col = lane % L;
  const int lo = blockIdx.x * p.chunk, hi = lo + min(p.chunk, p.s - lo);
  grid_dependency_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.ticket = 0;  // for the join, later in the stream
  // tokens outside every sequence: nothing of theirs counts
  const int first = p.offsets ? ld_plain(p.offsets) : 0, last = p.offsets ? ld_plain(p.offsets + p.B) : p.s;
  for (int i = threadIdx.x; i < hi - lo; i += kBlock)
    if (lo + i < first || lo + i >= last) p.lse[lo + i] = 0.f;
  int bad = 0;
  for (int b = p.offsets ? sequence_of(p.offsets, p.B, lo) : 0; b < p.B; ++b) {
    if (p.offsets && ld_plain(p.offsets + b) >= hi) break;
    const int2 r = piece_of(p.offsets, p.s, b, lo, hi);
    if (r.x >= r.y) continue;  // the same for the whole block
    for (int j = threadIdx.x; j < p.e; j += kBlock) s_count[j] = 0;
    __syncthreads();
    float acc[NI][V], zsum = 0.f;
    int tokens = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) acc[i][v] = 0.f;
    // i0, then a row's place o behind it: a token's number near 2^31 plus a step would not fit an int
    for (int i0 = warp * kRows * U; i0 < r.y - r.x; i0 += kWarps * kRows * U) {
      const int t0 = r.x + i0, left = r.y - t0;
      const float* x = p.logits + ((size_t)t0 + sub) * p.e;  // this lane's row of the first group
      // the loads of U row groups and of these tokens' ids travel together
      float f[U][NI][V];
      bool live[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int o = u * kRows + sub;
        live[u] = o < left && (!p.valid || ld_plain(p.valid + t0 + o) != 0);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int c = V * (col + L * i);
#pragma unroll
          for (int v = 0; v < V; ++v) f[u][i][v] = -CUDART_INF_F;
          if (live[u] && c < p.e) load_cols<V>(x + u * kRows * p.e + c, f[u][i]);
        }
      }
      const int n_ids = min(kRows * U, left) * p.k;
#pragma unroll 2
      for (int q = lane; q < n_ids; q += 32) {
        const int id = ld_plain(p.idx + (size_t)t0 * p.k + q);
        if (p.valid && ld_plain(p.valid + t0 + q / p.k) == 0) continue;
        if ((unsigned)id < (unsigned)p.e) atomicAdd(&s_count[id], 1);
        else if (id != -1) bad |= 2;
      }
      float sums[U], bases[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float top = -FLT_MAX;  // a mask of the type's lowest value counts as -inf
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int v = 0; v < V; ++v) top = fmaxf(top, f[u][i][v]);
        top = lanes_max<L>(top);
        const float base = top == -FLT_MAX ? 0.f : top;  // a row of masked experts: every exp below is 0
        const float sum = lanes_sum<L>(exponentials<NI * V>(&f[u][0][0], base));
        if (!(sum < CUDART_INF_F)) bad |= 1;  // a NaN or +inf makes it NaN
        // 0 for a row that takes no part; NaN stays
        const float inv = live[u] && sum != 0.f ? __fdividef(1.f, sum) : 0.f;
        if (live[u]) {
#pragma unroll
          for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) acc[i][v] = fmaf(f[u][i][v], inv, acc[i][v]);
        }
        sums[u] = live[u] ? sum : -1.f;
        bases[u] = base;
      }
      // lse of the U row groups: lane u of a row's lanes takes group u, so that the
      // logarithm is taken once (in rounds where a row has fewer lanes than U)
#pragma unroll
      for (int r0 = 0; r0 < U; r0 += L) {
        float sum = sums[r0], base = bases[r0];
#pragma unroll
        for (int u = r0 + 1; u < U && u < r0 + L; ++u) {
          sum = col == u - r0 ? sums[u] : sum;
          base = col == u - r0 ? bases[u] : base;
        }
        const int o = (r0 + col) * kRows + sub;
        if (col < U - r0 && col < L && o < left) {
          const bool some = sum > 0.f || sum != sum;
          const float lse = some ? base + logf(sum) : (sum < 0.f ? 0.f : -CUDART_INF_F);
          p.lse[t0 + o] = lse;
          if (some) zsum = fmaf(lse, lse, zsum);
          tokens += sum < 0.f ? 0 : 1;
        }
      }
    }
    // the warp's row groups, then the block's warps, in a fixed order
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int d = L; d < 32; d <<= 1) acc[i][v] += __shfl_xor_sync(0xffffffffu, acc[i][v], d);
        if (sub == 0) s_p[warp][V * (col + L * i) + v] = acc[i][v];
      }
    zsum = lanes_sum<32>(zsum);
    tokens = __reduce_add_sync(0xffffffffu, tokens);
    if (lane == 0) {
      s_z[warp] = zsum;
      s_t[warp] = tokens;
    }
    __syncthreads();
    const size_t slot = (size_t)blockIdx.x + b;
    for (int j = threadIdx.x; j < p.e; j += kBlock) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += s_p[w][j];
      p.pc.psum[slot * p.e + j] = sum;
      p.pc.count[slot * p.e + j] = s_count[j];
    }
    if (threadIdx.x == 0) {
      float z = 0.f;
      int n = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        z += s_z[w];
        n += s_t[w];
      }
      p.pc.zsum[slot] = z;
      p.pc.tokens[slot] = n;
    }
    __syncthreads();  // the shared sums are rewritten by the next piece
  }
  grid_dependents_launch();
  if (bad & 1) raise_status(p.status, MOE_DEV_NONFINITE);
  if (bad & 2) raise_status(p.status, MOE_DEV_BAD_ROUTE);
}

struct BalanceJoin {
  const int32_t* offsets;
  int s, e, k, B, chunk, cols;  // cols: blocks of 32 columns per sequence
  Pieces pc;
  int32_t* counts;
  float* mean_prob;
  float* coef;
  float* part;    // [B * cols] this block's share of e sum_j f_j P_j
  float* zpart;   // [B]
  int* tpart;     // [B] valid tokens
  unsigned* ticket;
  float* loss;    // [2]
  float* norm;    // [2] 1 / B', 1 / T
};

constexpr int kJoin = 1024;

// One block per sequence and 32 columns: the pieces, 32 threads a column, ten
// loads of each in flight, then a warp for each column; the last block to
// finish adds the sequences' losses in a fixed order.
__global__ void __launch_bounds__(kJoin) balance_join_kernel(const BalanceJoin p) {
  __shared__ float s_f[32][33];
  __shared__ int s_c[32][33];
  __shared__ float s_z[32], s_share[32];
  __shared__ int s_t[32];
  __shared__ float4 s_last_sums[32];
  __shared__ int s_last;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int b = (int)(blockIdx.x / (unsigned)p.cols), block = (int)(blockIdx.x - (unsigned)b * p.cols);
  grid_dependency_wait();
  int lo = 0, hi = p.s;
  if (p.offsets) {
    lo = max(0, ld_plain(p.offsets + b));
    hi = min(p.s, ld_plain(p.offsets + b + 1));
  }
  const int c0 = lo / p.chunk, c1 = lo < hi ? (hi - 1) / p.chunk + 1 : c0;  // the blocks that have a piece of it
  {
    const int col = block * 32 + tx;
    float sum = 0.f;
    int count = 0;
    if (col < p.e) {
      for (int q = c0 + ty; q < c1; q += 320) {
        float f[10];
        int n[10];
#pragma unroll
        for (int i = 0; i < 10; ++i) {
          const size_t at = ((size_t)min(q + 32 * i, c1 - 1) + b) * p.e + col;
          f[i] = q + 32 * i < c1 ? ld_plain(p.pc.psum + at) : 0.f;
          n[i] = q + 32 * i < c1 ? ld_plain(p.pc.count + at) : 0;
        }
#pragma unroll
        for (int i = 0; i < 10; ++i) {
          sum += f[i];
          count += n[i];
        }
      }
    }
    float z = 0.f;
    int tokens = 0;
    for (int c = c0 + threadIdx.x; c < c1; c += kJoin) {
      tokens += ld_plain(p.pc.tokens + (size_t)c + b);
      z += ld_plain(p.pc.zsum + (size_t)c + b);
    }
    s_f[ty][tx] = sum;
    s_c[ty][tx] = count;
    z = lanes_sum<32>(z);
    tokens = __reduce_add_sync(0xffffffffu, tokens);  // as integers: floats are exact to 2^24 only
    if (tx == 0) {
      s_z[ty] = z;
      s_t[ty] = tokens;
    }
  }
  __syncthreads();
  const int tokens = __reduce_add_sync(0xffffffffu, s_t[tx]);
  const int col = block * 32 + ty;  // this warp's column
  const float sum = lanes_sum<32>(s_f[tx][ty]);
  const int count = __reduce_add_sync(0xffffffffu, s_c[tx][ty]);
  const float inv_t = tokens > 0 ? 1.f / (float)tokens : 0.f;
  const float P = sum * inv_t, f = (float)count * inv_t / (float)p.k;
  if (tx == 0) {
    if (col < p.e) {
      p.counts[(size_t)b * p.e + col] = count;
      p.mean_prob[(size_t)b * p.e + col] = P;
      p.coef[(size_t)b * p.e + col] = (float)p.e * f * inv_t;
    }
    s_share[ty] = col < p.e ? (float)p.e * f * P : 0.f;
  }
  __syncthreads();
  auto write_losses = [&](float loss, float z, float sequences, float count) {
    const float per_seq = 1.f / fmaxf(sequences, 1.f), per_token = 1.f / fmaxf(count, 1.f);
    p.loss[0] = loss * per_seq;
    p.loss[1] = z * per_token;
    p.norm[0] = per_seq;
    p.norm[1] = per_token;
  };
  if (ty == 0) {
    const float share = lanes_sum<32>(s_share[tx]), z = lanes_sum<32>(s_z[tx]);
    if (tx == 0) {
      if (gridDim.x == 1) {  // there is nothing to add to it
        write_losses(share, z, tokens > 0 ? 1.f : 0.f, (float)tokens);
        s_last = 0;
      } else {
        p.part[(size_t)b * p.cols + block] = share;
        if (block == 0) {
          p.zpart[b] = z;
          p.tpart[b] = tokens;
        }
        __threadfence();
        s_last = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
      }
    }
  }
  grid_dependents_launch();
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  float4 all = make_float4(0.f, 0.f, 0.f, 0.f);  // loss, z, sequences with tokens, tokens
  for (int q = threadIdx.x; q < p.B; q += kJoin) {
    for (int c = 0; c < p.cols; ++c) all.x += __ldcg(p.part + (size_t)q * p.cols + c);
    all.y += __ldcg(p.zpart + q);
    const int n = __ldcg(p.tpart + q);
    all.z += n > 0 ? 1.f : 0.f;
    all.w += (float)n;
  }
  auto sum4 = [](float4 v) {
    return make_float4(lanes_sum<32>(v.x), lanes_sum<32>(v.y), lanes_sum<32>(v.z), lanes_sum<32>(v.w));
  };
  all = sum4(all);
  if (tx == 0) s_last_sums[ty] = all;
  __syncthreads();
  if (ty == 0) {
    all = sum4(s_last_sums[tx]);
    if (tx == 0) write_losses(all.x, all.y, all.z, all.w);
  }
}

struct BalanceBwd {
  const float* logits;
  const float* lse;
  const float* coef;
  const float* norm;
  const float* dloss;
  const uint8_t* valid;
  const int32_t* offsets;
  const float* add;
  float* dlogits;
  int s, e, B, chunk;
};

template <int V>
__device__ __forceinline__ void store_cols(float* p, const float* f) {
  if (V == 4) st_stream(reinterpret_cast<uint4*>(p), Vec<float>::from_float(f));
  else *p = f[0];
}

// Rows [lo, hi) get `add` or zeros: tokens outside every sequence.
template <int V>
__device__ __forceinline__ void copy_rows(const BalanceBwd& p, int lo, int hi) {
  for (long long q = (long long)lo * p.e + V * threadIdx.x; q < (long long)hi * p.e; q += V * kBlock) {
    float f[V];
#pragma unroll
    for (int v = 0; v < V; ++v) f[v] = 0.f;
    if (p.add) load_add<V>(p.add + q, f);
    store_cols<V>(p.dlogits + q, f);
  }
}

template <int V, int L, int NI>
__global__ void __launch_bounds__(kBlock, 2) balance_bwd_kernel(const BalanceBwd p) {
  constexpr int kRows = 32 / L, U = unroll_of(V, NI);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / L, col = lane % L;
  const int lo = blockIdx.x * p.chunk, hi = lo + min(p.chunk, p.s - lo);
  grid_dependency_wait();
  const float wl = ld_plain(p.dloss) * ld_plain(p.norm), wz = 2.f * ld_plain(p.dloss + 1) * ld_plain(p.norm + 1);
  if (p.offsets) {
    copy_rows<V>(p, lo, min(hi, max(lo, ld_plain(p.offsets))));
    copy_rows<V>(p, max(lo, min(hi, ld_plain(p.offsets + p.B))), hi);
  }
  for (int b = p.offsets ? sequence_of(p.offsets, p.B, lo) : 0; b < p.B; ++b) {
    if (p.offsets && ld_plain(p.offsets + b) >= hi) break;
    const int2 r = piece_of(p.offsets, p.s, b, lo, hi);
    if (r.x >= r.y) continue;
    float c[NI][V];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int j = V * (col + L * i) + v;
        c[i][v] = j < p.e ? wl * ld_plain(p.coef + (size_t)b * p.e + j) : 0.f;
      }
    for (int i0 = warp * kRows * U; i0 < r.y - r.x; i0 += kWarps * kRows * U) {
      const int t0 = r.x + i0, left = r.y - t0;
      float f[U][NI][V], g[U][NI][V], lse[U];
      bool some[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int o = u * kRows + sub;
        const bool live = o < left && (!p.valid || ld_plain(p.valid + t0 + o) != 0);
        lse[u] = o < left ? ld_plain(p.lse + t0 + o) : 0.f;
        some[u] = live && lse[u] != -CUDART_INF_F;  // a row of masked experts has no probabilities
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int o = u * kRows + sub;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int q = V * (col + L * i);
#pragma unroll
          for (int v = 0; v < V; ++v) f[u][i][v] = -CUDART_INF_F, g[u][i][v] = 0.f;
          if (o < left && q < p.e) {
            load_cols<V>(p.logits + (size_t)((unsigned)t0 + o) * p.e + q, f[u][i]);
            if (p.add) load_add<V>(p.add + (size_t)((unsigned)t0 + o) * p.e + q, g[u][i]);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int o = u * kRows + sub;
        // lse is rounded to its own last place: past 1e8 nothing of the sum's
        // logarithm is left in it.  Divided by the row's sum, p has that no more.
        const float sum = lanes_sum<L>(exponentials<NI * V>(&f[u][0][0], lse[u]));
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int v = 0; v < V; ++v) dot = fmaf(c[i][v], f[u][i][v], dot);
        const float inv = __fdividef(1.f, sum);  // in [1/256, 256]: lse is off by at most log e
        dot = lanes_sum<L>(dot) * inv;
        const float zt = wz * lse[u];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int q = V * (col + L * i);
          if (some[u]) {
#pragma unroll
            for (int v = 0; v < V; ++v) g[u][i][v] = fmaf(f[u][i][v] * inv, c[i][v] - dot + zt, g[u][i][v]);
          }
          if (o < left && q < p.e) store_cols<V>(p.dlogits + (size_t)((unsigned)t0 + o) * p.e + q, g[u][i]);
        }
      }
    }
  }
  grid_dependents_launch();
}

struct Shape {
  int V, L, NI;
};

// Lanes of a row: the fewest (a power of two) that hold it with one vector or
// element each; past 32 lanes each holds NI of them.
Shape shape_of(int e) {
  Shape h;
  h.V = e % 4 == 0 ? 4 : 1;
  const int n = e / h.V;
  h.L = 1;
  while (h.L < 32 && h.L < n) h.L *= 2;
  h.NI = 1;
  while (h.L * h.NI < n) h.NI *= 2;
  return h;
}

// Tokens of a block: at least one round of every warp, in at most
// kBalanceBlocks blocks, two an SM.
int chunk_of(int s, const Shape& h) {
  const int round = kWarps * (32 / h.L);
  long long c = ((long long)s + kBalanceBlocks - 1) / kBalanceBlocks;
  c = (c + round - 1) / round * round;
  return (int)c;
}

#define MOE_BALANCE_SHAPES(X)                                                                                  \
  X(4, 1, 1) X(4, 2, 1) X(4, 4, 1) X(4, 8, 1) X(4, 16, 1) X(4, 32, 1) X(4, 32, 2) X(1, 1, 1) X(1, 2, 1)        \
  X(1, 4, 1) X(1, 8, 1) X(1, 16, 1) X(1, 32, 1) X(1, 32, 2) X(1, 32, 4) X(1, 32, 8)

size_t up(size_t v) { return (v + 255) / 256 * 256; }

struct Plan {
  size_t psum, count, zsum, tokens, part, zpart, tpart, ticket, total;
};
Plan plan_of(int e, int B) {
  const size_t slots = (size_t)kBalanceBlocks + B, cols = (e + 31) / 32;
  Plan q;
  size_t at = 0;
  q.psum = at, at += up(slots * e * 4);
  q.count = at, at += up(slots * e * 4);
  q.zsum = at, at += up(slots * 4);
  q.tokens = at, at += up(slots * 4);
  q.part = at, at += up((size_t)B * cols * 4);
  q.zpart = at, at += up((size_t)B * 4);
  q.tpart = at, at += up((size_t)B * 4);
  q.ticket = at, at += up(4);
  q.total = at;
  return q;
}

}  // namespace

size_t balance_workspace(int e, int B) { return plan_of(e, B).total; }

cudaError_t launch_balance(const float* logits, const int32_t* idx, const uint8_t* valid, const int32_t* offsets,
                           int s, int e, int k, int B, float* loss, int32_t* counts, float* mean_prob, float* lse,
                           float* coef, float* norm, void* workspace, int32_t* status, cudaStream_t st) {
  char* ws = static_cast<char*>(workspace);
  const Plan q = plan_of(e, B);
  const Shape h = shape_of(e);
  const int chunk = s > 0 ? chunk_of(s, h) : 1;
  Pieces pc = {reinterpret_cast<float*>(ws + q.psum), reinterpret_cast<int*>(ws + q.count),
               reinterpret_cast<float*>(ws + q.zsum), reinterpret_cast<int*>(ws + q.tokens)};
  unsigned* ticket = reinterpret_cast<unsigned*>(ws + q.ticket);
  BalanceFwd p = {logits, idx, valid, offsets, s, e, k, B, chunk, lse, pc, ticket, status};
  const unsigned grid = s > 0 ? (unsigned)((s - 1) / chunk + 1) : 1u;  // no tokens: one block clears the ticket
  cudaError_t err = cudaErrorInvalidValue;
#define MOE_RUN(v, l, n) \
  if (h.V == v && h.L == l && h.NI == n) err = launch_chained(balance_kernel<v, l, n>, dim3(grid), dim3(kBlock), 0, st, p);
  MOE_BALANCE_SHAPES(MOE_RUN)
#undef MOE_RUN
  if (err != cudaSuccess) return err;
  const int cols = (e + 31) / 32;
  BalanceJoin j = {offsets, s, e, k, B, chunk, cols, pc, counts, mean_prob, coef,
                   reinterpret_cast<float*>(ws + q.part), reinterpret_cast<float*>(ws + q.zpart),
                   reinterpret_cast<int*>(ws + q.tpart), ticket, loss, norm};
  return launch_chained(balance_join_kernel, dim3((unsigned)cols * (unsigned)B), dim3(kJoin), 0, st, j);
}

cudaError_t launch_balance_bwd(const float* logits, const float* lse, const float* coef, const float* norm,
                               const float* dloss, const uint8_t* valid, const int32_t* offsets, const float* add,
                               int s, int e, int B, float* dlogits, cudaStream_t st) {
  const Shape h = shape_of(e);
  const int chunk = chunk_of(s, h);
  BalanceBwd p = {logits, lse, coef, norm, dloss, valid, offsets, add, dlogits, s, e, B, chunk};
  const unsigned grid = (unsigned)((s - 1) / chunk + 1);
  cudaError_t err = cudaErrorInvalidValue;
#define MOE_RUN(v, l, n) \
  if (h.V == v && h.L == l && h.NI == n) \
    err = launch_chained(balance_bwd_kernel<v, l, n>, dim3(grid), dim3(kBlock), 0, st, p);
  MOE_BALANCE_SHAPES(MOE_RUN)
#undef MOE_RUN
  return err;
}

}  // namespace moe
