// grouped_gemm.cu -- the expert-grouped GEMM that consumes the dispatched
// rows, on the 5th-generation tensor cores (tcgen05, TMEM accumulators,
// TMA tile loads), its fused form that gathers the token rows itself, and both
// for gated experts.
//
// DeepSpeed #8213 "Add an opt-in DeepEP transport for the AutoEP expert
// all-to-all", description: the dispatch groups arrivals by expert for the
// grouped GEMM, whose groups are bounded by offsets = cumsum(counts).
// Automodel #3684 "perf(moe): reuse the DeepEP dispatch layout on
// activation-checkpoint recompute": each expert's rows may be padded to a
// multiple (pad_multiple); nothing here needs it.
//
// Y[r] = A[r] . W[x]^T for every row r that a kept route to expert x owns,
// r in [offsets[x], offsets[x] + counts[x]).  A[r] is the dispatched row
// X[r] (moe_grouped_gemm) or the token row x[inv_row[r]] (fused dispatch:
// the dispatched buffer is never written or read).  bf16 operands,
// row-major, K contiguous; the accumulation is fp32 in TMEM.  Work units are row blocks
// of one expert's segment (256 rows on SM pairs, 128 on single SMs; the
// first at offsets[x], so a segment may start on any row) times
// 256-column tiles of N.
//
// Both forms run on pairs of SMs (grouped_gemm_pair_kernel, below): a
// cluster of two CTAs computes a 256-row block x 256 columns with
// tcgen05.mma.cta_group::2, each SM staging only its half of A and of B
// (two 64-wide K blocks per stage of a 3-stage ring).
// In the fused form the second CTA's gathered rows reach the MMA issuer
// through a 16-byte shared-to-shared bulk copy that counts on the first
// CTA's barrier: a per-K-block arrival with cluster-scope release instead
// held the paired fused GEMM to 0.56 PFLOP/s.  A TMA tile::gather4 of four
// rows per request was tried first for the fused form's A: correct, but at
// 33 copy requests per K-block it held the GEMM to a third of the tensor
// rate.  (A one-SM form with 128-row blocks came before the pairs and was
// measured 2-12 % slower on every shape; it is gone.  Short expert segments
// waste the tail of a 256-row block, but a 128-row block wastes the same
// tail rows, and where segments are short -- many experts, few rows each --
// streaming each expert's weights once bounds the GEMM anyway.)
// Every mbarrier wait is bounded on the global timer, each from its own start;
// a time-out records MOE_DEV_TIMEOUT and the roles wind down to the TMEM release.
#include "common.cuh"
#include "grouped.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace moe {

namespace {

constexpr int BM = 128, BN = 256, BK = 64;
constexpr int kTmemCols = 2 * BN;     // two fp32 accumulators of 128 lanes x 256 columns
// Epilogue warps of the gated form (4 in the plain one).  Its fused form has 4 too: with
// 8 beside the gathering warps 96 registers a thread do not do (16384 rows x 4096 x
// 2048, z kept: 357 us, 348 with 4).
constexpr int kGatedWarps = 8;
// Warps gathering the fused form's A rows: 8 (16 rows each) measured 1-4 %
// faster than 4 and 3 % faster than 16 (fewer registers per thread at 768
// threads); 2 were 20-30 % slower.
#ifndef MOE_GEMM_GATHER_WARPS
#define MOE_GEMM_GATHER_WARPS 8
#endif
constexpr int kGatherRows = BM / MOE_GEMM_GATHER_WARPS;  // A rows per gathering warp
static_assert(kGatherRows % 4 == 0 && kGatherRows >= 4, "a gathering warp copies 4 rows per instruction");
constexpr int kMaxE = 256;
// epilogue staging: per epilogue warp 32 rows x 64 bf16 columns, rows padded
// to 144 bytes (conflict-free 16-byte writes by row and reads by column)
constexpr int kStageRowBytes = 64 * 2 + 16;
constexpr int kEpiWarpBytes = 32 * kStageRowBytes;
constexpr int kEpiBytes = 4 * kEpiWarpBytes;
static_assert(kGatedWarps * kRowStage <= kEpiBytes, "the gated form's staging tiles fit in the same place");

struct GemmParams {
  const __nv_bfloat16* x;  // gather mode: token rows [s, K]
  const int32_t* offsets;
  const int32_t* counts;
  const int32_t* inv_row;  // gather mode: token of each owned row
  int e, rows, K, N;
  int s;                   // gather mode: token rows of x
  __nv_bfloat16* Y;
  int32_t* status;
  long long timeout_ns;  // of a single wait
  __nv_bfloat16* Z;      // gated form: [rows, 2N], or NULL
  int act;
};

// Shared-memory matrix descriptor: K-major, 128-byte swizzle (as TMA writes
// it), 8-row groups 1024 bytes apart.  The tile base is 1024-byte aligned.
__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3ffffu) >> 4);  // start address
  d |= (uint64_t)1 << 16;                    // leading byte offset (unused when swizzled)
  d |= (uint64_t)(1024 >> 4) << 32;          // stride byte offset
  d |= (uint64_t)1 << 46;                    // descriptor version
  d |= (uint64_t)2 << 61;                    // 128-byte swizzle
  return d;
}

// 16-byte asynchronous copy global -> shared (L2 only): copies src_bytes
// (0 or 16) from gsrc and fills the rest of the 16 bytes with zeros; with 0
// nothing is read.
__device__ __forceinline__ void cp_async16_zfill(uint32_t sdst, const void* gsrc, uint32_t src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sdst), "l"(gsrc), "r"(src_bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// One arrival on `bar` once every cp.async this thread issued so far has
// landed; the barrier's expected count includes it (.noinc).
__device__ __forceinline__ void cp_async_arrive_noinc(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// Drain one 128 x 256 fp32 accumulator to bf16 rows of Y.  Epilogue warp ew
// owns TMEM lanes 32ew .. 32ew+31 (rows r0 + 32ew ..); 64 columns at a time,
// each lane converts its row (nearest-even) into the warp's padded staging
// tile, then the warp stores it back out as 4 rows x 128 bytes per
// instruction.  Only rows below nvalid (owned by a route) are stored.
__device__ __forceinline__ void store_accumulator(uint32_t tcol, int ew, int lane, uint8_t* stage,
                                                  __nv_bfloat16* Y, int N, int r0, int n0, int nvalid) {
#pragma unroll 1
  for (int c2 = 0; c2 < BN / 64; ++c2) {
    uint4 out[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t v[32];
      tmem_ld32(tcol + (uint32_t)(64 * c2 + 32 * h), v);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[8 * q + i]);
        out[4 * h + q] = Vec<__nv_bfloat16>::from_float(f);
      }
    }
    uint4* srow = reinterpret_cast<uint4*>(stage + lane * kStageRowBytes);
#pragma unroll
    for (int q = 0; q < 8; ++q) srow[q] = out[q];
    __syncwarp();
    const int ch = lane & 7;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = 4 * i + (lane >> 3);
      const int col = n0 + 64 * c2 + 8 * ch;  // N % 8 == 0: a 16-byte chunk is wholly in or out
      if (32 * ew + row < nvalid && col < N) {
        const uint4 val = *reinterpret_cast<const uint4*>(stage + row * kStageRowBytes + ch * 16);
        *reinterpret_cast<uint4*>(Y + (size_t)(r0 + 32 * ew + row) * N + col) = val;
      }
    }
    __syncwarp();  // the staging tile is rewritten by the next 64 columns
  }
}

// Drain a gated unit's accumulator: columns [0, 128) are the gate's, [128, 256) the
// same columns of the factor.  Two warps (one) share 32 lanes, each with half (all)
// of the 128 columns of h, 32 at a time:
//   h = act(g) u,  and z = [g | u] where it is kept.
template <int kWarps>
__device__ __forceinline__ void store_gated(uint32_t tcol, int ew, int part, int lane, uint8_t* stage, const GemmParams& p,
                                            int r0, int n0, int nvalid) {
  constexpr int kChunks = 16 / kWarps;  // of 32 columns, this warp's share
  const int rows = nvalid - 32 * ew;
  if (rows <= 0) return;  // the whole warp
  const long long at = r0 + 32 * ew;
#pragma unroll 1
  for (int c = 0; c < kChunks; ++c) {
    const int j = 32 * (kChunks * part + c), col = n0 + j, cols = p.N - col;
    if (cols <= 0) return;
    uint32_t v[32], w[16];
    float g[32], u[32];
    tmem_ld32(tcol + (uint32_t)j, v);
#pragma unroll
    for (int i = 0; i < 32; ++i) g[i] = __uint_as_float(v[i]);
    tmem_ld32(tcol + (uint32_t)(BN / 2 + j), v);
#pragma unroll
    for (int i = 0; i < 32; ++i) u[i] = __uint_as_float(v[i]);
    if (p.Z) {
      pack_bf16(g, w);
      store_rows(stage, w, p.Z + at * 2 * p.N + col, 2LL * p.N, rows, cols, lane);
      pack_bf16(u, w);
      store_rows(stage, w, p.Z + at * 2 * p.N + p.N + col, 2LL * p.N, rows, cols, lane);
    }
    if (p.act != MOE_ACT_NONE) activate<32>(g, p.act);
#pragma unroll
    for (int i = 0; i < 32; ++i) g[i] *= u[i];
    pack_bf16(g, w);
    store_rows(stage, w, p.Y + at * p.N + col, p.N, rows, cols, lane);
  }
}

// Unit u -> expert x, the row block i of its segment and the column tile n0.
// blk[x] = row blocks of the experts before x.  An expert's units go in bands of
// kBand row blocks, the block fastest, so that the pairs that run at the same time
// share columns of W and rows of A in L2.  Gated, bands of 8: 16384 rows of 8
// experts, 4096 x 4096, 625 us (671 with 1).  The plain product keeps bands of 1, one
// block's column tiles one after another: bands of 8 made no difference but to the
// fused form on 131072 skewed rows, 4096 x 4096 (2780 us, 2875 with 8).
struct Unit {
  int x, i, n0;
};

template <int kBand>
__device__ __forceinline__ Unit decode_unit(int u, int ntn, const int* blk, int e, int width) {
  Unit t;
  t.x = expert_of(u / ntn, blk, e);
  const int r = u - blk[t.x] * ntn, band = r / (kBand * ntn), first = band * kBand;
  const int rows = min(kBand, blk[t.x + 1] - blk[t.x] - first), q = r - first * ntn, n = q / rows;
  t.i = first + q - n * rows;
  t.n0 = n * width;
  return t;
}

// ---- two-SM form (cta_group::2) ------------------------------------------
// A cluster of two CTAs on two SMs computes one 256 x 256 tile: CTA rank c
// holds rows 128c .. 128c+127 of the 256-row block (its A half) and columns
// 128c .. 128c+127 of the 256-column tile (its B half); one thread of rank
// 0 issues tcgen05.mma.cta_group::2 (M256 N256 K16), which reads both
// CTAs' shared memory at the same offsets and leaves each CTA's 128 rows
// of the fp32 result in its own TMEM.  Per SM and K-block only 32 KB move
// (48 KB in the one-SM form), so the ring holds six K-blocks.
//   both ranks, warp 0 lane 0: TMA of its A and B halves; the completion
//     bytes of both ranks are counted on rank 0's full barrier (the
//     .cta_group::2 form of the copy lets rank 1 signal it);
//   rank 0, warp 1 lane 0: MMA; its commits arrive on the empty / tfull
//     barriers of both ranks (multicast);
//   both ranks, warp 2: one collective TMEM allocation for the pair;
//   both ranks, warps 4..7: epilogue of its own rows, then an arrival on
//     rank 0's tempty barrier (remote for rank 1);
//   fused form, both ranks, warps 8..15: gather the CTA's 128 A rows, each
//     thread's copies arriving through cp.async.mbarrier.arrive.noinc;
//   fused form, rank 1, warp 1 lane 0: forwards each gathered stage to
//     rank 0's full barrier.
// A ring stage holds two 64-wide K blocks of this CTA's A and B halves (16 KB
// each per block), in a 3-stage ring: half the barrier round trips per MMA
// of one block per stage (measured 3-10 % faster for the plain form, 10-15 %
// for the fused one).
constexpr int kSubA = BM * BK * 2;              // 16 KB: 128 rows x 64 K of A, one swizzle atom column
constexpr int kSubB = (BN / 2) * BK * 2;        // 16 KB: 128 rows x 64 K of B
constexpr int kPairKB = 2;
constexpr int kPairStages = 3;
constexpr int kPairRingBytes = kPairStages * kPairKB * (kSubA + kSubB);  // 192 KB
constexpr int kPairSmemBytes = kPairRingBytes + kEpiBytes + 1024;
constexpr int BM2 = 2 * BM;                     // rows of a pair block

__device__ __forceinline__ uint32_t mma_idesc_pair() {
  uint32_t d = 0;
  d |= 1u << 4;                        // accumulator format: f32
  d |= 1u << 7;                        // A format: bf16
  d |= 1u << 10;                       // B format: bf16
  d |= (uint32_t)(BN >> 3) << 17;      // N / 8 (the pair's 256 columns)
  d |= (uint32_t)(BM2 >> 4) << 24;     // M / 16 (the pair's 256 rows)
  return d;
}

// Roles of a CTA: four control warps, the epilogue's, then the gathering ones.
template <bool kGather, bool kGated>
struct Roles {
  static constexpr int kEpiWarps = kGated && !kGather ? kGatedWarps : 4;
  static constexpr int kMain = 128 + 32 * kEpiWarps;
  static constexpr int kAll = kMain + (kGather ? 32 * MOE_GEMM_GATHER_WARPS : 0);
};

// kGated: W is [e, 2N, K], each expert's N gate rows and then its N factor rows; a
// unit is 256 rows x 128 columns of h, the first CTA holding the gate's 128 rows of
// W and the second the factor's, so that both land in the same row of TMEM.
template <bool kGather, bool kGated>
__global__ void __launch_bounds__(Roles<kGather, kGated>::kAll, 1)
    grouped_gemm_pair_kernel(const __grid_constant__ CUtensorMap tmA,
                             const __grid_constant__ CUtensorMap tmB, const GemmParams p) {
  constexpr int kPairABytes = kPairKB * kSubA;  // this CTA's 128 rows of A
  constexpr int kPairBBytes = kPairKB * kSubB;  // this CTA's 128 rows of B
  constexpr int kPairStageBytes = kPairABytes + kPairBBytes;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kPairStages], empty[kPairStages], tfull[2], tempty[2];
  __shared__ __align__(8) uint64_t gathered[kPairStages];  // fused form, rank 1: its gathered rows landed
  __shared__ __align__(8) uint64_t mma_drain;               // rank 0, after a time-out: its MMAs are done
  __shared__ __align__(16) uint8_t s_signal[16];             // fused form: source / target of rank 1's signal
  __shared__ uint32_t tmem_base;
  __shared__ int s_off[kMaxE + 1], s_cnt[kMaxE], s_blk[kMaxE + 1];
  __shared__ int s_err;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();  // 0 or 1 within the pair
  constexpr int kEpiWarps = Roles<kGather, kGated>::kEpiWarps, kMain = Roles<kGather, kGated>::kMain;
  constexpr int kWidth = kGated ? BN / 2 : BN;  // columns of Y (of h) a unit
  constexpr int kGatherWarps = MOE_GEMM_GATHER_WARPS;
  constexpr int kGatherArrivals = kGatherWarps * 32;  // one per gathering thread and stage
  // identical static layout in both CTAs: the dynamic buffer starts at the
  // same offset, so the MMA's descriptors address the same tiles in both
  uint8_t* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);

  if (threadIdx.x == 0) {
    s_err = 0;
    for (int i = 0; i < kPairStages; ++i) {
      // rank 0: its expect_tx arrival (both ranks' TMA bytes, and in the fused
      // form rank 1's 16-byte signal), plus its gathering threads' arrivals
      mbar_init(&full[i], kGather ? 1 + kGatherArrivals : 1);
      mbar_init(&empty[i], 1);  // the MMA commit, multicast to both ranks
      mbar_init(&gathered[i], kGatherArrivals);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 2 * kEpiWarps);  // rank 0: the epilogue warps of both ranks
    }
    mbar_init(&mma_drain, 1);
    fence_barrier_init();
  }
  __syncthreads();
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  grid_dependency_wait();  // all set-up is done: from here on memory of earlier kernels is read
  for (int x = threadIdx.x; x <= p.e; x += blockDim.x) s_off[x] = ld_plain(p.offsets + x);
  for (int x = threadIdx.x; x < p.e; x += blockDim.x) s_cnt[x] = ld_plain(p.counts + x);
  __syncthreads();
  if (warp == 3) prefix_blocks(s_cnt, s_blk, p.e, BM2, lane);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both ranks' barriers are initialised before any remote signal
  tc_fence_after();
  const uint32_t tbase = tmem_base;

  const int ntn = (p.N + kWidth - 1) / kWidth;  // the last column tile may be partial
  const int nunits = s_blk[p.e] * ntn;
  const int kblocks = (p.K + BK * kPairKB - 1) / (BK * kPairKB);  // per stage; columns past K read as zeros
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

  if (warp == 0 && lane == 0) {
    // ---- TMA producer (both ranks) ---------------------------------------
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = pair; u < nunits && ok; u += npairs) {
      const Unit t = decode_unit<kGated ? 8 : 1>(u, ntn, s_blk, p.e, kWidth);
      const int r0 = s_off[t.x] + BM2 * t.i + BM * (int)rank;
      for (int kb = 0; kb < kblocks; ++kb) {
        if (!mbar_wait_limited(&empty[stage], phase ^ 1u, p.timeout_ns)) {
          ok = false;
          break;
        }
        uint8_t* sa = smem + stage * kPairStageBytes;
        const uint32_t fb = mapa_shared(smem_addr(&full[stage]), 0);
        if (rank == 0) mbar_arrive_expect_tx(&full[stage], kGather ? 2 * kPairBBytes + 16 : 2 * kPairStageBytes);
#pragma unroll
        for (int q = 0; q < kPairKB; ++q) {
          const int kx = (kb * kPairKB + q) * BK;
          if (!kGather) tma_load_2d_pair(sa + q * kSubA, &tmA, kx, r0, fb);
          const int nrow = kGated ? (2 * t.x + (int)rank) * p.N + t.n0 : t.x * p.N + t.n0 + (BN / 2) * (int)rank;
          tma_load_2d_pair(sa + kPairABytes + q * kSubB, &tmB, kx, nrow, fb);
        }
        if (++stage == kPairStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // drain: every stage's last fill consumed, so no commit of rank 0 is
    // still on its way to this CTA's barriers when it leaves
    for (int i = 0; i < kPairStages && ok; ++i) {
      if (!mbar_wait_limited(&empty[stage], phase ^ 1u, p.timeout_ns)) ok = false;
      if (++stage == kPairStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (!ok) atomicOr(&s_err, 1);
  } else if (kGather && warp >= kMain / 32) {
    // ---- A gather (fused form, both ranks): this CTA's 128 rows ------------
    // Each lane copies 16 bytes of kGatherRows / 4 rows per K block (8 lanes per 128-byte
    // row, the swizzle as in the one-SM form), then hands its copies of the
    // stage to the stage's barrier (cp.async.mbarrier.arrive.noinc: one
    // arrival once they land) and runs on to the next free stage; waiting
    // for its own copies two stages later instead held the gather to a
    // shallow window and the fused GEMM 10-15 % lower.  Rank 0's threads
    // arrive on its full barrier, rank 1's on its own `gathered` barrier,
    // forwarded below; the waiter on each fences the async proxy.  A unit's
    // row-to-token indices are loaded while the previous unit is gathered.
    const int gw = warp - kMain / 32, chunk = lane & 7;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    // token of each of this lane's kGatherRows / 4 rows in unit u; -1 for rows no route owns
    auto unit_tokens = [&](int u, int* tok) {
      const Unit t = decode_unit<kGated ? 8 : 1>(u, ntn, s_blk, p.e, kWidth);
      const int r0 = s_off[t.x] + BM2 * t.i + BM * (int)rank;
      const int left = s_cnt[t.x] - BM2 * t.i - BM * (int)rank;
#pragma unroll
      for (int j = 0; j < kGatherRows / 4; ++j) {
        const int rr = kGatherRows * gw + 4 * j + (lane >> 3);
        tok[j] = -1;
        if (rr < left) {
          const int v = ld_plain(p.inv_row + r0 + rr);
          tok[j] = (unsigned)v < (unsigned)p.s ? v : 0;
        }
      }
    };
    int tok[kGatherRows / 4], ntok[kGatherRows / 4];
#pragma unroll
    for (int j = 0; j < kGatherRows / 4; ++j) ntok[j] = -1;  // after the last unit: nothing
    if (pair < nunits) unit_tokens(pair, tok);
    for (int u = pair; u < nunits && ok; u += npairs) {
      if (u + npairs < nunits) unit_tokens(u + npairs, ntok);  // in flight while this unit is gathered
      const __nv_bfloat16* src[kGatherRows / 4];
#pragma unroll
      for (int j = 0; j < kGatherRows / 4; ++j) src[j] = p.x + (size_t)(tok[j] < 0 ? 0 : tok[j]) * p.K + chunk * 8;
      for (int kb = 0; kb < kblocks; ++kb) {
        bool waited = true;
        if (lane == 0) waited = mbar_wait_limited(&empty[stage], phase ^ 1u, p.timeout_ns);
        if (!__shfl_sync(0xffffffffu, waited ? 1 : 0, 0)) {
          ok = false;
          break;
        }
        const uint32_t sa = smem_addr(smem + stage * kPairStageBytes);
#pragma unroll
        for (int q = 0; q < kPairKB; ++q) {
          const int kx = (kb * kPairKB + q) * BK;
#pragma unroll
          for (int j = 0; j < kGatherRows / 4; ++j) {
            // rows no route owns are not copied (their results are never stored)
            const int rr = kGatherRows * gw + 4 * j + (lane >> 3);
            if (tok[j] >= 0) {
              // columns past K: zeros, nothing read (the row's end may be the buffer's)
              const bool in_k = kx + chunk * 8 < p.K;
              cp_async16_zfill(sa + q * kSubA + rr * 128 + ((chunk ^ (rr & 7)) << 4), in_k ? src[j] + kx : src[j],
                               in_k ? 16u : 0u);
            }
          }
        }
        cp_async_arrive_noinc(rank == 0 ? &full[stage] : &gathered[stage]);
        if (++stage == kPairStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
#pragma unroll
      for (int j = 0; j < kGatherRows / 4; ++j) tok[j] = ntok[j];
    }
    cp_async_wait_all();  // nothing of this thread's stays in flight
    if (!ok && lane == 0) atomicOr(&s_err, 1);
  } else if (kGather && warp == 1 && lane == 0 && rank == 1) {
    // ---- forwarder (fused form, rank 1) ------------------------------------
    // Once all of this CTA's gathering warps have landed a stage, a 16-byte
    // shared-to-shared bulk copy into rank 0 counts on rank 0's full barrier:
    // an async-proxy signal, ordered after the gathered rows (fenced by
    // their writers, acquired here through the `gathered` barrier).
    const uint32_t sig_dst = mapa_shared(smem_addr(s_signal), 0);
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = pair; u < nunits && ok; u += npairs) {
      for (int kb = 0; kb < kblocks; ++kb) {
        if (!mbar_wait_limited(&gathered[stage], phase, p.timeout_ns)) {
          ok = false;
          break;
        }
        fence_proxy_async_smem();  // the rows landed by cp.async, before the async-proxy signal
        bulk_signal_s2s(sig_dst, s_signal, mapa_shared(smem_addr(&full[stage]), 0));
        if (++stage == kPairStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok) atomicOr(&s_err, 1);
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // ---- MMA issuer (rank 0) ----------------------------------------------
    const uint32_t idesc = mma_idesc_pair();
    int stage = 0, acc = 0;
    uint32_t phase = 0, tphase[2] = {0u, 0u};
    bool ok = true;
    for (int u = pair; u < nunits && ok; u += npairs) {
      if (!mbar_wait_cluster_limited(&tempty[acc], tphase[acc] ^ 1u, p.timeout_ns)) {
        ok = false;
        break;
      }
      tphase[acc] ^= 1u;
      tc_fence_after();
      const uint32_t dt = tbase + (uint32_t)(acc * BN);
      for (int kb = 0; kb < kblocks; ++kb) {
        if (!mbar_wait_cluster_limited(&full[stage], phase, p.timeout_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (kGather) fence_proxy_async_smem();  // this CTA's rows landed by cp.async
        const uint32_t sa = smem_addr(smem + stage * kPairStageBytes);
#pragma unroll
        for (int q = 0; q < kPairKB; ++q) {
          const uint64_t ad = smem_desc(sa + q * kSubA), bd = smem_desc(sa + kPairABytes + q * kSubB);
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            mma_bf16_pair(dt, ad + (uint64_t)(2 * kk), bd + (uint64_t)(2 * kk), idesc, (kb | q | kk) != 0);
        }
        mma_commit_pair(&empty[stage]);
        if (++stage == kPairStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      mma_commit_pair(&tfull[acc]);
      acc ^= 1;
    }
    if (!ok) {
      // a wait ran out: before this CTA (and, at the cluster barrier below,
      // its partner) leaves, let every MMA issued so far finish reading both
      // CTAs' shared memory -- one more commit, to this CTA only, arrives
      // after all of them and after the commits before it (bounded wait)
      mma_commit_pair(&mma_drain, 0x1);
      mbar_wait_limited(&mma_drain, 0, p.timeout_ns);
      atomicOr(&s_err, 1);
    }
  } else if (warp >= 4 && warp < 4 + kEpiWarps) {
    // ---- epilogue (both ranks): own 128 rows ------------------------------
    const int ew = warp & 3;
    const uint32_t te0 = mapa_shared(smem_addr(&tempty[0]), 0), te1 = mapa_shared(smem_addr(&tempty[1]), 0);
    int acc = 0;
    uint32_t tphase[2] = {0u, 0u};
    bool ok = true;
    for (int u = pair; u < nunits && ok; u += npairs) {
      const Unit t = decode_unit<kGated ? 8 : 1>(u, ntn, s_blk, p.e, kWidth);
      const int r0 = s_off[t.x] + BM2 * t.i + BM * (int)rank;
      const int left = s_cnt[t.x] - BM2 * t.i - BM * (int)rank;
      const int nvalid = left < 0 ? 0 : (left < BM ? left : BM);
      // every lane waits (and acquires) itself; the warp leaves together
      if (!__all_sync(0xffffffffu, mbar_wait_limited(&tfull[acc], tphase[acc], p.timeout_ns))) {
        ok = false;
        break;
      }
      tphase[acc] ^= 1u;
      tc_fence_after();
      const uint32_t tcol = tbase + ((uint32_t)(32 * ew) << 16) + (uint32_t)(acc * BN);
      uint8_t* stage_buf = smem + kPairStages * kPairStageBytes;
      if constexpr (kGated)
        store_gated<kEpiWarps>(tcol, ew, (warp - 4) >> 2, lane, stage_buf + (warp - 4) * kRowStage, p, r0, t.n0, nvalid);
      else
        store_accumulator(tcol, ew, lane, stage_buf + ew * kEpiWarpBytes, p.Y, p.N, r0, t.n0, nvalid);
      tc_fence_before();
      __syncwarp();  // every lane's TMEM reads are done
      if (lane == 0) {
        if (rank == 0) mbar_arrive(&tempty[acc]);
        else mbar_arrive_accumulator(acc ? te1 : te0);
      }
      acc ^= 1;
    }
    if (!ok) atomicOr(&s_err, 1);
  }

  grid_dependents_launch();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both ranks done with TMEM and with each other's barriers
  tc_fence_after();
  if (warp == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tbase),
                 "r"(kTmemCols)
                 : "memory");
  if (threadIdx.x == 0 && s_err) raise_status(p.status, MOE_DEV_TIMEOUT);
}

// 2-D bf16 row-major [outer, inner] tensor, box (BK inner) x box_rows, 128-B swizzle.
bool make_map(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer, uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {inner * 2};
  cuuint32_t box[2] = {BK, box_rows};
  cuuint32_t estride[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
            estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kGather, bool kGated = false>
cudaError_t launch_pair(const CUtensorMap& ma, const CUtensorMap& mb, const GemmParams& p,
                        const DeviceInfo& di, cudaStream_t st) {
  constexpr int kWidth = kGated ? BN / 2 : BN;
  static OncePerDevice once;
  cudaError_t err = once.run([] {
    return cudaFuncSetAttribute(grouped_gemm_pair_kernel<kGather, kGated>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kPairSmemBytes);
  });
  if (err != cudaSuccess) return err;
  // pair units: at most ceil(rows / 256) + e blocks of 256 rows, times the column tiles
  const long long units = (((long long)p.rows + BM2 - 1) / BM2 + p.e) * ((p.N + kWidth - 1) / kWidth);
  long long pairs = di.sms / 2;
  if (units < pairs) pairs = units;
  if (pairs < 1) pairs = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  cfg.blockDim = dim3(Roles<kGather, kGated>::kAll);
  cfg.dynamicSmemBytes = kPairSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, grouped_gemm_pair_kernel<kGather, kGated>, ma, mb, p);
}

GemmParams params(const int32_t* offsets, const int32_t* counts, int e, int rows, int K, int N,
                  void* Y, int32_t* status) {
  GemmParams p;
  p.x = nullptr;
  p.offsets = offsets;
  p.counts = counts;
  p.inv_row = nullptr;
  p.e = e;
  p.rows = rows;
  p.K = K;
  p.N = N;
  p.s = 0;
  p.Y = static_cast<__nv_bfloat16*>(Y);
  p.status = status;
  // the longest wait is the epilogue's, for a whole contraction: under 1 us for 128 of K when all is well
  p.timeout_ns = kWaitNs + 20000LL * (K / 128);
  p.Z = nullptr;
  p.act = MOE_ACT_NONE;
  return p;
}

}  // namespace

cudaError_t launch_grouped_gemm(const int32_t* offsets, const int32_t* counts, int e, int rows, int K,
                                int N, const void* X, const void* W, void* Y, int32_t* status,
                                const DeviceInfo& di, cudaStream_t st) {
  CUtensorMap ma, mb;
  if (!make_map(&ma, X, (uint64_t)K, (uint64_t)rows, BM) ||
      !make_map(&mb, W, (uint64_t)K, (uint64_t)e * (uint64_t)N, BN / 2))
    return cudaErrorInvalidValue;
  return launch_pair<false>(ma, mb, params(offsets, counts, e, rows, K, N, Y, status), di, st);
}

cudaError_t launch_dispatch_gemm(const int32_t* offsets, const int32_t* counts, const int32_t* inv_row,
                                 int e, int rows, int s, int K, int N, const void* x, const void* W,
                                 void* Y, int32_t* status, const DeviceInfo& di, cudaStream_t st) {
  CUtensorMap mb;
  GemmParams p = params(offsets, counts, e, rows, K, N, Y, status);
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.inv_row = inv_row;
  p.s = s;
  if (!make_map(&mb, W, (uint64_t)K, (uint64_t)e * (uint64_t)N, BN / 2)) return cudaErrorInvalidValue;
  return launch_pair<true>(mb, mb, p, di, st);  // A is gathered by threads: no A map
}

// Whether an expert product streams the weights through warp-level MMA, 16 rows at a
// time (few_gated_kernel), or goes by tiles of 256 rows.  The host knows the rows of
// all experts together, not their spread; where routing is skewed, an expert of many
// rows is streamed over and over.  Measured, tiles / streamed, even routing and
// skewed (Zipf 1.2): 64 experts of 2048 x 1408, a row an expert 84.0 / 73.9 and 48.0 /
// 43.9 us, two 116.8 / 103.7 and 57.5 / 58.5, four 127.9 / 122.7 and 69.4 / 82.1; 8
// experts of 4096 x 4096, two 91.7 / 75.9 and 76.6 / 58.5, eight 102.0 / 87.7 and 91.4
// / 93.2; 128 experts of 4096 x 512, two 164.2 / 139.0 and 62.2 / 67.9, four 178.1 /
// 165.1 and 78.4 / 94.3.  The worst case is every row on one expert: at most rows / 16 =
// e / 8 of its blocks are streamed, an eighth of what even routing streams, mostly from
// L2.  Two rows an expert, all on one: 64 experts of 2048 x 1408 15.4 / 21.3 us, 256 of
// them 16.7 / 76.8 (even routing 473.6 / 447.5); 256 of 4096 x 512 24.8 / 53.6 (353.9 /
// 301.9).
static bool few_rows(int rows, int e) { return rows <= kFewRows || rows <= 2LL * e; }

cudaError_t launch_grouped_gated(const int32_t* offsets, const int32_t* counts, int e, int rows, int K, int N, int act,
                                 const void* X, const void* W, void* H, void* Z, int32_t* status, const DeviceInfo& di,
                                 cudaStream_t st) {
  if (few_rows(rows, e))
    return launch_few_grouped(offsets, counts, nullptr, e, rows, 0, K, N, act, X, W, H, Z, status, di, st);
  CUtensorMap ma, mb;
  if (!make_map(&ma, X, (uint64_t)K, (uint64_t)rows, BM) ||
      !make_map(&mb, W, (uint64_t)K, 2 * (uint64_t)e * (uint64_t)N, BN / 2))
    return cudaErrorInvalidValue;
  GemmParams p = params(offsets, counts, e, rows, K, N, H, status);
  p.Z = static_cast<__nv_bfloat16*>(Z);
  p.act = act;
  return launch_pair<false, true>(ma, mb, p, di, st);
}

cudaError_t launch_dispatch_gated(const int32_t* offsets, const int32_t* counts, const int32_t* inv_row, int e, int rows,
                                  int s, int K, int N, int act, const void* x, const void* W, void* H, void* Z,
                                  int32_t* status, const DeviceInfo& di, cudaStream_t st) {
  if (few_rows(rows, e))
    return launch_few_grouped(offsets, counts, inv_row, e, rows, s, K, N, act, x, W, H, Z, status, di, st);
  CUtensorMap mb;
  GemmParams p = params(offsets, counts, e, rows, K, N, H, status);
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.inv_row = inv_row;
  p.s = s;
  p.Z = static_cast<__nv_bfloat16*>(Z);
  p.act = act;
  if (!make_map(&mb, W, (uint64_t)K, 2 * (uint64_t)e * (uint64_t)N, BN / 2)) return cudaErrorInvalidValue;
  return launch_pair<true, true>(mb, mb, p, di, st);
}

}  // namespace moe
