// grouped_bwd.cu -- backward of the product over the experts' row segments
//   Y[r] = X[r] W[x]^T,  r in [offsets[x], offsets[x] + counts[x])
// on the tensor cores:
//   dX[r] = dY[r] W[x]                        contracts over W's N rows
//   dW[x] = sum over x's rows of dY[r]^T X[r]  contracts over the rows
//
// One kernel form for both, on pairs of SMs as the forward product: tiles of 256 x 256, each
// CTA holding 128 rows of A and 128 columns of B, fp32 accumulators in TMEM, two
// of them, a ring of three stages of two 64-wide K blocks.  No operand is
// transposed in memory: where rows run along the other axis than the contracted
// one (W in dX, both operands in dW) the matrix descriptors say so.
//
// dX: units are row blocks of 256 of one expert times column tiles.  W is a
// three-dimensional tensor map [e][N][K], so that a K block past an expert's N
// rows reads zeros and not the next expert's weights.
//
// dW: units are tiles of one expert's dW; the contraction is as long as its
// segment.  A segment may end anywhere, and what follows it in memory is another
// expert's rows or was never written, so the last K block is cut: the MMAs stop
// at the last 16 rows that hold any of the segment, and of those 16 the rows past
// its end are overwritten with zeros in shared memory, in both operands (a NaN
// there would survive a zero in one), between the copy and the MMA.  Such a
// block's copies count on a barrier of each CTA (`tail`); a warp of each waits for
// it, writes the zeros, and arrives in the TMA's place on the barrier that the MMA
// waits for (the second CTA's word through the async proxy).  An expert without rows
// gets zeros.
//
// The accumulator drops the bits below its last place at every step of 16 terms, up
// to 2^-23 of the sum.  So a contraction of more than 2^17 terms hands it over every
// 2^17, and the epilogue adds these parts up in fp32: whatever the length, a sum of one
// sign is at most 2^-10 short, a quarter of what rounding to bf16 may take (2^22
// terms, in the mean: 2.6 % short in one accumulator, 0.07 % this way).  The running
// sums live in local memory: a part takes some 600 us, so their traffic does not matter,
// and short contractions keep their registers.  One expert of 2048 x 2048, dW: 131072
// rows 604 us, 2^20 rows 4.8 to 4.9 ms, 1.8 PFLOP/s both.
//
// Bound by the tensor cores where segments are long (1024 rows, 4096 x 1024: dX 1.69,
// dW 1.59 PFLOP/s), by memory where they are short (174 rows of 128 experts, 2816 x 704:
// dX 119 us, 5.6 TB/s; dW 125 us, 5.3 TB/s, against 84 for zeros alone), by the tiles'
// edges where they are uneven (64 experts of 6 to 768 rows, 16316 together, 2048 x 1408:
// dX 106 us, of which 86 for 25856 rows x 1536 columns of tiles, memory 71; dW 112 us).
//
//   warp 0 lane 0   TMA producer (both CTAs)
//   warp 1 lane 0   MMA issuer (the first CTA)
//   warp 2          TMEM allocation
//   warp 3          zeros behind a segment's end (dW)
//   warps 4..11     epilogue, two warps for each quarter of the TMEM lanes
// Every mbarrier wait is bounded on the global timer, each from its own start; a
// time-out records MOE_DEV_TIMEOUT and the roles wind down to the TMEM release.
#include "common.cuh"
#include "grouped.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace moe {

namespace {

typedef __nv_bfloat16 bf16;

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kKB = 2;                    // 64-wide K blocks a stage
constexpr int kStageK = 64 * kKB;
constexpr int kSub = 128 * 64 * 2;        // 16 KB: 128 rows (or columns) x 64
constexpr int kStage = kKB * 2 * kSub;    // A and B
constexpr int kStages = 3;
// a warp's staging tile: 32 rows x 64 columns (dW), 32 x 32 (dX)
template <bool kWeights>
constexpr int kPiece = kWeights ? 32 * 128 : kRowStage;
template <bool kWeights>
constexpr int kSmem = kStages * kStage + kEpiWarps * kPiece<kWeights> + 1024;
constexpr int kTile = 256;
constexpr int kTmemCols = 512;
constexpr int kMaxE = 256;
constexpr int kPartBlocks = (1 << 17) / kStageK;  // K blocks that one accumulator takes

struct Args {
  const int32_t* offsets;
  const int32_t* counts;
  int e;
  int M;     // dW: rows of an expert's dW (N of the product); dX: the contraction's length
  int cols;  // columns of the result (K of the product)
  bf16* out;
  int32_t* status;
  long long timeout_ns;  // of a single wait
};

struct Unit {
  int x, m0, n0;  // expert; first row of the pair's tile (within its segment, or within its dW); first column
  int blocks;     // K blocks of kStageK
  int count;      // rows of the expert
};

// The r-th unit of a pair.  dW's units are in order of falling length (their
// experts' rows), and every other round of them is dealt out in reverse, so that
// skewed routing leaves no pair with much more to do than another.
template <bool kWeights>
__device__ __forceinline__ int pick(int r, int pair, int pairs) {
  return r * pairs + (kWeights && (r & 1) ? pairs - 1 - pair : pair);
}

// order: dW's experts by falling count; dX: blk, row blocks of the experts before x.
template <bool kWeights>
__device__ __forceinline__ Unit unit_of(int u, const Args& p, const int* s_blk, const uint8_t* order, const int* s_cnt) {
  const int tn = (p.cols + kTile - 1) / kTile;
  Unit t;
  if constexpr (kWeights) {
    // an expert's tiles one after another, in bands of 8 rows of tiles, so that
    // those in flight share their operands in L2
    const int tm = (p.M + kTile - 1) / kTile;
    const int place = u / (tm * tn);
    t.x = order[place];
    const int r = u - place * tm * tn, band = r / (8 * tn), rows = min(8, tm - band * 8), q = r - band * 8 * tn, n = q / rows;
    t.m0 = (band * 8 + q - n * rows) * kTile;
    t.n0 = n * kTile;
    t.count = s_cnt[t.x];
    t.blocks = (t.count + kStageK - 1) / kStageK;
  } else {
    const int b = u / tn;
    t.x = expert_of(b, s_blk, p.e);
    t.m0 = kTile * (b - s_blk[t.x]);
    t.n0 = (u - b * tn) * kTile;
    t.count = s_cnt[t.x];
    t.blocks = (p.M + kStageK - 1) / kStageK;
  }
  return t;
}

__device__ __forceinline__ void tma_load_3d_pair(void* sdst, const CUtensorMap* map, int x, int y, int z, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(sdst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(mbar)
      : "memory");
}

struct Ring {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

// Rows of the last K block that hold some of the segment but end inside 16 of them.
__device__ __forceinline__ bool is_cut(const Unit& t, int kb) { return kb == t.blocks - 1 && (t.count & 15) != 0; }

template <bool kWeights>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_bwd_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ Args p) {
  extern __shared__ uint8_t smem_raw[];
  // full: the copies of both CTAs (two arrivals of the first CTA's producer; of a cut
  // block its zeroing warp's two, and 16 bytes from the second CTA's); tail: this
  // CTA's copies of a cut block
  __shared__ __align__(8) uint64_t full[kStages], empty[kStages], tail[kStages], tfull[2], tempty[2], drain;
  __shared__ __align__(16) uint8_t s_signal[16];  // source and target of the second CTA's word
  __shared__ uint32_t tmem_base;
  __shared__ int s_cnt[kMaxE], s_off[kWeights ? 1 : kMaxE], s_blk[kWeights ? 1 : kMaxE + 1];
  __shared__ uint8_t s_order[kWeights ? kMaxE : 1];
  __shared__ int s_err;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  uint8_t* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);

  if (threadIdx.x == 0) {
    s_err = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 2);
      mbar_init(&empty[i], 1);
      mbar_init(&tail[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 2 * kEpiWarps);
    }
    mbar_init(&drain, 1);
    fence_barrier_init();
  }
  __syncthreads();
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  grid_dependency_wait();  // from here on memory of earlier kernels is read
  for (int x = threadIdx.x; x < p.e; x += blockDim.x) {
    if (!kWeights) s_off[x] = ld_plain(p.offsets + x);
    s_cnt[x] = ld_plain(p.counts + x);
  }
  __syncthreads();
  if constexpr (kWeights) {
    for (int x = threadIdx.x; x < p.e; x += blockDim.x) {
      const int n = s_cnt[x];
      int place = 0;
      for (int y = 0; y < p.e; ++y) place += s_cnt[y] > n || (s_cnt[y] == n && y < x);
      s_order[place] = (uint8_t)x;
    }
  } else if (warp == 3) {
    prefix_blocks(s_cnt, s_blk, p.e, kTile, lane);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers exist before any remote signal
  tc_fence_after();
  const uint32_t tbase = tmem_base;

  const int tn = (p.cols + kTile - 1) / kTile;
  const int units = kWeights ? p.e * ((p.M + kTile - 1) / kTile) * tn : s_blk[p.e] * tn;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (warp == 0 && lane == 0) {
    // ---- TMA producer ------------------------------------------------------
    Ring r;
    bool ok = true;
    for (int i = 0, u = pair; u < units && ok; u = pick<kWeights>(++i, pair, pairs)) {
      const Unit t = unit_of<kWeights>(u, p, s_blk, s_order, s_cnt);
      const int m0 = t.m0 + 128 * (int)rank, n0 = t.n0 + 128 * (int)rank;
      const int first = kWeights ? ld_plain(p.offsets + t.x) : s_off[t.x];
      for (int kb = 0; kb < t.blocks; ++kb) {
        if (!mbar_wait_limited(&empty[r.stage], r.phase ^ 1u, p.timeout_ns)) {
          ok = false;
          break;
        }
        uint32_t fb;
        // the second half of a last block of at most 64 rows is not needed
        const bool both = !kWeights || t.count - kb * kStageK > 64;
        if (kWeights && is_cut(t, kb)) {
          fb = smem_addr(&tail[r.stage]);
          mbar_arrive_expect_tx(&tail[r.stage], both ? kStage : kStage / 2);
        } else {
          fb = mapa_shared(smem_addr(&full[r.stage]), 0);
          if (rank == 0) {
            mbar_arrive_expect_tx(&full[r.stage], both ? 2 * kStage : kStage);
            mbar_arrive(&full[r.stage]);
          }
        }
        uint8_t* sa = smem + r.stage * kStage;
#pragma unroll
        for (int q = 0; q < kKB; ++q) {
          const int k = kb * kStageK + 64 * q;
          if (q == 1 && !both) break;
          uint8_t* sb = sa + (kKB + q) * kSub;
          if constexpr (kWeights) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              tma_load_2d_pair(sa + q * kSub + g * 8192, &tmA, m0 + 64 * g, first + k, fb);
              tma_load_2d_pair(sb + g * 8192, &tmB, n0 + 64 * g, first + k, fb);
            }
          } else {
            tma_load_2d_pair(sa + q * kSub, &tmA, k, first + m0, fb);
#pragma unroll
            for (int g = 0; g < 2; ++g) tma_load_3d_pair(sb + g * 8192, &tmB, n0 + 64 * g, k, t.x, fb);
          }
        }
        r.next();
      }
    }
    // every stage's last fill consumed: nothing still arrives at this CTA's
    // barriers or shared memory when it leaves
    for (int i = 0; i < kStages && ok; ++i) {
      if (!mbar_wait_limited(&empty[r.stage], r.phase ^ 1u, p.timeout_ns)) ok = false;
      r.next();
    }
    if (!ok) atomicOr(&s_err, 1);
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // ---- MMA issuer ----------------------------------------------------------
    const uint32_t idesc = instr_desc<2, kTile, kWeights, true>();
    Ring r;
    int acc = 0;
    uint32_t tphase[2] = {0u, 0u};
    bool ok = true;
    for (int i = 0, u = pair; u < units && ok; u = pick<kWeights>(++i, pair, pairs)) {
      const Unit t = unit_of<kWeights>(u, p, s_blk, s_order, s_cnt);
      for (int kb0 = 0; kb0 < t.blocks && ok; kb0 += kPartBlocks) {
        if (!mbar_wait_cluster_limited(&tempty[acc], tphase[acc] ^ 1u, p.timeout_ns)) {
          ok = false;
          break;
        }
        tphase[acc] ^= 1u;
        tc_fence_after();
        const uint32_t dt = tbase + (uint32_t)(acc * kTile);
        const int kb1 = min(t.blocks, kb0 + kPartBlocks);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait_cluster_limited(&full[r.stage], r.phase, p.timeout_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_addr(smem + r.stage * kStage);
          const int left = kWeights ? t.count - kb * kStageK : kStageK;
#pragma unroll
          for (int q = 0; q < kKB; ++q) {
            const uint64_t ad = tile_desc<kWeights>(sa + q * kSub), bd = tile_desc<true>(sa + (kKB + q) * kSub);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              if (64 * q + 16 * kk < left)
                mma<2>(dt, ad + kk * kstep<kWeights>(), bd + kk * kstep<true>(), idesc, (kb > kb0) | (q | kk) != 0);
          }
          mma_commit_pair(&empty[r.stage]);
          r.next();
        }
        if (!ok) break;
        mma_commit_pair(&tfull[acc]);
        acc ^= 1;
      }
    }
    if (!ok) {
      // a wait ran out: let the MMAs issued so far finish reading shared memory
      // before the CTAs leave (one more commit, to this CTA only)
      mma_commit_pair(&drain, 0x1);
      mbar_wait_limited(&drain, 0, p.timeout_ns);
      atomicOr(&s_err, 1);
    }
  } else if (kWeights && warp == 3) {
    // ---- zeros behind a segment's end ------------------------------------------
    int pos = 0;  // ring position of the unit's first block
    uint32_t phases = 0;  // of each stage's tail barrier
    bool ok = true;
    for (int i = 0, u = pair; u < units && ok; u = pick<kWeights>(++i, pair, pairs)) {
      const Unit t = unit_of<kWeights>(u, p, s_blk, s_order, s_cnt);
      if (t.blocks == 0) continue;
      const int stage = (pos + t.blocks - 1) % kStages;
      pos = (pos + t.blocks) % kStages;
      if (!is_cut(t, t.blocks - 1)) continue;
      if (!__all_sync(0xffffffffu, mbar_wait_limited(&tail[stage], (phases >> stage) & 1u, p.timeout_ns))) {
        ok = false;
        break;
      }
      phases ^= 1u << stage;
      const int left = t.count - (t.blocks - 1) * kStageK, end = (left + 15) & ~15;
      // a row is 128 consecutive bytes in each of A's and B's two 64-wide parts
      const int part = lane >> 3, piece = lane & 7;
      for (int row = left; row < end; ++row) {
        uint8_t* at = smem + stage * kStage + ((part >> 1) * kKB + (row >> 6)) * kSub + (part & 1) * 8192 + (row & 63) * 128;
        *reinterpret_cast<uint4*>(at + piece * 16) = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        // the second CTA's word travels through the async proxy, behind its zeros (an
        // arrival with release at cluster scope instead: 128 experts of 2816 x 704 and
        // 174 rows 149 us)
        if (rank == 0) {
          mbar_arrive_expect_tx(&full[stage], 16);
          mbar_arrive(&full[stage]);
        } else {
          bulk_signal_s2s(mapa_shared(smem_addr(s_signal), 0), s_signal, mapa_shared(smem_addr(&full[stage]), 0));
        }
      }
    }
    if (!ok && lane == 0) atomicOr(&s_err, 1);
  } else if (warp >= 4) {
    // ---- epilogue --------------------------------------------------------------
    const int ew = warp & 3, half = (warp - 4) >> 2;
    uint8_t* stage_buf = smem + kStages * kStage + (warp - 4) * kPiece<kWeights>;
    const uint32_t te[2] = {mapa_shared(smem_addr(&tempty[0]), 0), mapa_shared(smem_addr(&tempty[1]), 0)};
    int acc = 0;
    uint32_t tphase[2] = {0u, 0u};
    bool ok = true;
    auto release = [&]() {  // this warp's reads of the accumulator are done
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) mbar_arrive(&tempty[acc]);
        else mbar_arrive_accumulator(te[acc]);
      }
    };
    for (int i = 0, u = pair; u < units && ok; u = pick<kWeights>(++i, pair, pairs)) {
      const Unit t = unit_of<kWeights>(u, p, s_blk, s_order, s_cnt);
      const int r0 = t.m0 + 128 * (int)rank + 32 * ew;
      const int rows = (kWeights ? p.M : t.count) - r0;
      const bool zeros = t.blocks == 0;
      auto filled = [&]() {  // the accumulator is ready; its address for this warp
        if (!__all_sync(0xffffffffu, mbar_wait_limited(&tfull[acc], tphase[acc], p.timeout_ns))) {
          ok = false;
          return;
        }
        tphase[acc] ^= 1u;
        tc_fence_after();
      };
      auto lanes_of = [&]() { return tbase + ((uint32_t)(32 * ew) << 16) + (uint32_t)(acc * kTile + 128 * half); };
      const bool parts = t.blocks > kPartBlocks;
      float sum[4][32];  // of the parts but the last
      if (parts) {
#pragma unroll 1
        for (int kb = 0; kb + kPartBlocks < t.blocks && ok; kb += kPartBlocks) {
          filled();
          if (!ok) break;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            tmem_ld32(lanes_of() + (uint32_t)(32 * c), v);
#pragma unroll
            for (int j = 0; j < 32; ++j) sum[c][j] = kb ? sum[c][j] + __uint_as_float(v[j]) : __uint_as_float(v[j]);
          }
          release();
          acc ^= 1;
        }
        if (!ok) break;
      }
      if (!zeros) filled();
      if (!ok) break;
      const uint32_t lanes = lanes_of();
      auto words = [&](int c, uint32_t (&w)[16]) {  // 32 columns of this lane's row
        if (zeros) {
#pragma unroll
          for (int j = 0; j < 16; ++j) w[j] = 0u;
          return;
        }
        uint32_t v[32];
        float f[32];
        tmem_ld32(lanes + (uint32_t)(32 * c), v);
#pragma unroll
        for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(v[j]);
        if (parts) {
#pragma unroll
          for (int j = 0; j < 32; ++j) f[j] += sum[c][j];
        }
        pack_bf16(f, w);
      };
      if constexpr (kWeights) {
        // 64 columns at a time through the staging tile, out by TMA, clipped at the
        // expert's edge (16-byte stores by lanes: 128 experts of 2816 x 704 and 174
        // rows, where little else is done, 217 us); the accumulator goes back as soon
        // as it is read
        uint32_t w[4][16];
#pragma unroll
        for (int c = 0; c < 4; ++c) words(c, w[c]);
        if (!zeros) release();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int col = t.n0 + 128 * half + 64 * c;
          if (rows <= 0 || col >= p.cols) break;  // the whole warp
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const uint32_t* v = w[2 * c + (q >> 2)] + 4 * (q & 3);
            *reinterpret_cast<uint4*>(stage_buf + lane * 128 + ((q ^ (lane & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&tmOut, stage_buf, col, r0, t.x);
            bulk_commit();
          }
        }
      } else {
        const long long first = (long long)s_off[t.x] + r0;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          const int col = t.n0 + 128 * half + 32 * c;
          if (rows <= 0 || col >= p.cols) break;  // the whole warp
          uint32_t w[16];
          words(c, w);
          store_rows(stage_buf, w, p.out + first * p.cols + col, p.cols, rows, p.cols - col, lane);
        }
        if (!zeros) release();
      }
      if (!zeros) acc ^= 1;
    }
    if (kWeights && lane == 0) bulk_wait_all();  // the stores have read the staging tile and are written
    if (!ok && lane == 0) atomicOr(&s_err, 1);
  }

  grid_dependents_launch();
  tc_fence_before();
  __syncthreads();
  if (s_err) {  // let copies in flight land before shared memory goes
    const uint64_t until = globaltimer_ns() + 200000;
    while (globaltimer_ns() < until) {
    }
  }
  cluster_sync_all();
  tc_fence_after();
  if (warp == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(kTmemCols) : "memory");
  if (threadIdx.x == 0 && s_err) raise_status(p.status, MOE_DEV_TIMEOUT);
}

// bf16 [outer][inner], contiguous; boxes of 64 x rows, 128-byte swizzle.
bool make_map(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer, uint32_t rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {inner * 2};
  cuuint32_t box[2] = {64, rows};
  cuuint32_t estride[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estride,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// bf16 [e][N][K]; boxes of 64 columns x rows of one expert.
bool make_weight_map(CUtensorMap* map, const void* base, uint64_t K, uint64_t N, uint64_t e, uint32_t rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {K, N, e};
  cuuint64_t strides[2] = {K * 2, K * N * 2};
  cuuint32_t box[3] = {64, rows, 1};
  cuuint32_t estride[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estride,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kWeights>
cudaError_t run(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& out, const Args& p, long long units, const DeviceInfo& di,
                cudaStream_t st) {
  static OncePerDevice once;
  cudaError_t err = once.run([] {
    return cudaFuncSetAttribute(grouped_bwd_kernel<kWeights>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<kWeights>);
  });
  if (err != cudaSuccess) return err;
  long long pairs = di.sms / 2;
  if (units < pairs) pairs = units;
  if (pairs < 1) pairs = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem<kWeights>;
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
  return cudaLaunchKernelEx(&cfg, grouped_bwd_kernel<kWeights>, ma, mb, out, p);
}

}  // namespace

cudaError_t launch_grouped_bwd(const int32_t* offsets, const int32_t* counts, int e, int rows, int K, int N, const void* dY,
                               const void* X, const void* W, void* dX, void* dW, int32_t* status, const DeviceInfo& di,
                               cudaStream_t st) {
  const long long tn = (K + kTile - 1) / kTile;
  CUtensorMap ma, mb;
  if (dX) {
    if (!make_map(&ma, dY, N, rows, 128) || !make_weight_map(&mb, W, K, N, e, 64)) return cudaErrorInvalidValue;
    // the longest wait is the epilogue's, for a whole contraction: under 1 us for 128 of it when all is well
    const Args p = {offsets, counts, e, N, K, static_cast<bf16*>(dX), status, kWaitNs + 20000LL * (N / kStageK)};
    cudaError_t err = run<false>(ma, mb, ma, p, (((long long)rows + kTile - 1) / kTile + e) * tn, di, st);
    if (err != cudaSuccess) return err;
  }
  if (dW) {
    CUtensorMap out;
    if (!make_map(&ma, dY, N, rows, 64) || !make_map(&mb, X, K, rows, 64) || !make_weight_map(&out, dW, K, N, e, 32))
      return cudaErrorInvalidValue;
    const Args p = {offsets, counts, e, N, K, static_cast<bf16*>(dW), status, kWaitNs + 20000LL * (rows / kStageK)};
    cudaError_t err = run<true>(ma, mb, out, p, e * ((long long)(N + kTile - 1) / kTile) * tn, di, st);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

}  // namespace moe
