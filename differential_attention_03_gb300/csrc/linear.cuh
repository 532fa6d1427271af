// Products with their epilogue on tcgen05 tensor cores (sm_103a):
//
//   z = A B^T (+ bias);  out = residual + act(z)          (kEpiBf16, kEpiF32)
//   g = x Wg^T, u = x Wu^T;  out = act(g) u               (kEpiGated, w_gu = [Wg; Wu])
//
// and, without bias, activation and residual, the two products of their
// backward pass.  An operand is K-major (the contraction contiguous: x and the
// weights of a forward) or MN-major (its other dimension contiguous: the
// weights in da = dz w, both operands in dw = dz^T a), so no transpose is
// ever stored.  bf16 operands, fp32 accumulation.
//
// Bound: the tensor cores (2 M N K flops; a 256-wide tile reads 1/128 byte of
// L2 a flop), or for short contractions the epilogue's stores.  8002 x 8192 x
// 2048: 139 to 142 us, 1.9 PFLOP/s; 510 to 520 cycles a K block, 512 of them MMAs.
// 8192 x 8192 x 64: 24 us, 5.6 TB/s of stores.
//
// One cluster of CG CTAs (an SM pair with CG = 2) per 128 CG x 256 tile,
// persistent over the tiles in groups of `group_m` row blocks, so that the
// CTAs at work share operands in L2.  From tile p.full on tiles are halves, of
// 128 CG x 128: a last round that would leave half of the clusters without
// work, or all of a small product (the host's choice, as is CG).  With CG = 2
// an MMA is M256 N256 K16 over both SMs' tensor cores: each CTA holds its 128
// rows of A and half of B, so a CTA's shared memory feeds half as many B bytes
// (8002 x 4096 x 2 x 10928, gated: 945 us on single SMs, 885 on pairs, at the time).
//   warps 0-7   (kEpiF32: 16 warps, 64 columns each) epilogue: warp w reads lanes 32 (w % 4) .. of the accumulator,
//               columns 128 (w / 4) .. (gated: 64 gate columns and their 64 up
//               columns).  32 rows of 128 bytes at a time leave through a
//               4 KB staging buffer a warp (128-byte swizzle) by TMA.  (16
//               warps in bf16 too: 4096 x 4096 x 512 with gelu and stored z 26
//               for 29 us, but 8192 x 1024 x 1024 18.4 for 15.3.)
//   then        TMA producer: per K block of 64 the A and B boxes into a ring.
//   last warp   TMEM allocator; MMA issuer (of the cluster's first CTA).
// TMEM: two 256-column accumulators: the epilogue of one tile overlaps the
// next one's main loop.  A programmatic dependent launch: barriers and TMEM are
// set up while the kernel before ends.
//
// kEpiF32: the tensor cores truncate as they add into fp32, which costs about
// 1e-9 relative an added value (measured: 1e-6 for a contraction of 1000,
// 9e-6 for 8192).  A result in bf16 does not see that; one in fp32 would, so
// its accumulators sum 512 values each and the epilogue warps add them up in
// registers, rounding to nearest (5e-7 in norm up to contractions of 65536; from
// millions of values on, the segments' own sums in fp32 count).  A bf16 result
// keeps one accumulator: 1e-3 at a million values, a quarter of its half step.
//
// Rows past M and contraction past K are zero-filled by TMA on load; rows past
// M and columns past N are not stored.
#pragma once

#include <cuda_bf16.h>

#include "act.cuh"
#include "linear_params.h"
#include "ptx.cuh"

#undef DA_BOUNDS_FILE
#define DA_BOUNDS_FILE 16

namespace da {

// ----------------------------------------------------------------- SM pairs
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address, in the cluster's shared window, of what `p` is in CTA `rank`.
__device__ __forceinline__ uint32_t map_to_rank(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// A load into this CTA's shared memory whose bytes count on the barrier at
// cluster address `bar` (its own or the pair's other CTA's).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  if (!DA_TMA_OK(smem_u32(dst), c0, c1, 0, 0)) return;
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}

template <int CG>
__device__ __forceinline__ void tmem_alloc_cg(uint32_t* dst, uint32_t ncols) {
  if (CG == 1) {
    tmem_alloc(dst, ncols);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_dealloc_cg(uint32_t taddr, uint32_t ncols) {
  if (CG == 1)
    tmem_dealloc(taddr, ncols);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Of a pair, from one lane: `commit` arrives on `bar` in both CTAs when the MMAs that the lane issued have completed.
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  if (!DA_MMA_OK(d_tmem, idesc)) return;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .b16 m;\n\tmov.b16 m, 3;\n\t"
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}

// The limit of a wait for an accumulator of `blocks` K blocks: a wait's own, and 4096 cycles a block (they take 270 to 450;
// from some 5 million blocks on, a weight gradient over 300 million rows, the contraction alone would pass the limit).
__device__ __forceinline__ uint64_t blocks_budget(int blocks) { return kWaitBudgetCycles + static_cast<uint64_t>(blocks) * 4096u; }

// ----------------------------------------------------------------- layout
// Epilogue warps: kEpiF32 holds sums in registers, 64 columns a thread (128 would spill: a warp may have 168).
__host__ __device__ constexpr int linear_epi_warps(int epi) { return epi == kEpiF32 ? 16 : 8; }

template <int CG, bool A_MN, bool B_MN, int EPI>
struct LinearCfg {
  static constexpr int BM = kLinBM, BN = kLinBN, BK = kLinBK;
  static constexpr int BN_CTA = BN / CG;  // rows of B that a CTA holds
  static constexpr int EPI_WARPS = linear_epi_warps(EPI), NTHREADS = (EPI_WARPS + 2) * 32;
  static constexpr int A_BYTES = BM * BK * 2;
  static constexpr int B_BYTES = BN_CTA * BK * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;  // 48 KB, a pair's CTA 32 KB
  static constexpr int STAGES = (229376 - EPI_WARPS * 4096) / STAGE_BYTES;  // 4, a pair 6; kEpiF32: 3 and 5
  // Where every tile is a half, its smaller slots: 6 and 8, kEpiF32 4 and 6.
  static constexpr int HALF_BYTES = A_BYTES + B_BYTES / 2;
  static constexpr int HALF_STAGES = STAGES * STAGE_BYTES / HALF_BYTES;
  static constexpr int OFF_STAGING = STAGES * STAGE_BYTES;
  static constexpr int OFF_BARS = OFF_STAGING + EPI_WARPS * 4096;
  static constexpr int NBARS = 2 * HALF_STAGES + 5;  // full, empty, acc_full[2], acc_empty[2], mma_done
  static constexpr int OFF_MISC = OFF_BARS + NBARS * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;  // + alignment slack
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t IDESC = idesc_bf16(BM * CG, BN, A_MN, B_MN), IDESC_HALF = idesc_bf16(BM * CG, BN / 2, A_MN, B_MN);
  static_assert(SMEM_BYTES <= 232448, "shared memory");
};

// What a cluster computes at step t of the persistent walk: rows from m (of CTA 0), accumulator columns from n0 (gated:
// gate columns), 256 or 128 accumulator columns.
struct LinTile {
  int mb, n0, cols;
};

// Tile t -> row block and column block, row blocks in groups of group_m.  From p.full on tiles come in halves: the last
// round, where it has work for no more than half of the clusters.
template <int EPI>
__device__ __forceinline__ LinTile linear_tile(const LinearParams& p, int t) {
  const bool half = t >= p.full;
  const int tile = half ? p.full + ((t - p.full) >> 1) : t;
  const int per_group = p.group_m * p.tiles_n;
  const int g = tile / per_group;
  const int first = g * p.group_m;
  const int gm = max(1, min(p.group_m, p.tiles_m - first));  // (a step past the last one is not used)
  const int r = tile - g * per_group;
  constexpr int BN = EPI == kEpiGated ? kLinBN / 2 : kLinBN;
  LinTile x;
  x.mb = first + r % gm;
  x.n0 = (r / gm) * BN + (half ? ((t - p.full) & 1) * (BN / 2) : 0);
  x.cols = half ? kLinBN / 2 : kLinBN;
  return x;
}

// ----------------------------------------------------------------- staging
// A warp's staging buffer: 32 rows x 128 bytes, 16-byte parts XORed by the row (the 128-byte swizzle of a tensor map).
// Part `q` of a row:
__device__ __forceinline__ uint4* stage_at(uint8_t* stg, int row, int q) {
  return reinterpret_cast<uint4*>(stg + row * 128 + ((q ^ (row & 7)) << 4));
}
// Global rows (`ld` bytes apart, `rows` of them and the first `bytes` bytes of each, a multiple of 16) to registers, 8
// lanes a row (lane = part lane % 8 of rows lane / 8 + 4 i), and from there into the buffer.
__device__ __forceinline__ void stage_load(uint4 (&r)[8], const uint8_t* src, long long ld, int rows, int bytes, int lane) {
  const int part = lane & 7;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = (lane >> 3) + 4 * i;
    r[i] = make_uint4(0, 0, 0, 0);
    if (row < rows && part * 16 < bytes) r[i] = *reinterpret_cast<const uint4*>(src + row * ld + part * 16);
  }
}
__device__ __forceinline__ void stage_put(uint8_t* stg, const uint4 (&r)[8], int lane) {
#pragma unroll
  for (int i = 0; i < 8; ++i) *stage_at(stg, (lane >> 3) + 4 * i, lane & 7) = r[i];
}
// The same without registers between; stage_copied: it has landed.
__device__ __forceinline__ void stage_copy(uint8_t* stg, const uint8_t* src, long long ld, int rows, int bytes, int lane) {
  const int part = lane & 7;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = (lane >> 3) + 4 * i;
    if (row < rows && part * 16 < bytes && DA_BOUNDS(row < 32))
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(stage_at(stg, row, part))), "l"(src + row * ld + part * 16)
                   : "memory");
  }
}
__device__ __forceinline__ void stage_copied() {
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
}
// Until the stores sent from the buffer have read it.
__device__ __forceinline__ void stage_free(int lane) {
  if (lane == 0) bulk_wait_read_all();
  __syncwarp();
}
// The buffer to columns from c0 of side c1, rows from r0: the tensor map drops what lies past its edges.
__device__ __forceinline__ void stage_send(const CUtensorMap* map, uint8_t* stg, int c0, int c1, int r0, int lane) {
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    if (DA_TMA_OK(smem_u32(stg), c0, c1, r0, 0))
      asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                       reinterpret_cast<uint64_t>(map)),
                   "r"(smem_u32(stg)), "r"(c0), "r"(c1), "r"(r0)
                   : "memory");
    bulk_commit_group();
  }
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ uint4 pack8_at(const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// This lane's row of 64 values as bf16, from column c0 of a side.  Whole lines leave by TMA: with 32-byte sectors straight
// from each lane a CTA's 64 KB took 5200 cycles (8192 x 8192 x 64: 47.6 us, in fp32 83.4; 34.5 and 50.2 so).  A second
// buffer a warp in place of a ring slot: no faster.
__device__ __forceinline__ void put_bf16_rows(uint8_t* stg, const float (&v)[64], const CUtensorMap* map, int c0, int side, int r0,
                                              int lane) {
  stage_free(lane);
#pragma unroll
  for (int q = 0; q < 8; ++q) *stage_at(stg, lane, q) = pack8_at(v + 8 * q);
  stage_send(map, stg, c0, side, r0, lane);
}

__device__ __forceinline__ void tmem_ld_wait16(uint32_t (&a)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]), "+r"(a[6]), "+r"(a[7]), "+r"(a[8]), "+r"(a[9]),
                 "+r"(a[10]), "+r"(a[11]), "+r"(a[12]), "+r"(a[13]), "+r"(a[14]), "+r"(a[15])
               :
               : "memory");
}

// 64 accumulator columns as floats.
__device__ __forceinline__ void load_cols64(uint32_t taddr, float (&v)[64]) {
  uint32_t a[32], b[32];
  tmem_ld32(taddr, a);
  tmem_ld32(taddr + 32, b);
  tmem_ld_wait2(a, b);
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    v[j] = __uint_as_float(a[j]);
    v[32 + j] = __uint_as_float(b[j]);
  }
}

// ----------------------------------------------------------------- epilogues
template <int N>
__device__ __forceinline__ void add_bias(float* v, const float* bias, int cols) {
#pragma unroll
  for (int q = 0; q < N / 4; ++q)
    if (4 * q < cols) {
      const float4 b = reinterpret_cast<const float4*>(bias)[q];
      v[4 * q] += b.x;
      v[4 * q + 1] += b.y;
      v[4 * q + 2] += b.z;
      v[4 * q + 3] += b.w;
    }
}

// 64 columns from column c0 (global) of the warp's 32 rows from row r0, `cols` columns of which exist.  res: the
// residual's rows as stage_load read them.
__device__ __forceinline__ void epilogue_bf16(const LinearParams& p, float (&v)[64], const uint4 (&res)[8], uint8_t* stg,
                                              int r0, int c0, int cols, int lane) {
  if (p.bias) add_bias<64>(v, p.bias + c0, cols);
  if (p.pre) put_bf16_rows(stg, v, &p.tm_pre, c0, 0, r0, lane);
  if (p.act != DIFFATTN_ACT_NONE)
    with_act(p.act, [&](auto tag) {
      act_all<decltype(tag)::value, 64, false>(v);
    });
  if (p.residual) {
    stage_free(lane);
    stage_put(stg, res, lane);
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const uint4 w = *stage_at(stg, lane, q);
      v[8 * q] += bf16_lo(w.x);
      v[8 * q + 1] += bf16_hi(w.x);
      v[8 * q + 2] += bf16_lo(w.y);
      v[8 * q + 3] += bf16_hi(w.y);
      v[8 * q + 4] += bf16_lo(w.z);
      v[8 * q + 5] += bf16_hi(w.z);
      v[8 * q + 6] += bf16_lo(w.w);
      v[8 * q + 7] += bf16_hi(w.w);
    }
  }
  put_bf16_rows(stg, v, &p.tm_out, c0, 0, r0, lane);
}

// Columns c0 .. c0 + 32 of an fp32 residual into the staging buffer.
__device__ __forceinline__ void fetch_f32(const LinearParams& p, uint8_t* stg, int r0, int c0, int rows, int cols, int lane) {
  stage_free(lane);
  stage_copy(stg, reinterpret_cast<const uint8_t*>(static_cast<const float*>(p.residual) + r0 * p.ldr + c0), p.ldr * 4, rows, cols * 4, lane);
}

// The same in fp32, 32 columns at a time; `rows` rows exist.  The first columns of a residual are on their way, unless
// the stored z needs the buffer first.
__device__ __forceinline__ void epilogue_f32(const LinearParams& p, float (&v)[64], uint8_t* stg, int r0, int c0, int rows,
                                             int cols, int lane) {
  if (p.bias) add_bias<64>(v, p.bias + c0, cols);
  if (p.pre) put_bf16_rows(stg, v, &p.tm_pre, c0, 0, r0, lane);
  if (p.act != DIFFATTN_ACT_NONE)
    with_act(p.act, [&](auto tag) {
      act_all<decltype(tag)::value, 64, true>(v);
    });
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (32 * h >= cols) break;
    if (p.residual) {
      if (h > 0 || p.pre) fetch_f32(p, stg, r0, c0 + 32 * h, rows, cols - 32 * h, lane);
      stage_copied();
    } else {
      stage_free(lane);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      float4* at = reinterpret_cast<float4*>(stage_at(stg, lane, q));
      const float* w = v + 32 * h + 4 * q;
      float4 x = make_float4(w[0], w[1], w[2], w[3]);
      if (p.residual) {
        const float4 y = *at;
        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
      }
      *at = x;
    }
    stage_send(&p.tm_out, stg, c0 + 32 * h, 0, r0, lane);
  }
}

// ----------------------------------------------------------------- kernel
template <int CG, bool A_MN, bool B_MN, int EPI>
__global__ void __launch_bounds__(LinearCfg<CG, A_MN, B_MN, EPI>::NTHREADS, 1)
    linear_kernel(const __grid_constant__ LinearParams p) {
  using C = LinearCfg<CG, A_MN, B_MN, EPI>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // (uniform to the compiler too)
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BARS);
  uint64_t* full = bars;                        // [stages] A and B of a K block landed (in both CTAs)
  uint64_t* empty = full + C::HALF_STAGES;      // [stages] the MMAs reading the slot completed
  uint64_t* acc_full = empty + C::HALF_STAGES;  // [2] every MMA of the accumulator completed
  uint64_t* acc_empty = acc_full + 2;           // [2] the epilogue (of both CTAs) has read the accumulator
  uint64_t* mma_done = acc_empty + 2;           // every MMA issued completed (abort drain)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);

  const int steps = p.full + 2 * (p.tiles_m * p.tiles_n - p.full);
  const int kblocks = (p.K + C::BK - 1) / C::BK;
  const int seg = EPI == kEpiF32 ? kLinSegBlocks : kblocks;  // K blocks an accumulator sums
  const int stages = p.full > 0 ? C::STAGES : C::HALF_STAGES, stage_bytes = p.full > 0 ? C::STAGE_BYTES : C::HALF_BYTES;
  const int cid = static_cast<int>(blockIdx.x) / CG, ncl = static_cast<int>(gridDim.x) / CG;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], CG * C::EPI_WARPS);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::EPI_WARPS + 1) tmem_alloc_cg<CG>(tmem_slot, C::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();
  tc_fence_after();
  LinTile x = linear_tile<EPI>(p, cid);
  if (warp == C::EPI_WARPS && elect_one()) {
    tma_prefetch_desc(&p.tm_a);
    tma_prefetch_desc(&p.tm_b);
  }
  grid_dep_wait();
  grid_dep_launch_dependents();  // (every CTA at work has its TMEM by now)
  const uint32_t tmem = *tmem_slot;
  const AbortState ab{abort_flag, p.status};

  if (warp == C::EPI_WARPS) {
    // ================================================================ producer
    // (The whole warp, one lane issuing: loops of one lane alone, ring slots divided out of a 64-bit count and a warp
    // index that the compiler took for divergent cost 470 to 600 cycles a K block, whatever its size; half tiles of
    // 300 x 2048 x 8192 took 41.9 us on single SMs and 38.9 on pairs, now 23.9 and 21.8, 300 and 270 cycles.)
    int slot = 0;
    uint32_t phase = 1;  // of `empty`; a slot's first use waits for nothing
    long long fill = 0;
    bool ok = true;
    for (int t = cid; ok && t < steps; t += ncl, x = linear_tile<EPI>(p, t)) {
      if (x.n0 >= p.N) continue;
      const int m0 = (x.mb * CG + static_cast<int>(rank)) * C::BM;
      const int part = x.cols / CG;  // rows of B that this CTA loads: gate columns and, N rows further, up columns if gated
      const uint32_t bytes = C::A_BYTES + static_cast<uint32_t>(part) * 128u;
      for (int kb = 0; kb < kblocks; ++kb, ++fill) {
        if (fill >= stages && !__all_sync(0xffffffffu, mbar_wait(&empty[slot], phase, ab))) {
          ok = false;
          break;
        }
        uint8_t* dst = smem + slot * stage_bytes;
        const uint32_t bar = CG == 2 ? map_to_rank(&full[slot], 0) : 0;
        const int k0 = kb * C::BK;
        if (elect_one() && DA_BOUNDS(k0 < p.K)) {
          if (rank == 0) mbar_arrive_expect_tx(&full[slot], CG * bytes);
          auto load = [&](uint8_t* to, const CUtensorMap* map, int c0, int c1) {
            if (CG == 2)
              tma_load_2d_pair(to, map, bar, c0, c1);
            else
              tma_load_2d(to, map, &full[slot], c0, c1);
          };
          // A box that starts past its tensor is filled with zeros, as one that ends past it.
          if (A_MN) {
            load(dst, &p.tm_a, m0, k0);
            load(dst + 8192, &p.tm_a, m0 + 64, k0);
          } else {
            load(dst, &p.tm_a, k0, m0);
          }
#pragma unroll
          for (int h = 0; h < C::BN_CTA / 64; ++h) {
            if (64 * h >= part) break;
            const int b = static_cast<int>(rank) * part + 64 * h;  // accumulator column of the box's first row
            // gated: the first half of the columns are gate rows, the second half their up rows
            const int nr = EPI == kEpiGated ? x.n0 + (2 * b < x.cols ? b : p.N + b - x.cols / 2) : x.n0 + b;
            if (B_MN)
              load(dst + C::A_BYTES + h * 8192, &p.tm_b, nr, k0);
            else
              load(dst + C::A_BYTES + h * 8192, &p.tm_b, k0, nr);
          }
        }
        __syncwarp();
        if (++slot == stages) slot = 0, phase ^= 1u;
      }
    }
    if (lane == 0) {
      // The commits of the last slots have arrived in this CTA (they come from the pair's first CTA).
      for (long long f = (fill > stages ? fill - stages : 0); ok && f < fill; ++f)
        ok = mbar_wait(&empty[f % stages], static_cast<uint32_t>(f / stages) & 1u, ab);
      if (*ab.flag && rank == 0) {
        // Aborted: the copies already issued land before the CTA exits.
        for (long long f = (fill > stages ? fill - stages : 0); f < fill; ++f)
          mbar_wait_drain(&full[f % stages], static_cast<uint32_t>(f / stages) & 1u, kWaitBudgetCycles);
      }
    }
    __syncwarp();
  } else if (warp == C::EPI_WARPS + 1) {
    // ================================================================ MMA issuer
    if (rank == 0) {
      // K-major: 128-byte rows, 8-row groups 1024 bytes apart.  MN-major: boxes of 64 x 64 (8 KB), groups of
      // eight k 1024 bytes apart inside one, the next 64 rows 8192 bytes further.
      const uint64_t dA = sdesc_sw128(smem_u32(smem), A_MN ? 8192 : 16, 1024);
      const uint64_t dB = sdesc_sw128(smem_u32(smem + C::A_BYTES), B_MN ? 8192 : 16, 1024);
      constexpr int KA = A_MN ? 2048 : 32, KB = B_MN ? 2048 : 32;  // bytes from one K16 step to the next
      auto waitp = [&](uint64_t* bar, uint32_t parity) -> bool {
        const bool r = __all_sync(0xffffffffu, mbar_wait(bar, parity, ab));
        tc_fence_after();
        return r;
      };
      int s = 0;
      uint32_t phase = 0;
      long long i = 0;  // accumulators of this cluster so far
      bool ok = true;
      for (int t = cid; ok && t < steps; t += ncl, x = linear_tile<EPI>(p, t)) {
          if (x.n0 >= p.N) continue;
        const uint32_t idesc = x.cols == C::BN ? C::IDESC : C::IDESC_HALF;
        for (int kb = 0, j = 0; ok && kb < kblocks; ++kb) {  // j: K blocks in the accumulator
          const int a = static_cast<int>(i & 1);
          const bool first = j == 0;
          // The epilogue of accumulator i - 2 has read these columns.
          if (first && i >= 2 && !waitp(&acc_empty[a], static_cast<uint32_t>((i >> 1) - 1) & 1u)) {
            ok = false;
            break;
          }
          if (!waitp(&full[s], phase)) {
            ok = false;
            break;
          }
          const uint64_t so = static_cast<uint64_t>((s * stage_bytes) >> 4);
          const uint32_t dacc = tmem + static_cast<uint32_t>(a * C::BN);
          const bool last = ++j == seg || kb == kblocks - 1;
          auto a_at = [&](int k) { return dA + so + static_cast<uint64_t>((k * KA) >> 4); };
          auto b_at = [&](int k) { return dB + so + static_cast<uint64_t>((k * KB) >> 4); };
          // (One lane for a whole block suits pairs, one elected for each instruction single SMs: half tiles of
          // 300 x 2048 x 8192 30.5 us against 33.5, and 23.9 against 29.0.)
          if (CG == 2) {
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < C::BK / 16; ++k) mma_pair(dacc, a_at(k), b_at(k), idesc, (!first || k > 0) ? 1u : 0u);
              tc_commit_pair(&empty[s]);
              if (last) tc_commit_pair(&acc_full[a]);
            }
            __syncwarp();
          } else {
#pragma unroll
            for (int k = 0; k < C::BK / 16; ++k) mma_ss_elect(dacc, a_at(k), b_at(k), idesc, (!first || k > 0) ? 1u : 0u);
            tc_commit_elect(&empty[s]);
            if (last) tc_commit_elect(&acc_full[a]);
          }
          if (++s == stages) s = 0, phase ^= 1u;
          if (last) {
            ++i;
            j = 0;
          }
        }
      }
      if (__any_sync(0xffffffffu, *ab.flag)) {
        // Aborted: the MMAs already issued complete before TMEM is freed.
        if (CG == 1)
          tc_commit_elect(mma_done);
        else if (elect_one())
          tc_commit_pair(mma_done);
        __syncwarp();
        mbar_wait_drain(mma_done, 0, kWaitBudgetCycles);
      }
    }
    __syncwarp();
  } else {
    // ================================================================ epilogue
    const int wq = warp & 3, half = warp >> 2;  // (kEpiF32: quarter)
    const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    uint8_t* stg = smem + C::OFF_STAGING + warp * 4096;
    const uint32_t empty0 = CG == 2 ? map_to_rank(&acc_empty[0], 0) : 0;
    const uint64_t wait_budget = EPI == kEpiF32 ? kWaitBudgetCycles : blocks_budget(kblocks);
    auto acc_wait = [&](long long i) -> bool {
      const bool got = __all_sync(0xffffffffu, mbar_wait(&acc_full[i & 1], static_cast<uint32_t>(i >> 1) & 1u, ab, wait_budget));
      tc_fence_after();
      return got;
    };
    auto acc_release = [&](long long i) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 2)
          mbar_arrive_cluster(empty0 + static_cast<uint32_t>(i & 1) * 8u);
        else
          mbar_arrive(&acc_empty[i & 1]);
      }
      __syncwarp();
    };
    long long i = 0;
    bool ok = true;
    for (int t = cid; ok && t < steps; t += ncl, x = linear_tile<EPI>(p, t)) {
      if (x.n0 >= p.N) continue;
      const int r0 = (x.mb * CG + static_cast<int>(rank)) * C::BM + wq * 32;
      const int rows = min(32, p.M - r0);  // (<= 0: none)
      if (EPI == kEpiGated) {
        // 64 gate columns and their up columns (a half tile has no more than 64)
        const int off = half * 64, width = x.cols >> 1, c0 = x.n0 + off, cols = off < width ? p.N - c0 : 0;
        if (!acc_wait(i)) break;
        const uint32_t acc = tl + static_cast<uint32_t>((i & 1) * C::BN + off);
        float g[64], u[64];
        if (off < width) {
          load_cols64(acc, g);
          load_cols64(acc + static_cast<uint32_t>(width), u);
        }
        acc_release(i);
        ++i;
        if (rows <= 0 || cols <= 0) continue;
        if (p.pre) {
          put_bf16_rows(stg, g, &p.tm_pre, c0, 0, r0, lane);
          put_bf16_rows(stg, u, &p.tm_pre, c0, 1, r0, lane);
        }
        with_act(p.act, [&](auto tag) {
          act_times<decltype(tag)::value, 64>(g, u);
        });
        put_bf16_rows(stg, g, &p.tm_out, c0, 0, r0, lane);
      } else if (EPI == kEpiF32) {
        const int off = half * 64, c0 = x.n0 + off, cols = off < x.cols ? p.N - c0 : 0;
        if (p.residual && !p.pre && rows > 0 && cols > 0) fetch_f32(p, stg, r0, c0, rows, cols, lane);
        float v[64];
        for (int kb = 0; kb < kblocks; kb += seg, ++i) {
          if (!acc_wait(i)) {
            ok = false;
            break;
          }
          if (off < x.cols) {
            const uint32_t acc = tl + static_cast<uint32_t>((i & 1) * C::BN + off);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t r[16];
              tmem_ld16(acc + 16 * q, r);
              tmem_ld_wait16(r);
#pragma unroll
              for (int j = 0; j < 16; ++j) v[16 * q + j] = kb == 0 ? __uint_as_float(r[j]) : v[16 * q + j] + __uint_as_float(r[j]);
            }
          }
          acc_release(i);
        }
        if (!ok) break;
        if (rows > 0 && cols > 0) epilogue_f32(p, v, stg, r0, c0, rows, cols, lane);
      } else {
        const int width = x.cols >> 1;  // accumulator columns of this half of the warps
        const int c0 = x.n0 + half * width, cols = min(width, p.N - c0);
        uint4 res[8];
        auto fetch = [&](int q) {
          if (p.residual && rows > 0 && cols > 64 * q)
            stage_load(res, reinterpret_cast<const uint8_t*>(static_cast<const __nv_bfloat16*>(p.residual) + r0 * p.ldr + c0 + 64 * q),
                       p.ldr * 2, rows, (cols - 64 * q) * 2, lane);
        };
        fetch(0);
        if (!acc_wait(i)) break;
        const uint32_t acc = tl + static_cast<uint32_t>((i & 1) * C::BN + half * width);
        float v[64];
        load_cols64(acc, v);
        if (width == 64) acc_release(i);
        if (rows > 0 && cols > 0) epilogue_bf16(p, v, res, stg, r0, c0, cols, lane);
        if (width > 64) {
          fetch(1);  // (earlier it costs registers that the activations need: 4096 x 4096 x 512, gelu, stored z: 36 for 31 us)
          load_cols64(acc + 64, v);
          acc_release(i);
          if (rows > 0 && cols > 64) epilogue_bf16(p, v, res, stg, r0, c0 + 64, cols - 64, lane);
        }
        ++i;
      }
    }
    if (lane == 0) bulk_wait_read_all();  // (the staging buffer lives until its stores have read it, aborted or not)
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();  // (no arrival or commit of the other CTA is on its way here any more)
  if (warp == C::EPI_WARPS + 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_cg<CG>(tmem, C::TMEM_COLS);
  }
}

}  // namespace da
