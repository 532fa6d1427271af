// The products of linear.cuh for few tokens (sm_103a): the weights stream
// through once, so HBM (or L2) bounds them, not the tensor cores.  Replayed from a
// graph, weights from HBM: 1 x 2048 x 2048 4.5 us (two of them the call's; from L2
// 3.6 to 4.0), 1 x 8192 x 2048 8.8, 16 x 8192 x 8192 22.9 (5.9 TB/s), 48 x 2048 x 2
// x 5464 10.2 to 11.0 (from L2 7.4 to 9.2), 512 x 2048 x 2048 8.0.
//
// A CTA owns `width` features (the MMA's columns; gated: width gate rows and
// their up rows) of up to 128 tokens (its rows; only p.nt of them are loaded, and
// rows past them multiply what lies behind in shared memory into accumulator
// rows that nothing reads).  A cluster of cs CTAs shares the contraction of
// one tile.  The host picks width and cs so that one round of CTAs covers the
// SMs evenly, whatever the model's width.
//   warps 0-7   accumulators (thread = token, half of the columns a warp) as
//               fp32 to the CTA of the cluster that finishes the feature (lg
//               groups of eight features each), through distributed shared
//               memory, 16 bytes a store; after one cluster barrier all warps
//               sum what came, in the order of the ranks, and do the epilogue.
//   warp 8      TMA producer: its first loads are under way before the CTA's
//               other warps have their barriers and TMEM.
//   warp 9      TMEM allocator and MMA issuer.
// A programmatic dependent launch: the CTAs come up while the kernel before
// them ends, and wait for its end before they touch global memory.
// Results repeat bit for bit (no atomics).
//
// kEpiF32 sums segments of 512 values of K at most, for the tensor cores'
// truncation (see linear.cuh): in accumulators of their own, where tensor memory
// has room for all of them, else taking turns in one or two.  Warps 0-7 then add
// each segment into running sums, in tensor memory too, while the next one's MMAs
// run: 1 x 32768 x 8192 81.5 us (bf16 out 80.5), 48 x 8192 x 8192 24.9 (23.3), 256 x
// 4096 x 16384 42.6 (37.5).  With all 8192 values in one accumulator results were
// off by 3e-5.  Not kept: narrower features in place of turns (88.9 and 29.7 us of
// the first two), running sums in shared memory (83.6 and 24.6, but the ring lost
// slots to them: 52.9 of the third).
#pragma once

#include "linear.cuh"
#include "vec8.cuh"

#undef DA_BOUNDS_FILE
#define DA_BOUNDS_FILE 15

namespace da {

constexpr int kFewEpiWarps = 8;
constexpr int kFewThreads = (kFewEpiWarps + 2) * 32;

__device__ __forceinline__ void store_cluster_f4(uint32_t addr, float a, float b, float c, float d) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

template <bool W_MN, int EPI>
__global__ void __launch_bounds__(kFewThreads, 2) linear_few_kernel(const __grid_constant__ LinearParams p) {
  constexpr int SIDES = EPI == kEpiGated ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // (uniform to the compiler too)

  // ---- shared memory: ring of [weights | tokens], partial sums, barriers
  const int wrows = p.width * SIDES;
  const uint32_t w_bytes = static_cast<uint32_t>(wrows) * 128u, stage_bytes = w_bytes + static_cast<uint32_t>(p.nt) * 128u;
  const int stages = p.stages;
  float* part = reinterpret_cast<float*>(smem + stages * stage_bytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + p.off_bars);
  uint64_t* full = bars;
  uint64_t* empty = full + stages;
  uint64_t* done = empty + stages;  // every MMA completed
  uint64_t* acc_full = done + 1;       // [2] segments taking turns: the accumulator's MMAs completed
  uint64_t* acc_empty = acc_full + 2;  // [2] ... it has been read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  // ---- work of this CTA: features, tokens, and its share of the contraction
  const int cs = p.cs, rank = cs > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int tile = static_cast<int>(blockIdx.x) / cs;
  const int f0 = (tile % p.tiles_n) * p.width, t0 = (tile / p.tiles_n) * p.nt;
  const int kblocks = (p.K + kLinBK - 1) / kLinBK;
  // K blocks rank, rank + cs, ...: what a cluster reads at one time lies together in the weights' rows.
  const int nkb = (kblocks - rank + cs - 1) / cs;  // >= 1
  const bool turns = EPI == kEpiF32 && p.turns;
  const int seg = EPI != kEpiF32 ? nkb : turns ? kLinSegBlocks : few_segment_blocks(nkb, wrows);  // K blocks of a segment
  const int segs = (nkb + seg - 1) / seg;
  const int accs = turns ? few_turns(wrows) : segs;
  uint32_t tmem_cols = 32;
  while (tmem_cols < static_cast<uint32_t>((accs + (turns ? 1 : 0)) * wrows)) tmem_cols *= 2;

  if (cs > 1) cluster_arrive();  // (waited for below: every CTA of the cluster has started)
  int fill = 0, slot = 0;
  uint32_t phase = 0;
  auto load = [&]() {
    const int k0 = (rank + fill * cs) * kLinBK;
    uint8_t* dst = smem + slot * stage_bytes;
    uint64_t* bar = &full[slot];
    ++fill;
    if (++slot == stages) {
      slot = 0;
      phase ^= 1u;
    }
    if (elect_one() && DA_BOUNDS(k0 < p.K && f0 < p.N && t0 < p.M)) {
      mbar_arrive_expect_tx(bar, stage_bytes);
      if (W_MN) {
        for (int j = 0; j < wrows; j += 64) tma_load_2d(dst + j * 128, &p.tm_a, bar, f0 + j, k0);
      } else {
        tma_load_2d(dst, &p.tm_a, bar, k0, f0);
        if (EPI == kEpiGated) tma_load_2d(dst + p.width * 128, &p.tm_a, bar, k0, p.N + f0);
      }
      tma_load_2d(dst + w_bytes, &p.tm_b, bar, k0, t0);
    }
    __syncwarp();
  };
  if (warp == kFewEpiWarps) {
    if (lane == 0) {
      for (int s = 0; s < stages; ++s) {
        mbar_init(&full[s], 1);
        mbar_init(&empty[s], 1);
      }
      mbar_init(done, 1);
      for (int a = 0; a < 2; ++a) {
        mbar_init(&acc_full[a], 1);
        mbar_init(&acc_empty[a], kFewEpiWarps);
      }
      *abort_flag = 0;
      fence_mbar_init();
    }
    __syncwarp();
    grid_dep_wait();
    const int first = min(nkb, stages);
    while (fill < first) load();
  } else if (warp == kFewEpiWarps + 1) {
    tmem_alloc(tmem_slot, tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_launch_dependents();  // (every CTA has its TMEM by the time the next kernel's come up)
  const uint32_t tmem = *tmem_slot;
  const AbortState ab{abort_flag, p.status};

  if (warp == kFewEpiWarps) {
    // ================================================================ producer
    while (fill < nkb) {
      if (!__all_sync(0xffffffffu, mbar_wait(&empty[slot], phase ^ 1u, ab))) break;
      load();
    }
    if (lane == 0) {
      if (*ab.flag)  // aborted: the copies already issued land before the CTA exits
        for (int f = max(0, fill - stages); f < fill; ++f)
          mbar_wait_drain(&full[f % stages], static_cast<uint32_t>(f / stages) & 1u, kWaitBudgetCycles);
    }
    __syncwarp();
  } else if (warp == kFewEpiWarps + 1) {
    // ================================================================ MMA issuer
    const uint64_t dX = sdesc_sw128(smem_u32(smem + w_bytes), 16, 1024);
    const uint64_t dW = sdesc_sw128(smem_u32(smem), W_MN ? 8192 : 16, 1024);
    constexpr int KW = W_MN ? 2048 : 32;
    const uint32_t idesc = idesc_bf16(128, 0, false, W_MN) | (static_cast<uint32_t>(wrows >> 3) << 17);
    int s = 0;
    bool landed = false;
    uint32_t ph = 0;
    auto block = [&](uint32_t dacc, bool more) {  // one K block; more: onto what the accumulator holds
      if (!__all_sync(0xffffffffu, landed) && !__all_sync(0xffffffffu, mbar_wait(&full[s], ph, ab))) return false;
      const int next = s + 1 == stages ? 0 : s + 1;
      landed = mbar_test(&full[next], next ? ph : ph ^ 1u);  // (known by the time that these MMAs are issued)
      tc_fence_after();
      const uint64_t so = static_cast<uint64_t>((s * stage_bytes) >> 4);
      if (!DA_BOUNDS_V(dacc - tmem + static_cast<uint32_t>(wrows) <= tmem_cols, dacc)) return false;
#pragma unroll
      for (int k = 0; k < kLinBK / 16; ++k)
        mma_ss_elect(dacc, dX + so + static_cast<uint64_t>((k * 32) >> 4), dW + so + static_cast<uint64_t>((k * KW) >> 4), idesc,
                     (more || k > 0) ? 1u : 0u);
      tc_commit_elect(&empty[s]);
      s = next;
      if (s == 0) ph ^= 1u;
      return true;
    };
    if (turns) {
      bool ok = true;
      int acc = 0;
      uint32_t acc_ph = 1;  // (an accumulator's first segment waits for nothing)
      for (int kb = 0; ok && kb < nkb; kb += seg) {
        if (!__all_sync(0xffffffffu, mbar_wait(&acc_empty[acc], acc_ph, ab))) break;
        const int to = min(seg, nkb - kb);
        for (int i = 0; ok && i < to; ++i) ok = block(tmem + static_cast<uint32_t>(acc * wrows), i > 0);
        tc_commit_elect(&acc_full[acc]);
        if (++acc == accs) acc = 0, acc_ph ^= 1u;
      }
    } else {
      int in_seg = 0;
      uint32_t dacc = tmem;
      for (int kb = 0; kb < nkb; ++kb) {
        if (!block(dacc, in_seg > 0)) break;
        if (++in_seg == seg) {
          in_seg = 0;
          dacc += static_cast<uint32_t>(wrows);
        }
      }
    }
    tc_commit_elect(done);
    if (__any_sync(0xffffffffu, *ab.flag)) mbar_wait_drain(done, 0, kWaitBudgetCycles);
    __syncwarp();
  }

  // ---- partial sums: [rank][token][lg groups][side][8], rows 16 bytes longer than their values (banks)
  const int groups = p.width >> 3, lg = p.lg;  // rank r finishes groups r lg .. of every token
  const int row_floats = lg * SIDES * 8 + 4;
  const int mt = min(p.nt, p.M - t0);
  const int wq = (warp & 3) * 32;  // first accumulator row of this warp
  // ---- what this CTA finishes: items of eight features of a token, i / ng by its high product (i < 2^16); the bias and
  // the residual of a thread's first item are on their way while the accumulators come
  const int ng = max(0, min(lg, groups - rank * lg));  // groups of this CTA
  const int items = mt * ng;
  const uint32_t over = 0xffffffffu / static_cast<uint32_t>(max(1, ng)) + 1u;
  auto token_of = [&](int i) { return ng == 1 ? i : static_cast<int>(__umulhi(static_cast<uint32_t>(i), over)); };
  float4 bias[2];
  uint4 res[2];
  auto fetch = [&](int i) {
    const int t = token_of(i), col = f0 + (rank * lg + i - t * ng) * 8;
    if (EPI == kEpiGated || i >= items || col >= p.N) return;
    if (p.bias) {
      bias[0] = reinterpret_cast<const float4*>(p.bias + col)[0];
      bias[1] = reinterpret_cast<const float4*>(p.bias + col)[1];
    }
    if (p.residual) {
      const uint4* at = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.residual) + ((t0 + t) * p.ldr + col) * (EPI == kEpiF32 ? 4 : 2));
      res[0] = at[0];
      if (EPI == kEpiF32) res[1] = at[1];
    }
  };
  grid_dep_wait();
  // groups of sixteen columns that a thread of warps 0-7 reads of its row: [first, last)
  const int pairs = wrows >> 4, first = warp < 4 ? 0 : (pairs + 1) >> 1, last = warp < 4 ? (pairs + 1) >> 1 : pairs;
  const int row = wq + lane;
  const uint32_t tl = tmem + (static_cast<uint32_t>(wq) << 16);
  const uint32_t running = static_cast<uint32_t>(accs * wrows);  // columns of the running sums, behind the accumulators
  if (turns && warp < kFewEpiWarps) {
    int acc = 0;
    uint32_t ph = 0;
    for (int j = 0; j < segs; ++j) {
      if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[acc], ph, ab))) break;
      tc_fence_after();
      for (int h = first; wq < mt && h < last; ++h) {
        if (!DA_BOUNDS_V(running + static_cast<uint32_t>(16 * h + 16) <= tmem_cols, h)) break;
        uint32_t a[16], b[16] = {};
        tmem_ld16(tl + static_cast<uint32_t>(acc * wrows + 16 * h), a);
        if (j > 0) tmem_ld16(tl + running + static_cast<uint32_t>(16 * h), b);
        tmem_ld_wait16x2(a, b);
#pragma unroll
        for (int k = 0; k < 16; ++k) a[k] = __float_as_uint(__uint_as_float(a[k]) + __uint_as_float(b[k]));
        tmem_st16(tl + running + static_cast<uint32_t>(16 * h), a);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[acc]);
      if (++acc == accs) acc = 0, ph ^= 1u;
    }
  }
  fetch(threadIdx.x);
  const bool go = warp < kFewEpiWarps && __all_sync(0xffffffffu, mbar_wait(done, 0, ab, blocks_budget(nkb)));
  if (cs > 1) cluster_wait();
  if (go && wq < mt) {
    // ================================================================ accumulators to the CTAs that finish them
    tc_fence_after();
    const uint32_t mine = smem_u32(part + (rank * p.nt + row) * row_floats);
    // groups of eight columns of this half of the warps
    int side = 0, g = 2 * first;
    if (SIDES == 2 && g >= groups) side = 1, g -= groups;
    int owner = g / lg, local = g - owner * lg;
    auto put = [&](const uint32_t* r) {
      uint32_t to = mine + static_cast<uint32_t>((local * SIDES + side) * 32);
      if (cs > 1) {
        asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(to) : "r"(owner));
        store_cluster_f4(to, __uint_as_float(r[0]), __uint_as_float(r[1]), __uint_as_float(r[2]), __uint_as_float(r[3]));
        store_cluster_f4(to + 16, __uint_as_float(r[4]), __uint_as_float(r[5]), __uint_as_float(r[6]), __uint_as_float(r[7]));
      } else {
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + 16), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
      }
    };
    auto next = [&]() {
      ++g;
      if (++local == lg) {
        local = 0;
        ++owner;
      }
      if (SIDES == 2 && g == groups) side = 1, g = 0, owner = 0, local = 0;
    };
    auto add_segments = [&](int c, uint32_t (&a)[16]) {
      for (int q = 1; q < segs; ++q) {
        if (!DA_BOUNDS_V(static_cast<uint32_t>(q * wrows + c + 16) <= tmem_cols, q)) break;
        uint32_t z[16];
        tmem_ld16(tl + static_cast<uint32_t>(q * wrows + c), z);
        tmem_ld_wait16x2(a, z);
#pragma unroll
        for (int j = 0; j < 16; ++j) a[j] = __float_as_uint(__uint_as_float(a[j]) + __uint_as_float(z[j]));
      }
    };
    constexpr int STEP = EPI == kEpiF32 ? 1 : 2;  // 16 or 32 columns a wait (an fp32 residual's registers leave no room for 32)
    const uint32_t from = turns ? tl + running : tl;
    for (int h = first; h < last; h += STEP) {
      if (!DA_BOUNDS_V(from - tl + static_cast<uint32_t>(16 * min(h + STEP, last)) <= tmem_cols, h)) break;
      uint32_t a[16], b[16] = {};
      tmem_ld16(from + static_cast<uint32_t>(16 * h), a);
      const bool more = STEP == 2 && h + 1 < last;
      if (more) tmem_ld16(from + static_cast<uint32_t>(16 * h + 16), b);
      tmem_ld_wait16x2(a, b);
      if (EPI == kEpiF32 && !turns) add_segments(16 * h, a);
      auto two = [&](const uint32_t* r) {
        if (row < mt) put(r);
        next();
        if (row < mt) put(r + 8);
        next();
      };
      two(a);
      if (more) two(b);
    }
  }
  tc_fence_before();
  __syncwarp();
  if (cs > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }

  // ================================================================ sum over the cluster, epilogue: eight features an item
  {
    auto sum8 = [&](int t, int g, int side, float (&v)[8]) {
      const float* at = part + t * row_floats + (g * SIDES + side) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.f;
#pragma unroll 4
      for (int c = 0; c < cs; ++c, at += p.nt * row_floats) {
        const float4 a = *reinterpret_cast<const float4*>(at), b = *reinterpret_cast<const float4*>(at + 4);
        v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
        v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
      }
    };
    for (int i = threadIdx.x; i < items; i += kFewThreads) {
      const int t = token_of(i), g = i - t * ng;
      const int col = f0 + (rank * lg + g) * 8;
      const long long row = t0 + t;
      if (col >= p.N || !DA_BOUNDS_V(row < p.M && col + 8 <= p.N, col)) continue;
      if (i >= kFewThreads) fetch(i);
      float v[8];
      sum8(t, g, 0, v);
      if (EPI == kEpiGated) {
        float u[8];
        sum8(t, g, 1, u);
        if (p.pre) {
          __nv_bfloat16* pre = p.pre + row * p.ldp + col;
          *reinterpret_cast<uint4*>(pre) = pack8(v);
          *reinterpret_cast<uint4*>(pre + p.N) = pack8(u);
        }
        with_act(p.act, [&](auto tag) {
          act_times<decltype(tag)::value, 8>(v, u);
        });
      } else {
        if (p.bias) {
          const float4 a = bias[0], b = bias[1];
          v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
          v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
        }
        if (p.pre) *reinterpret_cast<uint4*>(p.pre + row * p.ldp + col) = pack8(v);
        if (p.act != DIFFATTN_ACT_NONE)
          with_act(p.act, [&](auto tag) {
            act_all<decltype(tag)::value, 8, EPI == kEpiF32>(v);
          });
        if (p.residual) {
          float r[8];
          if (EPI == kEpiF32) {
            r[0] = __uint_as_float(res[0].x), r[1] = __uint_as_float(res[0].y), r[2] = __uint_as_float(res[0].z), r[3] = __uint_as_float(res[0].w);
            r[4] = __uint_as_float(res[1].x), r[5] = __uint_as_float(res[1].y), r[6] = __uint_as_float(res[1].z), r[7] = __uint_as_float(res[1].w);
          } else {
            unpack8(res[0], r);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] += r[j];
        }
      }
      if (EPI == kEpiF32) {
        float4* at = reinterpret_cast<float4*>(static_cast<float*>(p.out) + row * p.ldo + col);
        at[0] = make_float4(v[0], v[1], v[2], v[3]);
        at[1] = make_float4(v[4], v[5], v[6], v[7]);
      } else {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + row * p.ldo + col) = pack8(v);
      }
    }
  }

  if (warp == kFewEpiWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, tmem_cols);
  }
}

}  // namespace da
