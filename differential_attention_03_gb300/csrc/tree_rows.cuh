// Attention of drafted tokens over a key/value cache (tcgen05 tensor cores,
// TMA, mbarriers; sm_103a): up to 64 new tokens of a sequence, the nodes of a
// draft tree, against its cached keys.
//
// What it computes, for sequence b with L = lens[b] committed keys and the
// keys of its nt drafted tokens in cache rows L .. L + nt - 1:
//   token t sees key j  iff  j < L, or j = L + u with u < nt and bit u of its mask word
//   O_r = sum_j softmax_j(q_r . k_r[j] / sqrt d) v[j] over the keys it sees,   r = 1, 2
//   V1: out = (1 - lambda_init) gamma (O_1 - lambda O_2) / rms(O_1 - lambda O_2)
//   V2: out = O_1 - sigmoid(logit) O_2   (q_1, q_2 the query heads of a pair over one key head)
// A token that sees no key, or t >= nt, gets zeros.  One token is nt = 1.
//
// Rows.  A work unit is (sequence, key head, row tile); its 128 MMA rows are
// map 1's rows 0 .. 63 and map 2's 64 .. 127 (row = pair * T + token, pairs of
// a key head packed while they fit).  V1's maps have their own keys: the
// score tile is the sum of two MMAs whose A operands are [Q_1; 0] and
// [0; Q_2], windows of one shared buffer Q_1 | zeros | Q_2, so both maps'
// scores land stacked in one accumulator and one P V MMA serves both maps:
// each key and value byte is read once.  The half of the score MMAs that
// multiplies zeros is free, as HBM bounds the kernel: 128 keys of bf16 V1 at
// d = 128 are 128 KB, 5600 cycles of this SM's share of HBM, against 3072
// cycles of MMA (1024 of scores, 2048 of both terms of P).
//
// Formats.  bf16; FP8K: e4m3 keys with one scale a tensor, bf16 values; FP8:
// e4m3 keys and values with an fp32 scale a row.  8-bit operands are not
// converted: the query row is scaled by a power of two and split into two e4m3
// terms (hi + lo holds a bf16 value's eight bits), P into three e5m2 terms
// (three_e5m2x4), at twice the MMA rate.  A key's scale multiplies its scores; a
// value row's scale is folded into P before the split, and the reference
// maximum is that of score + log2(value scale), so that the largest
// contribution, not the largest weight, sits at the top of e5m2's range (a key
// with a large weight and a small value row would otherwise push every other
// weight towards its floor).
//
// Split.  The key tiles (128 keys) of all units form one line that is dealt
// out evenly, a contiguous range to each CTA, from the lengths on the device;
// a CTA writes one partial state (maximum, sum, unnormalised O) a unit it
// touches, and tree_combine_kernel merges a unit's states and finishes the
// rows.  So a ragged batch, one long sequence and many short ones all keep
// every SM streaming.
//
// Roles (640 threads, one CTA per SM): warp 0 TMA producer; warp 1 score
// MMAs; warp 2 P V MMAs; warp 3 value and key scales (FP8); warps 4-19
// softmax, four warps a lane quarter, each a quarter of a tile's key columns
// (quarters without rows only pass the barriers).  TMEM: O, then two score
// tiles, in which P replaces the scores where it has no tiles of its own.
//
// Rounding.  Weights meet bf16 values as two bf16 terms, 16 bits, and e4m3
// ones (whose own rounding is far coarser) as three e5m2 terms, 9 bits.  With
// one bf16 term, outputs over 8192 random keys were 2.5e-3 off the formula
// instead of 1.7e-3, which rounding the output itself is; the second term costs
// 0 to 5 % of a bf16 call's time.
// Scores, maxima, sums and O stay fp32.
//
// Measured (this kernel alone): bf16 V1 d128 B4 H12 T16 n8192 71 us (403 MB, 5.7
// TB/s; about 10 us of it are the way in and the last states' stores), V2 d128
// B4 H16 T8 47 us (269 MB); over 32768 keys HBM's rate (bf16 V1 d128 B8 H8 312
// us, 6.9 TB/s).  e4m3 with 64 tokens, V1 d128 H12 n65536: 124 us (415 MB, 3.3
// TB/s), bound by the softmax warps: 128 x 128 weights a tile are scaled,
// exponentiated and split for the 64 KB that the tile reads.  (Tried there: keys
// as the MMAs' rows with 64 columns, whose 32 columns a thread do not fit the
// registers, 216 us against 138; maxima exchanged only when one moves, and early
// looks at the barriers: no gain.)
#pragma once

#include "tree_common.cuh"

#undef DA_BOUNDS_FILE
#define DA_BOUNDS_FILE 13

namespace da {

template <int D, bool V2, int FMT>
struct TreeRowsCfg {
  static constexpr bool K8 = FMT != kCacheBf16, V8 = FMT == kCacheFp8;
  static constexpr int BN = 128;              // keys of a tile
  static constexpr int DV = V2 ? D : 2 * D;
  static constexpr int NMAP_K = V2 ? 1 : 2;   // key tensors
  static constexpr int NTERM = K8 ? 2 : 1;    // terms of a query row
  static constexpr int KROW = D * (K8 ? 1 : 2);         // bytes of a key row
  static constexpr int KBOXB = KROW < 128 ? KROW : 128;  // bytes of a key box row (its swizzle width)
  static constexpr int KBOX = KROW / KBOXB;
  static constexpr int VROW = DV * (V8 ? 1 : 2);
  static constexpr int VBOX = VROW / 128;
  static constexpr int VKEYS = kTreeValueKeys;  // of a value slot
  static constexpr int K_SLOT = BN * KROW, V_SLOT = VKEYS * VROW;
  static constexpr int QROWS = V2 ? 128 : 192;          // Q_even | Q_odd, or Q_1 | zeros | Q_2
  static constexpr int Q_TERM = QROWS * KROW;
  static constexpr int Q_BYTES = NTERM * Q_TERM;
  // Rings: about 160-176 KB in flight, split between keys and values.
  static constexpr int NK = (!V2 && D == 128) ? (K8 ? 4 : 2) : (!V2) ? (K8 ? (V8 ? 10 : 8) : 5) : (K8 ? 5 : 3);
  static constexpr int NV = (!V2 && D == 128) ? (V8 ? 6 : 3) : (!V2) ? (V8 ? 12 : (K8 ? 7 : 6)) : (V8 ? 11 : (K8 ? 6 : 5));
  static constexpr int NS = 6;  // scale buffers (FP8)
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = Q_BYTES;
  static constexpr int OFF_V = OFF_K + NK * K_SLOT;
  static constexpr int OFF_SC = OFF_V + NV * V_SLOT;           // float [NS][4][128]: key scales 1, 2, value scales, log2 of them
  static constexpr int OFF_XM = OFF_SC + (V8 ? NS * 4 * 128 * 4 : 0);  // float [2 tiles][4 warps][128]: maxima (at a segment's end: sums)
  static constexpr int OFF_QI = OFF_XM + 8 * 128 * 4;          // float [128]: inverse of the query row's power of two
  static constexpr int OFF_BARS = OFF_QI + 128 * 4;
  static constexpr int NBARS = 2 * NK + 2 * NV + 2 * NS + 2 + 2 + 2 + 2 + 1 + 2;
  static constexpr int OFF_MISC = OFF_BARS + NBARS * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 256 + 1024;
  // Tensor memory: O, two score tiles, and, where O leaves the room and P is e5m2 (DV = 128), a P tile of
  // 96 columns; else P takes the place of its scores.  P: first terms, then second, then third.
  static constexpr bool PSEP = DV == 128 && V8;
  static constexpr uint32_t TM_O = 0, TM_S = DV;
  static constexpr uint32_t TM_P = PSEP ? TM_S + 2 * BN : TM_S, P_STEP = PSEP ? 0 : BN;
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr int QK_STEPS = KROW / 32;
  static constexpr uint32_t IDESC_QK = K8 ? idesc_e4m3(128, BN) : idesc_bf16(128, BN, false, false);
  static constexpr uint32_t IDESC_PV = V8 ? (idesc_e4m3(128, DV) | kIdescA5 | (1u << 16)) : idesc_bf16(128, DV, false, true);
  static constexpr int NACT = 16;  // softmax warps: four a lane quarter
  static constexpr int NTHREADS = (4 + NACT) * 32;
  static_assert(SMEM_BYTES <= 232448, "shared memory");
  static_assert(DV + 2 * BN + (PSEP ? 96 : 0) <= 512, "tensor memory");
  static_assert(K_SLOT % 1024 == 0 && V_SLOT % 1024 == 0 && Q_TERM % 1024 == 0, "swizzled boxes start on 1 KB");
};

// 4-byte asynchronous copy to shared memory: `bytes` (4 or 0) of it from global, the rest zeros.
__device__ __forceinline__ void cp_async4(uint32_t dst, const float* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void mma_ts_f8_elect(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                uint32_t accumulate) {
  if (!DA_MMA_OK(d_tmem, idesc) || !DA_TMEM_A_OK(a_tmem)) return;
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// SPLIT: up to 32 rows a map stand twice, once for either half of a tile's keys, and the two are partial
// states of their own: half the keys a softmax thread.
template <int D, bool V2, int FMT, bool SPLIT>
__global__ void __launch_bounds__(640, 1) tree_rows_kernel(const __grid_constant__ TreeParams p) {
  using C = TreeRowsCfg<D, V2, FMT>;
  constexpr int DV = C::DV, BN = C::BN, NK = C::NK, NV = C::NV, NS = C::NS;
  static_assert(!SPLIT || FMT == kCacheFp8k, "only 8-bit keys with bf16 values stand twice");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BARS);
  uint64_t* kfull = bars;
  uint64_t* kempty = kfull + NK;
  uint64_t* vfull = kempty + NK;
  uint64_t* vempty = vfull + NV;
  uint64_t* sc_full = vempty + NV;
  uint64_t* sc_free = sc_full + NS;
  uint64_t* s_full = sc_free + NS;   // [2] scores of the tile in buffer s
  uint64_t* p_ready = s_full + 2;    // [2] P of the tile written over them
  uint64_t* pv_done = p_ready + 2;   // [2] its P V completed
  uint64_t* s_free = pv_done + 2;    // [2] (PSEP) its scores loaded
  uint64_t* q_full = s_free + 2;    // the segment's queries written
  uint64_t* drained = q_full + 1;    // [2] every MMA of an MMA warp completed (abort)
  uint8_t* misc = smem + C::OFF_MISC;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 4);
  int* start = reinterpret_cast<int*>(misc + 16);  // sequence, group of its units, tile; tiles in all
  unsigned long long* poison = reinterpret_cast<unsigned long long*>(misc + 32);  // [3] by segment
  long long* scratch = reinterpret_cast<long long*>(smem + C::OFF_XM);

  constexpr int NACT = C::NACT;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NK; ++s) {
      mbar_init(&kfull[s], 1);
      mbar_init(&kempty[s], 1);
    }
    for (int s = 0; s < NV; ++s) {
      mbar_init(&vfull[s], 1);
      mbar_init(&vempty[s], 1);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(&sc_full[s], 32);
      mbar_init(&sc_free[s], NACT);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_ready[s], NACT);
      mbar_init(&pv_done[s], 1);
      mbar_init(&s_free[s], NACT);
      mbar_init(&drained[s], 1);
    }
    mbar_init(q_full, NACT);
    *abort_flag = 0;
    poison[0] = poison[1] = poison[2] = 0;
    fence_mbar_init();
  }
  for (int i = threadIdx.x; i < C::Q_BYTES / 16; i += C::NTHREADS)  // (rows without a query, and V1's zeros)
    reinterpret_cast<uint4*>(smem + C::OFF_Q)[i] = make_uint4(0, 0, 0, 0);
  grid_dep_wait();  // (what came before it touches no global memory)
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }

  const int groups = p.H * p.mt / p.team;  // of units of a sequence
  tree_range(p, groups, scratch, start);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_launch_dependents();  // (every CTA holds its tensor memory: ptx.cuh)
  const uint32_t tmem = *tmem_slot;
  const int count = start[3];
  const AbortState ab{abort_flag, p.status};

  if (warp == 0) {
    // =============================================================== producer
    if (lane == 0) {
      tma_prefetch_desc(&p.tm_k1);
      if (!V2) tma_prefetch_desc(&p.tm_k2);
      tma_prefetch_desc(&p.tm_v);
      int kf = 0, vf = 0;
      bool ok = true;
      auto load_k = [&](const CUtensorMap* map, int b, int h, int key0) {
        const int s = kf % NK;
        const uint32_t use = static_cast<uint32_t>(kf / NK);
        if (use > 0 && !mbar_wait(&kempty[s], (use - 1) & 1u, ab)) return false;
        ++kf;
        mbar_arrive_expect_tx(&kfull[s], C::K_SLOT);
        uint8_t* dst = smem + C::OFF_K + s * C::K_SLOT;
        if (DA_BOUNDS_V(key0 < p.n && b < p.B && h < p.H, key0))
          for (int bx = 0; bx < C::KBOX; ++bx) tma_load_4d(dst + bx * BN * C::KBOXB, map, &kfull[s], bx * 64, h, key0, b);
        return true;
      };
      auto load_v = [&](int b, int h, int key0) {
        for (int part = 0; part < 2; ++part) {
          const int s = vf % NV;
          const uint32_t use = static_cast<uint32_t>(vf / NV);
          if (use > 0 && !mbar_wait(&vempty[s], (use - 1) & 1u, ab)) return false;
          ++vf;
          mbar_arrive_expect_tx(&vfull[s], C::V_SLOT);
          uint8_t* dst = smem + C::OFF_V + s * C::V_SLOT;
          if (DA_BOUNDS_V(b < p.B && h < p.H, key0))  // (a box past n reads zeros)
            for (int bx = 0; bx < C::VBOX; ++bx)
              tma_load_4d(dst + bx * C::VKEYS * 128, &p.tm_v, &vfull[s], bx * (C::V8 ? 128 : 64), h,
                          key0 + part * C::VKEYS, b);
        }
        return true;
      };
      int pb = 0, ph = 0, pk = -1;  // the tile whose values come after the next tile's keys
      TreeWalk w = walk_begin(p, count, start);
      while (ok && w.rem > 0) {
        const int seg = walk_seg(w);
        const int h = walk_unit(p, w) / p.mt;
        for (int i = 0; ok && i < seg; ++i) {
          const int key0 = (w.t + i) * BN;
          ok = load_k(&p.tm_k1, w.b, h, key0) && (V2 || load_k(&p.tm_k2, w.b, h, key0));
          if (ok && pk >= 0) ok = load_v(pb, ph, pk);
          pb = w.b;
          ph = h;
          pk = key0;
        }
        walk_next(p, groups, w, seg);
      }
      if (ok && pk >= 0) load_v(pb, ph, pk);
      if (*ab.flag) {  // aborted: let the copies already issued land before the CTA exits
        for (int f = (kf > NK ? kf - NK : 0); f < kf; ++f)
          mbar_wait_drain(&kfull[f % NK], static_cast<uint32_t>(f / NK) & 1u, kWaitBudgetCycles);
        for (int f = (vf > NV ? vf - NV : 0); f < vf; ++f)
          mbar_wait_drain(&vfull[f % NV], static_cast<uint32_t>(f / NV) & 1u, kWaitBudgetCycles);
      }
    }
    __syncwarp();
  } else if (warp == 1 || warp == 2) {
    // =============================================================== MMA issuers
    auto waitp = [&](uint64_t* bar, uint32_t parity) -> bool {
      const bool v = __all_sync(0xffffffffu, mbar_wait(bar, parity, ab));
      tc_fence_after();
      return v;
    };
    bool ok = true;
    // (descriptors and bounds broadcast and hoisted: see tree_cols.cuh)
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    uint32_t g = 0;  // tiles so far
    uint32_t slot = 0, phase = 0;
    TreeWalk w = walk_begin(p, count, start);
    for (uint32_t k = 0; ok && __shfl_sync(0xffffffffu, w.rem, 0) > 0; ++k) {
      const int seg = __shfl_sync(0xffffffffu, walk_seg(w), 0);
      if (warp == 1) {
        const uint64_t dk0 = sdesc_rows<C::KBOXB>(smem_u32(smem + C::OFF_K), 16);
        const uint64_t dq0 = sdesc_rows<C::KBOXB>(smem_u32(smem + C::OFF_Q), 16);
        ok = waitp(q_full, k & 1u);
        for (int i = 0; ok && i < seg; ++i, ++g) {
          const uint32_t s = g & 1u;
          // the buffer: its scores loaded, or (P in their place) their P V done
          if (g >= 2 && !waitp(C::PSEP ? &s_free[s] : &pv_done[s], ((g - 2) >> 1) & 1u)) ok = false;
          const uint32_t d = tm + C::TM_S + s * BN;
#pragma unroll
          for (int m = 0; m < C::NMAP_K; ++m) {
            if (ok && !waitp(&kfull[slot], phase)) ok = false;
            if (!ok) break;
            const uint32_t koff = slot * (C::K_SLOT >> 4);
#pragma unroll
            for (int term = 0; term < C::NTERM; ++term) {
#pragma unroll
              for (int st = 0; st < C::QK_STEPS; ++st) {
                // rows 0-127 or 64-191 of the shared query buffer
                const uint64_t a = desc_at(
                    dq0, (term * C::Q_TERM + m * 64 * C::KBOXB + (st >> 2) * (C::QROWS * 128) + (st & 3) * 32) >> 4);
                const uint64_t bd = desc_at(dk0, koff + (((st >> 2) * (BN * 128) + (st & 3) * 32) >> 4));
                const uint32_t acc = (m > 0 || term > 0 || st > 0) ? 1u : 0u;
                if constexpr (C::K8)
                  mma_ss_f8_elect(d, a, bd, C::IDESC_QK, acc);
                else
                  mma_ss_elect(d, a, bd, C::IDESC_QK, acc);
              }
            }
            tc_commit_elect(&kempty[slot]);
            if (++slot == NK) {
              slot = 0;
              phase ^= 1u;
            }
          }
          if (ok) tc_commit_elect(&s_full[s]);
        }
      } else {
        const uint64_t dv0 = sdesc_rows<128>(smem_u32(smem + C::OFF_V), C::VKEYS * 128);
        for (int i = 0; ok && i < seg; ++i, ++g) {
          const uint32_t s = g & 1u;
          if (!waitp(&p_ready[s], (g >> 1) & 1u)) ok = false;
          const uint32_t again = i > 0 ? 1u : 0u;
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            if (ok && !waitp(&vfull[slot], phase)) ok = false;
            if (!ok) break;
            constexpr int KS = C::V8 ? 32 : 16;  // keys of an MMA
            const uint32_t voff = slot * (C::V_SLOT >> 4);
#pragma unroll
            for (int kk = 0; kk < C::VKEYS / KS; ++kk) {
              const uint64_t b = desc_at(dv0, voff + ((kk * KS * 128) >> 4));
              const uint32_t col = tm + C::TM_P + s * C::P_STEP + 8u * (part * (C::VKEYS / KS) + kk);
              const uint32_t acc = (part > 0 || kk > 0) ? 1u : again;
              if constexpr (C::V8) {
                mma_ts_f8_elect(tm + C::TM_O, col, b, C::IDESC_PV, acc);
                mma_ts_f8_elect(tm + C::TM_O, col + 32u, b, C::IDESC_PV, 1u);
                mma_ts_f8_elect(tm + C::TM_O, col + 64u, b, C::IDESC_PV, 1u);
              } else {
                mma_ts_elect(tm + C::TM_O, col, b, C::IDESC_PV, acc);
                mma_ts_elect(tm + C::TM_O, col + 64u, b, C::IDESC_PV, 1u);
              }
            }
            tc_commit_elect(&vempty[slot]);
            if (++slot == NV) {
              slot = 0;
              phase ^= 1u;
            }
          }
          if (ok) tc_commit_elect(&pv_done[s]);
        }
      }
      walk_next(p, groups, w, seg);
    }
    tc_commit_elect(&drained[warp - 1]);
    if (*ab.flag) mbar_wait_drain(&drained[warp - 1], 0, kWaitBudgetCycles);
    __syncwarp();
  } else if (warp == 3) {
    // =============================================================== row scales (FP8)
    if constexpr (C::V8) {
      // Copies of kAhead tiles are in flight (a load a tile at a time would cost its whole latency a
      // tile); a lane then turns the scales it copied into what the softmax reads.
      constexpr int kAhead = 4;
      static_assert(NS > kAhead, "scale ring");
      TreeWalk a = walk_begin(p, count, start), w = a;
      int ai = 0, wi = 0;  // tile of the segment: the next to copy, the next to finish
      bool ok = true;
      float* const ring = reinterpret_cast<float*>(smem + C::OFF_SC);
      auto copy_next = [&](int f) {
        if (ok && f < count) {
          const int s = f % NS, use = f / NS;
          if (use > 0) ok = __all_sync(0xffffffffu, mbar_wait(&sc_free[s], static_cast<uint32_t>(use - 1) & 1u, ab));
          const size_t row = (static_cast<size_t>(a.b) * p.H + walk_unit(p, a) / p.mt) * p.n;
          const int key0 = (a.t + ai) * BN;
          const uint32_t dst = smem_u32(ring + s * 512);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = 32 * e + lane;
            const int in = key0 + j < a.len.end ? 4 : 0;  // (rows past the end: zeros)
            const size_t at = row + (in ? key0 + j : 0);
            cp_async4(dst + 4 * j, p.k1_scales + at, in);
            if (!V2) cp_async4(dst + 4 * (128 + j), p.k2_scales + at, in);
            cp_async4(dst + 4 * (256 + j), p.v_scales + at, in);
          }
          if (++ai == walk_seg(a)) {
            walk_next(p, groups, a, ai);
            ai = 0;
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      for (int f = 0; f < kAhead; ++f) copy_next(f);
      for (int g = 0; ok && g < count; ++g) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        float* dst = ring + (g % NS) * 512;
        const int key0 = (w.t + wi) * BN;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 32 * e + lane;
          const float x = dst[256 + j];
          // A value scale that is not finite makes its row NaN: for everybody (P is NaN), or, for a
          // drafted row, for the tokens that see it (marked by its log2, and weightless).
          const bool bad = !(fabsf(x) < INFINITY);
          const bool drafted = key0 + j >= w.len.L;
          // The scale, where P is split at, and the log2 that the reference maximum goes by: at
          // least kTreeLeastValueLog2, so that the sum of weights stays below fp32's end.
          dst[256 + j] = bad ? (drafted ? 0.f : __uint_as_float(0x7fffffffu)) : x * kTreeValueMult;
          dst[384 + j] = bad ? __uint_as_float(0x7fffffffu) : fmaxf(__log2f(x), kTreeLeastValueLog2);
        }
        mbar_arrive(&sc_full[g % NS]);
        if (++wi == walk_seg(w)) {
          walk_next(p, groups, w, wi);
          wi = 0;
        }
        copy_next(g + kAhead);
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
  } else {
    // =============================================================== softmax
    const int wq = warp & 3, qd = (warp - 4) >> 2;  // lane quarter, which of its four warps
    const int map = wq >> 1, sub = SPLIT ? (wq & 1) : 0;
    const bool act = C::V8 || SPLIT || 32 * (wq & 1) < p.R;  // the quarter has rows (e4m3 values: more than 32)
    {
      constexpr int NC = SPLIT ? 16 : 32;                      // key columns of this warp,
      const int col0 = SPLIT ? 64 * sub + 16 * qd : 32 * qd;   // from this one
      constexpr int OC = DV / 4;                               // output channels it rescales and writes
      const int r = SPLIT ? lane : (wq & 1) * 32 + lane;       // row of the map
      const bool valid = r < p.R;
      const int row = wq * 32 + lane;                          // MMA row
      const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32) << 16);
      const int pr = r / p.T, tok = r - pr * p.T;
      const int ti = threadIdx.x - 128;                        // index among the softmax threads
      constexpr int nth = NACT * 32;
      float* xm = reinterpret_cast<float*>(smem + C::OFF_XM);
      float* qi = reinterpret_cast<float*>(smem + C::OFF_QI);
      const float top = C::V8 ? kTreeRescale8Log2 : kTreeRescaleLog2;
      uint32_t g = 0;
      TreeWalk w = walk_begin(p, count, start);
      // (an aborted CTA walks on: every wait then returns at once, and no warp misses a named barrier)
      for (uint32_t k = 0; w.rem > 0; ++k) {
        const int seg = walk_seg(w);
        const int hm = walk_unit(p, w), h = hm / p.mt, mtile = hm - h * p.mt;
        // ---- the segment's queries (the previous segment's score MMAs have completed: every warp
        // here has seen its last s_full)
        const int pair0 = mtile * p.ppt, npair = min(p.ppt, p.pairs - pair0);
        constexpr int NCH = D / 8;  // 16-byte chunks of a bf16 query row
        for (int i0 = 0; i0 < 2 * p.R * NCH; i0 += nth) {
          const int i = i0 + ti;
          const int ch = i % NCH, rr = i / NCH;
          const int m = rr >= p.R, r2 = rr - m * p.R;
          const int pj = r2 / p.T, tj = r2 - pj * p.T;
          const bool in = i < 2 * p.R * NCH;
          const bool have = in && pj < npair && tj < w.len.nt;
          uint4 x = make_uint4(0, 0, 0, 0);
          if (have) {
            const size_t at = static_cast<size_t>(w.b) * p.T + tj;
            const __nv_bfloat16* src =
                V2 ? p.q1 + (at * (2 * p.pairs * p.H) + 2 * (h * p.pairs + pair0 + pj) + m) * D
                   : (m ? p.q2 : p.q1) + (at * p.H + h) * D;
            x = reinterpret_cast<const uint4*>(src)[ch];
          }
          const int qr = (V2 ? 64 : 128) * m + r2;  // row of the shared buffer
          uint8_t* q = smem + C::OFF_Q;
          if constexpr (!C::K8) {
            if (in) {
              uint8_t* dst = q + (ch >> 3) * (C::QROWS * 128) + swizzled<128>(qr, ch & 7);
              *reinterpret_cast<uint4*>(dst) = x;
            }
          } else {
            // The row scaled by a power of two that puts its largest magnitude in [128, 256), in
            // two e4m3 terms: exact for every element down to 2^-10 of the largest.
            const uint32_t u[4] = {x.x, x.y, x.z, x.w};
            float amax = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(u[e] << 16)), fabsf(__uint_as_float(u[e] & 0xffff0000u))));
#pragma unroll
            for (int o = 1; o < NCH; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const int sh = e4m3_shift(amax);
            uint2 hi, lo8;
            split_e4m3x8(x, sh, hi, lo8);
            if (in) {
              uint8_t* dst = q + swizzled<C::KBOXB>(qr, ch >> 1) + 8 * (ch & 1);
              *reinterpret_cast<uint2*>(dst) = hi;
              *reinterpret_cast<uint2*>(dst + C::Q_TERM) = lo8;
              if (SPLIT) {  // (the second copy of the rows)
                *reinterpret_cast<uint2*>(dst + 32 * C::KROW) = hi;
                *reinterpret_cast<uint2*>(dst + 32 * C::KROW + C::Q_TERM) = lo8;
              }
              if (ch == 0) qi[64 * m + r2] = __int_as_float((127 - sh) << 23);
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
        if (C::K8) named_bar_sync(5, nth);  // (every row's scale is written)
        float rc = p.scale_log2;
        if (C::K8) rc *= valid ? qi[64 * map + r] : 0.f;
        if (FMT == kCacheFp8k) rc *= (map && !V2) ? p.k2_scale : p.k1_scale;
        // (a finite number above zero, as hidden scores are minus infinity: below 2^-126 every score is as good as zero)
        if (C::K8) rc = fminf(fmaxf(rc, 0x1p-126f), 0x1.fffffep127f);
        // ---- what the row sees of the drafted tokens
        const unsigned long long see = valid ? tree_sees(p, w.b, tok, w.len) : 0ull;

        float m_used = -INFINITY, l = 0.f;
        // O times f (the first P V of a segment overwrites O).  It has to wait for the previous tile's P V,
        // still busy when the maxima are known: where P has tiles of its own, it comes last, behind the
        // weights (e4m3 V1 d64 B8 H16 T64 n32768: 464 us, 422 last); where P's place is the scores' it comes
        // first, so that their next MMAs are not held up (d128 B8 H8: 285 us, 296 last; all four with P in two
        // terms, now 431 and 297).
        auto scale_o = [&](float f) {
          mbar_wait(&pv_done[(g - 1) & 1u], ((g - 1) >> 1) & 1u, ab);
          __syncwarp();
          tc_fence_after();
#pragma unroll 1
          for (int q = 0; q < OC / 32; ++q) {
            uint32_t o[32];
            tmem_ld32(tl + C::TM_O + OC * qd + 32u * q, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
            tmem_st32(tl + C::TM_O + OC * qd + 32u * q, o);
          }
        };
        for (int i = 0; i < seg; ++i, ++g) {
          const uint32_t s = g & 1u;
          const int key0 = (w.t + i) * BN;
          const uint32_t tS = tl + C::TM_S + s * BN;
          mbar_wait(&s_full[s], (g >> 1) & 1u, ab);
          __syncwarp();
          tc_fence_after();
          const bool special = key0 + BN > w.len.L;  // the tile reaches into the drafted keys or past them
          float f = 1.f;                             // what O and the sum go by under a new reference
          if (act) {
            uint32_t x[NC];
            if constexpr (SPLIT)
              tmem_ld16(tS + col0, x);
            else
              tmem_ld32(tS + col0, x);
            const float* sc = reinterpret_cast<const float*>(smem + C::OFF_SC) + (g % NS) * 512 + col0;
            if constexpr (C::V8) {
              mbar_wait(&sc_full[g % NS], (g / NS) & 1u, ab);
              __syncwarp();
            }
            if constexpr (SPLIT)
              tmem_ld_wait16(x);
            else
              tmem_ld_wait(x);
            if constexpr (C::PSEP) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&s_free[s]);
            }
            // ---- scores
            const uint64_t rc2 = f2pack(rc, rc);
            float pm = -INFINITY;
            if constexpr (C::V8) {
#pragma unroll
              for (int c = 0; c < NC; c += 4) {
                const float4 ks = *reinterpret_cast<const float4*>(sc + 128 * ((map && !V2) ? 1 : 0) + c);
                const float4 lv = *reinterpret_cast<const float4*>(sc + 384 + c);
                float t0, t1, y0, y1;
                const uint64_t ta = mul2(f2pack(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), f2pack(ks.x, ks.y));
                const uint64_t tb = mul2(f2pack(__uint_as_float(x[c + 2]), __uint_as_float(x[c + 3])), f2pack(ks.z, ks.w));
                f2unpack(fma2(ta, rc2, f2pack(lv.x, lv.y)), y0, y1);
                pm = max3(pm, y0, y1);
                f2unpack(fma2(tb, rc2, f2pack(lv.z, lv.w)), y0, y1);
                pm = max3(pm, y0, y1);
                f2unpack(ta, t0, t1);
                x[c] = __float_as_uint(t0);
                x[c + 1] = __float_as_uint(t1);
                f2unpack(tb, t0, t1);
                x[c + 2] = __float_as_uint(t0);
                x[c + 3] = __float_as_uint(t1);
              }
            } else if (!special) {
#pragma unroll
              for (int c = 0; c < NC; c += 2) pm = max3(pm, __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
            }
            if (special) {  // hide what the row does not see
              const int rel = key0 + col0 - w.len.L;  // drafted token of the first column
              const uint32_t vis = static_cast<uint32_t>(
                  rel >= 64 ? 0ull : rel >= 0 ? see >> rel : rel <= -64 ? ~0ull : (see << -rel) | ((1ull << -rel) - 1ull));
              pm = -INFINITY;
#pragma unroll
              for (int c = 0; c < NC; ++c) {
                if (!((vis >> c) & 1u)) x[c] = __float_as_uint(-INFINITY);
                if constexpr (C::V8)
                  pm = fmaxf(pm, fmaf(__uint_as_float(x[c]), rc, sc[384 + c]));
                else
                  pm = fmaxf(pm, __uint_as_float(x[c]));
              }
            }
            if (!C::V8) pm *= rc;  // (0 < rc < infinity)
            // ---- the row's maximum over the quarter's four warps
            float* xg = xm + (g & 1u) * 512;
            xg[qd * 128 + row] = pm;
            named_bar_sync(1 + wq, 128);
            pm = fmaxf(max3(xg[row], xg[128 + row], xg[256 + row]), xg[384 + row]) - (C::V8 ? kTreeRoom8Log2 : 0.f);
            const float m_new = fmaxf(m_used, pm);
            if (__any_sync(0xffffffffu, m_new > m_used + top)) {
              f = (m_used == m_new) ? 1.f : ex2(m_used - m_new);
              l *= f;
              m_used = m_new;
              if (!C::PSEP && i > 0) scale_o(f);
            }
            const float ref = (m_used == -INFINITY) ? 0.f : m_used;
            // ---- weights
            const uint32_t tP = tl + C::TM_P + s * C::P_STEP;
            const uint64_t nb2 = f2pack(-ref, -ref);
            uint64_t acc[2] = {0, 0};
            if constexpr (C::V8) {
#pragma unroll
              for (int c0 = 0; c0 < NC; c0 += 16) {  // (16 columns' terms at a time, for the registers' sake)
                uint32_t t1[4], t2[4], t3[4];
#pragma unroll
                for (int c = c0; c < c0 + 16; c += 4) {
                  const float4 vs = *reinterpret_cast<const float4*>(sc + 256 + c);
                  float v[4];
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    float a0, a1;
                    f2unpack(fma2(f2pack(__uint_as_float(x[c + 2 * e]), __uint_as_float(x[c + 2 * e + 1])), rc2, nb2), a0, a1);
                    const uint64_t pw = f2pack(ex2(a0), ex2(a1));
                    acc[e] = add2(acc[e], pw);
                    f2unpack(mul2(pw, e ? f2pack(vs.z, vs.w) : f2pack(vs.x, vs.y)), v[2 * e], v[2 * e + 1]);
                  }
                  const int z = (c - c0) >> 2;
                  three_e5m2x4(v[0], v[1], v[2], v[3], t1[z], t2[z], t3[z]);
                }
                if (C::PSEP && c0 == 0 && g >= 1) {  // the P tile's last reader
                  mbar_wait(&pv_done[(g - 1) & 1u], ((g - 1) >> 1) & 1u, ab);
                  __syncwarp();
                  tc_fence_after();
                }
                tmem_st4(tP + 8u * qd + (c0 >> 2), t1);
                tmem_st4(tP + 32u + 8u * qd + (c0 >> 2), t2);
                tmem_st4(tP + 64u + 8u * qd + (c0 >> 2), t3);
              }
            } else {
              uint32_t hi[NC / 2], lo[NC / 2];
#pragma unroll
              for (int c = 0; c < NC; c += 2) {
                float a0, a1;
                f2unpack(fma2(f2pack(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), rc2, nb2), a0, a1);
                const float p0 = ex2(a0), p1 = ex2(a1);
                acc[(c >> 1) & 1] = add2(acc[(c >> 1) & 1], f2pack(p0, p1));
                hi[c >> 1] = pack_bf16x2(p0, p1);
                lo[c >> 1] = pack_bf16x2(p0 - __uint_as_float(hi[c >> 1] << 16), p1 - __uint_as_float(hi[c >> 1] & 0xffff0000u));
              }
              if constexpr (!SPLIT) {
                tmem_st16(tP + 16u * qd, hi);
                tmem_st16(tP + 64u + 16u * qd, lo);
              } else {
                const uint32_t zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                tmem_st8(tP + 32u * sub + 8u * qd, hi);
                tmem_st8(tP + 64u + 32u * sub + 8u * qd, lo);
                tmem_st8(tP + 32u * (sub ^ 1) + 8u * qd, zero);
                tmem_st8(tP + 64u + 32u * (sub ^ 1) + 8u * qd, zero);
              }
            }
            {
              float s0, s1;
              f2unpack(add2(acc[0], acc[1]), s0, s1);
              l += s0 + s1;
            }
          }
          if (special) {
            if (C::V8 && ti < BN && key0 + ti >= w.len.L && key0 + ti < w.len.end) {
              const float lv = *(reinterpret_cast<const float*>(smem + C::OFF_SC) + (g % NS) * 512 + 384 + ti);
              if (lv != lv) atomicOr(&poison[k % 3], 1ull << (key0 + ti - w.len.L));
            }
            // (the previous tile's P V first: the slots' earlier fills are then all used, so that the
            // parities below mean this tile's)
            if (g > 0) mbar_wait(&pv_done[(g - 1) & 1u], ((g - 1) >> 1) & 1u, ab);
#pragma unroll 1
            for (int part = 0; part < 2; ++part) {
              const uint32_t f = 2 * g + part;
              const int kp = key0 + part * C::VKEYS;
              if (w.len.L - kp >= C::VKEYS) continue;
              mbar_wait(&vfull[f % NV], (f / NV) & 1u, ab);
              __syncwarp();
              clean_values<C::VKEYS, C::VROW, C::V8>(smem + C::OFF_V + (f % NV) * C::V_SLOT, kp, w.len, &poison[k % 3], ti, nth);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (C::PSEP && i > 0 && __any_sync(0xffffffffu, f != 1.f)) scale_o(f);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&p_ready[s]);
            if (C::V8) mbar_arrive(&sc_free[g % NS]);
          }
          __syncwarp();
        }
        // ---- the segment's partial state
        mbar_wait(&pv_done[(g - 1) & 1u], ((g - 1) >> 1) & 1u, ab);
        __syncwarp();
        tc_fence_after();
        float* xl = xm + (g & 1u) * 512;
        xl[qd * 128 + row] = l;
        named_bar_sync(1 + wq, 128);
        if (qd == 0) l = (l + xl[128 + row]) + (xl[256 + row] + xl[384 + row]);
        named_bar_sync(1 + wq, 128);  // (the next segment's maxima go there)
        if (ti == 0) poison[(k + 2) % 3] = 0;
        const long long group = static_cast<long long>(w.b) * groups + w.grp;
        float* state = tree_state(p, group, static_cast<int>(blockIdx.x) / p.team, static_cast<int>(blockIdx.x) % p.team, DV);
        const int sm = 2 * sub + map;
        const bool here = valid && DA_BOUNDS_V(group < static_cast<long long>(p.B) * groups && r < kTreeRows, r);
        if (qd == 0 && here) {
          if (see & poison[k % 3]) l = __uint_as_float(0x7fffffffu);
          reinterpret_cast<float2*>(state)[sm * p.R + r] = make_float2(m_used, l);
        }
        float* o8 = state + tree_state_o(p.R, p.subs) + (static_cast<size_t>(sm) * p.R + r) * DV + OC * qd;
#pragma unroll 1
        for (int q = 0; act && q < OC / 32; ++q) {
          uint32_t o[32];
          tmem_ld32(tl + C::TM_O + OC * qd + 32u * q, o);
          tmem_ld_wait(o);
          if (here) {
#pragma unroll
            for (int c = 0; c < 4; ++c, o8 += 8) store8(o8, o + 8 * c);
          }
        }
        tc_fence_before();
        __syncwarp();
        walk_next(p, groups, w, seg);
      }
    }
  }

  // ---- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// Small tiles want SPLIT: 128 keys of e4m3 keys and bf16 values at DV = 128 are 48 KB, 2100 cycles of HBM, and
// the softmax's way through a tile is too long for that with 32 keys a thread (fp8k V1 d64 B8 H16 n32768, one
// token, 253 us split, 289 not).  Larger ones don't, as the second state of every row is written and merged
// (bf16 V1 d128 B4 H12 T16 n8192 79.0 us split, 76.9 not; T32 90.3 and 85.4; d64 B8 H16 T1 n32768 311 and 307).
template <int D, bool V2, int FMT>
cudaError_t launch_tree_rows(const TreeParams& p, cudaStream_t s) {
  using C = TreeRowsCfg<D, V2, FMT>;
  void (*kern)(TreeParams) = tree_rows_kernel<D, V2, FMT, false>;
  if constexpr (FMT == kCacheFp8k && C::DV == 128) {
    if (p.subs == 2) kern = tree_rows_kernel<D, V2, FMT, true>;
  }
  return launch_tree_pair<C::DV, V2>(kern, C::NTHREADS, C::SMEM_BYTES, C::V8 ? 1.f / kTreeValueMult : 1.f, p, s);
}

}  // namespace da
