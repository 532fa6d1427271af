// Attention of drafted tokens over a key/value cache (tcgen05 tensor cores,
// TMA, mbarriers; sm_103a): new tokens of a sequence, the nodes of a draft
// tree, against its cached keys, up to 32 rows (tokens times pairs) of a map
// over an fp8 cache (more, and the other formats: tree_rows.cuh).
//
// What it computes, for sequence b with L = lens[b] committed keys and the
// keys of its nt drafted tokens in cache rows L .. L + nt - 1:
//   token t sees key j  iff  j < L, or j = L + u with u < nt and bit u of its mask word
//   O_r = sum_j softmax_j(q_r . k_r[j] / sqrt d) v[j] over the keys it sees,   r = 1, 2
//   V1: out = (1 - lambda_init) gamma (O_1 - lambda O_2) / rms(O_1 - lambda O_2)
//   V2: out = O_1 - sigmoid(logit) O_2   (q_1, q_2 the query heads of a pair over one key head)
// A token that sees no key, or t >= nt, gets zeros.  One token is nt = 1.
//
// Orientation.  HBM bounds the step as long as few tokens share its bytes, so
// the MMAs take the cache as their 128 rows and the tokens as their columns:
//   S^T[key, token] = K Q^T,     O^T[channel, token] += V^T P^T,
// and cost what the tokens cost (8, 16 or 32 columns a map; a work unit is
// (sequence, key head, column tile), a V2 key head's pairs packed while they
// fit).  Both maps' columns lie side by side: V1's come from their own keys,
// V2's from one, and one V^T P^T serves both, so each key and value byte is
// read once.  A softmax thread then is a key: its scales and its place in the
// mask are its own registers.  (With tokens as rows, as in the forward, every
// thread needs every key's scales: three broadcast shared-memory reads a
// column, against which the MMAs' operands queued; e4m3 V1 d64 B8 H16 n32768,
// one token: 312 us; this way 188 us.)
//
// Softmax.  A column's reference maximum is shared memory's; scores come out
// as score - reference in one FMA, and only when some score of the tile is
// above it by more than a bound (one barrier with a vote a tile) do the warps
// reduce the column maxima, and rescale the sums and O^T.  Sums of weights
// stay in the threads' registers until the unit ends.
//
// Operands.  e4m3 keys and values with an fp32 scale a row, as the cache holds
// them: a query row is scaled by a power of two and split into two e4m3
// terms (hi + lo holds a bf16 value's eight bits; rows within a factor of
// eight of the largest share its power of two, and hold them down to 2^-7 of
// their own largest element instead of 2^-10), P into three e5m2 terms
// (three_e5m2x4).  A key's scale multiplies its scores; a value row's scale is
// folded into P before the split, and the reference is the maximum of score +
// log2(value scale), so that the largest contribution, not the largest weight,
// sits at the top of e5m2's range (a key with a large weight and a small value
// row would otherwise push every other weight towards its floor).
//
// Split.  The key tiles (128 keys) of all units form one line that is dealt
// out evenly, a contiguous range to each CTA, from the lengths on the device;
// a CTA writes a partial state (maximum, sum, unnormalised O) for each unit it
// touches, and tree_combine_kernel merges a unit's states and finishes the
// rows.  So a ragged batch, one long sequence and many short ones all keep
// every SM streaming.
//
// Roles (640 threads, one CTA per SM): warp 0 TMA producer; warp 1 score
// MMAs; warp 2 P V MMAs; warps 4-19 softmax, four warpgroups (one key a
// thread).  With 8 columns a map each is a stream (every fourth tile, with
// references, O^T and a partial state of its own, so that none waits for
// another) of both maps; with 16, a map of one of two streams; with 32, half
// the columns of a map.
//
// Measured (with the merge, replayed from a graph): one token V1 d64 B8 H16
// n32768 187 us (1.12 GB with the scales, 6.0 TB/s), V1 d128 B8 H8 172 us; 16
// tokens 180 us each; 32 tokens V1 d128 B8 H8 190 us (5.7 TB/s), V1 d64 B8 H16
// 261 us (4.3 TB/s), where the softmax warps bound it.
#pragma once

#include "tree_common.cuh"

#undef DA_BOUNDS_FILE
#define DA_BOUNDS_FILE 14

namespace da {

template <int D, bool V2, int TP>
struct TreeColsCfg {
  static constexpr int BN = 128;              // keys of a tile
  static constexpr int DV = V2 ? D : 2 * D;
  static constexpr int NMT = DV / 128;        // 128-channel MMAs of V^T
  static constexpr int NMAP_K = V2 ? 1 : 2;   // key tensors
  // Streams: tile g belongs to stream g % NSTREAM, which has its own references, O^T and P.  With 8
  // columns a map a warpgroup takes a stream's both maps, with 16 one map, with 32 half a map.
  static constexpr int NSTREAM = 32 / TP;
  static constexpr int NBUF = NSTREAM > 2 ? NSTREAM : 2;  // score tiles
  static constexpr int NC = 16;                 // columns of a softmax thread
  static constexpr int COLS = 2 * TP;           // columns of both maps
  // The terms of an operand stand side by side as columns, so that one MMA takes both.
  static constexpr int SCOLS = 2 * COLS;  // of a score tile: [map][term][TP]
  // P and O^T: [term][map][TP] with the three terms side by side, or, where tensor memory has no room for
  // them, two, and the third added to the first's O^T by MMAs of its own.
  static constexpr bool P3APART = TP == 32;
  static constexpr int PTERMS = P3APART ? 2 : 3;
  static constexpr int PCOLS = PTERMS * COLS;
  static constexpr int KROW = D;          // bytes of a key row (and its swizzle width)
  static constexpr int VROW = DV;
  static constexpr int VBOX = VROW / 128;
  static constexpr int VKEYS = kTreeValueKeys;  // of a value slot
  static constexpr int VF = BN / VKEYS;
  static constexpr int K_SLOT = BN * KROW, V_SLOT = VKEYS * VROW;
  // Query rows in shared memory, as the score MMAs' B operands: a V1 map's are its own rows.
  static constexpr int QROWS = SCOLS;
  static constexpr int QK_N = V2 ? SCOLS : 2 * TP;
  static constexpr int Q_BYTES = (QROWS * KROW + 1023) / 1024 * 1024;
  static constexpr int PROW = TP == 8 ? 64 : 128;      // bytes of a key's row of P^T (its swizzle width)
  static constexpr int P3ROW = P3APART ? COLS : 0;     // and of the third terms' own
  static constexpr int P_BYTES = BN * (PROW + P3ROW);  // of a stream
  // Rings: 160-168 KB in flight; some 14 KB stay free for a CTA of the merge, which is launched meanwhile.
  static constexpr int NK = D == 64 ? 10 : 5;
  static constexpr int NV = V_SLOT == 8192 ? (D == 64 ? 11 : 10) : 5;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_P = Q_BYTES;
  static constexpr int OFF_K = OFF_P + NSTREAM * P_BYTES;
  static constexpr int OFF_V = OFF_K + NK * K_SLOT;
  static constexpr int OFF_XM = OFF_V + NV * V_SLOT;    // float [4 warpgroups][4 warps][16]: maxima, sums
  static constexpr int OFF_AC = OFF_XM + 16 * 16 * 4;   // float [4 warpgroups][16]: minus the reference
  static constexpr int OFF_SEE = OFF_AC + 4 * 16 * 4;   // u64 [2 segments][32]: what a row's token sees of the drafts
  static constexpr int OFF_QS = OFF_SEE + 2 * 32 * 8;   // float [2 segments][64]: query rows' own factors
  static constexpr int OFF_QM = OFF_QS + 2 * 64 * 4;    // float [2 segments][64]: query rows' largest magnitudes
  static constexpr int OFF_BARS = OFF_QM + 2 * 64 * 4;
  static constexpr int NBARS = 2 * NK + 2 * NV + 4 * 4 + 1 + 2;
  static constexpr int OFF_MISC = OFF_BARS + NBARS * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 64 + 1024;
  static constexpr uint32_t TM_O = 0, TM_S = NSTREAM * NMT * PCOLS;  // O^T [stream][128 channels], the score tiles
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr int QK_STEPS = KROW / 32;
  static constexpr uint32_t IDESC_QK = idesc_e4m3(128, QK_N);
  static constexpr uint32_t IDESC_PV = idesc_e4m3(128, PCOLS) | kIdescB5 | (3u << 15);  // (V^T and P^T: both transposed)
  static constexpr uint32_t IDESC_P3 = idesc_e4m3(128, COLS) | kIdescB5 | (3u << 15);
  static constexpr int NSOFT = 16;              // softmax warps
  static constexpr int NARR = NSOFT / NSTREAM;  // of a stream
  static_assert(NSTREAM == tree_subs(kCacheFp8, DV, TP), "a partial state a stream");
  static constexpr int NTHREADS = (4 + NSOFT) * 32;
  static_assert(TP == 8 || TP == 16 || TP == 32, "columns of a map");
  static_assert(SMEM_BYTES <= 232448, "shared memory");
  static_assert(TM_S + NBUF * SCOLS <= 512, "tensor memory");
  static_assert(K_SLOT % 1024 == 0 && V_SLOT % 1024 == 0 && P_BYTES % 1024 == 0, "swizzled operands start on 1 KB");
  static_assert(QK_N % 16 == 0 && PCOLS % 16 == 0, "MMA columns");
  static_assert(PCOLS <= PROW && (P3ROW == 0 || P3ROW == 64), "P rows are one swizzle width");
};

constexpr float kTreeDead = -16384.f;  // minus the reference of a column without a token: weights of zero

// Lane l gets op over the warp's lanes of v[l % NC].
template <int NC, class Op>
__device__ __forceinline__ float lanes_reduce(const float (&v)[NC], int lane, Op op) {
  float t[NC / 2];
#pragma unroll
  for (int j = 0; j < NC / 2; ++j) {
    const bool up = (lane & (NC / 2)) != 0;
    const float send = up ? v[j] : v[j + NC / 2], keep = up ? v[j + NC / 2] : v[j];
    t[j] = op(keep, __shfl_xor_sync(0xffffffffu, send, NC / 2));
  }
#pragma unroll
  for (int s = NC / 4; s >= 1; s >>= 1) {
    const bool up = (lane & s) != 0;
#pragma unroll
    for (int j = 0; j < s; ++j) {
      const float send = up ? t[j] : t[j + s], keep = up ? t[j + s] : t[j];
      t[j] = op(keep, __shfl_xor_sync(0xffffffffu, send, s));
    }
  }
  if (NC == 16) t[0] = op(t[0], __shfl_xor_sync(0xffffffffu, t[0], 16));
  return t[0];
}

template <int D, bool V2, int TP>
__global__ void __launch_bounds__(640, 1) tree_cols_kernel(const __grid_constant__ TreeParams p) {
  using C = TreeColsCfg<D, V2, TP>;
  constexpr int DV = C::DV, BN = C::BN, NK = C::NK, NV = C::NV, NC = C::NC, COLS = C::COLS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BARS);
  uint64_t* kfull = bars;
  uint64_t* kempty = kfull + NK;
  uint64_t* vfull = kempty + NK;
  uint64_t* vempty = vfull + NV;
  uint64_t* s_full = vempty + NV;   // [NBUF] scores of the tile in buffer tile % NBUF
  uint64_t* s_free = s_full + 4;    // [NBUF] they are loaded
  uint64_t* p_ready = s_free + 4;   // [streams] P of the stream's tile written
  uint64_t* pv_done = p_ready + 4;  // [streams] its P V completed
  uint64_t* q_full = pv_done + 4;   // the segment's queries written
  uint64_t* drained = q_full + 1;   // [2] every MMA of an MMA warp completed (abort)
  uint8_t* misc = smem + C::OFF_MISC;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 4);
  int* start = reinterpret_cast<int*>(misc + 8);  // sequence, group of its units, tile; tiles in all
  unsigned long long* poison = reinterpret_cast<unsigned long long*>(misc + 24);  // [3] by segment
  long long* scratch = reinterpret_cast<long long*>(smem + C::OFF_XM);

  if (threadIdx.x == 0) {
    for (int s = 0; s < NK; ++s) {
      mbar_init(&kfull[s], 1);
      mbar_init(&kempty[s], 1);
    }
    for (int s = 0; s < NV; ++s) {
      mbar_init(&vfull[s], 1);
      mbar_init(&vempty[s], 1);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&s_free[s], C::NARR);
      mbar_init(&p_ready[s], C::NARR);
      mbar_init(&pv_done[s], 1);
    }
    mbar_init(&drained[0], 1);
    mbar_init(&drained[1], 1);
    mbar_init(q_full, C::NSOFT);
    *abort_flag = 0;
    poison[0] = poison[1] = poison[2] = 0;
    fence_mbar_init();
  }
  for (int i = threadIdx.x; i < C::Q_BYTES / 16; i += C::NTHREADS)  // (columns without a token)
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

  // Stream of the CTA's tile g, and its number in the stream.
  auto stream_of = [](uint32_t g) { return g % C::NSTREAM; };
  auto number_of = [](uint32_t g) { return g / C::NSTREAM; };

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
          tma_load_4d(dst, map, &kfull[s], 0, h, key0, b);
        return true;
      };
      auto load_v = [&](int b, int h, int key0) {
        for (int part = 0; part < C::VF; ++part) {
          const int s = vf % NV;
          const uint32_t use = static_cast<uint32_t>(vf / NV);
          if (use > 0 && !mbar_wait(&vempty[s], (use - 1) & 1u, ab)) return false;
          ++vf;
          mbar_arrive_expect_tx(&vfull[s], C::V_SLOT);
          uint8_t* dst = smem + C::OFF_V + s * C::V_SLOT;
          if (DA_BOUNDS_V(b < p.B && h < p.H, key0))  // (a box past n reads zeros)
            for (int bx = 0; bx < C::VBOX; ++bx)
              tma_load_4d(dst + bx * C::VKEYS * 128, &p.tm_v, &vfull[s], bx * 128, h,
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
    // Descriptors, loop bounds and accumulator addresses have to be known to be the same in the whole
    // warp (broadcast from lane 0, as they come from loaded lengths), and what moves from tile to tile
    // is one 32-bit word of each descriptor: an MMA whose operands were computed per lane between two
    // MMAs took 110-170 cycles to issue instead of 40.
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    uint32_t g = 0;       // tiles so far
    uint32_t slot = 0, phase = 0;  // of the ring
    TreeWalk w = walk_begin(p, count, start);
    for (uint32_t k = 0; ok && __shfl_sync(0xffffffffu, w.rem, 0) > 0; ++k) {
      const int seg = __shfl_sync(0xffffffffu, walk_seg(w), 0);
      if (warp == 1) {
        const uint64_t dk0 = sdesc_rows<C::KROW>(smem_u32(smem + C::OFF_K), 16);
        const uint64_t dq0 = sdesc_rows<C::KROW>(smem_u32(smem + C::OFF_Q), 16);
        ok = waitp(q_full, k & 1u);
        for (int i = 0; ok && i < seg; ++i, ++g) {
          const uint32_t s = g % C::NBUF;
          if (g >= C::NBUF && !waitp(&s_free[s], (g / C::NBUF - 1) & 1u)) ok = false;
#pragma unroll
          for (int m = 0; m < C::NMAP_K; ++m) {
            if (ok && !waitp(&kfull[slot], phase)) ok = false;
            if (!ok) break;
            const uint32_t d = tm + C::TM_S + s * C::SCOLS + m * 2 * TP;
            const uint32_t koff = slot * (C::K_SLOT >> 4);
#pragma unroll
            for (int st = 0; st < C::QK_STEPS; ++st) {
              const uint64_t a = desc_at(dk0, koff + ((st * 32) >> 4));
              const uint64_t bd = desc_at(dq0, (m * 2 * TP * C::KROW + st * 32) >> 4);
              mma_ss_f8_elect(d, a, bd, C::IDESC_QK, st > 0 ? 1u : 0u);
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
        const uint64_t dp0 = sdesc_rows<C::PROW>(smem_u32(smem + C::OFF_P), 16);
        const uint64_t dt0 = sdesc_rows<64>(smem_u32(smem + C::OFF_P + BN * C::PROW), 16);  // (P3APART: one stream)
        for (int i = 0; ok && i < seg; ++i, ++g) {
          const uint32_t st = stream_of(g);
          if (!waitp(&p_ready[st], number_of(g) & 1u)) ok = false;
          const uint32_t poff = st * (C::P_BYTES >> 4);
          const uint32_t again = i >= C::NSTREAM ? 1u : 0u;
#pragma unroll
          for (int part = 0; part < C::VF; ++part) {
            if (ok && !waitp(&vfull[slot], phase)) ok = false;
            if (!ok) break;
            const uint32_t voff = slot * (C::V_SLOT >> 4);
            constexpr int KS = 32;  // keys of an MMA
#pragma unroll
            for (int mt = 0; mt < C::NMT; ++mt) {
              const uint32_t d = tm + C::TM_O + (st * C::NMT + mt) * C::PCOLS;
#pragma unroll
              for (int kk = 0; kk < C::VKEYS / KS; ++kk) {
                // V^T: 128 channels are one box
                const uint64_t a = desc_at(dv0, voff + ((mt * C::VKEYS * 128 + kk * KS * 128) >> 4));
                const uint64_t bd = desc_at(dp0, poff + (((part * C::VKEYS + kk * KS) * C::PROW) >> 4));
                mma_ss_f8_elect(d, a, bd, C::IDESC_PV, (part > 0 || kk > 0) ? 1u : again);
                if constexpr (C::P3APART)
                  mma_ss_f8_elect(d, a, desc_at(dt0, ((part * C::VKEYS + kk * KS) * C::P3ROW) >> 4), C::IDESC_P3, 1u);
              }
            }
            tc_commit_elect(&vempty[slot]);
            if (++slot == NV) {
              slot = 0;
              phase ^= 1u;
            }
          }
          if (ok) tc_commit_elect(&pv_done[st]);
        }
      }
      walk_next(p, groups, w, seg);
    }
    tc_commit_elect(&drained[warp - 1]);
    if (*ab.flag) mbar_wait_drain(&drained[warp - 1], 0, kWaitBudgetCycles);
    __syncwarp();
  } else if (warp >= 4) {
    // =============================================================== softmax
    const int wq = warp & 3, wg = (warp - 4) >> 2;  // lane quarter (keys 32 wq .. of a tile), warpgroup
    constexpr bool BOTH = TP == 8;                     // the thread's 16 columns are both maps' 8
    const uint32_t stream = TP == 8 ? wg : TP == 16 ? wg >> 1 : 0;
    const int map = TP == 8 ? 0 : TP == 16 ? (wg & 1) : (wg >> 1);
    const int c0 = TP == 32 ? 16 * (wg & 1) : 0;         // first column of the map
    auto row_of = [&](int c) { return BOTH ? (c & 7) : c0 + c; };      // the thread's column c: its row,
    auto map_of = [&](int c) { return BOTH ? (c >> 3) : map; };        // its map
    const int key = 32 * wq + lane;                      // of the tile
    const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    const int ti = threadIdx.x - 128, nth = C::NSOFT * 32;           // among the softmax threads
    const int si = ti % (C::NARR * 32), nst = C::NARR * 32;            // among the stream's
    const int own = lane % NC;                           // the column this lane reduces
    float* xm = reinterpret_cast<float*>(smem + C::OFF_XM) + wg * 64;
    float* ac = reinterpret_cast<float*>(smem + C::OFF_AC) + wg * 16;
    const float top = kTreeRoom8Log2 + kTreeRescale8Log2;
    uint32_t g0 = 0;  // the segment's first tile
    TreeWalk w = walk_begin(p, count, start);
    // (an aborted CTA walks on: every wait then returns at once, and no warp misses a named barrier)
    for (uint32_t k = 0; w.rem > 0; ++k) {
      const int seg = walk_seg(w);
      const int hm = walk_unit(p, w), h = hm / p.mt, mtile = hm - h * p.mt;
      const int first = static_cast<int>((stream - g0) % C::NSTREAM);  // this stream's first tile of the segment
      // this thread's key and value scales of tile i of the segment
      const size_t srow = (static_cast<size_t>(w.b) * p.H + h) * p.n;
      const float* krow = ((map && !V2) ? p.k2_scales : p.k1_scales) + srow;
      const float* krow2 = (BOTH && !V2) ? p.k2_scales + srow : nullptr;
      const float* vrow = p.v_scales + srow;
      float ks_next = 0.f, ks2_next = 0.f, vs_next = 0.f;
      auto fetch_scales = [&](int i) {
        const int j = (w.t + i) * BN + key;
        const bool in = i < seg && j < w.len.end;
        ks_next = in ? krow[j] : 0.f;
        if (BOTH && !V2) ks2_next = in ? krow2[j] : 0.f;
        vs_next = in ? vrow[j] : 0.f;
      };
      fetch_scales(first);
      // ---- the segment's queries, once the previous segment's last score MMAs are done with theirs
      if (g0 > 0) {
        mbar_wait(&s_full[(g0 - 1) % C::NBUF], ((g0 - 1) / C::NBUF) & 1u, ab);
        __syncwarp();
      }
      const int pair0 = mtile * p.ppt, npair = min(p.ppt, p.pairs - pair0);
      unsigned long long* see = reinterpret_cast<unsigned long long*>(smem + C::OFF_SEE) + (k & 1u) * 32;
      float* qs = reinterpret_cast<float*>(smem + C::OFF_QS) + (k & 1u) * 64;
      float* qm = reinterpret_cast<float*>(smem + C::OFF_QM) + (k & 1u) * 64;
      constexpr int NCH = D / 8;  // 16-byte chunks of a bf16 query row
      auto query_chunk = [&](int i, int& m, int& r, int& ch) {  // chunk i of the rows' chunks: its map, row and place
        ch = i % NCH;
        const int rr = i / NCH;
        m = rr >= p.R;
        r = rr - m * p.R;
        const int pj = r / p.T, tj = r - pj * p.T;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (i < 2 * p.R * NCH && pj < npair && tj < w.len.nt) {
          const size_t at = static_cast<size_t>(w.b) * p.T + tj;
          const __nv_bfloat16* src = V2 ? p.q1 + (at * (2 * p.pairs * p.H) + 2 * (h * p.pairs + pair0 + pj) + m) * D
                                        : (m ? p.q2 : p.q1) + (at * p.H + h) * D;
          x = reinterpret_cast<const uint4*>(src)[ch];
        }
        return x;
      };
      const int nchunk = 2 * p.R * NCH;
      for (int i0 = 0; i0 < nchunk; i0 += nth) {  // the rows' largest magnitudes (NCH lanes a row)
        int m, r, ch;
        const uint4 x = query_chunk(i0 + ti, m, r, ch);
        const uint32_t u[4] = {x.x, x.y, x.z, x.w};
        float amax = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(u[e] << 16)), fabsf(__uint_as_float(u[e] & 0xffff0000u))));
#pragma unroll
        for (int o = 1; o < NCH; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (ch == 0 && i0 + ti < nchunk) qm[32 * m + r] = amax;
      }
      if (ti < 32) see[ti] = ti < p.R ? tree_sees(p, w.b, ti % p.T, w.len) : 0ull;
      // columns with a token, and their references
      auto live_col = [&](int c) {
        const int r = row_of(c), pj = r / p.T;
        return r < p.R && pj < npair && r - pj * p.T < w.len.nt;
      };
      const bool live = live_col(own);
      bool def = !live;  // this lane's column has a reference
      float ref = 0.f;
      if (wq == 0 && lane < NC) ac[own] = live ? 0.f : kTreeDead;
      named_bar_sync(5, nth);
      float rc = p.scale_log2;
      bool alike = true;  // the query rows share one power of two
      // Every row has its largest magnitude scaled into [128, 256); its two e4m3 terms are then exact
      // for elements down to 2^-10 of it.  Rows within a factor of eight of the largest take the
      // largest one's scale (exact down to 2^-7 of their own), which then is a constant of the tile.
      float big = 0.f, small = INFINITY;
      if (lane < p.R) {
        const float x0 = qm[lane], x1 = qm[32 + lane];
        big = fmaxf(x0, x1);
        small = fminf(x0 > 0.f ? x0 : INFINITY, x1 > 0.f ? x1 : INFINITY);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
        small = fminf(small, __shfl_xor_sync(0xffffffffu, small, o));
      }
      alike = small * 8.f >= big;
      const int all = e4m3_shift(big);
      for (int i = ti; i < nchunk; i += nth) {
        int m, r, ch;
        const uint4 x = query_chunk(i, m, r, ch);
        const int sh = alike ? all : e4m3_shift(qm[32 * m + r]);
        uint2 hi, lo;
        split_e4m3x8(x, sh, hi, lo);
        uint8_t* q = smem + C::OFF_Q + 8 * (ch & 1);
        *reinterpret_cast<uint2*>(q + swizzled<C::KROW>((2 * m) * TP + r, ch >> 1)) = hi;
        *reinterpret_cast<uint2*>(q + swizzled<C::KROW>((2 * m + 1) * TP + r, ch >> 1)) = lo;
        if (ch == 0) qs[32 * m + r] = __int_as_float((127 - sh) << 23);
      }
      if (alike) rc *= __int_as_float((127 - all) << 23);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
      named_bar_sync(5, nth);  // (qs)
      bool open = named_bar_any(1 + wg, !def);

      uint64_t l2[NC / 2];
#pragma unroll
      for (int c = 0; c < NC / 2; ++c) l2[c] = 0;
      bool any = false;     // the stream has had a tile of this segment
      uint32_t ready = 0;   // an early look at the next tile's barrier
      for (int i = first; i < seg; i += C::NSTREAM) {
        const uint32_t g = g0 + i, s = g % C::NBUF, nb = number_of(g);
        const int key0 = (w.t + i) * BN, j = key0 + key;
        const bool special = key0 + BN > w.len.L;  // the tile reaches into the drafted keys or past them
        float rk = rc, rk_b = rc, vs = 1.f, lv = 0.f;
        // A value scale that is not finite makes its row NaN: for everybody, or, for a drafted row,
        // for the tokens that see it (poison, and weightless).  The log2 the reference goes by is at
        // least kTreeLeastValueLog2, so that the sum of weights stays below fp32's end.
        rk *= ks_next;
        rk_b *= V2 ? ks_next : ks2_next;
        vs = vs_next;
        lv = fmaxf(__log2f(vs), kTreeLeastValueLog2);
        if (!(fabsf(vs) < INFINITY)) {
          vs = __uint_as_float(0x7fffffffu);
          lv = kTreeLeastValueLog2;
          if (j >= w.len.L) {
            atomicOr(&poison[k % 3], 1ull << (j - w.len.L));
            vs = 0.f;
          }
        }
        vs *= kTreeValueMult;
        fetch_scales(i + C::NSTREAM);
        if (!ready) mbar_wait(&s_full[s], (g / C::NBUF) & 1u, ab);
        __syncwarp();
        tc_fence_after();
        // (looked at now, needed when the weights are: a wait costs some 200 cycles even when it is over)
        const uint32_t pv_over = nb > 0 ? mbar_test(&pv_done[stream], (nb - 1) & 1u) : 1u;
        float x[NC];
        {
          const uint32_t ts = tl + C::TM_S + s * C::SCOLS;
          if constexpr (TP == 32) {
            uint32_t hi[16], lo[16];
            tmem_ld16(ts + map * 2 * TP + c0, hi);
            tmem_ld16(ts + map * 2 * TP + TP + c0, lo);
            tmem_ld_wait16x2(hi, lo);
#pragma unroll
            for (int c = 0; c < NC; ++c) x[c] = __uint_as_float(hi[c]) + __uint_as_float(lo[c]);
          } else {
            uint32_t raw[32];  // [map][term][8], or [term][16] of one map
            tmem_load(ts + map * 2 * TP, raw);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              const int a = BOTH ? (c >> 3) * 16 + (c & 7) : c;
              x[c] = __uint_as_float(raw[a]) + __uint_as_float(raw[a + TP]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[s]);
        if (!alike) {
#pragma unroll
          for (int c = 0; c < NC; ++c) x[c] *= qs[32 * map_of(c) + row_of(c)];
        }
        // ---- scores, less the references
        float pm = -INFINITY;
#pragma unroll
        for (int c = 0; c < NC; c += 4) {
          const float4 a = *reinterpret_cast<const float4*>(ac + c);
          const float rr = (BOTH && c >= 8) ? rk_b : rk;
          const uint64_t rk2 = f2pack(rr, rr);
          f2unpack(fma2(f2pack(x[c], x[c + 1]), rk2, f2pack(a.x, a.y)), x[c], x[c + 1]);
          f2unpack(fma2(f2pack(x[c + 2], x[c + 3]), rk2, f2pack(a.z, a.w)), x[c + 2], x[c + 3]);
          pm = max3(pm, x[c], x[c + 1]);
          pm = max3(pm, x[c + 2], x[c + 3]);
        }
        if (special && j >= w.len.L) {  // a drafted key, or none: hide it from who does not see it
          const int u = j - w.len.L;
          pm = -INFINITY;
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            if (j >= w.len.end || !((see[row_of(c)] >> u) & 1ull)) x[c] = -INFINITY;
            pm = fmaxf(pm, x[c]);
          }
        }
        float f = 1.f;     // what the reference of this lane's column rises by, as a factor on its O^T,
        bool fix = false;  // if there is some
        if (named_bar_any(1 + wg, open || pm + lv > top)) {
          // ---- new references: column maxima over the tile's keys
          float y[NC];
#pragma unroll
          for (int c = 0; c < NC; ++c) y[c] = x[c] + lv;
          const float mine = lanes_reduce<NC>(y, lane, [](float a, float b) { return fmaxf(a, b); });
          if (lane < NC) xm[wq * 16 + lane] = mine;
          named_bar_sync(1 + wg, 128);
          const float cm = fmaxf(fmaxf(xm[own], xm[16 + own]), fmaxf(xm[32 + own], xm[48 + own])) - kTreeRoom8Log2;
          float up = 0.f;  // how much the reference rises
          if (live && cm > -INFINITY && (!def || cm > 0.f)) up = cm;
          f = def ? ex2(-up) : 1.f;  // (before the first reference there is nothing to scale)
          ref += up;
          def = def || cm > -INFINITY;
          if (wq == 0 && lane < NC && live) ac[own] = -ref;
#pragma unroll
          for (int c = 0; c < NC; c += 2) {
            x[c] -= __shfl_sync(0xffffffffu, up, c);
            x[c + 1] -= __shfl_sync(0xffffffffu, up, c + 1);
            l2[c >> 1] = mul2(l2[c >> 1], f2pack(__shfl_sync(0xffffffffu, f, c), __shfl_sync(0xffffffffu, f, c + 1)));
          }
          fix = any;
          open = named_bar_any(1 + wg, !def);  // (and the references are in place)
        }
        // ---- weights
        uint32_t pk[3][NC / 4];
#pragma unroll
        for (int c = 0; c < NC; c += 4) {
          const uint64_t ea = f2pack(ex2(x[c]), ex2(x[c + 1])), eb = f2pack(ex2(x[c + 2]), ex2(x[c + 3]));
          l2[c >> 1] = add2(l2[c >> 1], ea);
          l2[(c >> 1) + 1] = add2(l2[(c >> 1) + 1], eb);
          float v0, v1, v2, v3;
          const uint64_t vs2 = f2pack(vs, vs);
          f2unpack(mul2(ea, vs2), v0, v1);
          f2unpack(mul2(eb, vs2), v2, v3);
          three_e5m2x4(v0, v1, v2, v3, pk[0][c >> 2], pk[1][c >> 2], pk[2][c >> 2]);
        }
        if (!pv_over) mbar_wait(&pv_done[stream], (nb - 1) & 1u, ab);  // the P tile's last reader
        __syncwarp();
        any = true;
        {
          // chunks of 16 bytes of the key's row: the columns' first terms, then all columns' second and third
          uint8_t* pt = smem + C::OFF_P + stream * C::P_BYTES;
          const int ch = (map * TP + c0) / 16;
#pragma unroll
          for (int e = 0; e < 3; ++e) {
            const uint32_t at = (C::P3APART && e == 2) ? BN * C::PROW + swizzled<64>(key, ch)
                                                       : swizzled<C::PROW>(key, ch + e * (COLS / 16));
            *reinterpret_cast<uint4*>(pt + at) = make_uint4(pk[e][0], pk[e][1], pk[e][2], pk[e][3]);
          }
        }
        if (fix) {  // (last of all, when the previous P V is over: V1 d64 B8 H16, 32 tokens, 286 us and 267 this way)
          tc_fence_after();
#pragma unroll 1
          for (int q = 0; q < C::PTERMS * C::NMT; ++q) {  // [128 channels][term]
            const uint32_t to = tl + C::TM_O + (stream * C::NMT * C::PCOLS + q * COLS) + map * TP + c0;
            uint32_t o[NC];
            tmem_load(to, o);
#pragma unroll
            for (int c = 0; c < NC; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * __shfl_sync(0xffffffffu, f, c));
            tmem_st16(to, o);
          }
          tmem_st_wait();
        }
        if (special) {
          // (the previous tile's P V first: the slots' earlier fills are then all used, so that the
          // parities below mean this tile's)
          if (g > 0) mbar_wait(&pv_done[stream_of(g - 1)], number_of(g - 1) & 1u, ab);
#pragma unroll 1
          for (int part = 0; part < C::VF; ++part) {
            const uint32_t fl = C::VF * g + part;
            const int kp = key0 + part * C::VKEYS;
            if (w.len.L - kp >= C::VKEYS) continue;
            mbar_wait(&vfull[fl % NV], (fl / NV) & 1u, ab);
            __syncwarp();
            clean_values<C::VKEYS, C::VROW, true>(smem + C::OFF_V + (fl % NV) * C::V_SLOT, kp, w.len, &poison[k % 3], si, nst);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready[stream]);
        const uint32_t gn = g + C::NSTREAM;
        ready = i + C::NSTREAM < seg ? mbar_test(&s_full[gn % C::NBUF], (gn / C::NBUF) & 1u) : 0u;
        ready = __all_sync(0xffffffffu, ready);
      }
      // ---- the stream's partial state of the segment
      const long long group = static_cast<long long>(w.b) * groups + w.grp;
      float* state = tree_state(p, group, static_cast<int>(blockIdx.x) / p.team, static_cast<int>(blockIdx.x) % p.team, DV);
      const bool here = DA_BOUNDS_V(group < static_cast<long long>(p.B) * groups && p.R <= TP, group);
      float l[NC];
#pragma unroll
      for (int c = 0; c < NC; c += 2) f2unpack(l2[c >> 1], l[c], l[c + 1]);
      const float lw = lanes_reduce<NC>(l, lane, [](float a, float b) { return a + b; });
      if (lane < NC) xm[wq * 16 + lane] = lw;
      if (any) {
        const uint32_t gl = g0 + first + (seg - 1 - first) / C::NSTREAM * C::NSTREAM;
        mbar_wait(&pv_done[stream], number_of(gl) & 1u, ab);
        __syncwarp();
        tc_fence_after();
      }
      named_bar_sync(1 + wg, 128);
      if (wq == 0 && lane < NC && row_of(own) < p.R && here) {
        float ls = (xm[lane] + xm[16 + lane]) + (xm[32 + lane] + xm[48 + lane]);
        if (see[row_of(own)] & poison[k % 3]) ls = __uint_as_float(0x7fffffffu);
        const int sm = static_cast<int>(stream) * 2 + map_of(own);
        reinterpret_cast<float2*>(state)[sm * p.R + row_of(own)] = make_float2((def && live) ? ref : -INFINITY, ls);
      }
      if (any) {
        float* o = state + tree_state_o(p.R, p.subs) + 32 * wq + lane;
#pragma unroll 1
        for (int mt = 0; mt < C::NMT; ++mt) {
          const uint32_t to = tl + C::TM_O + (stream * C::NMT + mt) * C::PCOLS + map * TP + c0;
          uint32_t a[NC], b[NC];
          tmem_load(to, a);
#pragma unroll
          for (int e = 1; e < C::PTERMS; ++e) {
            tmem_load(to + e * COLS, b);
#pragma unroll
            for (int c = 0; c < NC; ++c) a[c] = __float_as_uint(__uint_as_float(a[c]) + __uint_as_float(b[c]));
          }
#pragma unroll
          for (int c = 0; c < NC; ++c)
            if (row_of(c) < p.R && here)
              o[(static_cast<size_t>(stream * 2 + map_of(c)) * p.R + row_of(c)) * DV + 128 * mt] = __uint_as_float(a[c]);
        }
        tc_fence_before();
      }
      named_bar_sync(1 + wg, 128);  // (xm)
      if (ti == 0) poison[(k + 2) % 3] = 0;
      g0 += static_cast<uint32_t>(seg);
      walk_next(p, groups, w, seg);
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

template <int D, bool V2, int TP>
cudaError_t launch_tree_cols(const TreeParams& p, cudaStream_t s) {
  using C = TreeColsCfg<D, V2, TP>;
  return launch_tree_pair<C::DV, V2>(tree_cols_kernel<D, V2, TP>, C::NTHREADS, C::SMEM_BYTES, 1.f / kTreeValueMult, p, s);
}

}  // namespace da
