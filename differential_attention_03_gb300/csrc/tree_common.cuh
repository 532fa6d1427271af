// What the two tree-decode kernels share: the line of key tiles, descriptors,
// e5m2 weights in three terms, and the kernel that merges their partial states.
//
// A partial state holds, for each of `subs` subsets of a CTA's keys of a unit
// and each map: (reference maximum, sum of weights) of the R rows, then O of
// the rows, unnormalised: float2 [subs][2][R], then, from a 32-byte boundary,
// float [subs][2][R][DV].
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "cache_params.h"
#include "ptx.cuh"

#undef DA_BOUNDS_FILE
#define DA_BOUNDS_FILE 12

namespace da {

constexpr float kTreeRescaleLog2 = 8.f;    // bf16 P: how far a score may exceed the reference maximum
// e4m3 values: the reference sits at 2^8 on the scale that P is split at, 2^3 below the largest contribution
// when it is set, and moves once one is 2^4 above that: 2^15 at most (e5m2 ends at 57344 = 2^15.8).
constexpr float kTreeRoom8Log2 = 3.f, kTreeRescale8Log2 = 4.f;
constexpr float kTreeValueMult = 256.f;    // (a scale is at most 2^128 / 448: no overflow)
constexpr float kTreeLeastValueLog2 = -96.f;  // what a value row counts at least for the reference (sums stay below 2^128)

// A sequence's committed keys, its drafted tokens, the end of its keys and its tiles.
struct TreeLen {
  int L, nt, end, tiles;
};
__device__ __forceinline__ TreeLen tree_len(const TreeParams& p, int b) {
  TreeLen x;
  x.L = max(0, min(p.lens ? p.lens[b] : p.n - p.T, p.n));
  x.nt = max(0, min(p.ntok ? p.ntok[b] : p.T, p.T));
  x.end = min(p.n, x.L + x.nt);
  x.tiles = (x.end + 127) >> 7;
  return x;
}

// a / b of non-negative numbers; 64-bit division only where it is needed.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
  return a / b;
}

// Tiles of all sequences before `upto` and of all of them, per unit of a
// sequence (each has the same units), by the whole CTA; scratch of 2 * 32 + 2
// long longs.  Every thread returns with (before, total).
__device__ __forceinline__ void tree_prefix(const TreeParams& p, int upto, long long* scratch, long long& before,
                                            long long& total) {
  if (p.B <= 32) {  // (every warp for itself, without a barrier)
    const int lane = threadIdx.x & 31, x = lane < p.B ? tree_len(p, lane).tiles : 0;
    before = __reduce_add_sync(0xffffffffu, lane < upto ? x : 0);
    total = __reduce_add_sync(0xffffffffu, x);
    return;
  }
  long long a = 0, t = 0;
  for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
    const int x = tree_len(p, b).tiles;
    t += x;
    if (b < upto) a += x;
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, x);
    t += __shfl_xor_sync(0xffffffffu, t, x);
  }
  const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) {
    scratch[warp] = a;
    scratch[32 + warp] = t;
  }
  __syncthreads();
  before = total = 0;
  for (int w = 0; w < nw; ++w) {
    before += scratch[w];
    total += scratch[32 + w];
  }
  __syncthreads();
}

// Two floats as e4m3 codes (a in the low byte) and what the codes stand for.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 e4m3x2_value(uint32_t c) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c), __NV_E4M3)));
}

// Four non-negative floats of at most 2^15.8 as three e5m2 terms each.  An
// e5m2 code is the upper byte of an f16, so a term is that byte, and what is
// left an exact f16 subtraction; the last term rounds.  The three are within
// 2^-8.8 of the value, or 2^-16.8 absolute: 2^-28 of the largest contribution,
// so that weights too small to be told from zero do not add up to anything
// over any cache that fits the GPU.  (Two e4m3 terms hold the same bits, but
// end at 2^-17 of the largest: of 27000 keys 12 powers of e below one, 15 % of
// the sum was lost.)  Integer and f16 work, as the 8-bit conversion instructions
// take about 16 issue cycles each.  A NaN stays a NaN.
__device__ __forceinline__ void three_e5m2x4(float a, float b, float c, float d, uint32_t& t1, uint32_t& t2, uint32_t& t3) {
  uint32_t f0, f1;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(f0) : "f"(b), "f"(a));
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(f1) : "f"(d), "f"(c));
  t1 = __byte_perm(f0, f1, 0x7531);
  asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(f0) : "r"(f0 & 0xff00ff00u));
  asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(f1) : "r"(f1 & 0xff00ff00u));
  t2 = __byte_perm(f0, f1, 0x7531);
  asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(f0) : "r"(f0 & 0xff00ff00u));
  asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(f1) : "r"(f1 & 0xff00ff00u));
  t3 = __byte_perm(f0 + 0x00800080u, f1 + 0x00800080u, 0x7531);  // (a NaN, 0x7fff, does not carry into its neighbour)
}

// Instruction descriptor bits of kind::f8f6f4: A, or B, is e5m2 instead of e4m3.
constexpr uint32_t kIdescA5 = 1u << 7, kIdescB5 = 1u << 10;

// 32 lanes x 4 columns store.
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t (&v)[4]) {
  if (!DA_TMEM_OK(taddr, 4)) return;
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3])
               : "memory");
}

// Matrix descriptor over rows of `width` bytes (128, 64 or 32: the swizzle).
template <int WIDTH>
__device__ __forceinline__ uint64_t sdesc_rows(uint32_t saddr, uint32_t lbo) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>(((8 * WIDTH) >> 4) & 0x3FFFu) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(WIDTH == 128 ? 2 : WIDTH == 64 ? 4 : 6) << 61;
  return d;
}

// The descriptor `units` of 16 bytes further on (its address stays inside shared memory: no carry).
__device__ __forceinline__ uint64_t desc_at(uint64_t d, uint32_t units) {
  return (d & 0xffffffff00000000ull) | (static_cast<uint32_t>(d) + units);
}

// 16-byte chunk `ch` of row `row` in such a layout.
template <int WIDTH>
__device__ __forceinline__ uint32_t swizzled(int row, int ch) {
  const int x = WIDTH == 128 ? (ch ^ (row & 7)) : WIDTH == 64 ? (ch ^ ((row >> 1) & 3)) : (ch ^ ((row >> 2) & 1));
  return static_cast<uint32_t>(row * WIDTH + (x << 4));
}

// True in every thread of the 128 on named barrier `id` if `v` is true in any.
__device__ __forceinline__ bool named_bar_any(uint32_t id, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v)), "r"(id)
      : "memory");
  return r != 0;
}

// Waits for this thread's outstanding tcgen05.ld into 16 registers (tied in).
__device__ __forceinline__ void tmem_ld_wait16(uint32_t (&a)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]), "+r"(a[6]), "+r"(a[7]),
                 "+r"(a[8]), "+r"(a[9]), "+r"(a[10]), "+r"(a[11]), "+r"(a[12]), "+r"(a[13]), "+r"(a[14]), "+r"(a[15])
               :
               : "memory");
}

__device__ __forceinline__ void tmem_load(uint32_t t, uint32_t (&r)[32]) {
  tmem_ld32(t, r);
  tmem_ld_wait(r);
}
__device__ __forceinline__ void tmem_load(uint32_t t, uint32_t (&r)[16]) {
  tmem_ld16(t, r);
  tmem_ld_wait16(r);
}
__device__ __forceinline__ void tmem_store(uint32_t t, const uint32_t (&r)[32]) { tmem_st32(t, r); }
__device__ __forceinline__ void tmem_store(uint32_t t, const uint32_t (&r)[16]) { tmem_st16(t, r); }

// The line of tiles: sequence by sequence, group of `team` units by group,
// tile by tile; each team of CTAs takes a contiguous range of it, and CTA
// `lane` of the team unit `lane` of each group.  Neighbouring units are
// neighbouring heads, whose rows of a token lie side by side: read at about
// the same time they make whole DRAM bursts of rows as short as 64 bytes
// (e4m3 V1 d64 B8 H16 n32768: 199 us, each CTA for itself 240).
//
// The range of the CTA's team, from its place among the teams and the line's length W: the first tile and how many.
__device__ __forceinline__ int team_range(const TreeParams& p, long long W, long long& lo) {
  const long long G = min(static_cast<long long>(p.teams), max(W, 1ll));  // no team between two with tiles is without
  const int team = static_cast<int>(blockIdx.x) / p.team;
  lo = quotient(W * team, G);
  return team < G ? static_cast<int>(quotient(W * (team + 1), G) - lo) : 0;
}

// The sequence among 32 (this lane's has `mine` tiles of all groups) that tile `lo` falls in, whose place
// is written by its lane: sequence, group, tile.  `base`: tiles before the 32; returns with those after.
__device__ __forceinline__ bool find_start(int b, long long mine, int groups, long long lo, long long& base, int* start) {
  long long incl = mine;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, x);
    if ((threadIdx.x & 31) >= x) incl += y;
  }
  const long long excl = base + incl - mine;
  const bool here = lo >= excl && lo < excl + mine;
  if (here) {
    const int tiles = static_cast<int>(quotient(mine, groups));
    const int grp = static_cast<int>(quotient(lo - excl, tiles));
    start[0] = b;
    start[1] = grp;
    start[2] = static_cast<int>(lo - excl - static_cast<long long>(grp) * tiles);
  }
  base += __shfl_sync(0xffffffffu, incl, 31);
  return __any_sync(0xffffffffu, here);
}

// The CTA's range, by the whole CTA: start[0..2] are the sequence, its group and tile, start[3] the number
// of tiles; `scratch` 64 long longs, `start` four ints in shared memory.  The caller synchronises the CTA
// before it reads them.  Up to 32 sequences are warp 2's alone (one load a lane, no barrier: every CTA
// begins with this).
__device__ __forceinline__ void tree_range(const TreeParams& p, int groups, long long* scratch, int* start) {
  const int lane = threadIdx.x & 31;
  if (p.B <= 32) {
    if (threadIdx.x >> 5 != 2) return;
    const int tiles = lane < p.B ? tree_len(p, lane).tiles : 0;
    const int total = __reduce_add_sync(0xffffffffu, tiles);
    long long lo, base = 0;
    const int count = team_range(p, static_cast<long long>(total) * groups, lo);
    if (lane == 0) start[3] = count;
    if (count > 0) find_start(lane, static_cast<long long>(tiles) * groups, groups, lo, base, start);
    return;
  }
  long long before, total, lo, base = 0;
  tree_prefix(p, 0, scratch, before, total);
  const int count = team_range(p, total * groups, lo);
  if (threadIdx.x == 0) start[3] = count;
  if (threadIdx.x < 32 && count > 0)
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const long long mine = (b0 + lane < p.B) ? static_cast<long long>(tree_len(p, b0 + lane).tiles) * groups : 0;
      if (find_start(b0 + lane, mine, groups, lo, base, start)) break;
    }
}

// Every role walks the same segments: the CTA's tiles of one unit each.
struct TreeWalk {
  int b, grp, t, rem;  // sequence, group of units, tile, tiles left
  TreeLen len;
};
__device__ __forceinline__ TreeWalk walk_begin(const TreeParams& p, int count, const int* start) {
  TreeWalk w;
  w.rem = count;
  w.b = count > 0 ? start[0] : 0;
  w.grp = count > 0 ? start[1] : 0;
  w.t = count > 0 ? start[2] : 0;
  if (count > 0) w.len = tree_len(p, w.b);
  return w;
}
__device__ __forceinline__ int walk_seg(const TreeWalk& w) { return min(w.rem, w.len.tiles - w.t); }
__device__ __forceinline__ void walk_next(const TreeParams& p, int groups, TreeWalk& w, int seg) {
  w.rem -= seg;
  w.t = 0;
  if (w.rem <= 0) return;
  if (++w.grp == groups) {
    w.grp = 0;
    do {
      ++w.b;
      w.len = tree_len(p, w.b);
    } while (w.len.tiles == 0 && w.b + 1 < p.B);
  }
}

// The CTA's unit of its sequence in the group, and its partial state of it.
__device__ __forceinline__ int walk_unit(const TreeParams& p, const TreeWalk& w) {
  return w.grp * p.team + static_cast<int>(blockIdx.x) % p.team;
}
__device__ __forceinline__ float* tree_state(const TreeParams& p, long long group, int team, int lane, int dv) {
  return p.ws + (static_cast<size_t>(group + team) * p.team + lane) * tree_state_floats(p.R, p.subs, dv);
}

// Eight floats to a 32-byte boundary: a whole sector, where a lane has a row of its own.
__device__ __forceinline__ void store8(float* at, const uint32_t* x) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]),
               "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}

// What token `tok` of sequence b sees of the drafts in the cache.
__device__ __forceinline__ unsigned long long tree_sees(const TreeParams& p, int b, int tok, const TreeLen& len) {
  const int nt = len.end - len.L;
  unsigned long long s = p.mask ? p.mask[b * p.mask_sb + tok] : ((2ull << tok) - 1ull);
  if (nt < 64) s &= (1ull << nt) - 1ull;
  return s;
}

// Rows of a value tile's slot (VKEYS keys of VROW bytes, boxes of 128 bytes)
// that some token must not see, by `n` threads (this one is `i`): rows past
// the drafted ones hold whatever the cache held and are zeroed; a drafted row
// with a NaN or an infinity is zeroed and remembered in `poison`, so that it
// reaches only the tokens that see it.  kp: key of the slot's first row.
template <int VKEYS, int VROW, bool V8>
__device__ __forceinline__ void clean_values(uint8_t* slot, int kp, const TreeLen& len, unsigned long long* poison, int i,
                                             int n) {
  constexpr int RCH = VROW / 16;  // 16-byte chunks of a row
  const int r0 = max(0, len.L - kp);
  for (int x = i; x < (VKEYS - r0) * RCH; x += n) {
    const int vr = r0 + x / RCH, vc = x % RCH;
    uint4* at = reinterpret_cast<uint4*>(slot + (vc >> 3) * (VKEYS * 128) + vr * 128 + ((vc & 7) << 4));
    bool zero = kp + vr >= len.end;
    if (!zero) {
      const uint4 u = *at;
      const uint32_t v4[4] = {u.x, u.y, u.z, u.w};
      bool bad = false;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (V8) {  // e4m3: 0x7f, 0xff
          const uint32_t t7 = (v4[e] & 0x7f7f7f7fu) + 0x01010101u;
          bad |= (t7 & 0x80808080u) != 0;
        } else {
          bad |= (v4[e] & 0x7f80u) == 0x7f80u || (v4[e] & 0x7f800000u) == 0x7f800000u;
        }
      }
      if (bad) {
        atomicOr(poison, 1ull << (kp + vr - len.L));
        zero = true;
      }
    }
    if (zero) *at = make_uint4(0, 0, 0, 0);
  }
}

// The power of two (as its exponent) that puts a row's largest magnitude in [128, 256).
__device__ __forceinline__ int e4m3_shift(float amax) {
  const int bexp = (__float_as_int(amax) >> 23) & 0xff;
  return (amax > 0.f) ? max(-120, min(100, 134 - bexp)) : 0;  // (-120: the largest finite rows)
}

// Eight bf16 values times 2^sh as two e4m3 terms each.  An infinity becomes a NaN (the conversion would
// make it 448): its row's scores are infinite or NaN in the formula, so its softmax is NaN.
__device__ __forceinline__ void split_e4m3x8(const uint4& x, int sh, uint2& hi, uint2& lo) {
  const float mul = __int_as_float((127 + sh) << 23);
  const uint32_t u[4] = {x.x, x.y, x.z, x.w};
  uint32_t h[2], l[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    uint32_t a[2], b[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const float x0 = __uint_as_float(u[2 * e + z] << 16), x1 = __uint_as_float(u[2 * e + z] & 0xffff0000u);
      const float v0 = fmaf(x0, mul, x0 * 0.f), v1 = fmaf(x1, mul, x1 * 0.f);  // (infinity times 0)
      a[z] = e4m3x2(v0, v1);
      const float2 back = e4m3x2_value(a[z]);
      b[z] = e4m3x2(v0 - back.x, v1 - back.y);
    }
    h[e] = a[0] | (a[1] << 16);
    l[e] = b[0] | (b[1] << 16);
  }
  hi = make_uint2(h[0], h[1]);
  lo = make_uint2(l[0], l[1]);
}

// Merges the partial states of a unit and finishes one row a CTA.  A handful
// of dependent loads is all that it does, so it is built for latency: the
// states' maxima and sums by as many threads at once, and every state's O with
// nothing to wait for, the first ones beside the maxima.  The threads are
// kTreeMergers groups, each of which takes every kTreeMergers-th state, two
// channels a thread.  (Both kernels of a call of 5 tokens over 512 keys of 8
// V1 heads, d64, replayed from a graph: 14.3 us with one state after the other
// and the CTA's range found by all its warps, 9.7 us this way; one head's 512
// tiles on every SM: 140 and 30 us.  Four groups take 22 us there, but 85
// instead of 77 where 768 rows want to be on the SMs at once.)
constexpr int kTreeMaxStates = 160 * 4;  // of a unit: one a team and subset
constexpr int kTreeMergers = 2;

template <int DV, bool V2>
__global__ void __launch_bounds__(kTreeMergers * DV / 2) tree_combine_kernel(const __grid_constant__ TreeParams p, float o_mult) {
  grid_dep_launch_dependents();
  grid_dep_wait();
  constexpr int NG = DV / 2, NT = kTreeMergers * NG, NW = NT / 32;
  __shared__ long long scratch[64];
  __shared__ float2 ml[2][kTreeMaxStates];  // maximum and sum, then weight and whether there is one
  __shared__ float red[4 * NW + NG / 32];
  __shared__ float2 part[kTreeMergers][NG];
  const int HM = p.H * p.mt;
  const int unit = static_cast<int>(blockIdx.x) / p.R, r = static_cast<int>(blockIdx.x) - unit * p.R;
  const int b = unit / HM, hm = unit - b * HM;
  const int h = hm / p.mt, mtile = hm - h * p.mt;
  const int pj = r / p.T, t = r - pj * p.T;
  const int pair = mtile * p.ppt + pj;
  if (pair >= p.pairs) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = threadIdx.x / NG, i2 = threadIdx.x % NG;  // this thread's states and channels
  // what does not depend on the states, on its way
  const size_t orow = V2 ? (static_cast<size_t>(b) * p.T + t) * (p.H * p.pairs) + h * p.pairs + pair
                         : (static_cast<size_t>(b) * p.T + t) * p.H + h;
  const float coef = V2 ? 1.f / (1.f + expf(-p.lam_logits[b * p.sb + t * p.st + h * p.pairs + pair])) : *p.lambda;
  float2 g = make_float2(1.f, 1.f);
  if (!V2 && p.gamma) g = make_float2(p.gamma[2 * i2], p.gamma[2 * i2 + 1]);
  const TreeLen len = tree_len(p, b);
  long long before, total;
  tree_prefix(p, b, scratch, before, total);
  const bool any = len.tiles > 0 && t < len.nt;  // (the same for the whole CTA)
  float2 y = make_float2(0.f, 0.f);
  if (any) {
    const int groups = HM / p.team, grp = hm / p.team;
    const long long W = total * groups;
    const long long G = min(static_cast<long long>(p.teams), W);
    const long long s = before * groups + static_cast<long long>(grp) * len.tiles, e = s + len.tiles - 1;
    const int c0 = static_cast<int>(quotient((s + 1) * G - 1, W)), c1 = static_cast<int>(quotient((e + 1) * G - 1, W));
    const float* src = tree_state(p, static_cast<long long>(b) * groups + grp, c0, hm % p.team, DV);
    const size_t sf = p.team * tree_state_floats(p.R, p.subs, DV);
    const int n = (c1 - c0 + 1) * p.subs, shift = p.subs >> 1;  // (subs: 1, 2 or 4)
    const float* o = src + tree_state_o(p.R, p.subs) + static_cast<size_t>(r) * DV + 2 * i2;
    constexpr int U = 4;
    float2 v[U][2];
    auto load = [&](int k0) {  // O of states k0, k0 + kTreeMergers, ... (what is not there is not used)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * kTreeMergers;
        if (k >= n) continue;
        const float* at = o + (k >> shift) * sf + static_cast<size_t>(2 * (k & (p.subs - 1))) * p.R * DV;
        v[u][0] = *reinterpret_cast<const float2*>(at);
        v[u][1] = *reinterpret_cast<const float2*>(at + static_cast<size_t>(p.R) * DV);
      }
    };
    load(group);
    float M[2] = {-INFINITY, -INFINITY}, L[2] = {0.f, 0.f};
    for (int i = threadIdx.x; i < 2 * n; i += NT) {
      const int m = i >= n, k = i - m * n;
      const float2 x = reinterpret_cast<const float2*>(src + (k >> shift) * sf)[(2 * (k & (p.subs - 1)) + m) * p.R + r];
      ml[m][k] = x;
      M[0] = m ? M[0] : fmaxf(M[0], x.x);
      M[1] = m ? fmaxf(M[1], x.x) : M[1];
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) M[m] = fmaxf(M[m], __shfl_xor_sync(0xffffffffu, M[m], x));
      if (lane == 0) red[m * NW + warp] = M[m];
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      M[m] = red[m * NW];
#pragma unroll
      for (int i = 1; i < NW; ++i) M[m] = fmaxf(M[m], red[m * NW + i]);
    }
    for (int i = threadIdx.x; i < 2 * n; i += NT) {
      const int m = i >= n, k = i - m * n;
      const float2 x = ml[m][k];
      const bool none = x.x == -INFINITY && x.y == 0.f;  // nothing seen in this state
      const float top = m ? M[1] : M[0];
      const float w = none ? 0.f : (x.x == top) ? 1.f : ex2(x.x - top);
      ml[m][k].x = none ? -1.f : w;  // (a weight of -1: O is not there)
      const float lw = none ? 0.f : x.y * w;
      L[0] += m ? 0.f : lw;
      L[1] += m ? lw : 0.f;
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) L[m] += __shfl_xor_sync(0xffffffffu, L[m], x);
      if (lane == 0) red[(2 + m) * NW + warp] = L[m];
    }
    __syncthreads();
    float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    for (int k0 = group; k0 < n; k0 += U * kTreeMergers) {
      if (k0 != group) load(k0);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * kTreeMergers;
        if (k >= n) continue;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const float w = ml[m][k].x;
          if (w == -1.f) continue;
          acc[m].x = fmaf(v[u][m].x, w, acc[m].x);
          acc[m].y = fmaf(v[u][m].y, w, acc[m].y);
        }
      }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      L[m] = 0.f;
#pragma unroll
      for (int i = 0; i < NW; ++i) L[m] += red[(2 + m) * NW + i];
    }
    const float w1 = (L[0] == 0.f) ? 0.f : o_mult / L[0], w2 = (L[1] == 0.f) ? 0.f : -coef * o_mult / L[1];
    y = make_float2(acc[0].x * w1 + acc[1].x * w2, acc[0].y * w1 + acc[1].y * w2);
    part[group][i2] = y;
    __syncthreads();
    if (group == 0) {
#pragma unroll
      for (int i = 1; i < kTreeMergers; ++i) {
        y.x += part[i][i2].x;
        y.y += part[i][i2].y;
      }
    }
  }
  float rinv = 1.f;
  if (!V2) {
    if (group == 0) {
      float ss = y.x * y.x + y.y * y.y;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, x);
      if (lane == 0) red[4 * NW + warp] = ss;
    }
    __syncthreads();
    float tot = 0.f;
#pragma unroll
    for (int i = 0; i < NG / 32; ++i) tot += red[4 * NW + i];
    rinv = p.norm_mult * rsqrtf(tot * (1.f / DV) + p.eps);
  }
  if (group == 0 && DA_BOUNDS_V(b < p.B && t < p.T && h < p.H, t))
    reinterpret_cast<uint32_t*>(p.out + orow * DV)[i2] = pack_bf16x2(y.x * rinv * g.x, y.y * rinv * g.y);
}

// Launches a tree kernel and the merge, each a programmatic dependent of what precedes it.
template <int DV, bool V2>
cudaError_t launch_tree_pair(void (*kern)(TreeParams), int threads, int smem_bytes, float o_mult, const TreeParams& p,
                             cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.teams * p.team), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem_bytes);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, p);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cc = {};
  cc.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(p.B) * p.H * p.mt * p.R), 1, 1);
  cc.blockDim = dim3(kTreeMergers * DV / 2, 1, 1);
  cc.stream = s;
  cc.attrs = attr;
  cc.numAttrs = 1;
  return cudaLaunchKernelEx(&cc, tree_combine_kernel<DV, V2>, p, o_mult);
}

}  // namespace da
