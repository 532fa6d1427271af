// What the two tree-decode kernels share: the line of key tiles, descriptors,
// two-term e4m3 weights, and the kernel that merges their partial states.
//
// A partial state holds, for each of `subs` subsets of a CTA's keys of a unit
// and each map: (reference maximum, sum of weights) of the R rows, then O of
// the rows, unnormalised: float2 [subs][2][R], float [subs][2][R][DV].
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
constexpr float kTreeRescale8Log2 = 1.f;   // e4m3 P: the reference sits at 2^7, e4m3 ends at 448
constexpr float kTreeValueMult = 0.5f;     // 2^7, times two_e4m3x4's 2^-8

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

// Four non-negative floats, scaled to 2^-8 of what they stand for (at most
// 448 2^-8), as two e4m3 terms each: hi truncates, hi + lo is within 2^-8 of
// the value, or 2^-10 absolute, as a bf16 would be.  At that scale f16's
// exponent field is e4m3's, so a code is bits 7-13 of the f16: pairs of f16
// are shifted and masked as integers (the e4m3 conversion instructions take
// about 16 issue cycles each, and bounded the kernel: 372 us against 337 us
// at B8 H16 n32768 d64).  A NaN stays a NaN.
__device__ __forceinline__ void two_e4m3x4(float a, float b, float c, float d, uint32_t& hi, uint32_t& lo) {
  uint32_t f0, f1, r0, r1;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(f0) : "f"(b), "f"(a));
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(f1) : "f"(d), "f"(c));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r0) : "r"(f0), "r"(f0 & 0x7f807f80u));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r1) : "r"(f1), "r"(f1 & 0x7f807f80u));
  hi = __byte_perm(f0 << 1, f1 << 1, 0x7531);
  // (a NaN in one column must not carry into the next: its hi code says it already)
  lo = __byte_perm((r0 & 0x3fff3fffu) * 2 + 0x00800080u, (r1 & 0x3fff3fffu) * 2 + 0x00800080u, 0x7531);
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
// The CTA's range, by the whole CTA: its number of tiles; `scratch` 64 long longs, `start` three ints in shared memory.  The caller
// synchronises the CTA before it reads `start`.
__device__ __forceinline__ int tree_range(const TreeParams& p, int groups, long long* scratch, int* start) {
  long long before, total;
  tree_prefix(p, 0, scratch, before, total);
  const long long W = total * groups;
  const long long G = min(static_cast<long long>(p.teams), max(W, 1ll));  // no team between two with tiles is without
  const int team = static_cast<int>(blockIdx.x) / p.team;
  const long long lo = quotient(W * team, G), hi = quotient(W * (team + 1), G);
  const int count = team < G ? static_cast<int>(hi - lo) : 0;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x < 32 && count > 0) {  // the sequence that tile `lo` falls in: 32 sequences a step
    long long base = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const long long mine = (b0 + lane < p.B) ? static_cast<long long>(tree_len(p, b0 + lane).tiles) * groups : 0;
      long long incl = mine;
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, x);
        if (lane >= x) incl += y;
      }
      const long long excl = base + incl - mine;
      const bool here = lo >= excl && lo < excl + mine;
      if (here) {
        const int tiles = static_cast<int>(mine / groups);
        start[0] = b0 + lane;
        const int grp = static_cast<int>(quotient(lo - excl, tiles));
        start[1] = grp;
        start[2] = static_cast<int>(lo - excl - static_cast<long long>(grp) * tiles);
      }
      if (__any_sync(0xffffffffu, here)) break;
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  return count;
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
  return (amax > 0.f) ? max(-100, min(100, 134 - bexp)) : 0;
}

// Eight bf16 values times 2^sh as two e4m3 terms each.
__device__ __forceinline__ void split_e4m3x8(const uint4& x, int sh, uint2& hi, uint2& lo) {
  const float mul = __int_as_float((127 + sh) << 23);
  const uint32_t u[4] = {x.x, x.y, x.z, x.w};
  uint32_t h[2], l[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    uint32_t a[2], b[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const float v0 = __uint_as_float(u[2 * e + z] << 16) * mul;
      const float v1 = __uint_as_float(u[2 * e + z] & 0xffff0000u) * mul;
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

// Merges the partial states of a unit and finishes one row a CTA: two channels
// a thread.  A handful of dependent loads is all that it does, so it is built
// for latency: the states' maxima and sums by as many threads at once, then
// their weights, then every state's O with nothing to wait for in between
// (40 rows of 4 to 8 states: 14.4 us one state after the other, cold;
// 11 us this way).
constexpr int kTreeMaxStates = 160 * 4;  // of a unit: one a team and subset

template <int DV, bool V2>
__global__ void __launch_bounds__(DV / 2) tree_combine_kernel(const __grid_constant__ TreeParams p, float o_mult) {
  grid_dep_launch_dependents();
  grid_dep_wait();
  constexpr int NT = DV / 2;
  __shared__ long long scratch[64];
  __shared__ float2 ml[2][kTreeMaxStates];  // maximum and sum, then weight and whether there is one
  __shared__ float red[3 * NT / 32];
  const int HM = p.H * p.mt;
  const int unit = static_cast<int>(blockIdx.x) / p.R, r = static_cast<int>(blockIdx.x) - unit * p.R;
  const int b = unit / HM, hm = unit - b * HM;
  const int h = hm / p.mt, mtile = hm - h * p.mt;
  const int pj = r / p.T, t = r - pj * p.T;
  const int pair = mtile * p.ppt + pj;
  if (pair >= p.pairs) return;
  // what does not depend on the states, on its way
  const size_t orow = V2 ? (static_cast<size_t>(b) * p.T + t) * (p.H * p.pairs) + h * p.pairs + pair
                         : (static_cast<size_t>(b) * p.T + t) * p.H + h;
  const float coef = V2 ? 1.f / (1.f + expf(-p.lam_logits[b * p.sb + t * p.st + h * p.pairs + pair])) : *p.lambda;
  float2 g = make_float2(1.f, 1.f);
  if (!V2 && p.gamma) g = make_float2(p.gamma[2 * threadIdx.x], p.gamma[2 * threadIdx.x + 1]);
  const TreeLen len = tree_len(p, b);
  long long before, total;
  tree_prefix(p, b, scratch, before, total);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float y0 = 0.f, y1 = 0.f;
  if (len.tiles > 0 && t < len.nt) {  // (the same for the whole CTA)
    const int groups = HM / p.team, grp = hm / p.team;
    const long long W = total * groups;
    const long long G = min(static_cast<long long>(p.teams), W);
    const long long s = before * groups + static_cast<long long>(grp) * len.tiles, e = s + len.tiles - 1;
    const int c0 = static_cast<int>(quotient((s + 1) * G - 1, W)), c1 = static_cast<int>(quotient((e + 1) * G - 1, W));
    const float* src = tree_state(p, static_cast<long long>(b) * groups + grp, c0, hm % p.team, DV);
    const size_t sf = p.team * tree_state_floats(p.R, p.subs, DV);
    const int n = (c1 - c0 + 1) * p.subs;
    float M[2] = {-INFINITY, -INFINITY};
    for (int i = threadIdx.x; i < 2 * n; i += NT) {
      const int m = i >= n, k = i - m * n, c = k / p.subs, sub = k - c * p.subs;
      const float2 x = reinterpret_cast<const float2*>(src + c * sf)[(2 * sub + m) * p.R + r];
      ml[m][k] = x;
      M[m] = fmaxf(M[m], x.x);
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) M[m] = fmaxf(M[m], __shfl_xor_sync(0xffffffffu, M[m], x));
      if (lane == 0) red[m * (NT / 32) + warp] = M[m];
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      M[m] = red[m * (NT / 32)];
#pragma unroll
      for (int i = 1; i < NT / 32; ++i) M[m] = fmaxf(M[m], red[m * (NT / 32) + i]);
    }
    for (int i = threadIdx.x; i < 2 * n; i += NT) {
      const int m = i >= n, k = i - m * n;
      const float2 x = ml[m][k];
      const bool none = x.x == -INFINITY && x.y == 0.f;  // nothing seen in this state
      const float w = none ? 0.f : (x.x == M[m]) ? 1.f : ex2(x.x - M[m]);
      ml[m][k] = make_float2(none ? -1.f : w, none ? 0.f : x.y * w);  // (a weight of -1: O is not there)
    }
    __syncthreads();
    float L[2] = {0.f, 0.f}, a0[2] = {0.f, 0.f}, a1[2] = {0.f, 0.f};
    const float* o = src + p.subs * 4 * p.R + static_cast<size_t>(r) * DV;
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
      const int c = k / p.subs, sub = k - c * p.subs;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const float2 w = ml[m][k];
        float2 v = make_float2(0.f, 0.f);
        if (w.x != -1.f) v = reinterpret_cast<const float2*>(o + c * sf + static_cast<size_t>(2 * sub + m) * p.R * DV)[threadIdx.x];
        L[m] += w.y;
        a0[m] = fmaf(v.x, w.x, a0[m]);
        a1[m] = fmaf(v.y, w.x, a1[m]);
      }
    }
    const float w1 = (L[0] == 0.f) ? 0.f : o_mult / L[0], w2 = (L[1] == 0.f) ? 0.f : -coef * o_mult / L[1];
    y0 = a0[0] * w1 + a0[1] * w2;
    y1 = a1[0] * w1 + a1[1] * w2;
  }
  float rinv = 1.f;
  if (!V2) {
    float ss = y0 * y0 + y1 * y1;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, x);
    if (lane == 0) red[2 * (NT / 32) + warp] = ss;
    __syncthreads();
    float tot = 0.f;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) tot += red[2 * (NT / 32) + i];
    rinv = p.norm_mult * rsqrtf(tot * (1.f / DV) + p.eps);
  }
  if (DA_BOUNDS_V(b < p.B && t < p.T && h < p.H, t))
    reinterpret_cast<uint32_t*>(p.out + orow * DV)[threadIdx.x] = pack_bf16x2(y0 * rinv * g.x, y1 * rinv * g.y);
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
  cc.blockDim = dim3(DV / 2, 1, 1);
  cc.stream = s;
  cc.attrs = attr;
  cc.numAttrs = 1;
  return cudaLaunchKernelEx(&cc, tree_combine_kernel<DV, V2>, p, o_mult);
}

}  // namespace da
