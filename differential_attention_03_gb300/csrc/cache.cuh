// Rotary positions, the cache append (rotary, quantisation and the write in
// one pass) and the move of an accepted path inside the cache.
//
// Rotary: y = m R(pos theta) x on the first `rot` channels of each head, the
// rest unchanged.  A pair's angle is kept as a fraction of a turn, 2^64 units
// to the turn: position x units wraps modulo 2^64, which is the exact range
// reduction at any distance (in fp32 the product pos theta alone is off by
// 0.03 rad at position 10^6).  The remainder to the nearest quarter turn goes
// to sinpi / cospi in fp32.  One sine and cosine serve a position's every
// head and tensor: a CTA computes them once for its tokens into shared
// memory.  The backward pass is the rotation by the negative angle with the
// same m.
//
// Append: W / 16 lanes per (token, head) row, 16 channels a lane; a warp's rows
// are of one kind (queries, keys or values of one cache format), so that it
// runs one kind's code, and a row's largest magnitude is a few shuffles.
//
// All three kernels read and write each value once.  Measured: rotary fp32 V1
// d128, 8192 tokens of 48 heads (403 MB) 61 us, 6.55 TB/s, which is HBM's rate;
// bf16 V1 d64, 8192 tokens of 64 heads (134 MB) 25 us, 5.4 TB/s; append V2 d128
// fp8, 8002 padded tokens of 32 + 16 + 16 heads (173 MB) 37 us, 4.6 TB/s: a warp
// holds 32 bytes a lane in flight and nothing of its next rows while it rotates,
// finds the maximum and converts (some 200 instructions per 32 x 16 values, 57 %
// of the issue slots; staging a CTA's rows in shared memory by asynchronous
// copies took 10 % off 30000 unpadded tokens, but put 10 % on these, whose copies
// wait for ntok, and on a few hundred; two values an instruction in the maximum
// and the scaling changed nothing).  8000 unpadded tokens: V2 d128 bf16 45 us
// (262 MB), fp8k 44, fp8 46 (230 MB); V1 d64 H16 35, 34, 35.  A token 2.1 us one
// call after the other, the launch and two dependent loads; 300 tokens 3 to 4.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "cache_params.h"
#include "ptx.cuh"

#undef DA_BOUNDS_FILE
#define DA_BOUNDS_FILE 11

namespace da {

// m cos and m sin of pos * turns * 2^-64 turns.
__device__ __forceinline__ float2 rope_cos_sin(unsigned long long turns, int pos, float m) {
  const unsigned long long ph = turns * static_cast<unsigned long long>(static_cast<long long>(pos));
  const unsigned quarter = static_cast<unsigned>((ph + (1ull << 61)) >> 62);  // nearest quarter turn, mod 4
  const long long rem = static_cast<long long>(ph - (static_cast<unsigned long long>(quarter) << 62));
  float s, c;
  sincospif(static_cast<float>(rem) * 0x1p-63f, &s, &c);  // |remainder| <= an eighth of a turn
  const float cc = (quarter & 1) ? ((quarter & 2) ? s : -s) : ((quarter & 2) ? -c : c);
  const float ss = (quarter & 1) ? ((quarter & 2) ? -c : c) : ((quarter & 2) ? -s : s);
  return make_float2(cc * m, ss * m);
}

__device__ __forceinline__ void unpack_bf16x8(const uint4& w, float (&f)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// 16 bytes of a row as floats, and back.
template <bool F32>
struct RopeVec;
template <>
struct RopeVec<false> {
  static constexpr int N = 8, ES = 2;
  static __device__ __forceinline__ void get(const uint4& w, float (&f)[8]) { unpack_bf16x8(w, f); }
  static __device__ __forceinline__ uint4 put(const float (&f)[8]) { return pack_bf16x8(f); }
};
template <>
struct RopeVec<true> {
  static constexpr int N = 4, ES = 4;
  static __device__ __forceinline__ void get(const uint4& w, float (&f)[4]) {
    f[0] = __uint_as_float(w.x);
    f[1] = __uint_as_float(w.y);
    f[2] = __uint_as_float(w.z);
    f[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

// Element c of a row, as a float and back.
template <bool F32>
__device__ __forceinline__ float rope_get(const uint8_t* row, int c) {
  if constexpr (F32) return reinterpret_cast<const float*>(row)[c];
  else return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row)[c]);
}
template <bool F32>
__device__ __forceinline__ void rope_put(uint8_t* row, int c, float x) {
  if constexpr (F32) reinterpret_cast<float*>(row)[c] = x;
  else reinterpret_cast<__nv_bfloat16*>(row)[c] = __float2bfloat16_rn(x);
}

// a / n by the host's magic number 2^32 / n + 1 (0: plain division), exact while a times the
// magic number's excess stays below 2^32 / n: the host sees to it.
__device__ __forceinline__ unsigned fast_div(unsigned a, unsigned n, unsigned magic) {
  return magic ? __umulhi(a, magic) : a / n;
}

// VEC: 16-byte accesses (rows and the rotated part whole vectors); else
// element by element, for odd widths.  A work item is the two vectors (or
// elements) of one rotation, or one vector (element) to copy.
template <bool F32, bool VEC>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  grid_dep_launch_dependents();
  grid_dep_wait();
  using V = RopeVec<F32>;
  constexpr int N = V::N;
  __shared__ __align__(16) float2 cs[kRopeMaxTokens * 64];
  const int half = p.rope.rot >> 1;
  const long long tok0 = static_cast<long long>(blockIdx.x) * p.tokens_per_cta;
  const long long tokens = static_cast<long long>(p.B) * p.n;
  const int nt = static_cast<int>(min(static_cast<long long>(p.tokens_per_cta), tokens - tok0));
  for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
    const int t = i / half, f = i - t * half;
    const int pos = p.pos ? p.pos[tok0 + t] : static_cast<int>((tok0 + t) % p.n);
    float2 a = rope_cos_sin(p.rope.turns[f], pos, p.rope.mult);
    if (p.inverse) a.y = -a.y;
    cs[i] = a;
  }
  __syncthreads();
  // items of one head: `ri` rotations, then copies of the channels past rot
  const int step = VEC ? N : 1;
  const int ri = VEC ? (p.rope.inter ? p.rope.rot / N : half / N) : half;
  const int per_head = ri + (p.copy ? (p.d - p.rope.rot) / step : 0);
  const unsigned per_tok = static_cast<unsigned>(p.head_sum * per_head);
  const unsigned total = static_cast<unsigned>(nt) * per_tok;
  // Two items a turn, their loads before either is worked on.
  constexpr int U = 2;
  const unsigned stride = gridDim.y * kRopeThreads;
  for (unsigned i0 = blockIdx.y * kRopeThreads + threadIdx.x; i0 < total; i0 += U * stride) {
    const uint8_t* src[U];
    uint8_t* dst[U];
    const float2* a[U];
    int ca[U];
    bool turn[U], go[U];
    uint4 wa[U], wb[U];
    float x0[U], x1[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const unsigned i = i0 + u * stride;
      go[u] = i < total;
      const unsigned ii = go[u] ? i : 0u;
      const unsigned t = fast_div(ii, per_tok, p.magic_tok);
      const unsigned j = ii - t * per_tok;
      unsigned hh = fast_div(j, static_cast<unsigned>(per_head), p.magic_head);
      const int l = static_cast<int>(j - hh * per_head);
      int ten = 0;
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (ten == k && k + 1 < p.count && hh >= static_cast<unsigned>(p.heads[k])) {
          hh -= p.heads[k];
          ten = k + 1;
        }
      const size_t row = (static_cast<size_t>(tok0 + t) * p.heads[ten] + hh) * p.d;
      turn[u] = l < ri;
      go[u] = go[u] && (turn[u] || p.x[ten] != p.out[ten]) &&
              DA_BOUNDS_V(tok0 + t < tokens && hh < static_cast<unsigned>(p.heads[ten]), tok0 + t);
      a[u] = cs + t * half;
      src[u] = static_cast<const uint8_t*>(p.x[ten]) + row * V::ES;
      dst[u] = static_cast<uint8_t*>(p.out[ten]) + row * V::ES;
      if constexpr (VEC) {
        ca[u] = turn[u] ? l * N : p.rope.rot + (l - ri) * N;
        if (go[u]) {
          wa[u] = reinterpret_cast<const uint4*>(src[u])[ca[u] / N];
          if (turn[u] && !p.rope.inter) wb[u] = reinterpret_cast<const uint4*>(src[u])[(ca[u] + half) / N];
        }
      } else {
        ca[u] = turn[u] ? (p.rope.inter ? 2 * l : l) : p.rope.rot + (l - ri);
        a[u] += turn[u] ? l : 0;
        if (go[u]) {
          x0[u] = rope_get<F32>(src[u], ca[u]);
          if (turn[u]) x1[u] = rope_get<F32>(src[u], ca[u] + (p.rope.inter ? 1 : half));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!go[u]) continue;
      if constexpr (VEC) {
        uint4* out = reinterpret_cast<uint4*>(dst[u]);
        if (!turn[u]) {
          out[ca[u] / N] = wa[u];
          continue;
        }
        float xa[N];
        V::get(wa[u], xa);
        if (p.rope.inter) {
          float y[N];
#pragma unroll
          for (int e = 0; e < N; e += 2) {
            const float2 c = a[u][(ca[u] + e) >> 1];
            y[e] = xa[e] * c.x - xa[e + 1] * c.y;
            y[e + 1] = xa[e + 1] * c.x + xa[e] * c.y;
          }
          out[ca[u] / N] = V::put(y);
        } else {
          float xb[N], ya[N], yb[N];
          V::get(wb[u], xb);
#pragma unroll
          for (int e = 0; e < N; e += 2) {
            const float4 c = *reinterpret_cast<const float4*>(a[u] + ca[u] + e);
            ya[e] = xa[e] * c.x - xb[e] * c.y;
            yb[e] = xb[e] * c.x + xa[e] * c.y;
            ya[e + 1] = xa[e + 1] * c.z - xb[e + 1] * c.w;
            yb[e + 1] = xb[e + 1] * c.z + xa[e + 1] * c.w;
          }
          out[ca[u] / N] = V::put(ya);
          out[(ca[u] + half) / N] = V::put(yb);
        }
      } else {
        if (!turn[u]) {
          rope_put<F32>(dst[u], ca[u], x0[u]);
          continue;
        }
        const float2 c = *a[u];
        rope_put<F32>(dst[u], ca[u], x0[u] * c.x - x1[u] * c.y);
        rope_put<F32>(dst[u], ca[u] + (p.rope.inter ? 1 : half), x1[u] * c.x + x0[u] * c.y);
      }
    }
  }
}

// ----------------------------------------------------------------- append
__device__ __forceinline__ uint2 pack_e4m3x8(const float (&f)[8], float mul) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo =
        __nv_cvt_float2_to_fp8x2(make_float2(f[4 * h] * mul, f[4 * h + 1] * mul), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi =
        __nv_cvt_float2_to_fp8x2(make_float2(f[4 * h + 2] * mul, f[4 * h + 3] * mul), __NV_SATFINITE, __NV_E4M3);
    w[h] = lo | (hi << 16);
  }
  return make_uint2(w[0], w[1]);
}

// Largest magnitude of 8 numbers and m; a NaN stays one.
__device__ __forceinline__ float amax8(float m, const float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(m), "f"(fabsf(x[e])));
  return m;
}

enum AppendKind { kAppendQuery, kAppendKey, kAppendValue };

struct AppendShared {
  float cos[kAppendMaxTokens * 64], sin[kAppendMaxTokens * 64];  // [token][frequency]
  int at[kAppendMaxTokens];    // cache row of the token, -1: not written
  int seq[kAppendMaxTokens];   // its sequence
  int live[kAppendMaxTokens];  // whether the sequence has it
};

// The lane's channels of a rotated row in place: xa from channel ca, xb from cb.
__device__ __forceinline__ void append_turn(const AppendParams& p, const AppendShared& sh, bool halves, int t, int l,
                                            int ca, int cb, const __nv_bfloat16* src, float (&xa)[8], float (&xb)[8]) {
  const int rot = p.rope.rot, half = rot >> 1;
  const float *cs = sh.cos + t * half, *sn = sh.sin + t * half;
  if (halves) {
    if (16 * l >= rot) return;
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      const float4 c = *reinterpret_cast<const float4*>(cs + ca + e), s = *reinterpret_cast<const float4*>(sn + ca + e);
#pragma unroll
      for (int k = 0; k < 4; k += 2) {  // two pairs an instruction
        const float c0 = k ? c.z : c.x, c1 = k ? c.w : c.y, s0 = k ? s.z : s.x, s1 = k ? s.w : s.y;
        const uint64_t c2 = f2pack(c0, c1), s2 = f2pack(s0, s1), n2 = f2pack(-s0, -s1);
        const uint64_t x = f2pack(xa[e + k], xa[e + k + 1]), z = f2pack(xb[e + k], xb[e + k + 1]);
        f2unpack(fma2(z, n2, mul2(x, c2)), xa[e + k], xa[e + k + 1]);
        f2unpack(fma2(x, s2, mul2(z, c2)), xb[e + k], xb[e + k + 1]);
      }
    }
  } else if (p.rope.inter) {
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      const int ch = 16 * l + e;
      if (ch >= rot) break;
      const float c = cs[ch >> 1], s = sn[ch >> 1];
      float &u = e < 8 ? xa[e & 7] : xb[e & 7], &w = e < 8 ? xa[(e + 1) & 7] : xb[(e + 1) & 7];
      const float x0 = u, x1 = w;
      u = x0 * c - x1 * s;
      w = x1 * c + x0 * s;
    }
  } else {  // halves that do not end on 8 channels: the partner comes by its own load
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int ch = 16 * l + e;
      if (ch >= rot) break;
      const bool lo = ch < half;
      const float c = cs[lo ? ch : ch - half], s = sn[lo ? ch : ch - half];
      const float other = __bfloat162float(src[lo ? ch + half : ch - half]);
      float& x = e < 8 ? xa[e & 7] : xb[e & 7];
      x = lo ? x * c - other * s : x * c + other * s;
    }
  }
}

// 32 lanes' rows of one kind: W / 16 lanes a row, 16 channels a lane.
template <int W, int KIND, int FMT>
__device__ __forceinline__ void append_rows(const AppendParams& p, const AppendShared& sh, int tok0, int row0, int rows,
                                            bool halves) {
  constexpr int GL = W / 16;
  constexpr bool kCodes = KIND != kAppendQuery && FMT != kCacheBf16 && !(KIND == kAppendValue && FMT == kCacheFp8k);
  const int lane = threadIdx.x & 31, l = lane % GL;
  const int i = min(row0 + lane / GL, rows - 1);
  bool need = row0 + lane / GL < rows;
  const int heads = KIND == kAppendQuery ? p.Hq : p.H;
  const int per_tok = KIND == kAppendQuery ? p.nq * p.Hq : KIND == kAppendKey ? p.nk * p.H : p.H;
  const int t = static_cast<int>(fast_div(i, per_tok, p.magic[KIND]));
  const int j = i - t * per_tok;
  const bool second = KIND != kAppendValue && j >= heads;
  const int h = j - (second ? heads : 0);
  const __nv_bfloat16* src = KIND == kAppendValue ? p.v
                             : KIND == kAppendKey ? (second ? p.k[1] : p.k[0]) : (second ? p.q[1] : p.q[0]);
  const size_t in_row = static_cast<size_t>(tok0 + t) * heads + h;
  src += in_row * W;
  const int at = sh.at[t], b = sh.seq[t];
  const bool padding = KIND == kAppendQuery && !sh.live[t];
  if (KIND != kAppendQuery) need = need && at >= 0;
  // a lane of the rotated part holds both channels of its pairs
  const bool split = KIND != kAppendValue && halves && 16 * l < p.rope.rot;
  const int ca = split ? 8 * l : 16 * l, cb = split ? (p.rope.rot >> 1) + 8 * l : 16 * l + 8;
  uint4 wa = make_uint4(0, 0, 0, 0), wb = wa;
  if (need && !padding) {
    wa = *reinterpret_cast<const uint4*>(src + ca);
    wb = *reinterpret_cast<const uint4*>(src + cb);
  }
  if constexpr (KIND == kAppendQuery) {  // (padding tokens get zero queries)
    need = need && DA_BOUNDS_V(tok0 + t < p.B * p.T && h < p.Hq, t);
    if (p.rope.rot > 0 && !padding) {
      float xa[8], xb[8];
      unpack_bf16x8(wa, xa);
      unpack_bf16x8(wb, xb);
      append_turn(p, sh, halves, t, l, ca, cb, src, xa, xb);
      wa = pack_bf16x8(xa);
      wb = pack_bf16x8(xb);
    }
    if (need) {
      __nv_bfloat16* dst = (second ? p.qo[1] : p.qo[0]) + in_row * W;
      *reinterpret_cast<uint4*>(dst + ca) = wa;
      *reinterpret_cast<uint4*>(dst + cb) = wb;
    }
  } else {
    need = need && DA_BOUNDS_V(b < p.B && at < p.n && h < p.H, at);
    const size_t out_row = (static_cast<size_t>(b) * p.n + (at < 0 ? 0 : at)) * p.H + h;
    void* cache = KIND == kAppendValue ? p.vc : (second ? p.kc[1] : p.kc[0]);
    float xa[8], xb[8];
    const bool turned = KIND == kAppendKey && p.rope.rot > 0;
    if (kCodes || turned) {
      unpack_bf16x8(wa, xa);
      unpack_bf16x8(wb, xb);
      if (turned && need) append_turn(p, sh, halves, t, l, ca, cb, src, xa, xb);
    }
    if constexpr (kCodes) {
      float mul = second ? p.kinv[1] : p.kinv[0], scale = 0.f;
      if constexpr (FMT == kCacheFp8) {
        float m = amax8(amax8(0.f, xa), xb);
#pragma unroll
        for (int x = 1; x < GL; x <<= 1) {
          const float o = __shfl_xor_sync(0xffffffffu, m, x);
          asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(m), "f"(o));
        }
        // A row below 448 * 2^-126 keeps the smallest normal scale.  448 / top as 1.75 / (top 2^-8),
        // whose reciprocal neither over- nor underflows; one ulp off it at most.
        const float top = m < 448.f * 0x1p-126f ? 448.f * 0x1p-126f : m;
        scale = m == 0.f ? 0.f : top * (1.f / 448.f);
        float r;
        asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(top * 0x1p-8f));
        mul = 1.75f * r;
      }
      if (need) {
        uint8_t* dst = static_cast<uint8_t*>(cache) + out_row * W;
        const uint2 ea = pack_e4m3x8(xa, mul), eb = pack_e4m3x8(xb, mul);
        if (!split) {
          *reinterpret_cast<uint4*>(dst + ca) = make_uint4(ea.x, ea.y, eb.x, eb.y);
        } else {
          *reinterpret_cast<uint2*>(dst + ca) = ea;
          *reinterpret_cast<uint2*>(dst + cb) = eb;
        }
        if (FMT == kCacheFp8 && l == 0) {
          float* sc = KIND == kAppendValue ? p.vs : (second ? p.ks[1] : p.ks[0]);
          sc[(static_cast<size_t>(b) * p.H + h) * p.n + at] = scale;
        }
      }
    } else {
      if (turned) {
        wa = pack_bf16x8(xa);
        wb = pack_bf16x8(xb);
      }
      if (need) {
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(cache) + out_row * W;
        *reinterpret_cast<uint4*>(dst + ca) = wa;
        *reinterpret_cast<uint4*>(dst + cb) = wb;
      }
    }
  }
}

// A CTA's tokens' query, key and value rows, each kind in warps' loads of 32 / (W / 16) rows, so that a
// warp runs one kind's code.
template <int D, int DV, int FMT>
__global__ void __launch_bounds__(kAppendThreads, 4) cache_append_kernel(const __grid_constant__ AppendParams p) {
  grid_dep_launch_dependents();
  grid_dep_wait();
  __shared__ __align__(16) AppendShared sh;
  const int half = p.rope.rot >> 1;
  const int tok0 = static_cast<int>(blockIdx.x) * p.tokens_per_cta;
  const int nt = min(p.tokens_per_cta, p.B * p.T - tok0);
  for (int i = threadIdx.x; i < nt * max(half, 1); i += kAppendThreads) {
    const int t = half ? i / half : i, f = half ? i - t * half : 0;
    const int b = (tok0 + t) / p.T, tt = tok0 + t - b * p.T;
    const long long row = static_cast<long long>(p.lens ? p.lens[b] : 0) + tt;
    if (f == 0) {
      const bool lv = tt < (p.ntok ? p.ntok[b] : p.T);
      sh.live[t] = lv;
      sh.seq[t] = b;
      sh.at[t] = (lv && row >= 0 && row < p.n) ? static_cast<int>(row) : -1;
    }
    if (half) {
      const float2 c = rope_cos_sin(p.rope.turns[f], p.pos ? p.pos[tok0 + t] : static_cast<int>(row), p.rope.mult);
      sh.cos[i] = c.x;
      sh.sin[i] = c.y;
    }
  }
  __syncthreads();
  const bool halves = !p.rope.inter && half > 0 && (p.rope.rot & 15) == 0;
  constexpr int RK = 32 / (D / 16), RV = 32 / (DV / 16);  // rows a warp
  const int rq = nt * p.nq * p.Hq, rk = nt * p.nk * p.H, rv = nt * p.H;
  const int cq = (rq + RK - 1) / RK, ck = cq + (rk + RK - 1) / RK, cv = ck + (rv + RV - 1) / RV;
  constexpr int NW = kAppendThreads / 32;
  for (int c = blockIdx.y * NW + (threadIdx.x >> 5); c < cv; c += gridDim.y * NW) {
    if (c < cq) append_rows<D, kAppendQuery, FMT>(p, sh, tok0, c * RK, rq, halves);
    else if (c < ck) append_rows<D, kAppendKey, FMT>(p, sh, tok0, (c - cq) * RK, rk, halves);
    else append_rows<DV, kAppendValue, FMT>(p, sh, tok0, (c - ck) * RV, rv, halves);
  }
}

// ----------------------------------------------------------------- keep
// Rows lens[b] + path[b][i] of every cache tensor move to rows lens[b] + i, i
// in order.  A path ascends, so path[i] >= i: no row is written before it has
// been read, and each thread owns one 16-byte column of every row (its reads
// of a batch come before its writes).
__global__ void __launch_bounds__(kKeepThreads) cache_keep_kernel(const __grid_constant__ KeepParams p) {
  grid_dep_launch_dependents();
  grid_dep_wait();
  __shared__ int path[kKeepMaxPath];
  __shared__ int kept;
  const int b = blockIdx.x;
  const int len = p.lens[b];
  if (threadIdx.x < 32) {  // the longest ascending start of the path that stays inside the cache
    const int lane = threadIdx.x;
    int bad = kKeepMaxPath;
    const int want = min(p.nkeep[b], p.A);
    for (int i = lane; i < want; i += 32) {
      const int x = p.path[static_cast<size_t>(b) * p.A + i];
      const int before = i ? p.path[static_cast<size_t>(b) * p.A + i - 1] : -1;
      path[i] = x;
      if (x <= before || x >= kKeepMaxPath || static_cast<long long>(len) + x >= p.n) bad = min(bad, i);
    }
    bad = __reduce_min_sync(0xffffffffu, bad);
    if (lane == 0) {
      const int k = (len < 0) ? 0 : max(0, min(want, bad));
      kept = k;
      if (p.new_lens && blockIdx.y == 0) p.new_lens[b] = len + k;
    }
  }
  __syncthreads();
  const int k = kept;
  int first = 0;  // nodes that are in place already
  while (first < k && path[first] == first) ++first;
  if (first == k) return;
  const int step = gridDim.y * kKeepThreads, me = blockIdx.y * kKeepThreads + threadIdx.x;
  for (int ten = 0; ten < p.count; ++ten) {
    const size_t rb = static_cast<size_t>(p.row_bytes[ten]);
    uint8_t* base = static_cast<uint8_t*>(p.base[ten]) + (static_cast<size_t>(b) * p.n + len) * rb;
    for (int c = me; c < static_cast<int>(rb >> 4); c += step) {
      uint4* col = reinterpret_cast<uint4*>(base) + c;
      const size_t rs = rb >> 4;
      for (int i0 = first; i0 < k; i0 += 8) {
        uint4 w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (i0 + e < k) w[e] = col[rs * path[i0 + e]];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (i0 + e < k && DA_BOUNDS_V(len + i0 + e < p.n, i0 + e)) col[rs * (i0 + e)] = w[e];
      }
    }
    if (p.fmt == kCacheFp8)
      for (int h = me; h < p.H; h += step) {
        float* s = p.scales[ten] + (static_cast<size_t>(b) * p.H + h) * p.n + len;
        for (int i = first; i < k; ++i) s[i] = s[path[i]];
      }
  }
}

}  // namespace da
