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
// Append: one group of lanes per (token, head) row, 16 channels a lane; the
// row's largest magnitude is a few shuffles.  All three kernels read and
// write each value once and are bound by HBM, or by the launch when few.
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

// VEC: 16-byte accesses (rows and the rotated part whole vectors); else
// element by element, for odd widths.  A work item is the two vectors (or
// elements) of one rotation, or one vector (element) to copy.
template <bool F32, bool VEC>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  grid_dep_launch_dependents();
  grid_dep_wait();
  using V = RopeVec<F32>;
  constexpr int N = V::N;
  __shared__ float2 cs[kRopeMaxTokens * 64];
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
  const int per_tok = p.head_sum * per_head;
  const int total = nt * per_tok;
  for (int i = blockIdx.y * kRopeThreads + threadIdx.x; i < total; i += gridDim.y * kRopeThreads) {
    const int t = i / per_tok, j = i - t * per_tok;
    int hh = j / per_head;
    const int l = j - hh * per_head;
    int ten = 0;
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (ten == k && k + 1 < p.count && hh >= p.heads[k]) {
        hh -= p.heads[k];
        ten = k + 1;
      }
    const size_t row = (static_cast<size_t>(tok0 + t) * p.heads[ten] + hh) * p.d;
    const bool turn = l < ri;
    const bool inplace = p.x[ten] == p.out[ten];
    if (!turn && inplace) continue;
    const float2* a = cs + t * half;
    if (!DA_BOUNDS_V(tok0 + t < tokens && hh < p.heads[ten], tok0 + t)) continue;
    if constexpr (VEC) {
      const int ca = turn ? l * N : p.rope.rot + (l - ri) * N;
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.x[ten]) + row * V::ES);
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out[ten]) + row * V::ES);
      const uint4 wa = src[ca / N];
      if (!turn) {
        dst[ca / N] = wa;
        continue;
      }
      float xa[N];
      V::get(wa, xa);
      if (p.rope.inter) {
        float y[N];
#pragma unroll
        for (int e = 0; e < N; e += 2) {
          const float2 c = a[(ca + e) >> 1];
          y[e] = xa[e] * c.x - xa[e + 1] * c.y;
          y[e + 1] = xa[e + 1] * c.x + xa[e] * c.y;
        }
        dst[ca / N] = V::put(y);
      } else {
        float xb[N], ya[N], yb[N];
        V::get(src[(ca + half) / N], xb);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float2 c = a[ca + e];
          ya[e] = xa[e] * c.x - xb[e] * c.y;
          yb[e] = xb[e] * c.x + xa[e] * c.y;
        }
        dst[ca / N] = V::put(ya);
        dst[(ca + half) / N] = V::put(yb);
      }
    } else {
      const int c0 = turn ? (p.rope.inter ? 2 * l : l) : p.rope.rot + (l - ri);
      const int c1 = p.rope.inter ? c0 + 1 : c0 + half;
      if constexpr (F32) {
        const float* src = static_cast<const float*>(p.x[ten]) + row;
        float* dst = static_cast<float*>(p.out[ten]) + row;
        const float x0 = src[c0];
        if (!turn) {
          dst[c0] = x0;
          continue;
        }
        const float x1 = src[c1];
        const float2 c = a[l];
        dst[c0] = x0 * c.x - x1 * c.y;
        dst[c1] = x1 * c.x + x0 * c.y;
      } else {
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.x[ten]) + row;
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out[ten]) + row;
        if (!turn) {
          dst[c0] = src[c0];
          continue;
        }
        const float x0 = __bfloat162float(src[c0]), x1 = __bfloat162float(src[c1]);
        const float2 c = a[l];
        dst[c0] = __float2bfloat16_rn(x0 * c.x - x1 * c.y);
        dst[c1] = __float2bfloat16_rn(x1 * c.x + x0 * c.y);
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

// A row (token, tensor, head) is d / 16 (values: dv / 16) consecutive lanes of
// 16 channels each.  Order of a token's rows: queries, keys, values; every
// group starts at a multiple of its lanes (the host checks the widths).
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const __grid_constant__ AppendParams p) {
  grid_dep_launch_dependents();
  grid_dep_wait();
  __shared__ float2 cs[kAppendMaxTokens * 64];
  __shared__ int at[kAppendMaxTokens];   // cache row of the token, -1: not written
  __shared__ int live[kAppendMaxTokens];
  const int half = p.rope.rot >> 1;
  const long long tok0 = static_cast<long long>(blockIdx.x) * p.tokens_per_cta;
  const long long tokens = static_cast<long long>(p.B) * p.T;
  const int nt = static_cast<int>(min(static_cast<long long>(p.tokens_per_cta), tokens - tok0));
  for (int i = threadIdx.x; i < nt * max(half, 1); i += kAppendThreads) {
    const int t = half ? i / half : i, f = half ? i - t * half : 0;
    const int b = static_cast<int>((tok0 + t) / p.T), tt = static_cast<int>((tok0 + t) % p.T);
    const long long row = static_cast<long long>(p.lens ? p.lens[b] : 0) + tt;
    if (f == 0) {
      const bool lv = tt < (p.ntok ? p.ntok[b] : p.T);
      live[t] = lv;
      at[t] = (lv && row >= 0 && row < p.n) ? static_cast<int>(row) : -1;
    }
    if (half) cs[i] = rope_cos_sin(p.rope.turns[f], p.pos ? p.pos[tok0 + t] : static_cast<int>(row), p.rope.mult);
  }
  __syncthreads();
  const int gl = p.d >> 4, gv = p.dv >> 4;  // lanes of a query / key row, of a value row
  const int nrow = p.nq * p.Hq + p.nk * p.H;
  const int per_tok = nrow * gl + p.H * gv;
  const int total = nt * per_tok;
  // (whole warps iterate together: the row maxima are shuffles)
  for (int base = (blockIdx.y * kAppendThreads + (threadIdx.x & ~31)); base < total;
       base += gridDim.y * kAppendThreads) {
    const int i = min(base + static_cast<int>(threadIdx.x & 31), total - 1);
    const bool mine = base + static_cast<int>(threadIdx.x & 31) < total;
    const int t = i / per_tok;
    int j = i - t * per_tok;
    const long long tok = tok0 + t;
    const bool isv = j >= nrow * gl;
    int which = 0, h, l;
    bool isq = false;
    if (isv) {
      j -= nrow * gl;
      h = j / gv;
      l = j - h * gv;
    } else {
      h = j / gl;
      l = j - h * gl;
      isq = h < p.nq * p.Hq;
      if (isq) {
        which = h >= p.Hq;
        h -= which * p.Hq;
      } else {
        h -= p.nq * p.Hq;
        which = h >= p.H;
        h -= which * p.H;
      }
    }
    const int heads = isq ? p.Hq : p.H, width = isv ? p.dv : p.d;
    const __nv_bfloat16* src = isv ? p.v : isq ? (which ? p.q[1] : p.q[0]) : (which ? p.k[1] : p.k[0]);
    src += (static_cast<size_t>(tok) * heads + h) * width;
    const int row = at[t];
    const bool lv = live[t];
    const bool need = mine && (isq ? lv : row >= 0);
    // this lane's channels: 8 from ca, 8 from cb
    const bool split = !isv && !p.rope.inter && half > 0 && (p.rope.rot & 15) == 0;
    int ca = 16 * l, cb = 16 * l + 8;
    if (split) {
      const bool turn = 16 * l < p.rope.rot;
      ca = turn ? 8 * l : ca;
      cb = turn ? half + 8 * l : cb;
    }
    float xa[8], xb[8];
    if (need) {
      unpack_bf16x8(*reinterpret_cast<const uint4*>(src + ca), xa);
      unpack_bf16x8(*reinterpret_cast<const uint4*>(src + cb), xb);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) xa[e] = xb[e] = 0.f;
    }
    if (!isv && half > 0 && need) {
      const float2* a = cs + t * half;
      if (p.rope.inter) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          if (ca + e < p.rope.rot) {
            const float2 c = a[(ca + e) >> 1];
            const float x0 = xa[e], x1 = xa[e + 1];
            xa[e] = x0 * c.x - x1 * c.y;
            xa[e + 1] = x1 * c.x + x0 * c.y;
          }
          if (cb + e < p.rope.rot) {
            const float2 c = a[(cb + e) >> 1];
            const float x0 = xb[e], x1 = xb[e + 1];
            xb[e] = x0 * c.x - x1 * c.y;
            xb[e + 1] = x1 * c.x + x0 * c.y;
          }
        }
      } else if (split) {
        if (16 * l < p.rope.rot) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 c = a[ca + e];
            const float x0 = xa[e], x1 = xb[e];
            xa[e] = x0 * c.x - x1 * c.y;
            xb[e] = x1 * c.x + x0 * c.y;
          }
        }
      } else {  // halves that do not end on 8 channels: the partner comes by its own load
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int ch = 16 * l + e;
          if (ch >= p.rope.rot) continue;
          const bool lo = ch < half;
          const float2 c = a[lo ? ch : ch - half];
          const float other = __bfloat162float(src[lo ? ch + half : ch - half]);
          float& x = e < 8 ? xa[e & 7] : xb[e & 7];
          x = lo ? x * c.x - other * c.y : x * c.x + other * c.y;
        }
      }
    }
    if (isq) {  // (padding tokens get zero queries)
      if (mine && DA_BOUNDS_V(tok < tokens && h < p.Hq, tok)) {
        __nv_bfloat16* dst = (which ? p.qo[1] : p.qo[0]) + (static_cast<size_t>(tok) * p.Hq + h) * p.d;
        *reinterpret_cast<uint4*>(dst + ca) = pack_bf16x8(xa);
        *reinterpret_cast<uint4*>(dst + cb) = pack_bf16x8(xb);
      }
    }
    const int b = static_cast<int>(tok / p.T);
    const size_t crow = (static_cast<size_t>(b) * p.n + (row < 0 ? 0 : row)) * p.H + h;
    void* cache = isv ? p.vc : (which ? p.kc[1] : p.kc[0]);
    const bool write = need && !isq && DA_BOUNDS_V(b < p.B && row < p.n && h < p.H, row);
    if (p.fmt == kCacheBf16 || (isv && p.fmt == kCacheFp8k)) {
      if (write) {
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(cache) + crow * width;
        *reinterpret_cast<uint4*>(dst + ca) = pack_bf16x8(xa);
        *reinterpret_cast<uint4*>(dst + cb) = pack_bf16x8(xb);
      }
    } else {
      float mul = which ? p.kinv[1] : p.kinv[0];
      float scale = 0.f;
      if (p.fmt == kCacheFp8) {  // (uniform: every lane of the warp takes part)
        // largest magnitude as bits: a NaN or an infinity stays the largest
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          m = max(m, max(__float_as_uint(xa[e]) & 0x7fffffffu, __float_as_uint(xb[e]) & 0x7fffffffu));
        const int lanes = isv ? gv : gl;
#pragma unroll
        for (int x = 1; x < 16; x <<= 1) {
          const uint32_t o = __shfl_xor_sync(0xffffffffu, m, x);
          if (x < lanes) m = max(m, o);
        }
        const float amax = __uint_as_float(m);
        // a row below 448 * 2^-126 keeps the smallest normal scale (its inverse stays finite)
        const float top = (amax < 448.f * 0x1p-126f) ? 448.f * 0x1p-126f : amax;
        scale = (m == 0) ? 0.f : top / 448.f;
        mul = 448.f / top;
      }
      if (write) {
        uint8_t* dst = static_cast<uint8_t*>(cache) + crow * width;
        *reinterpret_cast<uint2*>(dst + ca) = pack_e4m3x8(xa, mul);
        *reinterpret_cast<uint2*>(dst + cb) = pack_e4m3x8(xb, mul);
        if (p.fmt == kCacheFp8 && l == 0) {
          float* sc = isv ? p.vs : (which ? p.ks[1] : p.ks[0]);
          sc[(static_cast<size_t>(b) * p.H + h) * p.n + row] = scale;
        }
      }
    }
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
