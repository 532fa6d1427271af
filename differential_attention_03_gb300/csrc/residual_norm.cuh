// The norms after and before a block, with its gate and residual scale, and
// their backward pass (sm_103a, CUDA cores).  Per row of width D:
//
//   p = post ? x / rms(x) gamma_post : x,      rms(x) = sqrt(mean x^2 + eps)
//   s = residual + scale gate p,               y = s / rms(s) gamma
//
// y is made from s before s is rounded.  Backward, from the gradients dy and
// ds and the stored s (n = s / rms(s), xh = x / rms(x)):
//   t  = ds + (dy gamma - n mean(dy gamma n)) / rms(s)     = dresidual
//   dgate = scale sum t p,  dp = scale gate t,  dgamma = sum dy n
//   post: dgamma_post = sum dp xh,  dx = (dp gamma_post - xh mean(dp gamma_post xh)) / rms(x)
//   else: dx = dp
//
// HBM-bound.  A worker (a warp for rows of up to 256 elements of 8-wide
// vectors, else a CTA) holds a whole row in registers, so that each tensor is
// read once whatever the number of reductions; sums are fp32.  Backward: a
// thread keeps its columns over all the rows of its worker, so the sums over
// rows stay in registers; each worker writes them once, and sum_parts_kernel
// joins the workers in a fixed order.
#pragma once

#include "block_params.h"
#include "ptx.cuh"
#include "vec8.cuh"

#undef DA_BOUNDS_FILE
#define DA_BOUNDS_FILE 14

namespace da {

template <int VEC>
__device__ __forceinline__ void load_vec(const __nv_bfloat16* p, float (&v)[VEC]) {
  if constexpr (VEC == 8)
    unpack8(*reinterpret_cast<const uint4*>(p), v);
  else
    v[0] = __bfloat162float(*p);
}
template <int VEC>
__device__ __forceinline__ void load_vec(const float* p, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    v[0] = *p;
  }
}
template <int VEC>
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&v)[VEC]) {
  if constexpr (VEC == 8)
    *reinterpret_cast<uint4*>(p) = pack8(v);
  else
    *p = __float2bfloat16_rn(v[0]);
}
template <int VEC>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *p = v[0];
  }
}

// Sums of two values over the worker's threads (every thread gets them).  buf: 2 x 32 floats a use, two uses in turn.
template <bool kWarp>
__device__ __forceinline__ float2 row_sums(float a, float b, float* buf, int& turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if (kWarp) return make_float2(a, b);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  float* at = buf + 64 * turn;  // (the other half may still be read by warps that lag behind)
  turn ^= 1;
  if (lane == 0) {
    at[warp] = a;
    at[32 + warp] = b;
  }
  __syncthreads();
  a = lane < nw ? at[lane] : 0.f;
  b = lane < nw ? at[32 + lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  return make_float2(a, b);
}

// NV vectors of VEC elements a thread; a worker's thread `t` of `nt` holds vectors t, t + nt, ...
template <typename TX, typename TS, int VEC, int NV, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 256 : 512) residual_norm_kernel(const NormParams p) {
  __shared__ float buf[128];
  int turn = 0;
  const int t = kWarp ? (threadIdx.x & 31) : threadIdx.x, nt = kWarp ? 32 : blockDim.x;
  const long long worker = kWarp ? blockIdx.x * 8ll + (threadIdx.x >> 5) : blockIdx.x;
  const long long workers = kWarp ? gridDim.x * 8ll : gridDim.x;
  const float inv_d = 1.f / static_cast<float>(p.D);
  const TX* x = static_cast<const TX*>(p.x);
  const TS* res = static_cast<const TS*>(p.residual);
  for (long long row = worker; row < p.rows; row += workers) {
    const long long at = row * p.D;
    float v[NV][VEC], r[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * nt) * VEC;
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = r[i][j] = 0.f;
      if (c < p.D) {
        load_vec<VEC>(x + at + c, v[i]);
        if (res) load_vec<VEC>(res + at + c, r[i]);
      }
    }
    float m = p.scale;
    if (p.post) {
      float q = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) q += v[i][j] * v[i][j];
      m *= rsqrtf(row_sums<kWarp>(q, 0.f, buf, turn).x * inv_d + p.eps);
    }
    const float* gate = p.gate ? p.gate + (row / p.group_rows) * p.D : nullptr;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * nt) * VEC;
      if (c < p.D) {
        float w[VEC];
        if (p.post && p.gamma_post) {
          load_vec<VEC>(p.gamma_post + c, w);
#pragma unroll
          for (int j = 0; j < VEC; ++j) v[i][j] *= w[j];
        }
        if (gate) {
          load_vec<VEC>(gate + c, w);
#pragma unroll
          for (int j = 0; j < VEC; ++j) v[i][j] *= w[j];
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          v[i][j] = r[i][j] + m * v[i][j];
          q += v[i][j] * v[i][j];
        }
        if (p.s_out && DA_BOUNDS_V(row < p.rows && c + VEC <= p.D, row))
          store_vec<VEC>(static_cast<TS*>(p.s_out) + at + c, v[i]);
      }
    }
    if (!p.norm) continue;
    const float rs = rsqrtf(row_sums<kWarp>(q, 0.f, buf, turn).x * inv_d + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * nt) * VEC;
      if (c < p.D) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[i][j] *= rs;
        if (p.gamma) {
          float w[VEC];
          load_vec<VEC>(p.gamma + c, w);
#pragma unroll
          for (int j = 0; j < VEC; ++j) v[i][j] *= w[j];
        }
        if (DA_BOUNDS_V(row < p.rows && c + VEC <= p.D, row)) store_vec<VEC>(static_cast<TX*>(p.y_out) + at + c, v[i]);
      }
    }
  }
}

template <typename TX, typename TS, int VEC, int NV, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 256 : 512) residual_norm_grad_kernel(const NormParams p) {
  __shared__ float buf[128];
  int turn = 0;
  const int t = kWarp ? (threadIdx.x & 31) : threadIdx.x, nt = kWarp ? 32 : blockDim.x;
  const long long worker = kWarp ? blockIdx.x * 8ll + (threadIdx.x >> 5) : blockIdx.x;
  const long long workers = kWarp ? gridDim.x * 8ll : gridDim.x;
  const float inv_d = 1.f / static_cast<float>(p.D);
  // pieces of this worker: a contiguous range
  const long long first = p.pieces * worker / workers, last = p.pieces * (worker + 1) / workers;
  float dga[NV][VEC], dgp[NV][VEC], dgt[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) dga[i][j] = dgp[i][j] = dgt[i][j] = 0.f;

  for (long long piece = first; piece < last; ++piece) {
    const long long g = piece / p.chunks, ch = piece - g * p.chunks;
    const long long row0 = g * p.group_rows + ch * p.chunk_rows;
    const long long row1 = min((g + 1) * p.group_rows, row0 + p.chunk_rows);
    const float* gate = p.gate ? p.gate + g * p.D : nullptr;
    for (long long row = row0; row < row1; ++row) {
      const long long at = row * p.D;
      float tt[NV][VEC];  // ds, then t = the gradient of s
      if (p.norm) {
        float sv[NV][VEC], dn[NV][VEC];
        float q = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (t + i * nt) * VEC;
#pragma unroll
          for (int j = 0; j < VEC; ++j) sv[i][j] = dn[i][j] = tt[i][j] = 0.f;
          if (c < p.D) {
            load_vec<VEC>(static_cast<const TS*>(p.s) + at + c, sv[i]);
            load_vec<VEC>(static_cast<const TX*>(p.dy) + at + c, dn[i]);
            if (p.ds) load_vec<VEC>(static_cast<const TS*>(p.ds) + at + c, tt[i]);
          }
        }
        float w[NV][VEC];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (t + i * nt) * VEC;
#pragma unroll
          for (int j = 0; j < VEC; ++j) w[i][j] = 1.f;
          if (p.gamma && c < p.D) load_vec<VEC>(p.gamma + c, w[i]);
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            q += sv[i][j] * sv[i][j];
            dot += dn[i][j] * w[i][j] * sv[i][j];
          }
        }
        const float2 sums = row_sums<kWarp>(q, dot, buf, turn);
        const float rs = rsqrtf(sums.x * inv_d + p.eps);
        const float mean = sums.y * rs * inv_d;  // of dn n
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float n = sv[i][j] * rs;
            dga[i][j] += dn[i][j] * n;
            tt[i][j] += rs * (dn[i][j] * w[i][j] - n * mean);
          }
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (t + i * nt) * VEC;
#pragma unroll
          for (int j = 0; j < VEC; ++j) tt[i][j] = 0.f;
          if (c < p.D && p.ds) load_vec<VEC>(static_cast<const TS*>(p.ds) + at + c, tt[i]);
        }
      }
      if (p.dresidual) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (t + i * nt) * VEC;
          if (c < p.D && DA_BOUNDS_V(row < p.rows && c + VEC <= p.D, row))
            store_vec<VEC>(static_cast<TS*>(p.dresidual) + at + c, tt[i]);
        }
      }
      // tt becomes the gradient of gate p; x joins
      float xv[NV][VEC];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (t + i * nt) * VEC;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          xv[i][j] = 0.f;
          tt[i][j] *= p.scale;
        }
        if (c < p.D && (p.post || p.part_gate)) load_vec<VEC>(static_cast<const TX*>(p.x) + at + c, xv[i]);
      }
      if (p.post) {
        float gv[NV][VEC], pv[NV][VEC];
        float q = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (t + i * nt) * VEC;
#pragma unroll
          for (int j = 0; j < VEC; ++j) gv[i][j] = pv[i][j] = 1.f;
          if (c < p.D) {
            if (gate) load_vec<VEC>(gate + c, gv[i]);
            if (p.gamma_post) load_vec<VEC>(p.gamma_post + c, pv[i]);
          }
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            q += xv[i][j] * xv[i][j];
            dot += tt[i][j] * gv[i][j] * pv[i][j] * xv[i][j];
          }
        }
        const float2 sums = row_sums<kWarp>(q, dot, buf, turn);
        const float rx = rsqrtf(sums.x * inv_d + p.eps);
        const float mean = sums.y * rx * inv_d;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (t + i * nt) * VEC;
          float out[VEC];
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float xh = xv[i][j] * rx, dp = tt[i][j] * gv[i][j];
            dgt[i][j] += tt[i][j] * xh * pv[i][j];
            dgp[i][j] += dp * xh;
            out[j] = rx * (dp * pv[i][j] - xh * mean);
          }
          if (p.dx && c < p.D && DA_BOUNDS_V(row < p.rows && c + VEC <= p.D, row))
            store_vec<VEC>(static_cast<TX*>(p.dx) + at + c, out);
        }
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (t + i * nt) * VEC;
          float gv[VEC];
#pragma unroll
          for (int j = 0; j < VEC; ++j) gv[j] = 1.f;
          if (gate && c < p.D) load_vec<VEC>(gate + c, gv);
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            dgt[i][j] += tt[i][j] * xv[i][j];
            gv[j] *= tt[i][j];
          }
          if (p.dx && c < p.D && DA_BOUNDS_V(row < p.rows && c + VEC <= p.D, row))
            store_vec<VEC>(static_cast<TX*>(p.dx) + at + c, gv);
        }
      }
    }
    if (p.part_gate) {
      const long long limit = p.pieces * p.D;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (t + i * nt) * VEC;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          if (c < p.D) DA_STORE(p.part_gate, (ch * p.groups + g) * p.D + c + j, limit, dgt[i][j]);
          dgt[i][j] = 0.f;
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (t + i * nt) * VEC;
    if (c >= p.D) continue;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      if (p.part_gamma) DA_STORE(p.part_gamma, worker * p.D + c + j, workers * p.D, dga[i][j]);
      if (p.part_post) DA_STORE(p.part_post, worker * p.D + c + j, workers * p.D, dgp[i][j]);
    }
  }
}

}  // namespace da
