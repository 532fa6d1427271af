// The element-wise part of the products' backward pass (sm_103a, CUDA cores):
//
//   dz = dy act'(z)                                    (kGated = false)
//   dg = dh u act'(g),  du = dh act(g)                 (kGated = true)
//   dbias[j] = sum over the rows of dz, in fp32 before dz is rounded
//
// dz (and [dg | du]) leave in bf16, the operand type of the products that
// follow.  HBM-bound: 6 bytes a value of z (gated 10); 8192 x 8192, gelu, with
// dbias 69 us (5.8 TB/s; silu 67), 8192 x 2 x 5464 97 (4.6; what lies in L2 aside).  A warp owns 256
// neighbouring columns (16 bytes a lane and tensor) and every eighth row of
// its CTA's chunk; the column sums stay in registers, are joined over the CTA's
// warps in shared memory and over the chunks by sum_parts_kernel, both in a
// fixed order, so that results repeat bit for bit.
#pragma once

#include "act.cuh"
#include "block_params.h"
#include "ptx.cuh"

#undef DA_BOUNDS_FILE
#define DA_BOUNDS_FILE 17

namespace da {

constexpr int kActGradThreads = 256;

// Eight bf16 values as pairs in fp32, and back.
__device__ __forceinline__ void pairs_of(const uint4& w, uint64_t (&v)[4]) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = f2pack(__uint_as_float(x[j] << 16), __uint_as_float(x[j] & 0xffff0000u));
}
__device__ __forceinline__ uint4 rounded(const uint64_t (&v)[4]) {
  uint32_t x[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float lo, hi;
    f2unpack(v[j], lo, hi);
    x[j] = pack_bf16x2(lo, hi);
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}

template <bool kGated, int ACT>
__global__ void __launch_bounds__(kActGradThreads) act_grad_kernel(const ActGradParams p) {
  __shared__ float sums[kGated ? 1 : 8][kGated ? 1 : 256];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = blockIdx.x * 256 + lane * 8;
  const int per = (p.M + p.chunks - 1) / p.chunks;
  const int r0 = blockIdx.y * per, r1 = min(p.M, r0 + per);
  grid_dep_wait();
  grid_dep_launch_dependents();
  uint64_t acc[4] = {0, 0, 0, 0};
  constexpr int IN = kGated ? 3 : ACT != DIFFATTN_ACT_NONE ? 2 : 1, RR = kGated ? 2 : 4;  // rows on their way at once
  if (col < p.N) {
    for (int r = r0 + warp; r < r1; r += 8 * RR) {
      uint4 in[RR][IN];
#pragma unroll
      for (int k = 0; k < RR; ++k) {
        const long long row = min(r + 8 * k, r1 - 1);  // (past the chunk: its last row again, which is not used)
        in[k][0] = *reinterpret_cast<const uint4*>(p.dy + row * p.ldy + col);
        if (IN > 1) in[k][IN > 1 ? 1 : 0] = *reinterpret_cast<const uint4*>(p.pre + row * p.ldp + col);
        if (IN > 2) in[k][IN > 2 ? 2 : 0] = *reinterpret_cast<const uint4*>(p.pre + row * p.ldp + p.N + col);
      }
#pragma unroll
      for (int k = 0; k < RR; ++k) {
        const int row = r + 8 * k;
        if (row >= r1) break;
        uint64_t dy[4];
        pairs_of(in[k][0], dy);
        if (kGated) {
          uint64_t g[4], u[4], value;
          pairs_of(in[k][IN > 1 ? 1 : 0], g);
          pairs_of(in[k][IN > 2 ? 2 : 0], u);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t slope = act_slope2<ACT, false>(g[j], value);
            g[j] = mul2(mul2(dy[j], u[j]), slope);
            u[j] = mul2(dy[j], value);
          }
          if (DA_BOUNDS_V(row < p.M && col + 8 <= p.N, row)) {
            *reinterpret_cast<uint4*>(p.dz + row * p.ldz + col) = rounded(g);
            *reinterpret_cast<uint4*>(p.dz + row * p.ldz + p.N + col) = rounded(u);
          }
        } else {
          if (ACT != DIFFATTN_ACT_NONE) {
            uint64_t z[4], value;
            pairs_of(in[k][IN > 1 ? 1 : 0], z);
#pragma unroll
            for (int j = 0; j < 4; ++j) dy[j] = mul2(dy[j], act_slope2<ACT, true>(z[j], value));
            if (DA_BOUNDS_V(row < p.M && col + 8 <= p.N, row)) *reinterpret_cast<uint4*>(p.dz + row * p.ldz + col) = rounded(dy);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[j] = add2(acc[j], dy[j]);
        }
      }
    }
  }
  if (!kGated && p.part) {
#pragma unroll
    for (int j = 0; j < 4; ++j) f2unpack(acc[j], sums[warp][lane * 8 + 2 * j], sums[warp][lane * 8 + 2 * j + 1]);
    __syncthreads();
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c < p.N) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) t += sums[w][threadIdx.x];
      DA_STORE(p.part, static_cast<long long>(blockIdx.y) * p.N + c, static_cast<long long>(p.chunks) * p.N, t);
    }
  }
}

// 32 columns a CTA; its 32 warps take every 32nd partial row, then add up in order.
__global__ void __launch_bounds__(1024) sum_parts_kernel(const SumParts p) {
  __shared__ float sums[32][33];
  const int k = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long col = static_cast<long long>(blockIdx.x) * 32 + lane;
  if (static_cast<long long>(blockIdx.x) * 32 >= p.width[k]) return;
  grid_dep_wait();
  float t = 0.f;
  if (col < p.width[k]) {
#pragma unroll 4
    for (int c = warp; c < p.count[k]; c += 32) t += p.part[k][c * p.width[k] + col];
  }
  sums[warp][lane] = t;
  __syncthreads();
  // (transposed: warp w adds up column w by shuffles, in a fixed order)
  t = sums[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  const long long out = static_cast<long long>(blockIdx.x) * 32 + warp;
  if (lane == 0 && out < p.width[k]) DA_STORE(p.dst[k], out, p.width[k], t);
}

}  // namespace da
