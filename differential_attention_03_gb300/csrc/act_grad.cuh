// The element-wise part of the products' backward pass (sm_103a, CUDA cores):
//
//   dz = dy act'(z)                                    (kGated = false)
//   dg = dh u act'(g),  du = dh act(g)                 (kGated = true)
//   dbias[j] = sum over the rows of dz, in fp32 before dz is rounded
//
// dz (and [dg | du]) leave in bf16, the operand type of the products that
// follow.  HBM-bound: 6 bytes a value of z (gated 10).  A warp owns 256
// neighbouring columns (16 bytes a lane and tensor) and every eighth row of
// its CTA's chunk; the column sums stay in registers, are joined over the CTA's
// warps in shared memory and over the chunks by sum_parts_kernel, both in a
// fixed order, so that results repeat bit for bit.
#pragma once

#include "act.cuh"
#include "block_params.h"
#include "ptx.cuh"
#include "vec8.cuh"

#undef DA_BOUNDS_FILE
#define DA_BOUNDS_FILE 13

namespace da {

constexpr int kActGradThreads = 256;

template <bool kGated, int ACT>
__global__ void __launch_bounds__(kActGradThreads) act_grad_kernel(const ActGradParams p) {
  __shared__ float sums[kGated ? 1 : 8][kGated ? 1 : 256];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = blockIdx.x * 256 + lane * 8;
  const int per = (p.M + p.chunks - 1) / p.chunks;
  const int r0 = blockIdx.y * per, r1 = min(p.M, r0 + per);
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (col < p.N) {
#pragma unroll 2
    for (int r = r0 + warp; r < r1; r += 8) {
      float dy[8];
      unpack8(*reinterpret_cast<const uint4*>(p.dy + r * p.ldy + col), dy);
      if (kGated) {
        float g[8], u[8], dg[8], du[8];
        unpack8(*reinterpret_cast<const uint4*>(p.pre + r * p.ldp + col), g);
        unpack8(*reinterpret_cast<const uint4*>(p.pre + r * p.ldp + p.N + col), u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float value;
          const float slope = act_slope<ACT>(g[j], value);
          dg[j] = dy[j] * u[j] * slope;
          du[j] = dy[j] * value;
        }
        if (DA_BOUNDS_V(r < p.M && col + 8 <= p.N, r)) {
          *reinterpret_cast<uint4*>(p.dz + r * p.ldz + col) = pack8(dg);
          *reinterpret_cast<uint4*>(p.dz + r * p.ldz + p.N + col) = pack8(du);
        }
      } else {
        if (ACT != DIFFATTN_ACT_NONE) {
          float z[8];
          unpack8(*reinterpret_cast<const uint4*>(p.pre + r * p.ldp + col), z);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float value;
            dy[j] *= act_slope<ACT>(z[j], value);
          }
          if (DA_BOUNDS_V(r < p.M && col + 8 <= p.N, r)) *reinterpret_cast<uint4*>(p.dz + r * p.ldz + col) = pack8(dy);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += dy[j];
      }
    }
  }
  if (!kGated && p.part) {
#pragma unroll
    for (int j = 0; j < 8; ++j) sums[warp][lane * 8 + j] = acc[j];
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
