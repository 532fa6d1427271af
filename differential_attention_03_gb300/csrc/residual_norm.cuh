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
// HBM-bound.  A worker holds a whole row in registers, so that each tensor is
// read once whatever the number of reductions; sums are fp32.  Three layouts:
//   kSubWarp  rows of up to 256 elements: 4 to 32 lanes a row, 16 bytes a lane.
//   kRing     wider rows of 16-byte multiples: a CTA a row, a vector or two a
//             thread; thread 0 keeps the next rows coming by bulk copies into a
//             ring in shared memory, so that loads never wait for reductions.
//   kPlain    rows of any other width: a CTA (up to 256 elements: a warp) a
//             row, single elements, plain loads.
// Backward: a CTA takes neighbouring rows and a thread keeps its columns over
// all of them, so the sums over rows stay in registers; each CTA writes them
// once (for a gate shared by a group of rows: once a group, or once a chunk of
// a large group), and sum_parts_kernel joins the CTAs in a fixed order.
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

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  if (!DA_BOUNDS_V((smem_u32(dst) & 15u) == 0 && (reinterpret_cast<uintptr_t>(src) & 15u) == 0 && (bytes & 15u) == 0, bytes)) return;
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// The threads that share a row: their number, this one's index, and sums over them (every one of them gets the sums).
template <int LAYOUT>
struct RowTeam {
  static constexpr bool kCta = LAYOUT == kRing || LAYOUT == kPlain;
  int t, nt, worker, workers;  // worker: of the CTA's
  float* buf;                  // CTA: 2 x 32 floats a use, two uses in turn
  int turn;

  __device__ __forceinline__ RowTeam(int lanes, float* b) : buf(b), turn(0) {
    nt = kCta ? blockDim.x : lanes;
    t = kCta ? threadIdx.x : (threadIdx.x & (lanes - 1));
    worker = kCta ? 0 : threadIdx.x / lanes;
    workers = kCta ? 1 : blockDim.x / lanes;
  }
  __device__ __forceinline__ float2 sums(float a, float b) {
    const int most = kCta ? 16 : nt >> 1;
    for (int o = most; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (!kCta) return make_float2(a, b);
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
};

// Rows on their way through shared memory.  Thread 0 issues; a slot is refilled when every thread has read it (a
// __syncthreads later).  A wait that runs out is recorded, and the kernel goes on: every later wait returns at once.
struct RowRing {
  const uint8_t* src[5];  // tensors, rows `bytes` long (0: none) and apart
  uint32_t bytes[5], off[5];
  uint32_t slot_bytes;
  uint8_t* slots;
  uint64_t* full;
  int stages;
  volatile int* abort_flag;
  long long next, end, step;  // rows still to issue
  int filled, used;

  // Every thread: where the slots lie; then thread 0 alone: start().
  __device__ __forceinline__ RowRing(uint8_t* smem, int stages_, long long first, long long end_, long long step_)
      : bytes{0, 0, 0, 0, 0}, slot_bytes(0), full(reinterpret_cast<uint64_t*>(smem)), stages(stages_), next(first), end(end_), step(step_),
        filled(0), used(0) {
    abort_flag = reinterpret_cast<volatile int*>(full + stages);
    slots = smem + 128;
  }
  __device__ __forceinline__ void add(int k, const void* tensor, uint32_t row_bytes) {
    src[k] = static_cast<const uint8_t*>(tensor);
    bytes[k] = row_bytes;
    off[k] = slot_bytes;
    slot_bytes += row_bytes;
  }
  __device__ __forceinline__ void issue() {
    if (next >= end) return;
    uint64_t* bar = &full[filled % stages];
    uint8_t* to = slots + (filled % stages) * slot_bytes;
    mbar_arrive_expect_tx(bar, slot_bytes);
#pragma unroll
    for (int k = 0; k < 5; ++k)
      if (bytes[k]) bulk_load(to + off[k], src[k] + next * bytes[k], bytes[k], bar);
    ++filled;
    next += step;
  }
  __device__ __forceinline__ void start() {
    for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  // Every thread: the next row's slot, landed.
  __device__ __forceinline__ const uint8_t* take(int* status) {
    mbar_wait(&full[used % stages], static_cast<uint32_t>(used / stages) & 1u, AbortState{abort_flag, status});
    const uint8_t* at = slots + (used % stages) * slot_bytes;
    ++used;
    return at;
  }
  // Thread 0, when no wait of the kernel is left.
  __device__ __forceinline__ void finish() {
    if (*abort_flag)
      for (int f = max(0, filled - stages); f < filled; ++f)
        mbar_wait_drain(&full[f % stages], static_cast<uint32_t>(f / stages) & 1u, kWaitBudgetCycles);
  }
};

// NV vectors of VEC elements a thread; thread t of a row's nt holds vectors t, t + nt, ...
template <typename TX, typename TS, int VEC, int NV, int LAYOUT>
__global__ void __launch_bounds__(512, 2) residual_norm_kernel(const NormParams p) {
  __shared__ float buf[128];
  extern __shared__ __align__(128) uint8_t smem[];
  RowTeam<LAYOUT> team(p.lanes, buf);
  const int t = team.t, nt = team.nt;
  const long long first = static_cast<long long>(blockIdx.x) * team.workers + team.worker;
  const long long step = static_cast<long long>(gridDim.x) * team.workers;
  const float inv_d = 1.f / static_cast<float>(p.D);
  const TX* x = static_cast<const TX*>(p.x);
  const TS* res = static_cast<const TS*>(p.residual);
  const bool row_gate = p.gate && p.group_rows == 1;
  RowRing ring(smem, p.stages, first, p.rows, step);
  if (LAYOUT == kRing) {
    ring.add(0, x, p.D * static_cast<uint32_t>(sizeof(TX)));
    ring.add(1, res, res ? p.D * static_cast<uint32_t>(sizeof(TS)) : 0u);
    ring.add(2, p.gate, row_gate ? p.D * 4u : 0u);
    if (threadIdx.x == 0) ring.start();
  }
  grid_dep_wait();
  if (LAYOUT == kRing) {
    if (threadIdx.x == 0)
      for (int s = 0; s < p.stages; ++s) ring.issue();
    __syncthreads();
  }
  grid_dep_launch_dependents();
  // Rows of a warp's teams go together (their shuffles are of the whole warp): as many turns as the first team's.
  const long long lead = LAYOUT == kSubWarp ? first - (threadIdx.x & 31) / nt : first;
  for (long long row = first, head = lead; head < p.rows; row += step, head += step) {
    const bool live = LAYOUT != kSubWarp || row < p.rows;
    const long long at = row * p.D;
    const uint8_t* slot = LAYOUT == kRing ? ring.take(p.status) : nullptr;
    const float* gate = p.gate ? p.gate + (row / p.group_rows) * p.D : nullptr;
    float v[NV][VEC], r[NV][VEC], w[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * nt) * VEC;
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = r[i][j] = 0.f, w[i][j] = 1.f;
      if (c < p.D && live) {
        if (LAYOUT == kRing) {
          load_vec<VEC>(reinterpret_cast<const TX*>(slot) + c, v[i]);
          if (res) load_vec<VEC>(reinterpret_cast<const TS*>(slot + ring.off[1]) + c, r[i]);
          if (row_gate)
            load_vec<VEC>(reinterpret_cast<const float*>(slot + ring.off[2]) + c, w[i]);
          else if (gate)
            load_vec<VEC>(gate + c, w[i]);
        } else {
          load_vec<VEC>(x + at + c, v[i]);
          if (res) load_vec<VEC>(res + at + c, r[i]);
          if (gate) load_vec<VEC>(gate + c, w[i]);
        }
      }
    }
    float m = p.scale;
    if (p.post) {
      float q = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) q += v[i][j] * v[i][j];
      m *= rsqrtf(team.sums(q, 0.f).x * inv_d + p.eps);
      if (LAYOUT == kRing && threadIdx.x == 0) ring.issue();
    }
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * nt) * VEC;
      if (c < p.D) {
        if (p.post && p.gamma_post) {
          float g[VEC];
          load_vec<VEC>(p.gamma_post + c, g);
#pragma unroll
          for (int j = 0; j < VEC; ++j) v[i][j] *= g[j];
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          v[i][j] = r[i][j] + m * (v[i][j] * w[i][j]);
          q += v[i][j] * v[i][j];
        }
        if (p.s_out && live && DA_BOUNDS_V(row < p.rows && c + VEC <= p.D, row))
          store_vec<VEC>(static_cast<TS*>(p.s_out) + at + c, v[i]);
      }
    }
    if (!p.norm) {
      if (LAYOUT == kRing && !p.post) {
        __syncthreads();
        if (threadIdx.x == 0) ring.issue();
      }
      continue;
    }
    const float rs = rsqrtf(team.sums(q, 0.f).x * inv_d + p.eps);
    if (LAYOUT == kRing && !p.post && threadIdx.x == 0) ring.issue();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * nt) * VEC;
      if (c < p.D && live) {
        float g[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) g[j] = 1.f;
        if (p.gamma) load_vec<VEC>(p.gamma + c, g);
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[i][j] *= rs * g[j];
        if (DA_BOUNDS_V(row < p.rows && c + VEC <= p.D, row)) store_vec<VEC>(static_cast<TX*>(p.y_out) + at + c, v[i]);
      }
    }
  }
  if (LAYOUT == kRing && threadIdx.x == 0) ring.finish();
}

// Sums a CTA's workers' columns and writes them: dst[c] (workers in order; one worker: its own values).
template <int VEC, int NV, int LAYOUT>
__device__ __forceinline__ void write_columns(const RowTeam<LAYOUT>& team, float (&v)[NV][VEC], float* dst, int D, float* scratch) {
  if (RowTeam<LAYOUT>::kCta) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (team.t + i * team.nt) * VEC;
      if (c < D) store_vec<VEC>(dst + c, v[i]);
    }
    return;
  }
  __syncthreads();  // (earlier readers of the scratch)
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (team.t + i * team.nt) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (c < D) scratch[team.worker * D + c + j] = v[i][j];
  }
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += blockDim.x) {
    float s = 0.f;
    for (int w = 0; w < team.workers; ++w) s += scratch[w * D + c];
    dst[c] = s;
  }
}

template <typename TX, typename TS, int VEC, int NV, int LAYOUT>
__global__ void __launch_bounds__(512) residual_norm_grad_kernel(const NormParams p) {
  __shared__ float buf[128];
  extern __shared__ __align__(128) uint8_t smem[];
  RowTeam<LAYOUT> team(p.lanes, buf);
  const int t = team.t, nt = team.nt;
  const float inv_d = 1.f / static_cast<float>(p.D);
  const bool row_gate = p.gate && p.gate_rows == p.rows;  // each row its own gate: no sum over rows
  // pieces of this CTA: neighbours, so that its rows are neighbours too
  const long long first = p.pieces * blockIdx.x / gridDim.x, last = p.pieces * (blockIdx.x + 1ll) / gridDim.x;
  auto piece_row = [&](long long piece) {
    const long long g = piece / p.chunks;
    return min(g * p.group_rows + (piece - g * p.chunks) * p.chunk_rows, (g + 1) * p.group_rows);
  };
  const bool need_x = p.post || p.part_gate;
  RowRing ring(smem, p.stages, piece_row(first), piece_row(last), 1);
  if (LAYOUT == kRing) {
    const uint32_t bx = p.D * static_cast<uint32_t>(sizeof(TX)), bs = p.D * static_cast<uint32_t>(sizeof(TS));
    ring.add(0, p.s, p.norm ? bs : 0u);
    ring.add(1, p.dy, p.norm ? bx : 0u);
    ring.add(2, p.ds, p.ds ? bs : 0u);
    ring.add(3, p.x, need_x ? bx : 0u);
    ring.add(4, p.gate, row_gate ? p.D * 4u : 0u);
    if (threadIdx.x == 0) ring.start();
  }
  grid_dep_wait();
  if (LAYOUT == kRing) {
    if (threadIdx.x == 0)
      for (int s = 0; s < p.stages; ++s) ring.issue();
    __syncthreads();
  }
  grid_dep_launch_dependents();
  // The parameters of this thread's columns stay in registers where a thread has eight of them; with 16 the sums take
  // those registers, and the parameters come from L1 for each row.
  constexpr bool kKeep = NV * VEC <= 8;
  constexpr int NK = kKeep ? NV : 1;
  float dga[NV][VEC], dgp[NV][VEC], dgt[NV][VEC], ga[NK][VEC], gp[NK][VEC], gv[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (t + i * nt) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      dga[i][j] = dgp[i][j] = dgt[i][j] = 0.f, gv[i][j] = 1.f;
      if (kKeep) ga[kKeep ? i : 0][j] = gp[kKeep ? i : 0][j] = 1.f;
    }
    if (kKeep && c < p.D) {
      if (p.gamma) load_vec<VEC>(p.gamma + c, ga[kKeep ? i : 0]);
      if (p.gamma_post) load_vec<VEC>(p.gamma_post + c, gp[kKeep ? i : 0]);
    }
  }
  auto column = [&](const float* from, float (&kept)[NK][VEC], int i, float (&out)[VEC]) {
    const int c = (t + i * nt) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) out[j] = kKeep ? kept[kKeep ? i : 0][j] : 1.f;
    if (!kKeep && from && c < p.D) load_vec<VEC>(from + c, out);
  };

  for (long long piece = first; piece < last; ++piece) {
    const long long g = piece / p.chunks, ch = piece - g * p.chunks;
    const long long row0 = piece_row(piece), row1 = min(row0 + p.chunk_rows, (g + 1) * p.group_rows);
    if (p.gate && !row_gate) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (t + i * nt) * VEC;
        if (c < p.D) load_vec<VEC>(p.gate + g * p.D + c, gv[i]);
      }
    }
    for (long long head = row0; head < row1; head += team.workers) {
      const long long row = head + team.worker;
      const bool live = LAYOUT == kRing || LAYOUT == kPlain || row < row1;
      const long long at = row * p.D;
      const uint8_t* slot = LAYOUT == kRing ? ring.take(p.status) : nullptr;
      const TS* s_row = LAYOUT == kRing ? reinterpret_cast<const TS*>(slot) : static_cast<const TS*>(p.s) + at;
      const TX* dy_row = LAYOUT == kRing ? reinterpret_cast<const TX*>(slot + ring.off[1]) : static_cast<const TX*>(p.dy) + at;
      const TS* ds_row = LAYOUT == kRing ? reinterpret_cast<const TS*>(slot + ring.off[2]) : static_cast<const TS*>(p.ds) + at;
      const TX* x_row = LAYOUT == kRing ? reinterpret_cast<const TX*>(slot + ring.off[3]) : static_cast<const TX*>(p.x) + at;
      const float* gate_row = LAYOUT == kRing ? reinterpret_cast<const float*>(slot + ring.off[4]) : p.gate + at;
      float tt[NV][VEC];  // ds, then t = the gradient of s, then that of gate p
      float xv[NV][VEC];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (t + i * nt) * VEC;
#pragma unroll
        for (int j = 0; j < VEC; ++j) tt[i][j] = xv[i][j] = 0.f;
        if (c < p.D && live) {
          if (p.ds) load_vec<VEC>(ds_row + c, tt[i]);
          if (need_x) load_vec<VEC>(x_row + c, xv[i]);
          if (row_gate) load_vec<VEC>(gate_row + c, gv[i]);
        }
      }
      if (p.norm) {
        float sv[NV][VEC], dn[NV][VEC];
        float q = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (t + i * nt) * VEC;
#pragma unroll
          for (int j = 0; j < VEC; ++j) sv[i][j] = dn[i][j] = 0.f;
          if (c < p.D && live) {
            load_vec<VEC>(s_row + c, sv[i]);
            load_vec<VEC>(dy_row + c, dn[i]);
          }
          float gk[VEC];
          column(p.gamma, ga, i, gk);
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            q += sv[i][j] * sv[i][j];
            dot += dn[i][j] * gk[j] * sv[i][j];
          }
        }
        const float2 sums = team.sums(q, dot);
        const float rs = rsqrtf(sums.x * inv_d + p.eps);
        const float mean = sums.y * rs * inv_d;  // of dn n
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          float gk[VEC];
          column(p.gamma, ga, i, gk);
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float n = sv[i][j] * rs;
            dga[i][j] += dn[i][j] * n;
            tt[i][j] += rs * (dn[i][j] * gk[j] - n * mean);
          }
        }
      } else if (LAYOUT == kRing) {
        __syncthreads();
      }
      if (LAYOUT == kRing && threadIdx.x == 0) ring.issue();  // (every thread has read the slot)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (t + i * nt) * VEC;
        if (p.dresidual && c < p.D && live && DA_BOUNDS_V(row < p.rows && c + VEC <= p.D, row))
          store_vec<VEC>(static_cast<TS*>(p.dresidual) + at + c, tt[i]);
#pragma unroll
        for (int j = 0; j < VEC; ++j) tt[i][j] *= p.scale;
      }
      float rx = 1.f, mean = 0.f;
      if (p.post) {
        float q = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          float gk[VEC];
          column(p.gamma_post, gp, i, gk);
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            q += xv[i][j] * xv[i][j];
            dot += tt[i][j] * gv[i][j] * gk[j] * xv[i][j];
          }
        }
        const float2 sums = team.sums(q, dot);
        rx = rsqrtf(sums.x * inv_d + p.eps);
        mean = sums.y * rx * inv_d;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (t + i * nt) * VEC;
        float out[VEC], dg[VEC], gk[VEC];
        column(p.gamma_post, gp, i, gk);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float xh = xv[i][j] * rx, dp = tt[i][j] * gv[i][j];  // (without the norm rx = 1, mean = 0, gp = 1)
          dg[j] = tt[i][j] * xh * gk[j];
          if (!row_gate) dgt[i][j] += dg[j];
          dgp[i][j] += dp * xh;
          out[j] = rx * (dp * gk[j] - xh * mean);
        }
        if (c < p.D && live && DA_BOUNDS_V(row < p.rows && c + VEC <= p.D, row)) {
          if (p.dx) store_vec<VEC>(static_cast<TX*>(p.dx) + at + c, out);
          if (row_gate && p.part_gate) store_vec<VEC>(p.part_gate + at + c, dg);
        }
      }
    }
    if (p.part_gate && !row_gate) {
      if (DA_BOUNDS_V((ch * p.groups + g + 1) * p.D <= p.pieces * p.D, ch))
        write_columns<VEC, NV, LAYOUT>(team, dgt, p.part_gate + (ch * p.groups + g) * p.D, p.D, reinterpret_cast<float*>(smem));
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) dgt[i][j] = 0.f;
    }
  }
  const long long mine = static_cast<long long>(blockIdx.x) * p.D;
  if (p.part_gamma) write_columns<VEC, NV, LAYOUT>(team, dga, p.part_gamma + mine, p.D, reinterpret_cast<float*>(smem));
  if (p.part_post) write_columns<VEC, NV, LAYOUT>(team, dgp, p.part_post + mine, p.D, reinterpret_cast<float*>(smem));
  if (LAYOUT == kRing && threadIdx.x == 0) ring.finish();
}

}  // namespace da
