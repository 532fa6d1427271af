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
//             ring in shared memory, so that loads never wait for reductions (a
//             warp of its own for them would take a quarter of the registers
//             from the others: 17 warps an SM instead of 16).
//   kPlain    rows of any other width: a CTA (up to 256 elements: a warp) a
//             row, two or single elements at a time, plain loads.
// Backward: a CTA takes neighbouring rows and a thread keeps its columns over
// all of them, so the sums over rows stay in registers; each CTA writes them
// once (for a gate shared by a group of rows: once a group, or once a chunk of
// a large group), and sum_parts_kernel joins the CTAs in a fixed order.
// 8002 x 4096 on an fp32 stream, both norms, a gate a sequence: 65 us forward
// (6.0 TB/s); 16384 x 2048 in bf16, a gate, both norms: 73 us backward (5.5 TB/s).
// 16777 x 1000 in bf16, the same: 25 us (5.4 TB/s), 43 backward; of odd width,
// 16760 x 1001: 103 and 197 us, bound by instructions on single elements.
#pragma once

#include "act.cuh"
#include "block_params.h"
#include "ptx.cuh"
#include "vec8.cuh"

#undef DA_BOUNDS_FILE
#define DA_BOUNDS_FILE 18

namespace da {

// VEC elements of a thread in fp32: pairs, which an instruction takes at once, or a single one.
template <int VEC>
struct Row {
  static constexpr int N = VEC / 2;
  uint64_t v[N];
  __device__ __forceinline__ void fill(float x) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = f2pack(x, x);
  }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = f2pack(__uint_as_float(x[j] << 16), __uint_as_float(x[j] & 0xffff0000u));
  }
  __device__ __forceinline__ void load(const float* p) {
    const ulonglong2 a = reinterpret_cast<const ulonglong2*>(p)[0], b = reinterpret_cast<const ulonglong2*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const {
    uint32_t x[4];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float lo, hi;
      f2unpack(v[j], lo, hi);
      x[j] = pack_bf16x2(lo, hi);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(x[0], x[1], x[2], x[3]);
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<ulonglong2*>(p)[0] = make_ulonglong2(v[0], v[1]);
    reinterpret_cast<ulonglong2*>(p)[1] = make_ulonglong2(v[2], v[3]);
  }
  __device__ __forceinline__ float dot(const Row& o) const {
    uint64_t t = mul2(v[0], o.v[0]);
#pragma unroll
    for (int j = 1; j < N; ++j) t = fma2(v[j], o.v[j], t);
    float lo, hi;
    f2unpack(t, lo, hi);
    return lo + hi;
  }
  __device__ __forceinline__ float square() const { return dot(*this); }
  static __device__ __forceinline__ uint64_t mul(uint64_t a, uint64_t b) { return mul2(a, b); }
  static __device__ __forceinline__ uint64_t fma(uint64_t a, uint64_t b, uint64_t c) { return fma2(a, b, c); }
  static __device__ __forceinline__ uint64_t all(float x) { return f2pack(x, x); }
};
template <>
struct Row<2> {
  static constexpr int N = 1;
  uint64_t v[1];
  __device__ __forceinline__ void fill(float x) { v[0] = f2pack(x, x); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
    v[0] = f2pack(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  __device__ __forceinline__ void load(const float* p) { v[0] = *reinterpret_cast<const uint64_t*>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const {
    float lo, hi;
    f2unpack(v[0], lo, hi);
    *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(lo, hi);
  }
  __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<uint64_t*>(p) = v[0]; }
  __device__ __forceinline__ float dot(const Row& o) const {
    float lo, hi;
    f2unpack(mul2(v[0], o.v[0]), lo, hi);
    return lo + hi;
  }
  __device__ __forceinline__ float square() const { return dot(*this); }
  static __device__ __forceinline__ uint64_t mul(uint64_t a, uint64_t b) { return mul2(a, b); }
  static __device__ __forceinline__ uint64_t fma(uint64_t a, uint64_t b, uint64_t c) { return fma2(a, b, c); }
  static __device__ __forceinline__ uint64_t all(float x) { return f2pack(x, x); }
};
template <>
struct Row<1> {
  static constexpr int N = 1;
  float v[1];
  __device__ __forceinline__ void fill(float x) { v[0] = x; }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v[0] = __bfloat162float(*p); }
  __device__ __forceinline__ void load(const float* p) { v[0] = *p; }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *p = __float2bfloat16_rn(v[0]); }
  __device__ __forceinline__ void store(float* p) const { *p = v[0]; }
  __device__ __forceinline__ float dot(const Row& o) const { return v[0] * o.v[0]; }
  __device__ __forceinline__ float square() const { return v[0] * v[0]; }
  static __device__ __forceinline__ float mul(float a, float b) { return a * b; }
  static __device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }
  static __device__ __forceinline__ float all(float x) { return x; }
};

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
  float* buf;                  // CTA: 4 x 32 values a use, two uses in turn; those of warps that the CTA lacks stay zero
  int turn;

  __device__ __forceinline__ RowTeam(int lanes, float* b) : buf(b), turn(0) {
    nt = kCta ? blockDim.x : lanes;
    t = kCta ? threadIdx.x : (threadIdx.x & (lanes - 1));
    worker = kCta ? 0 : threadIdx.x / lanes;
    workers = kCta ? 1 : blockDim.x / lanes;
    if (kCta)
      for (int k = threadIdx.x; k < 256; k += blockDim.x) buf[k] = 0.f;
  }
  // Sums of each of v over the row's threads; every thread gets them.
  template <int N>
  __device__ __forceinline__ void sums(float (&v)[N]) {
    if (kCta) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    } else {
      for (int o = nt >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
      return;
    }
    float* at = buf + turn;  // (the other half may still be read by warps that lag behind)
    turn ^= 128;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int k = 0; k < N; ++k) at[32 * k + (threadIdx.x >> 5)] = v[k];
    }
    __syncthreads();
    const int nw = nt >> 5;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float4* from = reinterpret_cast<const float4*>(at + 32 * k);
      float4 x = from[0];
      for (int w = 4; w < nw; w += 4) {
        const float4 y = from[w >> 2];
        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
      }
      v[k] = (x.x + x.y) + (x.z + x.w);
    }
  }
};

// Rows on their way through shared memory: slot k holds the k-th row ahead.  Thread 0 refills a slot once every thread
// has read it (a barrier later).  A wait that runs out is recorded, and the kernel goes on: every later wait returns at
// once.
struct RowRing {
  static constexpr int kBytes = 128;  // barriers and flag, before the slots
  const uint8_t* src[5];  // tensors, rows `bytes` long (0: none) and apart
  uint32_t bytes[5], off[5];
  uint32_t slot_bytes;
  uint8_t* smem;
  int stages, slot;
  uint32_t phase;
  int* status;

  __device__ __forceinline__ RowRing(uint8_t* smem_, int stages_, int* status_)
      : bytes{0, 0, 0, 0, 0}, slot_bytes(0), smem(smem_), stages(stages_), slot(0), phase(0), status(status_) {}
  __device__ __forceinline__ uint64_t* full(int s) const { return reinterpret_cast<uint64_t*>(smem) + s; }
  __device__ __forceinline__ AbortState ab() const {
    return AbortState{reinterpret_cast<volatile int*>(smem + 8 * kNormMaxStages), status};
  }
  __device__ __forceinline__ void add(int k, const void* tensor, uint32_t row_bytes) {
    src[k] = static_cast<const uint8_t*>(tensor);
    bytes[k] = row_bytes;
    off[k] = slot_bytes;
    slot_bytes += row_bytes;
  }
  __device__ __forceinline__ void init() {  // one thread, before a __syncthreads
    for (int s = 0; s < stages; ++s) mbar_init(full(s), 1);
    *ab().flag = 0;
    fence_mbar_init();
  }
  __device__ __forceinline__ void load(int s, long long row) {
    mbar_arrive_expect_tx(full(s), slot_bytes);
    uint8_t* to = smem + kBytes + s * slot_bytes;
#pragma unroll
    for (int k = 0; k < 5; ++k)
      if (bytes[k]) bulk_load(to + off[k], src[k] + static_cast<uint64_t>(static_cast<uint32_t>(row)) * bytes[k], bytes[k], full(s));
  }
  // Thread 0: the first rows (first, first + step, ...).
  __device__ __forceinline__ void start(long long first, long long end, long long step) {
    for (int s = 0; s < stages && first + s * step < end; ++s) load(s, first + s * step);
  }
  // Every thread: the slot of the k-th row ahead, landed.
  __device__ __forceinline__ int take_slot(int k) const {
    const bool over = slot + k >= stages;
    const int s = slot + k - (over ? stages : 0);
    mbar_wait(full(s), phase ^ (over ? 1u : 0u), ab());
    return s;
  }
  __device__ __forceinline__ const uint8_t* take(int k = 0) const { return smem + kBytes + take_slot(k) * slot_bytes; }
  // Every thread, a barrier after its last read of the slot: row `ahead` into it, if there is one.
  __device__ __forceinline__ void refill(long long ahead, long long end) {
    if (threadIdx.x == 0 && ahead < end) load(slot, ahead);
    if (++slot == stages) {
      slot = 0;
      phase ^= 1u;
    }
  }
  // Thread 0, aborted: what is still on its way lands before the CTA exits; `rows`: of the CTA.
  __device__ __forceinline__ void drain(long long rows) const {
    if (*ab().flag)
      for (long long f = rows > stages ? rows - stages : 0; f < rows; ++f)
        mbar_wait_drain(full(static_cast<int>(f % stages)), static_cast<uint32_t>(f / stages) & 1u, kWaitBudgetCycles);
  }
};

// Rows whose sum of squares leaves fp32's range (elements above 1e17) are summed again scaled by this power of two.
constexpr float kSmall = 8.271806125530277e-25f;  // 2^-80
__device__ __forceinline__ bool overflowed(float q) { return q > 3.4028234e38f; }
template <int VEC>
__device__ __forceinline__ Row<VEC> scaled(Row<VEC> r, float k) {
#pragma unroll
  for (int j = 0; j < Row<VEC>::N; ++j) r.v[j] = Row<VEC>::mul(r.v[j], Row<VEC>::all(k));
  return r;
}

// NV vectors of VEC elements a thread; thread t of a row's nt holds vectors t, t + nt, ...
template <typename TX, typename TS, int VEC, int NV, int LAYOUT>
__global__ void __launch_bounds__(LAYOUT == kRing || LAYOUT == kPlain ? 512 : 256, LAYOUT == kRing ? 1 : LAYOUT == kPlain ? 2 : 4)
    residual_norm_kernel(const NormParams p) {
  using R = Row<VEC>;
  __shared__ __align__(16) float buf[256];
  extern __shared__ __align__(128) uint8_t smem[];
  RowTeam<LAYOUT> team(p.lanes, buf);
  const int t = team.t, nt = team.nt;
  const long long first = static_cast<long long>(blockIdx.x) * team.workers + team.worker;
  const long long step = static_cast<long long>(gridDim.x) * team.workers;
  const float inv_d = 1.f / static_cast<float>(p.D);
  const bool row_gate = p.gate && p.group_rows == 1;
  const bool group_gate = p.gate && !row_gate;
  const bool has_res = p.residual != nullptr;
  RowRing ring(smem, p.stages, p.status);
  if (LAYOUT == kRing) {
    ring.add(0, p.x, p.D * static_cast<uint32_t>(sizeof(TX)));
    ring.add(1, p.residual, has_res ? p.D * static_cast<uint32_t>(sizeof(TS)) : 0u);
    ring.add(2, p.gate, row_gate ? p.D * 4u : 0u);
    if (threadIdx.x == 0) ring.init();
  }
  grid_dep_wait();
  if (LAYOUT == kRing && threadIdx.x == 0) ring.start(first, p.rows, step);
  if (RowTeam<LAYOUT>::kCta) __syncthreads();
  grid_dep_launch_dependents();
  // What multiplies a column in every row stays in registers.
  constexpr bool kKeep = VEC == 8;
  R kept[kKeep ? NV : 1], kept_y[kKeep ? NV : 1];
  auto column = [&](int c, R& w, long long group) {  // gamma_post, and the group's gate
    w.fill(1.f);
    if (p.gamma_post) w.load(p.gamma_post + c);
    if (group_gate) {
      R g;
      g.load(p.gate + group * p.D + c);
#pragma unroll
      for (int j = 0; j < R::N; ++j) w.v[j] = R::mul(w.v[j], g.v[j]);
    }
  };
  auto column_y = [&](int c, R& w) {
    w.fill(1.f);
    if (p.gamma) w.load(p.gamma + c);
  };
  if (kKeep) {
#pragma unroll
    for (int i = 0; i < (kKeep ? NV : 1); ++i) {
      const int c = (t + i * nt) * VEC;
      if (c < p.D) column_y(c, kept_y[i]);
    }
  }
  long long group = -1;  // whose gate is in `kept`
  // Rows of a warp's teams go together (their shuffles are of the whole warp): as many turns as the first team's.
  const long long lead = LAYOUT == kSubWarp ? first - (threadIdx.x & 31) / nt : first;
  long long at = first * p.D;
  for (long long row = first, head = lead; head < p.rows; row += step, head += step, at += step * p.D) {
    const bool live = LAYOUT != kSubWarp || row < p.rows;
    auto mine = [&](int i) { return (t + i * nt) * VEC < p.D && live; };  // whether this thread has vector i
    const uint8_t* slot = LAYOUT == kRing ? ring.take() : nullptr;
    const TX* x_row = LAYOUT == kRing ? reinterpret_cast<const TX*>(slot) : static_cast<const TX*>(p.x) + at;
    const TS* r_row = LAYOUT == kRing ? reinterpret_cast<const TS*>(slot + ring.off[1]) : static_cast<const TS*>(p.residual) + at;
    const float* g_row = LAYOUT == kRing ? reinterpret_cast<const float*>(slot + ring.off[2]) : p.gate + at;
    if (live) {
      const long long now = group_gate ? static_cast<uint32_t>(row) / static_cast<uint32_t>(p.group_rows) : 0;
      if (now != group) {
        group = now;
        if (kKeep) {
#pragma unroll
          for (int i = 0; i < (kKeep ? NV : 1); ++i)
            if ((t + i * nt) * VEC < p.D) column((t + i * nt) * VEC, kept[i], group);
        }
      }
    }
    R v[NV], r[NV], w[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * nt) * VEC;
      if (mine(i)) {
        v[i].load(x_row + c);
        r[i].fill(0.f);
        if (has_res) r[i].load(r_row + c);
        if (row_gate) w[i].load(g_row + c);
      }
    }
    // One over rms(v), from this thread's share of the sum of squares.
    auto inverse_rms = [&](float share) {
      float q[1] = {share};
      team.sums(q);
      float r = rsqrtf(q[0] * inv_d + p.eps);
      const bool over = overflowed(q[0]);
      if (RowTeam<LAYOUT>::kCta ? over : __any_sync(0xffffffffu, over)) {
        q[0] = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (mine(i)) q[0] += scaled(v[i], kSmall).square();
        team.sums(q);
        if (over) r = rsqrtf(q[0] * inv_d) * kSmall;
      }
      return r;
    };
    float m = p.scale;
    if (p.post) {
      float q = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (mine(i)) q += v[i].square();
      m *= inverse_rms(q);
      if (LAYOUT == kRing) ring.refill(row + p.stages * step, p.rows);
    }
    float q = 0.f;
    const auto mm = R::all(m);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * nt) * VEC;
      if (!mine(i)) continue;
      R k;
      if (kKeep)
        k = kept[kKeep ? i : 0];
      else
        column(c, k, group);
      // (normed before gamma and the gate, which may take a large element past fp32)
#pragma unroll
      for (int j = 0; j < R::N; ++j) v[i].v[j] = R::mul(v[i].v[j], mm);
      if (row_gate) {
#pragma unroll
        for (int j = 0; j < R::N; ++j) v[i].v[j] = R::mul(v[i].v[j], w[i].v[j]);
      }
#pragma unroll
      for (int j = 0; j < R::N; ++j) v[i].v[j] = R::fma(v[i].v[j], k.v[j], r[i].v[j]);
      q += v[i].square();
      if (p.s_out && DA_BOUNDS_V(row < p.rows && c + VEC <= p.D, row)) v[i].store(static_cast<TS*>(p.s_out) + at + c);
    }
    if (!p.norm) {
      if (LAYOUT == kRing && !p.post) {
        __syncthreads();
        ring.refill(row + p.stages * step, p.rows);
      }
      continue;
    }
    const auto rs = R::all(inverse_rms(q));
    if (LAYOUT == kRing && !p.post) ring.refill(row + p.stages * step, p.rows);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * nt) * VEC;
      if (!mine(i)) continue;
      R k;
      if (kKeep)
        k = kept_y[kKeep ? i : 0];
      else
        column_y(c, k);
#pragma unroll
      for (int j = 0; j < R::N; ++j) v[i].v[j] = R::mul(v[i].v[j], R::mul(rs, k.v[j]));
      if (DA_BOUNDS_V(row < p.rows && c + VEC <= p.D, row)) v[i].store(static_cast<TX*>(p.y_out) + at + c);
    }
  }
  if (LAYOUT == kRing && threadIdx.x == 0) ring.drain((p.rows - first + step - 1) / step);
}

// Sums a CTA's workers' columns and writes them: dst[c] (workers in order; one worker: its own values).
template <int VEC, int NV, int LAYOUT>
__device__ __forceinline__ void write_columns(const RowTeam<LAYOUT>& team, const Row<VEC> (&v)[NV], float* dst, int D, float* scratch) {
  if (!RowTeam<LAYOUT>::kCta) __syncthreads();  // (earlier readers of the scratch)
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (team.t + i * team.nt) * VEC;
    if (c < D) v[i].store((RowTeam<LAYOUT>::kCta ? dst : scratch + team.worker * D) + c);
  }
  if (RowTeam<LAYOUT>::kCta) return;
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += blockDim.x) {
    float s = 0.f;
    for (int w = 0; w < team.workers; ++w) s += scratch[w * D + c];
    dst[c] = s;
  }
}

template <typename TX, typename TS, int VEC, int NV, int LAYOUT>
__global__ void __launch_bounds__(LAYOUT == kRing || LAYOUT == kPlain ? 512 : 256, LAYOUT == kRing || LAYOUT == kPlain ? 1 : 2)
    residual_norm_grad_kernel(const NormParams p) {
  using R = Row<VEC>;
  __shared__ __align__(16) float buf[256];
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
  const bool need_x = p.post || p.part_gate, has_ds = p.ds != nullptr;
  RowRing ring(smem, p.stages, p.status);
  if (LAYOUT == kRing) {
    const uint32_t bx = p.D * static_cast<uint32_t>(sizeof(TX)), bs = p.D * static_cast<uint32_t>(sizeof(TS));
    ring.add(0, p.s, p.norm ? bs : 0u);
    ring.add(1, p.dy, p.norm ? bx : 0u);
    ring.add(2, p.ds, has_ds ? bs : 0u);
    ring.add(3, p.x, need_x ? bx : 0u);
    ring.add(4, p.gate, row_gate ? p.D * 4u : 0u);
    if (threadIdx.x == 0) ring.init();
  }
  grid_dep_wait();
  const long long end = piece_row(last);
  if (LAYOUT == kRing && threadIdx.x == 0) ring.start(piece_row(first), end, 1);
  if (RowTeam<LAYOUT>::kCta) __syncthreads();
  grid_dep_launch_dependents();
  // kHold: a row's values and the parameters of a thread's columns stay in registers, every load of a row issued at its
  // start.  Rows of the ring (16 elements a thread here): only t is held across the reductions; s, dy and x are read from
  // the slot again, gamma from L1, and gamma_post with the group's gate from shared memory where it has room (all three
  // from L1, which they overfill: 2730 x 6144 in bf16 100 us, 78 so; 4088 x 4104 on an fp32 stream 140 and 110).
  // dga: sums of dy n.  u: sums of t xh over a piece (with a gate a row: of t gate xh), of which gamma_post times is the
  // gate's gradient and the gate times gamma_post's; the latter's sums over pieces are in shared memory.
  constexpr bool kHold = LAYOUT != kRing;
  constexpr int NH = kHold ? NV : 1;
  R dga[NV], u[NV], kept_ga[NH], kept_c[NH];
  float* post_sums = reinterpret_cast<float*>(smem + p.off_post) + (RowTeam<LAYOUT>::kCta ? 0 : team.worker * p.D);
  float* combined_row = reinterpret_cast<float*>(smem + p.off_combined);  // (a thread's own columns)
  auto column = [&](const float* from, int i) -> R {
    R w;
    w.fill(1.f);
    if (from) w.load(from + (t + i * nt) * VEC);
    return w;
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (t + i * nt) * VEC;
    dga[i].fill(0.f);
    u[i].fill(0.f);
    if (p.part_post && c < p.D) u[i].store(post_sums + c);
    if (kHold && c < p.D) kept_ga[kHold ? i : 0] = column(p.gamma, i);
  }
  const auto scale = R::all(p.scale);

  for (long long piece = first; piece < last; ++piece) {
    const long long g = piece / p.chunks, ch = piece - g * p.chunks;
    const long long row0 = piece_row(piece), row1 = min(row0 + p.chunk_rows, (g + 1) * p.group_rows);
    const float* group_gate = p.gate && !row_gate ? p.gate + g * p.D : nullptr;
    auto combined = [&](int i) -> R {  // gamma_post, and the group's gate
      R w = column(p.gamma_post, i);
      if (group_gate) {
        const R gv = column(group_gate, i);
#pragma unroll
        for (int j = 0; j < R::N; ++j) w.v[j] = R::mul(w.v[j], gv.v[j]);
      }
      return w;
    };
    if (kHold) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if ((t + i * nt) * VEC < p.D) kept_c[kHold ? i : 0] = combined(i);
    } else if (p.off_combined >= 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if ((t + i * nt) * VEC < p.D) combined(i).store(combined_row + (t + i * nt) * VEC);
    }
    auto gamma_of = [&](int i) -> R { return kHold ? kept_ga[kHold ? i : 0] : column(p.gamma, i); };
    auto c_of = [&](int i) -> R {
      if (kHold) return kept_c[kHold ? i : 0];
      if (p.off_combined < 0) return combined(i);
      R w;
      w.load(combined_row + (t + i * nt) * VEC);
      return w;
    };
    long long at = (row0 + team.worker) * p.D;
    for (long long head = row0; head < row1; head += team.workers, at += static_cast<long long>(team.workers) * p.D) {
      const long long row = head + team.worker;
      const bool live = RowTeam<LAYOUT>::kCta || row < row1;
      auto mine = [&](int i) { return (t + i * nt) * VEC < p.D && live; };  // whether this thread has vector i
      const uint8_t* slot = LAYOUT == kRing ? ring.take() : nullptr;
      const TS* s_row = LAYOUT == kRing ? reinterpret_cast<const TS*>(slot) : static_cast<const TS*>(p.s) + at;
      const TX* dy_row = LAYOUT == kRing ? reinterpret_cast<const TX*>(slot + ring.off[1]) : static_cast<const TX*>(p.dy) + at;
      const TS* ds_row = LAYOUT == kRing ? reinterpret_cast<const TS*>(slot + ring.off[2]) : static_cast<const TS*>(p.ds) + at;
      const TX* x_row = LAYOUT == kRing ? reinterpret_cast<const TX*>(slot + ring.off[3]) : static_cast<const TX*>(p.x) + at;
      const float* gate_row = LAYOUT == kRing ? reinterpret_cast<const float*>(slot + ring.off[4]) : p.gate + at;
      R tt[NV];  // t = the gradient of s, then that of gate p
      R held_s[NH], held_dy[NH], held_x[NH], held_g[NH];
      if (kHold) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (t + i * nt) * VEC, h = kHold ? i : 0;
          if (!mine(i)) continue;
          tt[i].fill(0.f);
          held_x[h].fill(0.f);
          if (p.norm) {
            held_s[h].load(s_row + c);
            held_dy[h].load(dy_row + c);
          }
          if (has_ds) tt[i].load(ds_row + c);
          if (need_x) held_x[h].load(x_row + c);
          if (row_gate) held_g[h].load(gate_row + c);
        }
      }
      auto s_of = [&](int i) -> R {
        if (kHold) return held_s[kHold ? i : 0];
        R w;
        w.load(s_row + (t + i * nt) * VEC);
        return w;
      };
      auto dy_of = [&](int i) -> R {
        if (kHold) return held_dy[kHold ? i : 0];
        R w;
        w.load(dy_row + (t + i * nt) * VEC);
        return w;
      };
      auto x_of = [&](int i) -> R {
        if (kHold) return held_x[kHold ? i : 0];
        R w;
        w.fill(0.f);
        if (need_x) w.load(x_row + (t + i * nt) * VEC);
        return w;
      };
      auto gate_of = [&](int i) -> R {
        if (kHold) return held_g[kHold ? i : 0];
        R w;
        w.load(gate_row + (t + i * nt) * VEC);
        return w;
      };
      float r = 0.f, mean = 0.f;  // one over rms(s); minus the mean of dn n, over rms(s)
      // From partial(k, sums), which adds this thread's share of the sums of (k v)^2 and of d (k v): one over rms(v), and
      // minus the mean of d v / rms(v), over rms(v).
      auto statistics = [&](auto&& partial) {
        float sums[2] = {0.f, 0.f};
        partial(1.f, sums);
        team.sums(sums);
        r = rsqrtf(sums[0] * inv_d + p.eps);
        mean = -(sums[1] * r * inv_d) * r;
        const bool over = overflowed(sums[0]);
        if (RowTeam<LAYOUT>::kCta ? over : __any_sync(0xffffffffu, over)) {
          sums[0] = sums[1] = 0.f;
          partial(kSmall, sums);
          team.sums(sums);
          if (over) {
            const float q = rsqrtf(sums[0] * inv_d);
            r = q * kSmall;
            mean = -(sums[1] * q * inv_d) * r;
          }
        }
      };
      if (p.norm)
        statistics([&](float k, float (&sums)[2]) {
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            if (!mine(i)) continue;
            const R ga = gamma_of(i), sv = scaled(s_of(i), k);
            R dn = dy_of(i);
#pragma unroll
            for (int j = 0; j < R::N; ++j) dn.v[j] = R::mul(dn.v[j], ga.v[j]);
            sums[0] += sv.square();
            sums[1] += sv.dot(dn);
          }
        });
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (t + i * nt) * VEC;
        if (!mine(i)) continue;
        R& tk = tt[i];
        if (!kHold) {
          tk.fill(0.f);
          if (has_ds) tk.load(ds_row + c);
        }
        if (p.norm) {
          const auto rs = R::all(r), m = R::all(mean);
          const R ga = gamma_of(i), sv = s_of(i), dn = dy_of(i);
#pragma unroll
          for (int j = 0; j < R::N; ++j) {
            const auto n = R::mul(sv.v[j], rs);
            dga[i].v[j] = R::fma(dn.v[j], n, dga[i].v[j]);
            tk.v[j] = R::fma(R::mul(dn.v[j], ga.v[j]), rs, R::fma(n, m, tk.v[j]));
          }
        }
        if (p.dresidual && DA_BOUNDS_V(row < p.rows && c + VEC <= p.D, row)) tk.store(static_cast<TS*>(p.dresidual) + at + c);
#pragma unroll
        for (int j = 0; j < R::N; ++j) tk.v[j] = R::mul(tk.v[j], scale);
      }
      r = 1.f, mean = 0.f;
      if (p.post)  // of x
        statistics([&](float k, float (&sums)[2]) {
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            if (!mine(i)) continue;
            const R cv = c_of(i), xv = scaled(x_of(i), k);
            R d;
#pragma unroll
            for (int j = 0; j < R::N; ++j) d.v[j] = R::mul(tt[i].v[j], cv.v[j]);
            if (row_gate) {
              const R gv = gate_of(i);
#pragma unroll
              for (int j = 0; j < R::N; ++j) d.v[j] = R::mul(d.v[j], gv.v[j]);
            }
            sums[0] += xv.square();
            sums[1] += xv.dot(d);
          }
        });
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (t + i * nt) * VEC;
        if (!mine(i)) continue;
        const auto rx = R::all(r), m = R::all(mean);
        const R cv = c_of(i);
        R out, xh = x_of(i), dp = tt[i];
        if (row_gate) {
          const R gv = gate_of(i);
#pragma unroll
          for (int j = 0; j < R::N; ++j) dp.v[j] = R::mul(dp.v[j], gv.v[j]);
        }
#pragma unroll
        for (int j = 0; j < R::N; ++j) {
          // (without the norm rx = 1, m = 0, and c is the gate alone)
          xh.v[j] = R::mul(xh.v[j], rx);
          u[i].v[j] = R::fma(dp.v[j], xh.v[j], u[i].v[j]);
          out.v[j] = R::fma(R::mul(dp.v[j], cv.v[j]), rx, R::mul(xh.v[j], m));
        }
        const bool in = DA_BOUNDS_V(row < p.rows && c + VEC <= p.D, row);
        if (p.dx && in) out.store(static_cast<TX*>(p.dx) + at + c);
        if (row_gate && p.part_gate && in) {
#pragma unroll
          for (int j = 0; j < R::N; ++j) xh.v[j] = R::mul(R::mul(tt[i].v[j], xh.v[j]), cv.v[j]);
          xh.store(p.part_gate + at + c);
        }
      }
      if (LAYOUT == kRing) {
        __syncthreads();  // (every thread has read the slot)
        ring.refill(row + p.stages, end);
      }
    }
    if (p.part_post) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (t + i * nt) * VEC;
        if (c >= p.D) continue;
        R sum;
        sum.load(post_sums + c);
        const R gv = column(group_gate, i);  // (with a gate a row it is in u)
#pragma unroll
        for (int j = 0; j < R::N; ++j) sum.v[j] = R::fma(u[i].v[j], gv.v[j], sum.v[j]);
        sum.store(post_sums + c);
      }
    }
    if (p.part_gate && !row_gate) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if ((t + i * nt) * VEC >= p.D) continue;
        const R w = column(p.gamma_post, i);
#pragma unroll
        for (int j = 0; j < R::N; ++j) u[i].v[j] = R::mul(u[i].v[j], w.v[j]);
      }
      if (DA_BOUNDS_V((ch * p.groups + g + 1) * p.D <= p.pieces * p.D, ch))
        write_columns<VEC, NV, LAYOUT>(team, u, p.part_gate + (ch * p.groups + g) * p.D, p.D, reinterpret_cast<float*>(smem));
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) u[i].fill(0.f);
  }
  const long long out = static_cast<long long>(blockIdx.x) * p.D;
  if (p.part_gamma) write_columns<VEC, NV, LAYOUT>(team, dga, p.part_gamma + out, p.D, reinterpret_cast<float*>(smem));
  if (p.part_post) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if ((t + i * nt) * VEC < p.D) u[i].load(post_sums + (t + i * nt) * VEC);
    write_columns<VEC, NV, LAYOUT>(team, u, p.part_post + out, p.D, reinterpret_cast<float*>(smem));
  }
  if (LAYOUT == kRing && threadIdx.x == 0) ring.drain(end - piece_row(first));
}

// ----------------------------------------------------------------- the backward pass of wide rows
// residual_norm_grad_kernel's work for rows of 16-byte multiples up to 4096 with dy given, which is bound by
// instructions (16384 x 2048 took 496 a warp and row, 104 us): two rows at once, whose four sums share one butterfly and
// one barrier, and whose parameters stay in registers; no branch in a row depends on the thread (threads past the row
// compute its first columns again and count for nothing): 73 us.

// Sums of four values over the warp: lane l gets that of value (l >> 3) & 3.
__device__ __forceinline__ float warp_sum4(float a, float b, float c, float d) {
  const int lane = threadIdx.x & 31;
  const bool hi = lane & 16, mid = lane & 8;
  float x = hi ? c : a, y = hi ? d : b;
  x += __shfl_xor_sync(0xffffffffu, hi ? a : c, 16);
  y += __shfl_xor_sync(0xffffffffu, hi ? b : d, 16);
  float z = mid ? y : x;
  z += __shfl_xor_sync(0xffffffffu, mid ? x : y, 8);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  return z;
}
// The same over the CTA (up to 16 warps; buf: 64 floats that nothing else uses until the next but one barrier).
__device__ __forceinline__ float4 cta_sum4(float a, float b, float c, float d, float* buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const float z = warp_sum4(a, b, c, d);
  if ((lane & 7) == 0) buf[16 * (lane >> 3) + warp] = z;  // [value][warp]
  __syncthreads();
  // lane: value lane / 8, warps lane % 8 and 8 more
  const int w = lane & 7;
  const float* at = buf + 16 * (lane >> 3) + w;
  float t = w < nw ? at[0] : 0.f;
  if (w + 8 < nw) t += at[8];
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  return make_float4(__shfl_sync(0xffffffffu, t, 0), __shfl_sync(0xffffffffu, t, 8), __shfl_sync(0xffffffffu, t, 16),
                     __shfl_sync(0xffffffffu, t, 24));
}

template <typename T>
__device__ __forceinline__ void load_shared8(Row<8>& r, uint32_t addr) {
  if (sizeof(T) == 2) {
    uint32_t x[4];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(addr));
#pragma unroll
    for (int j = 0; j < 4; ++j) r.v[j] = f2pack(__uint_as_float(x[j] << 16), __uint_as_float(x[j] & 0xffff0000u));
  } else {
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(r.v[0]), "=l"(r.v[1]) : "r"(addr));
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(r.v[2]), "=l"(r.v[3]) : "r"(addr + 16));
  }
}

template <typename TX, typename TS, bool POST>
__global__ void __launch_bounds__(512) residual_norm_grad_pairs_kernel(const NormParams p) {
  using R = Row<8>;
  __shared__ float buf[128];
  extern __shared__ __align__(128) uint8_t smem[];
  const float inv_d = 1.f / static_cast<float>(p.D);
  const bool row_gate = p.gate && p.gate_rows == p.rows;
  const long long first = p.pieces * blockIdx.x / gridDim.x, last = p.pieces * (blockIdx.x + 1ll) / gridDim.x;
  auto piece_row = [&](long long piece) {
    const long long g = piece / p.chunks;
    return min(g * p.group_rows + (piece - g * p.chunks) * p.chunk_rows, (g + 1) * p.group_rows);
  };
  const bool need_x = POST || p.part_gate, has_ds = p.ds != nullptr;
  RowRing ring(smem, p.stages, p.status);
  const uint32_t bx = p.D * static_cast<uint32_t>(sizeof(TX)), bs = p.D * static_cast<uint32_t>(sizeof(TS));
  ring.add(0, p.s, bs);
  ring.add(1, p.dy, bx);
  ring.add(2, p.ds, has_ds ? bs : 0u);
  ring.add(3, p.x, need_x ? bx : 0u);
  ring.add(4, p.gate, row_gate ? p.D * 4u : 0u);
  if (threadIdx.x == 0) ring.init();
  grid_dep_wait();
  const long long start = piece_row(first), end = piece_row(last);
  if (threadIdx.x == 0) ring.start(start, end, 1);
  __syncthreads();
  grid_dep_launch_dependents();

  const bool mine = static_cast<int>(threadIdx.x) * 8 < p.D;
  const int c = mine ? threadIdx.x * 8 : 0;
  const uint32_t base = smem_u32(smem) + RowRing::kBytes;
  const uint32_t o_s = c * sizeof(TS), o_dy = ring.off[1] + c * sizeof(TX), o_ds = ring.off[2] + c * sizeof(TS),
                 o_x = ring.off[3] + c * sizeof(TX), o_g = ring.off[4] + c * 4;
  R dga, u, ga, cv;
  dga.fill(0.f);
  u.fill(0.f);
  ga.fill(1.f);
  if (p.gamma) ga.load(p.gamma + c);
  float* post_sums = reinterpret_cast<float*>(smem + p.off_post);
  if (p.part_post && mine) u.store(post_sums + c);
  const auto scale = R::all(p.scale);

  for (long long piece = first; piece < last; ++piece) {
    const long long g = piece / p.chunks, ch = piece - g * p.chunks;
    const long long row0 = piece_row(piece), row1 = min(row0 + p.chunk_rows, (g + 1) * p.group_rows);
    R gv;  // the group's gate
    gv.fill(1.f);
    if (p.gate && !row_gate) gv.load(p.gate + g * p.D + c);
    cv.fill(1.f);
    if (POST && p.gamma_post) cv.load(p.gamma_post + c);
#pragma unroll
    for (int j = 0; j < 4; ++j) cv.v[j] = mul2(cv.v[j], gv.v[j]);
    long long at = row0 * p.D + c;
    // Rows row and, with RR = 2, row + 1.
    auto rows_at_once = [&](long long row, auto count) {
      constexpr int RR = decltype(count)::value;
      R tt[RR];
      uint32_t slot[RR];
      float q[2], dot[2], r[2], mean[2];
      // From partial(k, f, q, dot), this thread's share of the sums of (f v)^2 and of d (f v) of row k: one over rms(v), and
      // minus the mean of d v / rms(v), over rms(v).
      auto statistics = [&](auto&& partial, float* at) {
        q[1] = dot[1] = 0.f;
#pragma unroll
        for (int k = 0; k < RR; ++k) {
          partial(k, 1.f, q[k], dot[k]);
          if (!mine) q[k] = dot[k] = 0.f;
        }
        float4 sums = cta_sum4(q[0], dot[0], q[1], dot[1], at);
        q[0] = sums.x, dot[0] = sums.y, q[1] = sums.z, dot[1] = sums.w;
        const bool over = overflowed(q[0]) || overflowed(q[1]);
#pragma unroll
        for (int k = 0; k < RR; ++k) {
          r[k] = rsqrtf(q[k] * inv_d + p.eps);
          mean[k] = -(dot[k] * r[k] * inv_d) * r[k];
        }
        if (over) {  // (the same for every thread)
          __syncthreads();
          float w[2] = {0.f, 0.f}, e[2] = {0.f, 0.f};
          for (int k = 0; k < RR; ++k) {
            partial(k, kSmall, w[k], e[k]);
            if (!mine) w[k] = e[k] = 0.f;
          }
          sums = cta_sum4(w[0], e[0], w[1], e[1], at);
          w[0] = sums.x, e[0] = sums.y, w[1] = sums.z, e[1] = sums.w;
          for (int k = 0; k < RR; ++k)
            if (overflowed(q[k])) {
              const float s = rsqrtf(w[k] * inv_d);
              r[k] = s * kSmall;
              mean[k] = -(e[k] * s * inv_d) * r[k];
            }
        }
      };
#pragma unroll
      for (int k = 0; k < RR; ++k) slot[k] = base + ring.take_slot(k) * ring.slot_bytes;
      statistics(
          [&](int k, float f, float& square, float& dots) {
            R sv, dn;
            load_shared8<TS>(sv, slot[k] + o_s);
            load_shared8<TX>(dn, slot[k] + o_dy);
            if (f != 1.f) sv = scaled(sv, f);
#pragma unroll
            for (int j = 0; j < 4; ++j) dn.v[j] = mul2(dn.v[j], ga.v[j]);
            square = sv.square();
            dots = sv.dot(dn);
          },
          buf);
#pragma unroll
      for (int k = 0; k < RR; ++k) {
        const auto rs = R::all(r[k]), m = R::all(mean[k]);
        R sv, dn;
        tt[k].fill(0.f);
        if (has_ds) load_shared8<TS>(tt[k], slot[k] + o_ds);
        load_shared8<TS>(sv, slot[k] + o_s);
        load_shared8<TX>(dn, slot[k] + o_dy);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t n = mul2(sv.v[j], rs);
          dga.v[j] = fma2(dn.v[j], n, dga.v[j]);
          tt[k].v[j] = fma2(mul2(dn.v[j], ga.v[j]), rs, fma2(n, m, tt[k].v[j]));
        }
        if (p.dresidual && mine && DA_BOUNDS_V(row + k < p.rows && c + 8 <= p.D, row)) tt[k].store(static_cast<TS*>(p.dresidual) + at + k * p.D);
#pragma unroll
        for (int j = 0; j < 4; ++j) tt[k].v[j] = mul2(tt[k].v[j], scale);
      }
      if (POST)  // of x
        statistics(
            [&](int k, float f, float& square, float& dots) {
              R xv, d;
              load_shared8<TX>(xv, slot[k] + o_x);
              if (f != 1.f) xv = scaled(xv, f);
#pragma unroll
              for (int j = 0; j < 4; ++j) d.v[j] = mul2(tt[k].v[j], cv.v[j]);
              if (row_gate) {
                R gr;
                load_shared8<float>(gr, slot[k] + o_g);
#pragma unroll
                for (int j = 0; j < 4; ++j) d.v[j] = mul2(d.v[j], gr.v[j]);
              }
              square = xv.square();
              dots = xv.dot(d);
            },
            buf + 64);
#pragma unroll
      for (int k = 0; k < RR; ++k) {
        const auto rx = R::all(POST ? r[k] : 1.f), m = R::all(POST ? mean[k] : 0.f);
        R xh, out;
        xh.fill(0.f);
        if (need_x) load_shared8<TX>(xh, slot[k] + o_x);
        uint64_t dp[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) dp[j] = tt[k].v[j];
        if (row_gate) {
          R gr;
          load_shared8<float>(gr, slot[k] + o_g);
#pragma unroll
          for (int j = 0; j < 4; ++j) dp[j] = mul2(dp[j], gr.v[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (POST) xh.v[j] = mul2(xh.v[j], rx);
          u.v[j] = fma2(dp[j], xh.v[j], u.v[j]);
          out.v[j] = mul2(dp[j], cv.v[j]);
          if (POST) out.v[j] = fma2(out.v[j], rx, mul2(xh.v[j], m));
        }
        const bool in = mine && DA_BOUNDS_V(row + k < p.rows && c + 8 <= p.D, row);
        if (p.dx && in) out.store(static_cast<TX*>(p.dx) + at + k * p.D);
        if (row_gate && p.part_gate) {
#pragma unroll
          for (int j = 0; j < 4; ++j) xh.v[j] = mul2(mul2(tt[k].v[j], xh.v[j]), cv.v[j]);
          if (in) xh.store(p.part_gate + at + k * p.D);
        }
      }
      __syncthreads();  // (every thread has read the slots)
#pragma unroll
      for (int k = 0; k < RR; ++k) ring.refill(row + k + p.stages, end);
      at += RR * static_cast<long long>(p.D);
    };
    long long row = row0;
    for (; row + 1 < row1; row += 2) rows_at_once(row, ActTag<2>{});
    if (row < row1) rows_at_once(row, ActTag<1>{});

    if (p.part_post && mine) {
      R sum;
      sum.load(post_sums + c);
#pragma unroll
      for (int j = 0; j < 4; ++j) sum.v[j] = fma2(u.v[j], gv.v[j], sum.v[j]);  // (with a gate a row it is in u)
      sum.store(post_sums + c);
    }
    if (p.part_gate && !row_gate) {
      R w;
      w.fill(1.f);
      if (POST && p.gamma_post) w.load(p.gamma_post + c);
#pragma unroll
      for (int j = 0; j < 4; ++j) w.v[j] = mul2(u.v[j], w.v[j]);
      if (mine && DA_BOUNDS_V((ch * p.groups + g + 1) * p.D <= p.pieces * p.D, ch)) w.store(p.part_gate + (ch * p.groups + g) * p.D + c);
    }
    u.fill(0.f);
  }
  const long long out = static_cast<long long>(blockIdx.x) * p.D + c;
  if (p.part_gamma && mine) dga.store(p.part_gamma + out);
  if (p.part_post && mine) {
    u.load(post_sums + c);
    u.store(p.part_post + out);
  }
  if (threadIdx.x == 0) ring.drain(end - start);
}

}  // namespace da
