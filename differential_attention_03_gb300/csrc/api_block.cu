// C entry points of what stands around the attention layer in a block: the
// products with their epilogue, the gated feed-forward product, the norms with
// gate and residual, and their backward passes: argument validation, TMA
// descriptors, launch shapes.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "block_params.h"
#include "diffattn.h"
#include "host.h"
#include "launch.h"
#include "linear_params.h"

namespace {

namespace dh = da::host;

diffattn_status fail(diffattn_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return dh::error(s, buf);
}

diffattn_status cuda_fail(cudaError_t e, const char* fn) {
  return fail(DIFFATTN_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
}

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

int sms_or_default() {
  const int s = dh::sms();
  return s > 0 ? s : 152;
}

// ---- overlap
// A tensor of a call: `rows` rows of `width` bytes, `ld` bytes apart.
struct Span {
  const void* at;
  long long rows, width, ld;
};

Span flat(const void* at, long long bytes) { return Span{at, 1, bytes, bytes}; }

bool overlap(const Span& a, const Span& b) {
  if (!a.at || !b.at || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  const uintptr_t xn = x + static_cast<uintptr_t>((a.rows - 1) * a.ld + a.width);
  const uintptr_t yn = y + static_cast<uintptr_t>((b.rows - 1) * b.ld + b.width);
  if (x >= yn || y >= xn) return false;
  // Rows of the same stride that lie side by side: b's columns behind a's, and the next row of a behind b's.
  const long long ld = a.rows > 1 ? a.ld : b.ld;
  if ((a.rows == 1 || a.ld == ld) && (b.rows == 1 || b.ld == ld) && a.width <= ld && b.width <= ld) {
    const long long off = static_cast<long long>((y >= x ? (y - x) % static_cast<uintptr_t>(ld)
                                                         : (static_cast<uintptr_t>(ld) - (x - y) % static_cast<uintptr_t>(ld)) %
                                                               static_cast<uintptr_t>(ld)));
    if (off >= a.width && off + b.width <= ld) return false;
  }
  return true;
}

// What a call writes overlaps nothing else of it.
diffattn_status disjoint(const char* fn, const Span* written, int nw, const Span* read, int nr) {
  for (int i = 0; i < nw; ++i) {
    for (int j = 0; j < nr; ++j)
      if (overlap(written[i], read[j])) return fail(DIFFATTN_ERR_SHAPE, "%s: an output overlaps an input", fn);
    for (int j = 0; j < i; ++j)
      if (overlap(written[i], written[j])) return fail(DIFFATTN_ERR_SHAPE, "%s: outputs overlap", fn);
  }
  return DIFFATTN_OK;
}

// ---- arguments of the products
bool bad_act(int act) { return act < DIFFATTN_ACT_NONE || act > DIFFATTN_ACT_SILU; }
bool bad_dtype(int dt) { return dt != DIFFATTN_BF16 && dt != DIFFATTN_F32; }

// A matrix of rows `width` wide, `ld` apart, elements of `es` bytes: aligned for 16-byte accesses.
diffattn_status check_rows(const char* fn, const char* name, const void* at, long long width, long long ld, int es) {
  if (!at) return fail(DIFFATTN_ERR_NULL, "%s: %s is NULL", fn, name);
  if (!aligned(at, 16)) return fail(DIFFATTN_ERR_ALIGN, "%s: %s must be 16-byte aligned", fn, name);
  if (ld < width || ld % (16 / es) != 0 || ld > (1ll << 36))
    return fail(DIFFATTN_ERR_SHAPE, "%s: row stride %lld of %s: at least %lld, a multiple of %d", fn, ld, name, width, 16 / es);
  return DIFFATTN_OK;
}

diffattn_status check_workspace(const char* fn, const void* ws, size_t bytes, size_t need) {
  if (need == 0) return DIFFATTN_OK;
  if (!ws) return fail(DIFFATTN_ERR_NULL, "%s: NULL workspace", fn);
  if (bytes < need) return fail(DIFFATTN_ERR_SHAPE, "%s: workspace of %zu bytes, %zu needed", fn, bytes, need);
  if (!aligned(ws, 256)) return fail(DIFFATTN_ERR_ALIGN, "%s: workspace not 256-byte aligned", fn);
  return DIFFATTN_OK;
}

// 2-D map over bf16 rows: box = 64 columns (128 bytes, swizzled) x box_rows rows; zeros past the edges.
diffattn_status map_rows(CUtensorMap* m, const void* base, long long rows, long long cols, long long ld, int box_rows) {
  dh::EncodeTiled enc;
  diffattn_status s = dh::encoder(&enc);
  if (s != DIFFATTN_OK) return s;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(DIFFATTN_ERR_CUDA, "cuTensorMapEncodeTiled failed (CUresult %d)", (int)r);
  return DIFFATTN_OK;
}

// 3-D map for stores of 32 rows x 128 bytes (swizzled) into rows of `sides` parts of `cols` columns; what lies past an
// edge is dropped.
diffattn_status map_out(CUtensorMap* m, void* base, long long rows, int sides, long long cols, long long ld, bool f32) {
  dh::EncodeTiled enc;
  diffattn_status s = dh::encoder(&enc);
  if (s != DIFFATTN_OK) return s;
  const cuuint64_t es = f32 ? 4 : 2;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(sides), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(sides > 1 ? cols : ld) * es, static_cast<cuuint64_t>(ld) * es};
  const cuuint32_t box[3] = {f32 ? 32u : 64u, 1, 32};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(DIFFATTN_ERR_CUDA, "cuTensorMapEncodeTiled failed (CUresult %d)", (int)r);
  return DIFFATTN_OK;
}

enum class Kind { kForward, kGated, kDgrad, kWgrad };

constexpr int kGroupRows = 2048;  // rows of a group of the tile walk

// A product: out [M, N] over a contraction of K.  x: the token rows [M, K] (wgrad: [K, M]); w: [N, K] (gated [2 N, K];
// dgrad and wgrad [K, N]), rows ldx and ldw apart.
struct Product {
  Kind kind;
  int epi;
  const void* x;
  const void* w;
  long long ldx, ldw;
};

// linear_kernel's tiles in clusters of cg CTAs.
long long tile_count(const Product& q, const da::LinearParams& p, int cg) {
  const int bn = q.kind == Kind::kGated ? da::kLinBN / 2 : da::kLinBN;
  return ((p.M + da::kLinBM * cg - 1ll) / (da::kLinBM * cg)) * ((p.N + bn - 1ll) / bn);
}

// Tiles before the ones that come in halves: those of whole rounds, if half of the clusters or fewer have work after them.
long long full_tiles(long long tiles, long long clusters) {
  const long long rest = tiles % clusters;
  return 2 * rest <= clusters ? tiles - rest : tiles;
}

// How linear_kernel's tiles are laid out: SM pairs or single SMs, tiles before the ones that come in halves, and an
// estimate of the time.
struct TilePlan {
  int cg;
  long long full;
  double cost;
};

// Estimates in us, fitted to whole and half tiles on pairs and single SMs over 64 products from 160 x 1024 x 512 to
// 1000 x 2048 x 8192 and 16384 x 512 x 512 with inputs beyond L2 on a GB300 (the choice takes 0.3 % more than the best of
// the four on average, 3 % at worst): a K block takes so long, or what the CTAs of its round draw from L2 at 20 MB a
// us; a tile at least its epilogue; beside them what a call costs.  (Pairs throughout, halves in the last round alone:
// 777 x 1024 x 1024 8.9 us, 2048 x 1024 x 1024 9.0, 4096 x 256 x 256 5.6; single SMs' halves 5.5, 5.7 and 3.4.)
TilePlan make_tile_plan(const Product& q, const da::LinearParams& p, int sms) {
  static const double block[2][2] = {{0.318, 0.191}, {0.261, 0.145}}, call[2][2] = {{3.7, 2.75}, {5.55, 4.8}};
  static const double least[2] = {1.35, 0.57};  // [whole, half]
  const int kblocks = (p.K + da::kLinBK - 1) / da::kLinBK;
  TilePlan best = {};
  for (int cg = 1; cg <= 2; ++cg) {
    const long long tiles = tile_count(q, p, cg), clusters = sms / cg;
    auto rounds = [&](long long n, int half) {
      const double bytes = (da::kLinBM + da::kLinBN / cg / (half ? 2 : 1)) * da::kLinBK * 2.0;
      auto round = [&](long long at_work) {
        return std::max(kblocks * std::max(block[cg - 1][half], bytes * at_work * cg / 20e6), least[half]);
      };
      return n / clusters * round(clusters) + (n % clusters ? round(n % clusters) : 0.0);
    };
    for (int half = 0; half <= 1; ++half) {
      const long long full = half ? 0 : full_tiles(tiles, clusters);
      const double cost = call[cg - 1][half] + rounds(full, 0) + rounds(2 * (tiles - full), 1);
      if (best.cg == 0 || cost < best.cost) best = TilePlan{cg, full, cost};
    }
  }
  return best;
}

// Clusters of cs CTAs of linear_few_kernel, one CTA an SM, that run at once: clusters of 4 and 8 do not fill every SM.
int cluster_slots(int cs, int sms) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][4];
  int dev = 0;
  if (cs <= 2 || cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return std::max(1, sms / cs);
  std::atomic<int>& slot = known[dev][cs == 4 ? 2 : 3];
  int n = slot.load();
  if (n == 0) {
    if (da::linear_few_clusters(cs, &n) != cudaSuccess || n < 1) {
      cudaGetLastError();
      n = std::max(1, sms / cs);
    }
    slot.store(n);
  }
  return n;
}

// How the products for few tokens lay their work out; nt = 0: linear_kernel's tiles suit it better.
struct FewPlan {
  int nt, width, cs, lg, stages, off_bars, turns, smem;
  long long tiles;
};

// Estimates in us, fitted to a sweep of widths and clusters over 54 products from 1 x 1024 x 1024 to 2048 x 1024 x 1024
// and 16 x 8192 x 8192, weights beyond L2, on a GB300 (the choice takes 0.6 % more than the best width and cluster on
// average, 7 % at worst; between it and linear_kernel's tiles 0.7 % and 7 %): HBM 6.1 MB a us together with an SM's own
// stream (167 KB a us, dgrad's boxes 143; at least 0.105 us a K block; all together 32 MB a us), what a cluster's CTAs
// hand each other (12.7 KB a us), the epilogue, and what a call costs.
FewPlan make_few_plan(const Product& q, const da::LinearParams& p, int sms, double least) {
  FewPlan best = {};
  if (q.kind == Kind::kWgrad) return best;
  const int sides = q.kind == Kind::kGated ? 2 : 1;
  const int nt = p.M >= 128 ? 128 : (p.M + 15) / 16 * 16;
  const long long ttiles = (p.M + nt - 1ll) / nt;
  const int kblocks = (p.K + da::kLinBK - 1) / da::kLinBK;
  const int step = q.kind == Kind::kDgrad ? 64 : sides == 2 ? 8 : 16, most = 256 / sides;
  const double hbm = 2.0 * sides * p.N * p.K / 6.1e6, draw = q.kind == Kind::kDgrad ? 143e3 : 167e3;
  if (ttiles * p.N > 0x7fffffffll) return best;
  for (int cs = 1; cs <= 8 && cs <= kblocks; cs *= 2) {
    const int at_once = cluster_slots(cs, sms);
    const int nkb = (kblocks + cs - 1) / cs;
    for (int width = step; width <= most && width < p.N + step; width += step) {
      const int wrows = width * sides, lg = (width / 8 + cs - 1) / cs;
      // fp32 outputs: segments of kLinSegBlocks, more than tensor memory has accumulators for, take turns in them.
      const bool turns = q.epi == da::kEpiF32 && da::few_segment_blocks(nkb, wrows) > da::kLinSegBlocks;
      if (turns && da::few_turns(wrows) == 0) continue;
      const long long tiles = ttiles * ((p.N + width - 1) / width);
      const double rounds = static_cast<double>((tiles + at_once - 1) / at_once);
      const double stream = rounds * nkb * std::max({(wrows + nt) * 128.0 / draw, (wrows + nt) * 128.0 * std::min<long long>(tiles, at_once) * cs / 32e6, 0.105});
      const double end = (cs > 1 ? 0.28 + nt * wrows * (4.0 / 12.7e3) * (cs - 1) / cs : 0.0) + std::min(p.M, nt) * lg * sides * 0.001 + wrows * 0.0031;
      const double cost = 1.8 + std::sqrt(stream * stream + hbm * hbm) + rounds * end + (rounds - 1) * 0.4;
      if (cost >= least) continue;
      // ring, partial sums (and, behind the last slot's token rows, what an MMA of 128 rows reads), barriers
      const int stage = (wrows + nt) * 128, part = std::max(cs * nt * (lg * sides * 8 + 4) * 4, (128 - nt) * 128);
      const int budget = (rounds > 1 ? 113 * 1024 : da::kFewMaxSmem) - 1024 - part - 512;
      const int stages = std::min({nkb, budget / stage, 24});
      if (stages < 1 || (stages < 3 && stages < nkb)) continue;
      least = cost;
      best.nt = nt, best.width = width, best.cs = cs, best.lg = lg, best.stages = stages, best.tiles = tiles;
      best.off_bars = stages * stage + part;
      best.turns = turns ? 1 : 0;
      best.smem = best.off_bars + (2 * stages + 5) * 8 + 16 + 1024;
    }
  }
  return best;
}

struct Plan {
  FewPlan few;
  TilePlan tile;
};

// The plans of the sizes that this thread asked for last.
Plan product_plan(const Product& q, const da::LinearParams& p, int sms) {
  struct Known {
    int kind, epi, M, N, K, sms;
    Plan plan;
  };
  constexpr unsigned kEntries = 64;
  static thread_local Known known[kEntries];  // (sms = 0: none yet)
  const int kind = static_cast<int>(q.kind);
  const unsigned h = static_cast<unsigned>(p.M) * 2654435761u ^ static_cast<unsigned>(p.N) * 40503u ^ static_cast<unsigned>(p.K) * 9973u ^
                     static_cast<unsigned>(4 * kind + q.epi) * 131u;
  Known& k = known[(h >> 7) % kEntries];
  if (k.sms != sms || k.kind != kind || k.epi != q.epi || k.M != p.M || k.N != p.N || k.K != p.K) {
    const TilePlan t = make_tile_plan(q, p, sms);
    k = Known{kind, q.epi, p.M, p.N, p.K, sms, {make_few_plan(q, p, sms, p.M > 128 ? t.cost : 1e30), t}};
  }
  return k.plan;
}

// Sizes of a product whose indexes, to the end of the last tile, do not fit 31 bits.
bool past_31_bits(int M, int N, int K) {
  return M + 2ll * da::kLinBM > 0x7fffffffll || 2ll * N + 2 * da::kLinBN > 0x7fffffffll || static_cast<long long>(K) + da::kLinBK > 0x7fffffffll;
}

// Descriptors, tiles, status word and launch of a product whose sizes and epilogue are in p.
diffattn_status launch_product(const char* fn, const Product& q, da::LinearParams& p, cudaStream_t s) {
  diffattn_status st = dh::status_address(&p.status);
  if (st != DIFFATTN_OK) return st;
  const int sms = sms_or_default();
  if (past_31_bits(p.M, p.N, p.K)) return fail(DIFFATTN_ERR_SHAPE, "%s: too large", fn);
  const bool x_mn = q.kind == Kind::kWgrad, w_mn = x_mn || q.kind == Kind::kDgrad;
  const long long wrows = q.kind == Kind::kGated ? 2ll * p.N : p.N;
  auto map_w = [&](CUtensorMap* m, int box) {
    return w_mn ? map_rows(m, q.w, p.K, p.N, q.ldw, 64) : map_rows(m, q.w, wrows, p.K, q.ldw, box);
  };
  auto map_x = [&](CUtensorMap* m, int box) {
    return x_mn ? map_rows(m, q.x, p.K, p.M, q.ldx, 64) : map_rows(m, q.x, p.M, p.K, q.ldx, box);
  };
  cudaError_t e;
  const Plan plan = product_plan(q, p, sms);
  const FewPlan& f = plan.few;
  if (f.nt) {
    p.nt = f.nt, p.width = f.width, p.cs = f.cs, p.lg = f.lg, p.stages = f.stages, p.off_bars = f.off_bars, p.turns = f.turns;
    p.tiles_n = (p.N + f.width - 1) / f.width;
    if ((st = map_w(&p.tm_a, f.width)) != DIFFATTN_OK) return st;
    if ((st = map_x(&p.tm_b, f.nt)) != DIFFATTN_OK) return st;
    if (f.tiles * f.cs > 0x7fffffffll) return fail(DIFFATTN_ERR_SHAPE, "%s: too large", fn);
    e = da::launch_linear_few(p, q.epi, w_mn, static_cast<int>(f.tiles * f.cs), f.smem, s);
  } else {
    const int bn = q.kind == Kind::kGated ? da::kLinBN / 2 : da::kLinBN;
    p.tiles_n = (p.N + bn - 1) / bn;
    const int cg = plan.tile.cg;
    const int bm = da::kLinBM * cg;
    p.tiles_m = (p.M + bm - 1) / bm;
    p.group_m = kGroupRows / bm;
    const long long tiles = tile_count(q, p, cg), clusters = sms / cg;
    if (2 * tiles > 0x7fffffffll - sms) return fail(DIFFATTN_ERR_SHAPE, "%s: too large", fn);
    p.full = static_cast<int>(plan.tile.full);
    if ((st = map_x(&p.tm_a, 128)) != DIFFATTN_OK) return st;
    if ((st = map_w(&p.tm_b, 64)) != DIFFATTN_OK) return st;
    if ((st = map_out(&p.tm_out, p.out, p.M, 1, p.N, p.ldo, q.epi == da::kEpiF32)) != DIFFATTN_OK) return st;
    if (p.pre && (st = map_out(&p.tm_pre, p.pre, p.M, q.kind == Kind::kGated ? 2 : 1, p.N, p.ldp, false)) != DIFFATTN_OK) return st;
    const int grid = static_cast<int>(std::min(p.full + 2 * (tiles - p.full), clusters)) * cg;
    e = q.kind == Kind::kDgrad   ? da::launch_linear_dgrad(p, cg, grid, s)
        : q.kind == Kind::kWgrad ? da::launch_linear_wgrad(p, q.epi, cg, grid, s)
                                 : da::launch_linear_fwd(p, q.epi, cg, grid, s);
  }
  if (e != cudaSuccess) return cuda_fail(e, fn);
  dh::count_launches(1);
  return DIFFATTN_OK;
}

// out [M, N] = dz [M, C] w [C, N], bf16.
diffattn_status dgrad(const char* fn, int M, int N, int C, const void* dz, long long ldz, const void* w, void* out,
                      cudaStream_t s) {
  da::LinearParams p;
  memset(&p, 0, sizeof(p));
  p.M = M, p.N = N, p.K = C;
  p.out = out, p.ldo = N;
  return launch_product(fn, Product{Kind::kDgrad, da::kEpiBf16, dz, w, ldz, N}, p, s);
}

// out [M, N] = dz^T a with dz [C, M] and a [C, N].
diffattn_status wgrad(const char* fn, int M, int N, int C, const void* dz, long long ldz, const void* a, long long lda,
                      void* out, diffattn_dtype dt, cudaStream_t s) {
  da::LinearParams p;
  memset(&p, 0, sizeof(p));
  p.M = M, p.N = N, p.K = C;
  p.out = out, p.ldo = N;
  return launch_product(fn, Product{Kind::kWgrad, dt == DIFFATTN_F32 ? da::kEpiF32 : da::kEpiBf16, dz, a, ldz, lda}, p, s);
}

// Sizes of a backward pass whose kernels' 32-bit indexes (a step past the last row, chunk or column block) do not overflow.
bool too_large(int M, int N, int K) { return M > 0x7ffe0000 || N > 0x3fff0000 || K > 0x3fff0000; }

// Row chunks of the element-wise kernels: some eight CTAs an SM, at least 32 rows each.
int act_grad_chunks(int M, int N) {
  const long long across = (N + 255ll) / 256;
  const long long want = (152 * 8 + across - 1) / across, most = (M + 31ll) / 32;
  return static_cast<int>(std::max(1ll, std::min({want, most, 65535ll})));
}

// Row chunks of the bias gradient.  Up to 64 rows are one chunk, whose column sums need no second kernel (64 x 8192, gelu:
// 5.9 us; 3.9 so; 128 x 1024 3.9, so 6.2).
int bias_chunks(int M, int N) { return M <= 64 ? 1 : act_grad_chunks(M, N); }

// Workspace of diffattn_linear_backward: the bias gradient's partial sums, then dz.
size_t bias_parts_bytes(int M, int N) { return round256(static_cast<size_t>(bias_chunks(M, N)) * N * 4); }
size_t linear_workspace(int M, int N, bool bent, bool dbias) {
  return (dbias && bias_chunks(M, N) > 1 ? bias_parts_bytes(M, N) : 0) + (bent ? round256(static_cast<size_t>(M) * N * 2) : 0);
}

diffattn_status act_grad(const char* fn, const da::ActGradParams& p, bool gated, cudaStream_t s) {
  const cudaError_t e = da::launch_act_grad(p, gated, s);
  if (e != cudaSuccess) return cuda_fail(e, fn);
  dh::count_launches(1);
  return DIFFATTN_OK;
}

diffattn_status sum_parts(const char* fn, const da::SumParts& p, cudaStream_t s) {
  const cudaError_t e = da::launch_sum_parts(p, s);
  if (e != cudaSuccess) return cuda_fail(e, fn);
  dh::count_launches(1);
  return DIFFATTN_OK;
}

diffattn_status zero(const char* fn, void* at, size_t bytes, cudaStream_t s) {
  if (!at || !bytes) return DIFFATTN_OK;
  const cudaError_t e = cudaMemsetAsync(at, 0, bytes, s);
  return e == cudaSuccess ? DIFFATTN_OK : cuda_fail(e, fn);
}

size_t dtype_bytes(int dt) { return dt == DIFFATTN_F32 ? 4 : 2; }

}  // namespace

extern "C" {

int diffattn_debug_product_plan(int kind, int M, int N, int K, int f32, int* plan) {
  if (kind < 0 || kind > 3 || M < 1 || N < 1 || K < 1 || !plan || past_31_bits(M, N, K)) return 0;
  da::LinearParams p;
  memset(&p, 0, sizeof(p));
  p.M = M, p.N = N, p.K = K;
  const bool gated = static_cast<Kind>(kind) == Kind::kGated;
  const Product q = {static_cast<Kind>(kind), gated ? da::kEpiGated : f32 ? da::kEpiF32 : da::kEpiBf16, nullptr, nullptr, 0, 0};
  const Plan x = product_plan(q, p, sms_or_default());
  const int cg = x.tile.cg;
  if (x.few.nt) {
    const int blocks = ((K + da::kLinBK - 1) / da::kLinBK + x.few.cs - 1) / x.few.cs;
    const int seg = !f32 ? blocks : x.few.turns ? da::kLinSegBlocks : da::few_segment_blocks(blocks, x.few.width);
    const int row[6] = {x.few.cs, x.few.width, x.few.nt, x.few.lg, x.few.stages, seg * da::kLinBK};
    memcpy(plan, row, sizeof(row));
    return 1;
  }
  const int row[6] = {cg, static_cast<int>(x.tile.full), static_cast<int>(tile_count(q, p, cg) - x.tile.full), 0, 0,
                      f32 ? da::kLinSegBlocks * da::kLinBK : (K + da::kLinBK - 1) / da::kLinBK * da::kLinBK};
  memcpy(plan, row, sizeof(row));
  return 2;
}

diffattn_status diffattn_linear(int M, int N, int K, const void* a, long long lda, const void* w, const float* bias,
                                diffattn_activation act, const void* residual, long long ldr, diffattn_dtype out_dt,
                                void* out, long long ldo, void* pre, void* stream) {
  const char* fn = "diffattn_linear";
  if (M < 0 || N < 0 || K < 1) return fail(DIFFATTN_ERR_SHAPE, "%s: bad sizes M=%d N=%d K=%d", fn, M, N, K);
  if (N % 8 != 0 || K % 8 != 0)
    return fail(DIFFATTN_ERR_SHAPE, "%s: N and K must be multiples of 8 (16-byte rows; got N=%d K=%d)", fn, N, K);
  if (bad_act(act)) return fail(DIFFATTN_ERR_DTYPE, "%s: unknown activation %d", fn, (int)act);
  if (bad_dtype(out_dt)) return fail(DIFFATTN_ERR_DTYPE, "%s: the output must be bf16 or fp32", fn);
  if (M == 0 || N == 0) return dh::success();
  const int es = static_cast<int>(dtype_bytes(out_dt));
  diffattn_status st;
  if ((st = check_rows(fn, "a", a, K, lda, 2)) != DIFFATTN_OK) return st;
  if ((st = check_rows(fn, "w", w, K, K, 2)) != DIFFATTN_OK) return st;
  if ((st = check_rows(fn, "out", out, N, ldo, es)) != DIFFATTN_OK) return st;
  if (residual && (st = check_rows(fn, "residual", residual, N, ldr, es)) != DIFFATTN_OK) return st;
  if (pre && (st = check_rows(fn, "pre", pre, N, N, 2)) != DIFFATTN_OK) return st;
  if (!aligned(bias, 16)) return fail(DIFFATTN_ERR_ALIGN, "%s: bias must be 16-byte aligned", fn);
  {
    const long long n = N, k = K;
    const bool in_place = residual == out && ldr == ldo;
    const Span wr[2] = {{out, M, n * es, ldo * es}, {pre, M, n * 2, n * 2}};
    const Span rd[4] = {{a, M, k * 2, lda * 2}, {w, N, k * 2, k * 2}, flat(bias, n * 4),
                        {in_place ? nullptr : residual, M, n * es, ldr * es}};
    if ((st = disjoint(fn, wr, 2, rd, 4)) != DIFFATTN_OK) return st;
    if (in_place && overlap(wr[1], wr[0])) return fail(DIFFATTN_ERR_SHAPE, "%s: an output overlaps an input", fn);
  }
  da::LinearParams p;
  memset(&p, 0, sizeof(p));
  p.bias = bias;
  p.residual = residual;
  p.out = out;
  p.pre = static_cast<__nv_bfloat16*>(pre);
  p.ldr = ldr, p.ldo = ldo, p.ldp = N;
  p.M = M, p.N = N, p.K = K, p.act = act;
  const Product q = {Kind::kForward, out_dt == DIFFATTN_F32 ? da::kEpiF32 : da::kEpiBf16, a, w, lda, K};
  if ((st = launch_product(fn, q, p, static_cast<cudaStream_t>(stream))) != DIFFATTN_OK) return st;
  return dh::success();
}

size_t diffattn_linear_backward_workspace(int M, int N, int K) {
  return diffattn_linear_backward_workspace_for(M, N, K, DIFFATTN_ACT_RELU, 1);
}

size_t diffattn_linear_backward_workspace_for(int M, int N, int K, diffattn_activation act, int dbias) {
  if (M < 1 || N < 1 || K < 1 || bad_act(act)) return 0;
  return linear_workspace(M, N, act != DIFFATTN_ACT_NONE, dbias != 0);
}

diffattn_status diffattn_linear_backward(int M, int N, int K, const void* a, long long lda, const void* w, const void* dy,
                                         long long ldy, const void* pre, diffattn_activation act, void* da_, void* dw,
                                         diffattn_dtype dw_dt, float* dbias, void* workspace, size_t workspace_bytes,
                                         void* stream) {
  const char* fn = "diffattn_linear_backward";
  if (M < 0 || N < 0 || K < 1) return fail(DIFFATTN_ERR_SHAPE, "%s: bad sizes M=%d N=%d K=%d", fn, M, N, K);
  if (N % 8 != 0 || K % 8 != 0)
    return fail(DIFFATTN_ERR_SHAPE, "%s: N and K must be multiples of 8 (16-byte rows; got N=%d K=%d)", fn, N, K);
  if (bad_act(act)) return fail(DIFFATTN_ERR_DTYPE, "%s: unknown activation %d", fn, (int)act);
  if (bad_dtype(dw_dt)) return fail(DIFFATTN_ERR_DTYPE, "%s: dw must be bf16 or fp32", fn);
  if (too_large(M, N, K)) return fail(DIFFATTN_ERR_SHAPE, "%s: too large", fn);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t wes = dtype_bytes(dw_dt);
  diffattn_status st;
  if (N > 0 && dw && (st = check_rows(fn, "dw", dw, K, K, static_cast<int>(wes))) != DIFFATTN_OK) return st;
  if (!aligned(dbias, 4)) return fail(DIFFATTN_ERR_ALIGN, "%s: dbias must be 4-byte aligned", fn);
  if (M > 0 && da_ && (st = check_rows(fn, "da", da_, K, K, 2)) != DIFFATTN_OK) return st;
  if (M == 0 || N == 0) {  // sums over nothing
    if (N > 0 && (st = zero(fn, dw, static_cast<size_t>(N) * K * wes, s)) != DIFFATTN_OK) return st;
    if (N > 0 && (st = zero(fn, dbias, static_cast<size_t>(N) * 4, s)) != DIFFATTN_OK) return st;
    if (M > 0 && (st = zero(fn, da_, static_cast<size_t>(M) * K * 2, s)) != DIFFATTN_OK) return st;
    return dh::success();
  }
  if (!da_ && !dw && !dbias) return dh::success();
  const bool bent = act != DIFFATTN_ACT_NONE;
  if (dw && (st = check_rows(fn, "a", a, K, lda, 2)) != DIFFATTN_OK) return st;
  if (da_ && (st = check_rows(fn, "w", w, K, K, 2)) != DIFFATTN_OK) return st;
  if ((st = check_rows(fn, "dy", dy, N, ldy, 2)) != DIFFATTN_OK) return st;
  if (bent && (st = check_rows(fn, "pre", pre, N, N, 2)) != DIFFATTN_OK) return st;
  const size_t need = linear_workspace(M, N, bent, dbias != nullptr);
  if ((st = check_workspace(fn, workspace, workspace_bytes, need)) != DIFFATTN_OK) return st;
  {
    const long long n = N, k = K;
    const Span wr[4] = {{da_, M, k * 2, k * 2}, flat(dw, n * k * static_cast<long long>(wes)), flat(dbias, n * 4),
                        flat(workspace, static_cast<long long>(need))};
    const Span rd[4] = {{dw ? a : nullptr, M, k * 2, lda * 2}, {da_ ? w : nullptr, N, k * 2, k * 2}, {dy, M, n * 2, ldy * 2},
                        {bent ? pre : nullptr, M, n * 2, n * 2}};
    if ((st = disjoint(fn, wr, 4, rd, 4)) != DIFFATTN_OK) return st;
  }
  const void* dz = dy;
  long long ldz = ldy;
  if (bent || dbias) {
    da::ActGradParams p;
    memset(&p, 0, sizeof(p));
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.dy = static_cast<const __nv_bfloat16*>(dy);
    p.pre = static_cast<const __nv_bfloat16*>(pre);
    p.ldy = ldy, p.ldp = N, p.ldz = N;
    p.M = M, p.N = N, p.act = act, p.chunks = dbias ? bias_chunks(M, N) : act_grad_chunks(M, N);
    p.part = dbias;
    if (dbias && p.chunks > 1) p.part = reinterpret_cast<float*>(ws), ws += bias_parts_bytes(M, N);
    p.dz = bent ? reinterpret_cast<__nv_bfloat16*>(ws) : nullptr;
    if ((st = act_grad(fn, p, false, s)) != DIFFATTN_OK) return st;
    if (dbias && p.chunks > 1) {
      da::SumParts q;
      memset(&q, 0, sizeof(q));
      q.part[0] = p.part, q.dst[0] = dbias, q.width[0] = N, q.count[0] = p.chunks;
      if ((st = sum_parts(fn, q, s)) != DIFFATTN_OK) return st;
    }
    if (bent) dz = p.dz, ldz = N;
  }
  if (da_ && (st = dgrad(fn, M, K, N, dz, ldz, w, da_, s)) != DIFFATTN_OK) return st;
  if (dw && (st = wgrad(fn, N, K, M, dz, ldz, a, lda, dw, dw_dt, s)) != DIFFATTN_OK) return st;
  return dh::success();
}

diffattn_status diffattn_gated_linear(int M, int D, int F, const void* x, long long ldx, const void* w_gu,
                                      diffattn_activation act, void* h, long long ldh, void* gu, void* stream) {
  const char* fn = "diffattn_gated_linear";
  if (M < 0 || F < 0 || D < 1) return fail(DIFFATTN_ERR_SHAPE, "%s: bad sizes M=%d D=%d F=%d", fn, M, D, F);
  if (D % 8 != 0 || F % 8 != 0)
    return fail(DIFFATTN_ERR_SHAPE, "%s: D and F must be multiples of 8 (16-byte rows; got D=%d F=%d)", fn, D, F);
  if (bad_act(act)) return fail(DIFFATTN_ERR_DTYPE, "%s: unknown activation %d", fn, (int)act);
  if (M == 0 || F == 0) return dh::success();
  if (F > 0x3fffffff) return fail(DIFFATTN_ERR_SHAPE, "%s: too large", fn);
  diffattn_status st;
  if ((st = check_rows(fn, "x", x, D, ldx, 2)) != DIFFATTN_OK) return st;
  if ((st = check_rows(fn, "w_gu", w_gu, D, D, 2)) != DIFFATTN_OK) return st;
  if ((st = check_rows(fn, "h", h, F, ldh, 2)) != DIFFATTN_OK) return st;
  if (gu && (st = check_rows(fn, "gu", gu, 2ll * F, 2ll * F, 2)) != DIFFATTN_OK) return st;
  {
    const long long d = D, f = F;
    const Span wr[2] = {{h, M, f * 2, ldh * 2}, {gu, M, f * 4, f * 4}};
    const Span rd[2] = {{x, M, d * 2, ldx * 2}, {w_gu, 2 * f, d * 2, d * 2}};
    if ((st = disjoint(fn, wr, 2, rd, 2)) != DIFFATTN_OK) return st;
  }
  da::LinearParams p;
  memset(&p, 0, sizeof(p));
  p.out = h;
  p.pre = static_cast<__nv_bfloat16*>(gu);
  p.ldo = ldh, p.ldp = 2ll * F;
  p.M = M, p.N = F, p.K = D, p.act = act;
  const Product q = {Kind::kGated, da::kEpiGated, x, w_gu, ldx, D};
  if ((st = launch_product(fn, q, p, static_cast<cudaStream_t>(stream))) != DIFFATTN_OK) return st;
  return dh::success();
}

size_t diffattn_gated_linear_backward_workspace(int M, int D, int F) {
  if (M < 1 || D < 1 || F < 1) return 0;
  return round256(static_cast<size_t>(M) * F * 4);
}

diffattn_status diffattn_gated_linear_backward(int M, int D, int F, const void* x, long long ldx, const void* w_gu,
                                               const void* gu, const void* dh_, long long ldh, diffattn_activation act,
                                               void* dx, void* dw, diffattn_dtype dw_dt, void* workspace,
                                               size_t workspace_bytes, void* stream) {
  const char* fn = "diffattn_gated_linear_backward";
  if (M < 0 || F < 0 || D < 1) return fail(DIFFATTN_ERR_SHAPE, "%s: bad sizes M=%d D=%d F=%d", fn, M, D, F);
  if (D % 8 != 0 || F % 8 != 0)
    return fail(DIFFATTN_ERR_SHAPE, "%s: D and F must be multiples of 8 (16-byte rows; got D=%d F=%d)", fn, D, F);
  if (bad_act(act)) return fail(DIFFATTN_ERR_DTYPE, "%s: unknown activation %d", fn, (int)act);
  if (bad_dtype(dw_dt)) return fail(DIFFATTN_ERR_DTYPE, "%s: dw must be bf16 or fp32", fn);
  if (too_large(M, F, D)) return fail(DIFFATTN_ERR_SHAPE, "%s: too large", fn);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t wes = dtype_bytes(dw_dt);
  diffattn_status st;
  if (F > 0 && dw && (st = check_rows(fn, "dw", dw, D, D, static_cast<int>(wes))) != DIFFATTN_OK) return st;
  if (M > 0 && dx && (st = check_rows(fn, "dx", dx, D, D, 2)) != DIFFATTN_OK) return st;
  if (M == 0 || F == 0) {
    if (F > 0 && (st = zero(fn, dw, static_cast<size_t>(2) * F * D * wes, s)) != DIFFATTN_OK) return st;
    if (M > 0 && (st = zero(fn, dx, static_cast<size_t>(M) * D * 2, s)) != DIFFATTN_OK) return st;
    return dh::success();
  }
  if (!dx && !dw) return dh::success();
  if (dw && (st = check_rows(fn, "x", x, D, ldx, 2)) != DIFFATTN_OK) return st;
  if (dx && (st = check_rows(fn, "w_gu", w_gu, D, D, 2)) != DIFFATTN_OK) return st;
  if ((st = check_rows(fn, "gu", gu, 2ll * F, 2ll * F, 2)) != DIFFATTN_OK) return st;
  if ((st = check_rows(fn, "dh", dh_, F, ldh, 2)) != DIFFATTN_OK) return st;
  const size_t need = diffattn_gated_linear_backward_workspace(M, D, F);
  if ((st = check_workspace(fn, workspace, workspace_bytes, need)) != DIFFATTN_OK) return st;
  {
    const long long d = D, f = F;
    const Span wr[3] = {{dx, M, d * 2, d * 2}, flat(dw, 2 * f * d * static_cast<long long>(wes)),
                        flat(workspace, static_cast<long long>(need))};
    const Span rd[4] = {{dw ? x : nullptr, M, d * 2, ldx * 2}, flat(dx ? w_gu : nullptr, 4 * f * d),
                        flat(gu, 4ll * M * f), {dh_, M, f * 2, ldh * 2}};
    if ((st = disjoint(fn, wr, 3, rd, 4)) != DIFFATTN_OK) return st;
  }
  da::ActGradParams p;
  memset(&p, 0, sizeof(p));
  p.dy = static_cast<const __nv_bfloat16*>(dh_);
  p.pre = static_cast<const __nv_bfloat16*>(gu);
  p.dz = static_cast<__nv_bfloat16*>(workspace);
  p.ldy = ldh, p.ldp = 2ll * F, p.ldz = 2ll * F;
  p.M = M, p.N = F, p.act = act, p.chunks = std::min((M + 31) / 32, 65535);  // (8192 x 5464: 8 CTAs an SM 115 us, 37 so 107)
  if ((st = act_grad(fn, p, true, s)) != DIFFATTN_OK) return st;
  if (dx && (st = dgrad(fn, M, D, 2 * F, workspace, 2ll * F, w_gu, dx, s)) != DIFFATTN_OK) return st;
  if (dw && (st = wgrad(fn, 2 * F, D, M, workspace, 2ll * F, x, ldx, dw, dw_dt, s)) != DIFFATTN_OK) return st;
  return dh::success();
}

}  // extern "C"

// ----------------------------------------------------------------- norms
namespace {

// How a row of D elements is laid over threads.  Rows of 16-byte multiples: vectors of 8 elements, a power of two of
// lanes up to 256 elements, above a CTA a row with one or two vectors a thread: forward two above 512 elements;
// backward one (of two rows at once) up to 4096, as 512 threads are the most.  Other rows: eight elements a thread up to
// 4096, sixteen above, in pairs where the width is even (sixteen forward too: 16760 x 1001 150 us, with eight and twice
// the warps 103).
da::NormShape norm_shape(int D, bool grad) {
  da::NormShape h;
  h.vec = D % 8 == 0 ? 8 : D % 2 == 0 ? 2 : 1;
  const int per = D > (grad || h.vec < 8 ? 4096 : 512) ? 16 : 8;  // elements a thread
  h.nv = per / h.vec;
  h.lanes = 32;
  if (D <= 256) {
    h.layout = h.vec == 8 ? da::kSubWarp : da::kPlainWarp;
    h.threads = 256;
    h.nv = 8 / h.vec;
    if (h.vec == 8)
      for (h.lanes = 4; h.lanes * 8 < D;) h.lanes *= 2;
  } else {
    h.layout = h.vec == 8 ? da::kRing : da::kPlain;
    h.threads = ((D + per - 1) / per + 31) / 32 * 32;
  }
  return h;
}

bool norm_row_cta(const da::NormShape& h) { return h.layout == da::kRing || h.layout == da::kPlain; }
int norm_workers(const da::NormShape& h) { return norm_row_cta(h) ? 1 : h.threads / h.lanes; }

// Ring slots and dynamic shared memory where rows take `slot` bytes (and a CTA `extra` more), for up to `ctas` CTAs an
// SM: some 128 KB an SM on its way.  Returns how many CTAs an SM then holds.
int norm_ring(const da::NormShape& h, long long slot, long long extra, int ctas, int* stages, int* smem) {
  *stages = 0;
  *smem = 0;
  if (h.layout != da::kRing) return ctas;
  while (ctas > 1 && slot + extra > da::kNormMaxSmem / ctas - 1152) --ctas;
  const long long room = da::kNormMaxSmem / ctas - 1152 - extra;
  *stages = static_cast<int>(std::max(1ll, std::min({static_cast<long long>(da::kNormMaxStages), room / slot, std::max(4ll, (128ll * 1024 / ctas) / slot)})));
  *smem = static_cast<int>(128 + *stages * slot);
  return ctas;
}

diffattn_status norm_common(const char* fn, int dt, int sdt, int rows, int D, const float* gate, int gate_rows) {
  if (bad_dtype(dt) || bad_dtype(sdt) || (dt == DIFFATTN_F32 && sdt != DIFFATTN_F32))
    return fail(DIFFATTN_ERR_DTYPE, "%s: types: both bf16, both fp32, or bf16 on an fp32 stream", fn);
  if (rows < 0 || D < 1) return fail(DIFFATTN_ERR_SHAPE, "%s: bad sizes rows=%d D=%d", fn, rows, D);
  if (D > da::kNormMaxD) return fail(DIFFATTN_ERR_UNSUPPORTED, "%s: D at most %d (got %d)", fn, da::kNormMaxD, D);
  if (gate && (gate_rows < 1 || rows % gate_rows != 0))
    return fail(DIFFATTN_ERR_SHAPE, "%s: rows (%d) must be a multiple of gate_rows (%d)", fn, rows, gate_rows);
  return DIFFATTN_OK;
}

cudaError_t launch_norm(const da::NormParams& p, const da::NormShape& h, int dt, int sdt, bool grad, int grid, int smem,
                        cudaStream_t s) {
  if (dt == DIFFATTN_F32) return da::launch_norm_f32(p, h, grad, grid, smem, s);
  return sdt == DIFFATTN_F32 ? da::launch_norm_mixed(p, h, grad, grid, smem, s) : da::launch_norm_bf16(p, h, grad, grid, smem, s);
}

// Pieces of the backward pass: runs of rows that are summed over together.  A CTA takes neighbouring pieces.
struct NormPlan {
  long long groups, group_rows, chunk_rows, pieces;
  int chunks, grid;
};

// CTAs an SM of the backward kernel: 512 threads together (128 registers each), eight CTAs at most.
int norm_grad_per_sm(const da::NormShape& h) { return std::max(1, std::min(8, 512 / h.threads)); }

NormPlan norm_plan(int rows, int D, int gate_rows) {
  NormPlan n;
  const da::NormShape h = norm_shape(D, true);
  const int workers = norm_workers(h);
  n.groups = gate_rows > 0 && gate_rows < rows ? gate_rows : 1;
  n.group_rows = rows / n.groups;
  const long long want = std::max<long long>(1, std::min<long long>((rows - 1ll + workers) / workers, 152 * norm_grad_per_sm(h)));
  // A piece a CTA where groups are few; several smaller pieces a CTA where whole groups would leave CTAs unequal.
  const long long pieces = 2 * n.groups <= want ? want / n.groups : n.groups < 4 * want ? (4 * want + n.groups - 1) / n.groups : 1;
  const long long chunks = std::max(1ll, std::min(pieces, (n.group_rows + workers - 1) / workers));
  n.chunk_rows = (n.group_rows + chunks - 1) / chunks;
  n.chunks = static_cast<int>((n.group_rows + n.chunk_rows - 1) / n.chunk_rows);
  n.pieces = n.groups * n.chunks;
  n.grid = static_cast<int>(std::min(n.pieces, want));
  return n;
}

}  // namespace

extern "C" {

diffattn_status diffattn_residual_norm(diffattn_dtype dt, diffattn_dtype stream_dt, int rows, int D, const void* x,
                                       const void* residual, const float* gate, int gate_rows, float scale, int post,
                                       const float* gamma_post, const float* gamma, float eps, void* s_out, void* y,
                                       void* stream) {
  const char* fn = "diffattn_residual_norm";
  diffattn_status st = norm_common(fn, dt, stream_dt, rows, D, gate, gate_rows);
  if (st != DIFFATTN_OK) return st;
  if (!std::isfinite(scale)) return fail(DIFFATTN_ERR_SHAPE, "%s: scale not finite", fn);
  if (gamma_post && !post) return fail(DIFFATTN_ERR_SHAPE, "%s: gamma_post without post", fn);
  if (rows == 0) return dh::success();
  if (!s_out && !y) return fail(DIFFATTN_ERR_SHAPE, "%s: neither s nor y wanted", fn);
  if (gamma && !y) return fail(DIFFATTN_ERR_SHAPE, "%s: gamma without y", fn);
  if (!x) return fail(DIFFATTN_ERR_NULL, "%s: x is NULL", fn);
  for (const void* q : {x, residual, static_cast<const void*>(s_out), static_cast<const void*>(y),
                        static_cast<const void*>(gate), static_cast<const void*>(gamma_post), static_cast<const void*>(gamma)})
    if (!aligned(q, 16)) return fail(DIFFATTN_ERR_ALIGN, "%s: tensors must be 16-byte aligned", fn);
  const long long v = static_cast<long long>(rows) * D, xe = dtype_bytes(dt), se = dtype_bytes(stream_dt);
  {
    const Span wr[2] = {flat(s_out, v * se), flat(y, v * xe)};
    const Span rd[5] = {flat(x, v * xe), flat(residual == s_out ? nullptr : residual, v * se),
                        flat(gate, gate ? 4ll * gate_rows * D : 0), flat(gamma_post, 4ll * D), flat(gamma, 4ll * D)};
    if ((st = disjoint(fn, wr, 2, rd, 5)) != DIFFATTN_OK) return st;
  }
  da::NormParams p;
  memset(&p, 0, sizeof(p));
  p.x = x, p.residual = residual, p.gate = gate, p.gamma_post = gamma_post, p.gamma = gamma;
  p.s_out = s_out, p.y_out = y;
  p.rows = rows, p.D = D;
  p.gate_rows = gate ? gate_rows : 0;
  p.groups = gate ? gate_rows : 1;
  p.group_rows = rows / p.groups;
  p.scale = scale, p.eps = eps > 0.f ? eps : 1e-5f;
  p.post = post ? 1 : 0, p.norm = y ? 1 : 0;
  if ((st = dh::status_address(&p.status)) != DIFFATTN_OK) return st;
  const da::NormShape h = norm_shape(D, false);
  const int workers = norm_workers(h);
  p.lanes = h.lanes;
  // As many CTAs as an SM holds at once, by its registers, which warps take in fours; each walks its rows.  (A CTA more
  // than fit and it runs alone behind the others: 16777 x 1000 37 us, not 25.)
  const int fit = h.layout != da::kRing ? 1024 : h.nv == 1 ? 640 : 512;  // threads: at 64, 96 and 116 registers
  int smem;
  const int per_sm = norm_ring(h, D * (xe + (residual ? se : 0) + (gate && p.group_rows == 1 ? 4 : 0)), 0,
                               std::max(1, std::min(16, fit / h.threads)), &p.stages, &smem);
  const int grid = static_cast<int>(std::min<long long>((rows - 1ll + workers) / workers, static_cast<long long>(sms_or_default()) * per_sm));
  const cudaError_t e = launch_norm(p, h, dt, stream_dt, false, grid, smem, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, fn);
  dh::count_launches(1);
  return dh::success();
}

size_t diffattn_residual_norm_backward_workspace(int rows, int D, int gate_rows) {
  if (rows < 1 || D < 1 || gate_rows < 0) return 0;
  const NormPlan n = norm_plan(rows, D, gate_rows);
  return 2 * round256(static_cast<size_t>(n.grid) * D * 4) +
         (gate_rows > 0 && gate_rows < rows && n.chunks > 1 ? round256(static_cast<size_t>(n.pieces) * D * 4) : 0);
}

diffattn_status diffattn_residual_norm_backward(diffattn_dtype dt, diffattn_dtype stream_dt, int rows, int D,
                                                const void* x, const void* s_in, const void* dy, const void* ds,
                                                const float* gate, int gate_rows, float scale, int post,
                                                const float* gamma_post, const float* gamma, float eps, void* dx,
                                                void* dresidual, float* dgate, float* dgamma_post, float* dgamma,
                                                void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "diffattn_residual_norm_backward";
  diffattn_status st = norm_common(fn, dt, stream_dt, rows, D, gate, gate_rows);
  if (st != DIFFATTN_OK) return st;
  if (!std::isfinite(scale)) return fail(DIFFATTN_ERR_SHAPE, "%s: scale not finite", fn);
  if (dgate && !gate) return fail(DIFFATTN_ERR_SHAPE, "%s: dgate without gate", fn);
  if ((dgamma_post || gamma_post) && !post) return fail(DIFFATTN_ERR_SHAPE, "%s: dgamma_post or gamma_post without post", fn);
  for (const void* q : {x, s_in, dy, ds, static_cast<const void*>(gate), static_cast<const void*>(gamma_post),
                        static_cast<const void*>(gamma), static_cast<const void*>(dx), static_cast<const void*>(dresidual),
                        static_cast<const void*>(dgate), static_cast<const void*>(dgamma_post), static_cast<const void*>(dgamma)})
    if (!aligned(q, 16)) return fail(DIFFATTN_ERR_ALIGN, "%s: tensors must be 16-byte aligned", fn);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if ((st = zero(fn, dgamma, 4ull * D, s)) != DIFFATTN_OK) return st;
    if ((st = zero(fn, dgamma_post, 4ull * D, s)) != DIFFATTN_OK) return st;
    if (gate && (st = zero(fn, dgate, 4ull * D * gate_rows, s)) != DIFFATTN_OK) return st;
    return dh::success();
  }
  if (!dy && !ds) return fail(DIFFATTN_ERR_NULL, "%s: neither dy nor ds", fn);
  if ((dgamma || gamma) && !dy) return fail(DIFFATTN_ERR_SHAPE, "%s: dgamma or gamma without dy", fn);
  if (dy && !s_in) return fail(DIFFATTN_ERR_NULL, "%s: s is NULL", fn);
  if (!x && (post || dgate)) return fail(DIFFATTN_ERR_NULL, "%s: x is NULL", fn);
  if (!dx && !dresidual && !dgate && !dgamma_post && !dgamma) return dh::success();
  const NormPlan n = norm_plan(rows, D, gate ? gate_rows : 0);
  const size_t need = diffattn_residual_norm_backward_workspace(rows, D, gate ? gate_rows : 0);
  if ((st = check_workspace(fn, workspace, workspace_bytes, need)) != DIFFATTN_OK) return st;
  const long long v = static_cast<long long>(rows) * D, xe = dtype_bytes(dt), se = dtype_bytes(stream_dt);
  const long long gb = gate ? 4ll * gate_rows * D : 0;
  {
    const Span wr[6] = {flat(dx, v * xe), flat(dresidual, v * se), flat(dgate, gb), flat(dgamma_post, 4ll * D),
                        flat(dgamma, 4ll * D), flat(workspace, static_cast<long long>(need))};
    const Span rd[7] = {flat(x, v * xe), flat(s_in, v * se), flat(dy, v * xe), flat(ds == dresidual ? nullptr : ds, v * se),
                        flat(gate, gb), flat(gamma_post, 4ll * D), flat(gamma, 4ll * D)};
    if ((st = disjoint(fn, wr, 6, rd, 7)) != DIFFATTN_OK) return st;
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const size_t part = round256(static_cast<size_t>(n.grid) * D * 4);
  da::NormParams p;
  memset(&p, 0, sizeof(p));
  p.x = x, p.s = s_in, p.dy = dy, p.ds = ds, p.gate = gate, p.gamma_post = gamma_post, p.gamma = gamma;
  p.dx = dx, p.dresidual = dresidual;
  p.part_gamma = dgamma ? reinterpret_cast<float*>(ws) : nullptr;
  p.part_post = dgamma_post ? reinterpret_cast<float*>(ws + part) : nullptr;
  p.part_gate = !dgate ? nullptr : n.chunks > 1 ? reinterpret_cast<float*>(ws + 2 * part) : dgate;
  const bool row_gate = gate && gate_rows == rows;
  if (row_gate) p.part_gate = dgate;
  p.rows = rows, p.gate_rows = gate ? gate_rows : 0;
  p.group_rows = n.group_rows, p.groups = n.groups, p.chunk_rows = n.chunk_rows, p.pieces = n.pieces;
  p.chunks = n.chunks, p.D = D;
  p.scale = scale, p.eps = eps > 0.f ? eps : 1e-5f;
  p.post = post ? 1 : 0, p.norm = dy ? 1 : 0;
  if ((st = dh::status_address(&p.status)) != DIFFATTN_OK) return st;
  const da::NormShape h = norm_shape(D, true);
  p.lanes = h.lanes;
  int smem;
  const long long slot = D * ((dy ? xe + se : 0) + (ds ? se : 0) + (post || dgate ? xe : 0) + (row_gate ? 4 : 0));
  // gamma_post times the gate in shared memory too, where that leaves two slots.
  const bool combined = h.layout == da::kRing && h.nv == 2 && (gamma_post || (gate && !row_gate)) && 2 * slot + 8ll * D <= da::kNormMaxSmem - 1152;
  norm_ring(h, slot, (combined ? 8ll : 4ll) * D, norm_grad_per_sm(h), &p.stages, &smem);
  // Behind the ring: gamma_post times the gate, and sums for dgamma_post.  Rows of warps: two such arrays a worker (those
  // sums, and room to join them).
  p.off_combined = combined ? smem : -1;
  if (combined) smem += 4 * D;
  if (!norm_row_cta(h)) smem = norm_workers(h) * D * 4;
  p.off_post = smem;
  smem += norm_workers(h) * D * 4;
  const cudaError_t e = launch_norm(p, h, dt, stream_dt, true, n.grid, smem, s);
  if (e != cudaSuccess) return cuda_fail(e, fn);
  dh::count_launches(1);
  da::SumParts q;
  memset(&q, 0, sizeof(q));
  int k = 0;
  auto add = [&](const float* from, float* to, long long width, long long count) {
    q.part[k] = from, q.dst[k] = to, q.width[k] = width, q.count[k] = static_cast<int>(count);
    ++k;
  };
  if (dgamma) add(p.part_gamma, dgamma, D, n.grid);
  if (dgamma_post) add(p.part_post, dgamma_post, D, n.grid);
  if (dgate && !row_gate && n.chunks > 1) add(p.part_gate, dgate, static_cast<long long>(n.groups) * D, n.chunks);
  if (k > 0 && (st = sum_parts(fn, q, s)) != DIFFATTN_OK) return st;
  return dh::success();
}

}  // extern "C"
