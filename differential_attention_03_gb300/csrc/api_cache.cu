// C entry points of the rotary positions, the cache append, the tree decode
// and the cache keep: argument validation, TMA descriptors, launch shapes.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "cache_params.h"
#include "diffattn.h"
#include "host.h"

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

bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + bn && y < x + an;
}

// A tensor of a call.
struct Span {
  const void* at;
  size_t bytes;
};

// What a call writes may overlap nothing else of the call: rows are read and written by threads of their own.
diffattn_status disjoint(const char* fn, const Span* written, int nw, const Span* read, int nr) {
  for (int i = 0; i < nw; ++i) {
    const Span& w = written[i];
    if (!w.at || w.bytes == 0) continue;
    for (int j = 0; j < nr; ++j)
      if (read[j].at && read[j].bytes && overlap(w.at, w.bytes, read[j].at, read[j].bytes))
        return fail(DIFFATTN_ERR_SHAPE, "%s: an output or the cache overlaps an input", fn);
    for (int j = 0; j < i; ++j)
      if (written[j].at && written[j].bytes && overlap(w.at, w.bytes, written[j].at, written[j].bytes))
        return fail(DIFFATTN_ERR_SHAPE, "%s: outputs or cache tensors overlap", fn);
  }
  return DIFFATTN_OK;
}

int sms_or_default() {
  const int s = dh::sms();
  return s > 0 ? s : 148;
}

// 2^32 / n + 1, by whose high product fast_div divides numbers up to `most` by n exactly; 0 where it would not.
unsigned division_magic(unsigned long long n, unsigned long long most) {
  if (n < 2 || most >= (1ull << 32)) return 0;  // (n = 1: 2^32 + 1 does not fit)
  const unsigned long long m = (1ull << 32) / n + 1;
  return (m * n - (1ull << 32)) * most < (1ull << 32) ? static_cast<unsigned>(m) : 0;
}

// 4-D map over a contiguous [B, n, heads, W] tensor of bf16 or bytes: box =
// `box_bytes` (64 or 128, the swizzle) of a row x 1 head x `rows` tokens.
// `side` heads are read side by side at about the same time: L2 fetches what
// they ask for together (256 bytes at most).  Fetching more brings rows that
// are gone again before their reader comes, fetching less leaves DRAM with
// short bursts: e4m3 V1 d64 B8 H16 n32768, a 64-byte row a head, 8 side by
// side: 223 us at 64 bytes, 199 us at 256; alone 240 us at 64, 338 us at 256.
diffattn_status cache_map(CUtensorMap* m, const void* base, int B, int n, int heads, int W, int es, int box_bytes,
                          int rows, int side) {
  dh::EncodeTiled enc;
  diffattn_status s = dh::encoder(&enc);
  if (s != DIFFATTN_OK) return s;
  const cuuint64_t row = static_cast<cuuint64_t>(W) * es;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(W), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(n),
                              static_cast<cuuint64_t>(B)};
  const cuuint64_t strides[3] = {row, row * heads, row * heads * n};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(box_bytes / es), 1, static_cast<cuuint32_t>(rows), 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r =
      enc(m, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base),
          dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
          box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
          row * side >= 256   ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
          : row * side >= 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                              : CU_TENSOR_MAP_L2_PROMOTION_L2_64B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(DIFFATTN_ERR_CUDA, "cuTensorMapEncodeTiled failed (CUresult %d)", (int)r);
  return DIFFATTN_OK;
}

// A rotation as the kernels take it; NULL: none.
diffattn_status rope_turns(const char* fn, const diffattn_rope_spec* rope, int d, da::RopeTurns* out) {
  memset(out, 0, sizeof(*out));
  out->mult = 1.f;
  if (!rope) return DIFFATTN_OK;
  if (rope->rot_dim < 2 || rope->rot_dim > d || rope->rot_dim > 128 || (rope->rot_dim & 1))
    return fail(DIFFATTN_ERR_SHAPE, "%s: rot_dim %d: even, from 2 to the head width %d", fn, rope->rot_dim, d);
  if (!std::isfinite(rope->mult)) return fail(DIFFATTN_ERR_SHAPE, "%s: the rotary factor is not finite", fn);
  out->rot = rope->rot_dim;
  out->inter = rope->interleaved ? 1 : 0;
  out->mult = rope->mult;
  for (int i = 0; i < rope->rot_dim / 2; ++i) out->turns[i] = rope->turns[i];
  return DIFFATTN_OK;
}

bool bad_format(int fmt) {
  return fmt != DIFFATTN_CACHE_BF16 && fmt != DIFFATTN_CACHE_FP8K && fmt != DIFFATTN_CACHE_FP8;
}

diffattn_status check_scales(const char* fn, int fmt, int nk, int n, const float* ks, const float* const* kscales,
                             const float* vscales) {
  if (fmt == DIFFATTN_CACHE_FP8K)
    for (int i = 0; i < nk; ++i)
      if (!(std::isfinite(ks[i]) && ks[i] > 0.f && std::isfinite(1.f / ks[i])))
        return fail(DIFFATTN_ERR_SHAPE, "%s: key scales must be finite and positive, as must their reciprocals", fn);
  if (fmt == DIFFATTN_CACHE_FP8 && n > 0) {  // (an empty cache has no rows to point to)
    for (int i = 0; i < nk; ++i) {
      if (!kscales[i]) return fail(DIFFATTN_ERR_NULL, "%s: NULL key row scales", fn);
      if (!aligned(kscales[i], 4)) return fail(DIFFATTN_ERR_ALIGN, "%s: row scales must be 4-byte aligned", fn);
    }
    if (!vscales) return fail(DIFFATTN_ERR_NULL, "%s: NULL value row scales", fn);
    if (!aligned(vscales, 4)) return fail(DIFFATTN_ERR_ALIGN, "%s: row scales must be 4-byte aligned", fn);
  }
  return DIFFATTN_OK;
}

// nk key tensors (V1 two, V2 one), as many query tensors or none.
diffattn_status append(const char* fn, diffattn_cache_format fmt, int B, int T, int Hq, int H, int n, int d, int dv,
                       int nk, const void* const* q, const void* const* k, const void* v,
                       const diffattn_rope_spec* rope, const int* positions, const int* lens, const int* ntok,
                       void* const* qo, void* const* kc, void* vc, const float* ks, float* const* kscales,
                       float* vscales, void* stream) {
  if (bad_format(fmt)) return fail(DIFFATTN_ERR_DTYPE, "%s: unknown cache format %d", fn, (int)fmt);
  if (B < 0 || T < 0 || Hq < 0 || H < 0 || n < 0 || d < 1)
    return fail(DIFFATTN_ERR_SHAPE, "%s: bad sizes B=%d T=%d Hq=%d H=%d n=%d d=%d", fn, B, T, Hq, H, n, d);
  if (B == 0 || T == 0) return dh::success();
  const bool hasq = q[0] != nullptr || (nk == 2 && q[1] != nullptr);
  if (H == 0 && Hq > 0 && hasq) return fail(DIFFATTN_ERR_SHAPE, "%s: Hq = %d queries without a key head", fn, Hq);
  if (H == 0) return dh::success();
  if (nk == 2 ? (d != 64 && d != 128) : d != 128)
    return fail(DIFFATTN_ERR_UNSUPPORTED, "%s: d = %d", fn, d);
  for (int i = 0; i < nk; ++i) {
    if (!k[i] || (n > 0 && !kc[i])) return fail(DIFFATTN_ERR_NULL, "%s: NULL key pointer", fn);
    if (hasq && (!q[i] || !qo[i])) return fail(DIFFATTN_ERR_NULL, "%s: NULL query pointer", fn);
  }
  if (!v || (n > 0 && !vc)) return fail(DIFFATTN_ERR_NULL, "%s: NULL value pointer", fn);
  const float* ksc[2] = {kscales[0], kscales[1]};
  diffattn_status st = check_scales(fn, fmt, nk, n, ks, ksc, vscales);
  if (st != DIFFATTN_OK) return st;
  for (int i = 0; i < nk; ++i)
    if (!aligned(k[i], 16) || !aligned(kc[i], 16) || (hasq && (!aligned(q[i], 16) || !aligned(qo[i], 16))))
      return fail(DIFFATTN_ERR_ALIGN, "%s: tensors must be 16-byte aligned", fn);
  if (!aligned(v, 16) || !aligned(vc, 16)) return fail(DIFFATTN_ERR_ALIGN, "%s: tensors must be 16-byte aligned", fn);
  {
    Span w[8], r[8];
    int nw = 0, nr = 0;
    const size_t tok = static_cast<size_t>(B) * T, rows = static_cast<size_t>(B) * n * H;
    const size_t kes = fmt == DIFFATTN_CACHE_BF16 ? 2 : 1, ves = fmt == DIFFATTN_CACHE_FP8 ? 1 : 2;
    for (int i = 0; i < nk; ++i) {
      r[nr++] = {k[i], tok * H * d * 2};
      w[nw++] = {kc[i], rows * d * kes};
      if (fmt == DIFFATTN_CACHE_FP8) w[nw++] = {kscales[i], rows * 4};
      if (hasq) {
        r[nr++] = {q[i], tok * Hq * d * 2};
        w[nw++] = {qo[i], tok * Hq * d * 2};
      }
    }
    r[nr++] = {v, tok * H * dv * 2};
    r[nr++] = {positions, tok * 4};
    r[nr++] = {lens, static_cast<size_t>(B) * 4};
    r[nr++] = {ntok, static_cast<size_t>(B) * 4};
    w[nw++] = {vc, rows * dv * ves};
    if (fmt == DIFFATTN_CACHE_FP8) w[nw++] = {vscales, rows * 4};
    if ((st = disjoint(fn, w, nw, r, nr)) != DIFFATTN_OK) return st;
  }
  da::AppendParams p;
  memset(&p, 0, sizeof(p));
  if ((st = rope_turns(fn, rope, d, &p.rope)) != DIFFATTN_OK) return st;
  for (int i = 0; i < nk; ++i) {
    p.k[i] = static_cast<const __nv_bfloat16*>(k[i]);
    p.kc[i] = kc[i];
    p.ks[i] = kscales[i];
    p.kinv[i] = fmt == DIFFATTN_CACHE_FP8K ? 1.f / ks[i] : 1.f;
    if (hasq) {
      p.q[i] = static_cast<const __nv_bfloat16*>(q[i]);
      p.qo[i] = static_cast<__nv_bfloat16*>(qo[i]);
    }
  }
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.vc = vc;
  p.vs = vscales;
  p.pos = positions;
  p.lens = lens;
  p.ntok = ntok;
  p.B = B;
  p.T = T;
  p.Hq = Hq;
  p.H = H;
  p.n = n;
  p.d = d;
  p.dv = dv;
  p.nk = nk;
  p.nq = hasq ? nk : 0;
  p.fmt = fmt;
  const long long tokens = static_cast<long long>(B) * T;
  const long long lanes = (static_cast<long long>(p.nq) * Hq + static_cast<long long>(nk) * H) * (d / 16) +
                          static_cast<long long>(H) * (dv / 16);
  if (tokens > 0x7fffffffll || lanes > 0xfffffffll)
    return fail(DIFFATTN_ERR_SHAPE, "%s: too many tokens or heads", fn);
  // Several tokens a CTA once there are 24 CTAs an SM, for the angles' sake (the padded prefill of
  // 8002 tokens: 2 tokens a CTA 37.4 us, 6 38.4, 1 46.7); with few tokens, several CTAs a token.
  const int sms = sms_or_default();
  p.tokens_per_cta = static_cast<int>(std::min<long long>(da::kAppendMaxTokens, std::max<long long>(1, tokens / (24 * sms))));
  const long long of[3] = {static_cast<long long>(p.nq) * Hq, static_cast<long long>(nk) * H, H};
  for (int k = 0; k < 3; ++k) p.magic[k] = division_magic(of[k], of[k] * p.tokens_per_cta);
  const int gx = static_cast<int>((tokens + p.tokens_per_cta - 1) / p.tokens_per_cta);
  const long long most = (lanes * p.tokens_per_cta + da::kAppendThreads - 1) / da::kAppendThreads;
  const int gy = static_cast<int>(std::max<long long>(1, std::min<long long>({most, 2ll * sms / gx, 65535ll})));
  const cudaError_t e = da::launch_cache_append(p, gx, gy, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, fn);
  dh::count_launches(1);
  return dh::success();
}

diffattn_status keep(const char* fn, diffattn_cache_format fmt, int B, int A, int H, int n, int d, int dv, int nk,
                     void* const* kc, void* vc, float* const* kscales, float* vscales, const int* lens,
                     const int* path, const int* nkeep, int* new_lens, void* stream) {
  if (bad_format(fmt)) return fail(DIFFATTN_ERR_DTYPE, "%s: unknown cache format %d", fn, (int)fmt);
  if (B < 0 || A < 0 || H < 0 || n < 0 || d < 1)
    return fail(DIFFATTN_ERR_SHAPE, "%s: bad sizes B=%d A=%d H=%d n=%d d=%d", fn, B, A, H, n, d);
  if (A > da::kKeepMaxPath)
    return fail(DIFFATTN_ERR_UNSUPPORTED, "%s: paths of at most %d nodes (got %d)", fn, da::kKeepMaxPath, A);
  if (B == 0) return dh::success();
  if (nk == 2 ? (d != 64 && d != 128) : d != 128)
    return fail(DIFFATTN_ERR_UNSUPPORTED, "%s: d = %d", fn, d);
  const bool empty = n == 0 || H == 0;  // (no rows to point to; new_lens is written all the same)
  if ((!empty && !vc) || !lens || !nkeep || (A > 0 && !path)) return fail(DIFFATTN_ERR_NULL, "%s: NULL pointer", fn);
  for (int i = 0; i < nk; ++i)
    if (!empty && !kc[i]) return fail(DIFFATTN_ERR_NULL, "%s: NULL pointer", fn);
  const float one[2] = {1.f, 1.f};
  const float* ksc[2] = {kscales[0], kscales[1]};
  diffattn_status st = check_scales(fn, fmt, nk, empty ? 0 : n, one, ksc, vscales);
  if (st != DIFFATTN_OK) return st;
  da::KeepParams p;
  memset(&p, 0, sizeof(p));
  p.count = nk + 1;
  for (int i = 0; i <= nk; ++i) {
    p.base[i] = i < nk ? kc[i] : vc;
    p.scales[i] = i < nk ? kscales[i] : vscales;
    const bool wide = fmt == DIFFATTN_CACHE_BF16 || (i == nk && fmt == DIFFATTN_CACHE_FP8K);
    const long long rb = static_cast<long long>(H) * (i < nk ? d : dv) * (wide ? 2 : 1);
    if (rb > 0x3fffffffll) return fail(DIFFATTN_ERR_SHAPE, "%s: too many heads", fn);
    p.row_bytes[i] = static_cast<int>(rb);
    if (!aligned(p.base[i], 16)) return fail(DIFFATTN_ERR_ALIGN, "%s: tensors must be 16-byte aligned", fn);
  }
  {
    // (every CTA of a sequence reads lens, path and nkeep for itself, one of them writes new_lens)
    Span w[7];
    int nw = 0;
    const size_t rows = static_cast<size_t>(B) * n;
    for (int i = 0; i <= nk; ++i) {
      w[nw++] = {p.base[i], rows * p.row_bytes[i]};
      if (fmt == DIFFATTN_CACHE_FP8) w[nw++] = {p.scales[i], rows * H * 4};
    }
    const size_t ints = sizeof(int) * static_cast<size_t>(B);
    w[nw++] = {new_lens, ints};
    const Span r[3] = {{lens, ints}, {path, ints * A}, {nkeep, ints}};
    if ((st = disjoint(fn, w, nw, r, 3)) != DIFFATTN_OK) return st;
  }
  p.B = B;
  p.A = A;
  p.H = H;
  p.n = n;
  p.fmt = fmt;
  p.lens = lens;
  p.path = path;
  p.nkeep = nkeep;
  p.new_lens = new_lens;
  const int widest = std::max(p.row_bytes[0], p.row_bytes[nk]) / 16;
  const int gy = std::max(1, std::min((widest + da::kKeepThreads - 1) / da::kKeepThreads, 65535));
  const cudaError_t e = da::launch_cache_keep(p, gy, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, fn);
  dh::count_launches(1);
  return dh::success();
}

// CTAs the tree decode's key tiles are dealt to, at most (its workspace has a state for each).
constexpr int kTreeMaxCtas = 160;
constexpr int kTreeTeam = 8;  // CTAs of a team, at most

struct TreeShape {
  int pairs, ppt, mt, R;
  long long units;  // all sequences
};

TreeShape tree_shape(int B, int T, int H, int pairs) {
  TreeShape s;
  s.pairs = pairs;
  s.ppt = std::max(1, std::min(pairs, da::kTreeRows / std::max(1, T)));
  s.mt = (pairs + s.ppt - 1) / s.ppt;
  s.R = s.ppt * T;
  s.units = static_cast<long long>(B) * H * s.mt;
  return s;
}

size_t tree_workspace(int B, int T, int H, int pairs, int dv) {
  const TreeShape s = tree_shape(B, T, H, pairs);
  return (static_cast<size_t>(s.units) + kTreeMaxCtas) * da::tree_state_floats(s.R, da::tree_subs_most(s.R), dv) * sizeof(float) +
         16;  // (states start on 32 bytes)
}

diffattn_status tree(const char* fn, bool v2, diffattn_cache_format fmt, int B, int T, int H, int pairs, int n, int d,
                     const void* q1, const void* q2, const void* k1, const void* k2, const float* ks,
                     const float* const* kscales, const void* v, const float* vscales, const int* lens,
                     const int* ntok, const unsigned long long* mask, long long mask_sb, da::TreeParams& p, void* out,
                     void* workspace, size_t workspace_bytes, void* stream) {
  if (bad_format(fmt)) return fail(DIFFATTN_ERR_DTYPE, "%s: unknown cache format %d", fn, (int)fmt);
  const int dv = v2 ? d : 2 * d, nk = v2 ? 1 : 2;
  if (v2 ? d != 128 : (d != 64 && d != 128)) return fail(DIFFATTN_ERR_UNSUPPORTED, "%s: d = %d", fn, d);
  if (T > da::kTreeRows)
    return fail(DIFFATTN_ERR_UNSUPPORTED, "%s: at most %d drafted tokens a sequence (got %d)", fn, da::kTreeRows, T);
  if (n == 0) k1 = k2 = v = out;  // (an empty cache still needs valid maps; no key is read)
  if (!q1 || (!v2 && !q2) || !k1 || (!v2 && !k2) || !v || !out) return fail(DIFFATTN_ERR_NULL, "%s: NULL pointer", fn);
  diffattn_status st = check_scales(fn, fmt, nk, n, ks, kscales, vscales);
  if (st != DIFFATTN_OK) return st;
  if (!aligned(q1, 16) || !aligned(q2, 16) || !aligned(k1, 16) || !aligned(k2, 16) || !aligned(v, 16) ||
      !aligned(out, 16))
    return fail(DIFFATTN_ERR_ALIGN, "%s: tensors must be 16-byte aligned", fn);
  if (!aligned(mask, 8)) return fail(DIFFATTN_ERR_ALIGN, "%s: mask words must be 8-byte aligned", fn);
  const TreeShape sh = tree_shape(B, T, H, pairs);
  const long long tiles = sh.units * ((static_cast<long long>(n) + 127) / 128);
  if (sh.units * sh.R > 0x7fffffffll || tiles > 0x7fffffffll)
    return fail(DIFFATTN_ERR_SHAPE, "%s: too many (sequence, head) pairs or keys", fn);
  if (!workspace) return fail(DIFFATTN_ERR_NULL, "%s: NULL workspace", fn);
  const size_t need = tree_workspace(B, T, H, pairs, dv);
  if (workspace_bytes < need)
    return fail(DIFFATTN_ERR_SHAPE, "%s: workspace of %zu bytes, %zu needed", fn, workspace_bytes, need);
  if (!aligned(workspace, 16)) return fail(DIFFATTN_ERR_ALIGN, "%s: workspace must be 16-byte aligned", fn);
  {
    // (out is written when the queries and the cache have been read, beside what the second kernel reads)
    const size_t rows = static_cast<size_t>(B) * n * H, tok = static_cast<size_t>(B) * T, ints = sizeof(int) * static_cast<size_t>(B);
    const size_t kes = fmt == DIFFATTN_CACHE_BF16 ? 2 : 1, ves = fmt == DIFFATTN_CACHE_FP8 ? 1 : 2;
    const size_t rowscales = fmt == DIFFATTN_CACHE_FP8 ? rows * 4 : 0;
    const Span w[2] = {{out, tok * H * pairs * dv * 2}, {workspace, need}};
    const Span r[12] = {{k1, rows * d * kes}, {k2, v2 ? 0 : rows * d * kes}, {v, rows * dv * ves},
                        {kscales[0], rowscales}, {kscales[1], v2 ? 0 : rowscales}, {vscales, rowscales},
                        {lens, ints}, {ntok, ints}, {mask, 8 * (static_cast<size_t>(mask_sb) * (B - 1) + T)},
                        {p.lambda, 4}, {p.gamma, 4 * static_cast<size_t>(dv)},
                        {p.lam_logits, p.sb < 0 || p.st < 0 ? 0 : 4 * static_cast<size_t>(p.sb * (B - 1) + p.st * (T - 1) + static_cast<long long>(H) * pairs)}};
    const Span q[2] = {{q1, tok * H * pairs * (v2 ? 2 : 1) * d * 2}, {q2, tok * H * d * 2}};
    if ((st = disjoint(fn, w, 2, r, 12)) != DIFFATTN_OK || (st = disjoint(fn, w + 1, 1, q, 2)) != DIFFATTN_OK) return st;
  }
  int* status = nullptr;
  if ((st = dh::status_address(&status)) != DIFFATTN_OK) return st;
  // Neighbouring heads side by side: their rows of a token are neighbours in memory.
  p.team = 1;
  while (p.team < kTreeTeam && H * sh.mt % (2 * p.team) == 0) p.team *= 2;
  const int ctas = std::min(sms_or_default(), kTreeMaxCtas);
  p.teams = static_cast<int>(std::max<long long>(1, std::min<long long>(tiles / p.team, ctas / p.team)));
  const bool k8 = fmt != DIFFATTN_CACHE_BF16, v8 = fmt == DIFFATTN_CACHE_FP8;
  const int nn = n > 0 ? n : 1;
  const int side = std::max(1, p.team / sh.mt);  // heads
  const int kbox = (k8 && d == 64) ? 64 : 128;
  if ((st = cache_map(&p.tm_k1, k1, B, nn, H, d, k8 ? 1 : 2, kbox, 128, side)) != DIFFATTN_OK) return st;
  if (!v2 && (st = cache_map(&p.tm_k2, k2, B, nn, H, d, k8 ? 1 : 2, kbox, 128, side)) != DIFFATTN_OK) return st;
  if ((st = cache_map(&p.tm_v, v, B, nn, H, dv, v8 ? 1 : 2, 128, da::kTreeValueKeys, side)) != DIFFATTN_OK) return st;
  p.q1 = static_cast<const __nv_bfloat16*>(q1);
  p.q2 = static_cast<const __nv_bfloat16*>(q2);
  p.k1_scales = kscales[0];
  p.k2_scales = kscales[1];
  p.v_scales = vscales;
  p.k1_scale = ks[0];
  p.k2_scale = ks[1];
  p.lens = lens;
  p.ntok = ntok;
  p.mask = mask;
  p.mask_sb = mask_sb;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.B = B;
  p.T = T;
  p.H = H;
  p.n = n;
  p.pairs = sh.pairs;
  p.ppt = sh.ppt;
  p.mt = sh.mt;
  p.R = sh.R;
  p.subs = da::tree_subs(fmt, dv, sh.R);
  p.ws = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(workspace) + 31) & ~uintptr_t(31));
  p.status = status;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = v2 ? da::launch_tree_v2_d128(p, fmt, s)
                           : d == 64 ? da::launch_tree_v1_d64(p, fmt, s) : da::launch_tree_v1_d128(p, fmt, s);
  if (e != cudaSuccess) return cuda_fail(e, fn);
  dh::count_launches(2);
  return dh::success();
}

constexpr double kTwoPi = 6.283185307179586476925286766559;

}  // namespace

extern "C" {

diffattn_status diffattn_rope_from_frequencies(diffattn_rope_spec* rope, int rot_dim, int interleaved,
                                               const double* frequencies, float mult) {
  const char* fn = "diffattn_rope_from_frequencies";
  if (!rope || !frequencies) return fail(DIFFATTN_ERR_NULL, "%s: NULL pointer", fn);
  if (rot_dim < 2 || rot_dim > 128 || (rot_dim & 1))
    return fail(DIFFATTN_ERR_SHAPE, "%s: rot_dim %d: even, from 2 to 128", fn, rot_dim);
  if (!std::isfinite(mult)) return fail(DIFFATTN_ERR_SHAPE, "%s: the factor is not finite", fn);
  memset(rope, 0, sizeof(*rope));
  rope->rot_dim = rot_dim;
  rope->interleaved = interleaved ? 1 : 0;
  rope->mult = mult;
  for (int i = 0; i < rot_dim / 2; ++i) {
    if (!std::isfinite(frequencies[i])) return fail(DIFFATTN_ERR_SHAPE, "%s: frequency %d is not finite", fn, i);
    double f = frequencies[i] / kTwoPi;
    f -= std::floor(f);
    if (f >= 1.0) f = 0.0;  // (a tiny negative frequency rounds up to one turn)
    rope->turns[i] = static_cast<unsigned long long>(f * 18446744073709551616.0);
  }
  return dh::success();
}

diffattn_status diffattn_rope_init(diffattn_rope_spec* rope, int rot_dim, int interleaved, double base,
                                   diffattn_rope_scaling scaling, double factor, int original_context,
                                   double beta_fast, double beta_slow) {
  const char* fn = "diffattn_rope_init";
  if (!rope) return fail(DIFFATTN_ERR_NULL, "%s: NULL pointer", fn);
  if (rot_dim < 2 || rot_dim > 128 || (rot_dim & 1))
    return fail(DIFFATTN_ERR_SHAPE, "%s: rot_dim %d: even, from 2 to 128", fn, rot_dim);
  if (!(base > 1.0) || !std::isfinite(base)) return fail(DIFFATTN_ERR_SHAPE, "%s: the base must be above 1", fn);
  if (scaling != DIFFATTN_ROPE_NONE && scaling != DIFFATTN_ROPE_LINEAR && scaling != DIFFATTN_ROPE_NTK &&
      scaling != DIFFATTN_ROPE_YARN)
    return fail(DIFFATTN_ERR_DTYPE, "%s: unknown scaling %d", fn, (int)scaling);
  if (scaling != DIFFATTN_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
    return fail(DIFFATTN_ERR_SHAPE, "%s: the scaling factor must be at least 1", fn);
  if (scaling == DIFFATTN_ROPE_NTK && rot_dim < 4)
    return fail(DIFFATTN_ERR_SHAPE, "%s: ntk scaling needs rot_dim of at least 4", fn);
  if (scaling == DIFFATTN_ROPE_YARN && (original_context < 1 || !(beta_fast > 0.0) || !(beta_slow > 0.0)))
    return fail(DIFFATTN_ERR_SHAPE, "%s: yarn scaling needs the original context and both betas positive", fn);
  const double r = rot_dim;
  if (scaling == DIFFATTN_ROPE_NTK) base *= std::pow(factor, r / (r - 2.0));
  double low = 0.0, high = 1.0;
  if (scaling == DIFFATTN_ROPE_YARN) {
    // the pair that makes `beta` turns over the original context
    low = std::max(0.0, std::floor(r * std::log(original_context / (beta_fast * kTwoPi)) / (2.0 * std::log(base))));
    high = std::min(r - 1.0, std::ceil(r * std::log(original_context / (beta_slow * kTwoPi)) / (2.0 * std::log(base))));
  }
  double th[64];
  for (int i = 0; i < rot_dim / 2; ++i) {
    th[i] = std::pow(base, -2.0 * i / r);
    if (scaling == DIFFATTN_ROPE_LINEAR) th[i] /= factor;
    if (scaling == DIFFATTN_ROPE_YARN) {
      const double w = std::min(1.0, std::max(0.0, (i - low) / std::max(high - low, 0.001)));
      th[i] = th[i] * (1.0 - w) + th[i] / factor * w;
    }
  }
  const double mult = scaling == DIFFATTN_ROPE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
  return diffattn_rope_from_frequencies(rope, rot_dim, interleaved, th, static_cast<float>(mult));
}

diffattn_status diffattn_rope(diffattn_dtype dt, int B, int n, int d, int count, const void* const* x,
                              const int* heads, const diffattn_rope_spec* rope, const int* positions, int inverse,
                              void* const* out, void* stream) {
  const char* fn = "diffattn_rope";
  if (dt != DIFFATTN_F32 && dt != DIFFATTN_BF16) return fail(DIFFATTN_ERR_DTYPE, "%s: bad dtype %d", fn, (int)dt);
  if (B < 0 || n < 0 || d < 1 || count < 0) return fail(DIFFATTN_ERR_SHAPE, "%s: bad sizes B=%d n=%d d=%d", fn, B, n, d);
  if (count > 4) return fail(DIFFATTN_ERR_UNSUPPORTED, "%s: at most 4 tensors a call (got %d)", fn, count);
  if (B == 0 || n == 0 || count == 0) return dh::success();
  if (!x || !heads || !out || !rope) return fail(DIFFATTN_ERR_NULL, "%s: NULL pointer", fn);
  if (d > 128) return fail(DIFFATTN_ERR_UNSUPPORTED, "%s: d = %d above 128", fn, d);
  const bool f32 = dt == DIFFATTN_F32;
  const size_t es = f32 ? 4 : 2;
  da::RopeParams p;
  memset(&p, 0, sizeof(p));
  diffattn_status st = rope_turns(fn, rope, d, &p.rope);
  if (st != DIFFATTN_OK) return st;
  const int N = f32 ? 4 : 8;  // elements of a 16-byte access
  bool vec = d % N == 0 && p.rope.rot % (p.rope.inter ? N : 2 * N) == 0;
  long long head_sum = 0;
  for (int i = 0; i < count; ++i) {
    if (heads[i] < 0) return fail(DIFFATTN_ERR_SHAPE, "%s: %d heads", fn, heads[i]);
    if (heads[i] > 0 && (!x[i] || !out[i])) return fail(DIFFATTN_ERR_NULL, "%s: NULL tensor", fn);
    if (!aligned(x[i], es) || !aligned(out[i], es) || (!f32 && (!aligned(x[i], 16) || !aligned(out[i], 16))))
      return fail(DIFFATTN_ERR_ALIGN, "%s: bf16 tensors must be 16-byte aligned, fp32 ones 4-byte", fn);
    if (!aligned(x[i], 16) || !aligned(out[i], 16)) vec = false;
    p.x[i] = x[i];
    p.out[i] = out[i];
    p.heads[i] = heads[i];
    if (x[i] != out[i]) p.copy = 1;
    head_sum += heads[i];
  }
  // an output may be its own input, and may not overlap anything else of the call
  for (int i = 0; i < count; ++i)
    for (int j = 0; j < count; ++j) {
      const size_t ni = static_cast<size_t>(B) * n * heads[i] * d * es, nj = static_cast<size_t>(B) * n * heads[j] * d * es;
      if ((i != j || x[i] != out[j]) && overlap(out[j], nj, x[i], ni) && ni && nj)
        return fail(DIFFATTN_ERR_SHAPE, "%s: an output overlaps an input other than its own", fn);
      if (i < j && overlap(out[i], ni, out[j], nj) && ni && nj)
        return fail(DIFFATTN_ERR_SHAPE, "%s: outputs overlap", fn);
      if (i == j && positions && ni && overlap(out[i], ni, positions, sizeof(int) * static_cast<size_t>(B) * n))
        return fail(DIFFATTN_ERR_SHAPE, "%s: an output overlaps the positions", fn);
    }
  if (head_sum == 0) return dh::success();
  const long long tokens = static_cast<long long>(B) * n;
  const long long items = head_sum * d;  // of a token, at most
  if (tokens > 0x7fffffffll || items > 0xfffffffll)
    return fail(DIFFATTN_ERR_SHAPE, "%s: too many tokens or heads", fn);
  p.count = count;
  p.head_sum = static_cast<int>(head_sum);
  p.B = B;
  p.n = n;
  p.d = d;
  p.inverse = inverse ? 1 : 0;
  p.pos = positions;
  // Tokens a CTA as for the append (fp32 V1 d128, 8192 tokens: 2 a CTA 61.4 us, 6 64.4).
  const int sms = sms_or_default();
  p.tokens_per_cta = static_cast<int>(std::min<long long>(da::kRopeMaxTokens, std::max<long long>(1, tokens / (24 * sms))));
  const int gx = static_cast<int>((tokens + p.tokens_per_cta - 1) / p.tokens_per_cta);
  const long long per_head = vec ? d / N : d;
  {
    const int ri = vec ? (p.rope.inter ? p.rope.rot / N : p.rope.rot / 2 / N) : p.rope.rot / 2;
    const long long ph = ri + (p.copy ? (d - p.rope.rot) / (vec ? N : 1) : 0);
    p.magic_tok = division_magic(head_sum * ph, head_sum * ph * p.tokens_per_cta);
    p.magic_head = division_magic(ph, head_sum * ph);
  }
  const long long most = (head_sum * per_head * p.tokens_per_cta + da::kRopeThreads - 1) / da::kRopeThreads;
  const int gy = static_cast<int>(std::max<long long>(1, std::min<long long>({most, 2ll * sms / gx, 65535ll})));
  const cudaError_t e = da::launch_rope(p, f32, vec, gx, gy, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, fn);
  dh::count_launches(1);
  return dh::success();
}

diffattn_status diffattn_cache_append(diffattn_cache_format fmt, int B, int T, int H, int n, int d, const void* q1,
                                      const void* q2, const void* k1, const void* k2, const void* v,
                                      const diffattn_rope_spec* rope, const int* positions, const int* lens,
                                      const int* ntok, void* q1_out, void* q2_out, void* k1_cache, void* k2_cache,
                                      void* v_cache, float k1_scale, float k2_scale, float* k1_scales,
                                      float* k2_scales, float* v_scales, void* stream) {
  const void* q[2] = {q1, q2};
  const void* k[2] = {k1, k2};
  void* qo[2] = {q1_out, q2_out};
  void* kc[2] = {k1_cache, k2_cache};
  const float ks[2] = {k1_scale, k2_scale};
  float* kscales[2] = {k1_scales, k2_scales};
  return append("diffattn_cache_append", fmt, B, T, H, H, n, d, 2 * d, 2, q, k, v, rope, positions, lens, ntok, qo,
                kc, v_cache, ks, kscales, v_scales, stream);
}

diffattn_status diffattn_v2_cache_append(diffattn_cache_format fmt, int B, int T, int Hq, int Hkv, int n, int d,
                                         const void* q, const void* k, const void* v, const diffattn_rope_spec* rope,
                                         const int* positions, const int* lens, const int* ntok, void* q_out,
                                         void* k_cache, void* v_cache, float k_scale, float* k_scales,
                                         float* v_scales, void* stream) {
  const void* qa[2] = {q, nullptr};
  const void* ka[2] = {k, nullptr};
  void* qo[2] = {q_out, nullptr};
  void* kc[2] = {k_cache, nullptr};
  const float ks[2] = {k_scale, 1.f};
  float* kscales[2] = {k_scales, nullptr};
  return append("diffattn_v2_cache_append", fmt, B, T, Hq, Hkv, n, d, d, 1, qa, ka, v, rope, positions, lens, ntok,
                qo, kc, v_cache, ks, kscales, v_scales, stream);
}

diffattn_status diffattn_cache_keep(diffattn_cache_format fmt, int B, int A, int H, int n, int d, void* k1_cache,
                                    void* k2_cache, void* v_cache, float* k1_scales, float* k2_scales,
                                    float* v_scales, const int* lens, const int* path, const int* nkeep,
                                    int* new_lens, void* stream) {
  void* kc[2] = {k1_cache, k2_cache};
  float* kscales[2] = {k1_scales, k2_scales};
  return keep("diffattn_cache_keep", fmt, B, A, H, n, d, 2 * d, 2, kc, v_cache, kscales, v_scales, lens, path, nkeep,
              new_lens, stream);
}

diffattn_status diffattn_v2_cache_keep(diffattn_cache_format fmt, int B, int A, int Hkv, int n, int d, void* k_cache,
                                       void* v_cache, float* k_scales, float* v_scales, const int* lens,
                                       const int* path, const int* nkeep, int* new_lens, void* stream) {
  void* kc[2] = {k_cache, nullptr};
  float* kscales[2] = {k_scales, nullptr};
  return keep("diffattn_v2_cache_keep", fmt, B, A, Hkv, n, d, d, 1, kc, v_cache, kscales, v_scales, lens, path, nkeep,
              new_lens, stream);
}

size_t diffattn_tree_decode_workspace(int B, int T, int H, int d) {
  if (B < 1 || T < 1 || H < 1 || d < 1 || T > da::kTreeRows) return 0;
  return tree_workspace(B, T, H, 1, 2 * d);
}

diffattn_status diffattn_tree_decode(diffattn_cache_format fmt, int B, int T, int H, int n, int d, const void* q1,
                                     const void* q2, const void* k1, const void* k2, float k1_scale, float k2_scale,
                                     const float* k1_scales, const float* k2_scales, const void* v,
                                     const float* v_scales, const int* lens, const int* ntok,
                                     const unsigned long long* mask, long long mask_sb, const float* lambda,
                                     float lambda_init, const float* gamma, float eps, void* out, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  const char* fn = "diffattn_tree_decode";
  if (B < 0 || T < 0 || H < 0 || n < 0 || d < 1 || mask_sb < 0)
    return fail(DIFFATTN_ERR_SHAPE, "%s: bad sizes B=%d T=%d H=%d n=%d d=%d", fn, B, T, H, n, d);
  if (B == 0 || T == 0 || H == 0) return dh::success();
  if (!lambda) return fail(DIFFATTN_ERR_NULL, "%s: NULL lambda", fn);
  if (!std::isfinite(lambda_init)) return fail(DIFFATTN_ERR_SHAPE, "%s: lambda_init not finite", fn);
  da::TreeParams p;
  memset(&p, 0, sizeof(p));
  p.lambda = lambda;
  p.gamma = gamma;
  p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(d)));
  p.norm_mult = 1.f - lambda_init;
  p.eps = eps <= 0.f ? 1e-5f : eps;
  const float ks[2] = {k1_scale, k2_scale};
  const float* kscales[2] = {k1_scales, k2_scales};
  return tree(fn, false, fmt, B, T, H, 1, n, d, q1, q2, k1, k2, ks, kscales, v, v_scales, lens, ntok, mask, mask_sb, p,
              out, workspace, workspace_bytes, stream);
}

size_t diffattn_v2_tree_decode_workspace(int B, int T, int Hq, int Hkv, int d) {
  if (B < 1 || T < 1 || Hkv < 1 || d < 1 || T > da::kTreeRows || Hq < 2 * Hkv || Hq % (2 * Hkv)) return 0;
  return tree_workspace(B, T, Hkv, Hq / Hkv / 2, d);
}

diffattn_status diffattn_v2_tree_decode(diffattn_cache_format fmt, int B, int T, int Hq, int Hkv, int n, int d,
                                        const void* q, const void* k, float k_scale, const float* k_scales,
                                        const void* v, const float* v_scales, const int* lens, const int* ntok,
                                        const unsigned long long* mask, long long mask_sb, const float* lam_logits,
                                        long long sb, long long st, float softmax_scale, void* out, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  const char* fn = "diffattn_v2_tree_decode";
  if (B < 0 || T < 0 || Hq < 0 || Hkv < 0 || n < 0 || d < 1 || mask_sb < 0)
    return fail(DIFFATTN_ERR_SHAPE, "%s: bad sizes B=%d T=%d Hq=%d Hkv=%d n=%d d=%d", fn, B, T, Hq, Hkv, n, d);
  if (B == 0 || T == 0 || Hq == 0) return dh::success();
  if (Hkv < 1 || Hq % (2 * Hkv))
    return fail(DIFFATTN_ERR_SHAPE, "%s: Hq = %d must be an even multiple of Hkv = %d", fn, Hq, Hkv);
  if (!lam_logits) return fail(DIFFATTN_ERR_NULL, "%s: NULL lam_logits", fn);
  if (!std::isfinite(softmax_scale)) return fail(DIFFATTN_ERR_SHAPE, "%s: softmax_scale not finite", fn);
  da::TreeParams p;
  memset(&p, 0, sizeof(p));
  p.lam_logits = lam_logits;
  p.sb = sb;
  p.st = st;
  const double scale = softmax_scale > 0.f ? softmax_scale : 1.0 / std::sqrt(static_cast<double>(d));
  p.scale_log2 = static_cast<float>(1.4426950408889634 * scale);
  p.norm_mult = 1.f;
  const float ks[2] = {k_scale, k_scale};
  const float* kscales[2] = {k_scales, nullptr};
  return tree(fn, true, fmt, B, T, Hkv, Hq / Hkv / 2, n, d, q, nullptr, k, nullptr, ks, kscales, v, v_scales, lens,
              ntok, mask, mask_sb, p, out, workspace, workspace_bytes, stream);
}

}  // extern "C"
