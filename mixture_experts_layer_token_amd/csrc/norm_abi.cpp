// C-ABI entry points of the norm of rows and of the norm and clipping of gradients: argument validation, then the launches.
#include <algorithm>
#include <cmath>
#include <vector>

#include "norm.hpp"

namespace moe {
namespace {

bool aligned(const void* p, size_t n) { return (uintptr_t)p % n == 0; }
size_t dt_bytes(int dt) { return dt == MOE_BF16 ? 2 : 4; }

constexpr int kMaxRows = 1 << 24, kMaxH = 1 << 20, kMaxTensors = 1 << 16;

int check_norm(const moe_norm_desc* d, const char* fn) {
  if (!d) return fail(MOE_ERR_INVALID, "%s: null moe_norm_desc", fn);
  if (d->rows < 0 || d->rows > kMaxRows) return fail(MOE_ERR_INVALID, "%s: rows=%d out of 0..1<<24", fn, d->rows);
  if (d->H < 1 || d->H > kMaxH) return fail(MOE_ERR_INVALID, "%s: H=%d out of 1..1<<20", fn, d->H);
  if (d->rms != 0 && d->rms != 1) return fail(MOE_ERR_INVALID, "%s: rms=%d", fn, d->rms);
  if (!dtype_valid(d->dt) || !dtype_valid(d->pdt)) return fail(MOE_ERR_INVALID, "%s: bad dtype %d / %d", fn, d->dt, d->pdt);
  if (!(d->eps >= 0.f) || !std::isfinite(d->eps)) return fail(MOE_ERR_INVALID, "%s: eps=%g", fn, (double)d->eps);
  constexpr int64_t kMaxLd = (int64_t)1 << 40;
  if ((d->ldx && (d->ldx < d->H || d->ldx > kMaxLd)) || (d->ldy && (d->ldy < d->H || d->ldy > kMaxLd)))
    return fail(MOE_ERR_INVALID, "%s: row strides %lld, %lld shorter than a row", fn, (long long)d->ldx, (long long)d->ldy);
  return MOE_OK;
}

NormArgs norm_args(const moe_norm_desc* d, const void* x, const void* weight) {
  NormArgs a = {};
  a.rows = d->rows, a.H = d->H, a.rms = d->rms, a.eps = d->eps;
  a.x = x, a.weight = weight;
  a.ldx = d->ldx ? d->ldx : d->H, a.ldy = d->ldy ? d->ldy : d->H;
  a.par_bf16 = d->pdt == MOE_BF16;
  return a;
}

// everything about the list; written: whether results are asked for
int check_tensors(const char* fn, const moe_tensor* t, int n, bool written) {
  if (n < 0 || n > kMaxTensors) return fail(MOE_ERR_INVALID, "%s: n=%d out of 0..1<<16", fn, n);
  if (n > 0 && !t) return fail(MOE_ERR_INVALID, "%s: null list", fn);
  int64_t total = 0;
  for (int i = 0; i < n; ++i) {
    if (!dtype_valid(t[i].dt)) return fail(MOE_ERR_INVALID, "%s: tensor %d: bad dtype %d", fn, i, t[i].dt);
    if (t[i].numel < 0 || t[i].numel > ((int64_t)1 << 40))
      return fail(MOE_ERR_INVALID, "%s: tensor %d: numel=%lld out of 0..1<<40", fn, i, (long long)t[i].numel);
    total += t[i].numel;
    if (t[i].numel > 0 && !t[i].src) return fail(MOE_ERR_INVALID, "%s: tensor %d: null pointer", fn, i);
    if (!aligned(t[i].src, dt_bytes(t[i].dt)) || !aligned(t[i].dst, dt_bytes(t[i].dt)))
      return fail(MOE_ERR_INVALID, "%s: tensor %d: pointer not aligned to its element type", fn, i);
  }
  if (total > ((int64_t)1 << 40)) return fail(MOE_ERR_INVALID, "%s: more than 1<<40 elements", fn);
  if (!written) return MOE_OK;
  // A result may be its own gradient in place; anything else that overlaps it (the same gradient named twice among them) would
  // be read or scaled twice in an order that nothing fixes.
  struct Span {
    uintptr_t lo, hi;
    int i, out;
  };
  std::vector<Span> spans;
  for (int i = 0; i < n; ++i) {
    const size_t bytes = (size_t)t[i].numel * dt_bytes(t[i].dt);
    if (!bytes) continue;
    const bool in_place = t[i].dst == t[i].src;
    spans.push_back({(uintptr_t)t[i].src, (uintptr_t)t[i].src + bytes, i, in_place});
    if (t[i].dst && !in_place) spans.push_back({(uintptr_t)t[i].dst, (uintptr_t)t[i].dst + bytes, i, 1});
  }
  std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
  // of the spans that began earlier, the one that ends last, and the result that ends last
  const Span *any = nullptr, *out = nullptr;
  for (const Span& s : spans) {
    const Span* hit = s.out ? any : out;
    if (hit && hit->hi > s.lo) return fail(MOE_ERR_INVALID, "%s: tensors %d and %d overlap", fn, hit->i, s.i);
    if (!any || s.hi > any->hi) any = &s;
    if (s.out && (!out || s.hi > out->hi)) out = &s;
  }
  return MOE_OK;
}

int grad_norm_call(const char* fn, const moe_tensor* t, int n, bool clip, float max_norm, float* norm, void* ws,
                   size_t ws_bytes, void* stream) {
  int rc;
  try {
    rc = check_tensors(fn, t, n, clip);
  } catch (...) {
    return fail(MOE_ERR_INVALID, "%s: out of host memory", fn);
  }
  if (rc != MOE_OK) return rc;
  if (clip && (!(max_norm > 0.f) || !std::isfinite(max_norm))) return fail(MOE_ERR_INVALID, "%s: max_norm=%g", fn, (double)max_norm);
  if (!norm || !aligned(norm, 4)) return fail(MOE_ERR_INVALID, "%s: null or misaligned norm", fn);
  const size_t need = grad_norm_workspace(n);
  if (!ws || ws_bytes < need || !aligned(ws, 256))
    return fail(MOE_ERR_WORKSPACE, "%s: workspace of %zu bytes (need %zu, 256-byte aligned)", fn, ws ? ws_bytes : 0, need);
  return launch_grad_norm(t, n, clip, max_norm, norm, (double*)ws, (hipStream_t)stream);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_norm(const moe_norm_desc* d, const void* x, const void* weight, const void* bias, void* y, float* stats,
                        void* stream) {
  const char* fn = "moe_norm";
  int rc = check_norm(d, fn);
  if (rc != MOE_OK || d->rows == 0) return rc;
  const size_t b = dt_bytes(d->dt), p = dt_bytes(d->pdt);
  if (!x || !y) return fail(MOE_ERR_INVALID, "%s: null pointer", fn);
  if (!aligned(x, b) || !aligned(y, b) || !aligned(weight, p) || !aligned(bias, p) || !aligned(stats, 4))
    return fail(MOE_ERR_INVALID, "%s: pointer not aligned to its element type", fn);
  NormArgs a = norm_args(d, x, weight);
  a.bias = bias, a.y = y, a.stats = stats;
  return launch_norm(a, d->dt, (hipStream_t)stream);
}

extern "C" size_t moe_norm_workspace(int rows, int H) {
  if (rows < 1 || rows > kMaxRows || H < 1 || H > kMaxH) return 0;
  return norm_workspace(rows, H);
}

extern "C" int moe_norm_grad(const moe_norm_desc* d, const void* dy, const void* x, const void* weight, const float* stats,
                             const void* add, void* dx, void* dweight, void* dbias, void* ws, size_t ws_bytes,
                             void* stream) {
  const char* fn = "moe_norm_grad";
  int rc = check_norm(d, fn);
  if (rc != MOE_OK) return rc;
  const size_t b = dt_bytes(d->dt), p = dt_bytes(d->pdt);
  if (d->rows > 0 && (!dy || !x || !stats || !dx)) return fail(MOE_ERR_INVALID, "%s: null pointer", fn);
  if (!aligned(dy, b) || !aligned(x, b) || !aligned(add, b) || !aligned(dx, b) || !aligned(weight, p) ||
      !aligned(dweight, p) || !aligned(dbias, p) || !aligned(stats, 4))
    return fail(MOE_ERR_INVALID, "%s: pointer not aligned to its element type", fn);
  const size_t need = moe_norm_workspace(d->rows, d->H);
  if (need && (!ws || ws_bytes < need || !aligned(ws, 256)))
    return fail(MOE_ERR_WORKSPACE, "%s: workspace of %zu bytes (need %zu, 256-byte aligned)", fn, ws ? ws_bytes : 0, need);
  NormArgs a = norm_args(d, x, weight);
  a.dy = dy, a.add = add, a.dx = dx, a.dweight = dweight, a.dbias = dbias;
  a.stats = const_cast<float*>(stats);
  const size_t part = (size_t)norm_parts(d->rows, d->H) * 2 * d->H;
  a.part = dweight || dbias ? (float*)ws : nullptr;
  a.sums = (float*)ws + part;
  return launch_norm_grad(a, d->dt, (hipStream_t)stream);
}

extern "C" size_t moe_grad_norm_workspace(int n) { return n < 0 || n > kMaxTensors ? 0 : grad_norm_workspace(n); }

extern "C" int moe_grad_norm(const moe_tensor* t, int n, float* norm, void* ws, size_t ws_bytes, void* stream) {
  return grad_norm_call("moe_grad_norm", t, n, false, 0.f, norm, ws, ws_bytes, stream);
}

extern "C" int moe_clip_grad_norm(const moe_tensor* t, int n, float max_norm, float* norm, void* ws, size_t ws_bytes,
                                  void* stream) {
  return grad_norm_call("moe_clip_grad_norm", t, n, true, max_norm, norm, ws, ws_bytes, stream);
}
