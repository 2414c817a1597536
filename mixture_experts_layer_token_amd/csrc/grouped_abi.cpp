// C-ABI entry points of the grouped products over plain weights, of the 8-bit operators, of the SwiGLU gate
// and of the combine's gradient: argument validation, then the launches.
#include "grouped.hpp"
#include "rowwise.hpp"

namespace moe {
namespace {

bool aligned(const void* p, size_t n) { return (uintptr_t)p % n == 0; }
size_t dt_bytes(int dt) { return dt == MOE_BF16 ? 2 : 4; }

// everything about the descriptor; bytes: of an x / w element
int check_grouped(const moe_grouped* g, const char* fn) {
  if (!g) return fail(MOE_ERR_INVALID, "%s: null moe_grouped", fn);
  if (g->rows < 0 || g->rows > (1 << 24)) return fail(MOE_ERR_INVALID, "%s: rows=%d out of 0..1<<24", fn, g->rows);
  if (g->E < 1 || g->E > 1024) return fail(MOE_ERR_INVALID, "%s: E=%d out of 1..1024", fn, g->E);
  if (g->N < 1 || g->N > (1 << 20) || g->K < 1 || g->K > (1 << 20))
    return fail(MOE_ERR_INVALID, "%s: N=%d, K=%d out of 1..1<<20", fn, g->N, g->K);
  if (g->perm_src && (g->k < 1 || g->k > 16 || g->x_rows < 0 || g->x_rows > (1 << 24)))
    return fail(MOE_ERR_INVALID, "%s: k=%d, x_rows=%d", fn, g->k, g->x_rows);
  constexpr int64_t kMaxLd = (int64_t)1 << 40;
  if ((g->ldx && (g->ldx < g->K || g->ldx > kMaxLd)) || (g->ldw && (g->ldw < g->K || g->ldw > kMaxLd)) ||
      (g->ldy && (g->ldy < g->N || g->ldy > kMaxLd)))
    return fail(MOE_ERR_INVALID, "%s: row strides %lld, %lld, %lld shorter than a row", fn, (long long)g->ldx,
                (long long)g->ldw, (long long)g->ldy);
  const int64_t ldw = g->ldw ? g->ldw : g->K;
  if (g->w_stride && (g->w_stride < (g->N - 1) * ldw + g->K || g->w_stride > kMaxLd))
    return fail(MOE_ERR_INVALID, "%s: expert stride %lld shorter than a matrix", fn, (long long)g->w_stride);
  if (!g->offsets || !aligned(g->offsets, 4) || !aligned(g->perm_src, 4))
    return fail(MOE_ERR_INVALID, "%s: null or misaligned offsets or perm_src", fn);
  return MOE_OK;
}

GroupArgs group_args(const moe_grouped* g, const void* x, const void* w, const void* y, int out_dt) {
  GroupArgs a = {};
  a.x = x, a.w = w, a.y = y;
  a.offsets = g->offsets, a.perm_src = g->perm_src;
  a.k = g->perm_src ? g->k : 1;
  a.k_inv = a.k > 1 ? (unsigned)((0x100000000ULL + a.k - 1) / a.k) : 0;
  a.x_rows = g->perm_src ? g->x_rows : g->rows;
  a.rows = g->rows, a.E = g->E, a.N = g->N, a.K = g->K;
  a.ldx = g->ldx ? g->ldx : g->K;
  a.ldy = g->ldy ? g->ldy : g->N;
  a.ldw = g->ldw ? g->ldw : g->K;
  a.w_stride = g->w_stride ? g->w_stride : a.ldw * g->N;
  a.out_bf16 = out_dt == MOE_BF16;
  return a;
}

// x, w, y in the roles of the forward product; `out` is the one that is written
int grouped_call(const char* fn, const moe_grouped* g, int op, int dt, const void* x, const void* w, const void* y,
                 int out_dt, void* ws, size_t ws_bytes, void* stream) {
  if (!dtype_valid(dt) || !dtype_valid(out_dt)) return fail(MOE_ERR_INVALID, "%s: bad dtype %d / %d", fn, dt, out_dt);
  int rc = check_grouped(g, fn);
  if (rc != MOE_OK) return rc;
  const bool dw = op == kOpDw;
  const bool need_w = dw || g->rows > 0, need_xy = g->rows > 0;
  if ((need_w && !w) || (need_xy && (!y || (!x && !(g->perm_src && g->x_rows == 0)))))
    return fail(MOE_ERR_INVALID, "%s: null pointer", fn);
  const size_t in = dt_bytes(dt), out = dt_bytes(out_dt);
  if (!aligned(x, op == kOpDx ? out : in) || !aligned(w, dw ? out : in) || !aligned(y, op == kOpY ? out : in))
    return fail(MOE_ERR_INVALID, "%s: pointer not aligned to its element type", fn);
  const size_t need = moe_grouped_workspace(dt, g->rows, g->N, g->K, g->E);
  if (need && (!ws || ws_bytes < need || !aligned(ws, 256)))
    return fail(MOE_ERR_WORKSPACE, "%s: workspace of %zu bytes (need %zu, 256-byte aligned)", fn, ws ? ws_bytes : 0,
                need);
  if (g->rows == 0 && !dw) return MOE_OK;
  GroupArgs a = group_args(g, x, w, y, out_dt);
  if (op == kOpDx) a.perm_src = nullptr;  // dx has one row per grouped row
  return launch_grouped(a, op, dt == MOE_BF16 ? kBf16 : kF32, ws, (hipStream_t)stream);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_grouped_workspace(int dt, int rows, int N, int K, int E) {
  if (!dtype_valid(dt) || rows < 0 || N < 1 || K < 1 || E < 1 || E > 1024) return 0;
  return grouped_workspace(dt == MOE_BF16 ? kBf16 : kF32, rows, N, K, E);
}

extern "C" int moe_grouped_gemm(const moe_grouped* g, int dt, const void* x, const void* w, void* y, int ydt, void* ws,
                                size_t ws_bytes, void* stream) {
  return grouped_call("moe_grouped_gemm", g, kOpY, dt, x, w, y, ydt, ws, ws_bytes, stream);
}

extern "C" int moe_grouped_gemm_dx(const moe_grouped* g, int dt, const void* dy, const void* w, void* dx, int dxdt,
                                   void* ws, size_t ws_bytes, void* stream) {
  moe_grouped h;
  if (g) {
    h = *g;
    h.perm_src = nullptr;
  }
  return grouped_call("moe_grouped_gemm_dx", g ? &h : nullptr, kOpDx, dt, dx, w, dy, dxdt, ws, ws_bytes, stream);
}

extern "C" int moe_grouped_gemm_dw(const moe_grouped* g, int dt, const void* dy, const void* x, void* dw, int dwdt,
                                   void* ws, size_t ws_bytes, void* stream) {
  return grouped_call("moe_grouped_gemm_dw", g, kOpDw, dt, x, dw, dy, dwdt, ws, ws_bytes, stream);
}

extern "C" int moe_grouped_gemm_i8(const moe_grouped* g, const int8_t* q, const float* q_scale, const int8_t* w,
                                   const float* w_scale, void* y, int ydt, void* stream) {
  const char* fn = "moe_grouped_gemm_i8";
  if (!dtype_valid(ydt)) return fail(MOE_ERR_INVALID, "%s: bad dtype %d", fn, ydt);
  int rc = check_grouped(g, fn);
  if (rc != MOE_OK) return rc;
  if (g->K > 131071) return fail(MOE_ERR_UNSUPPORTED, "%s: K=%d above 131071 (int32 sums)", fn, g->K);
  const bool no_x = g->perm_src && g->x_rows == 0;
  if (g->rows > 0 && (!w || !w_scale || !y || (!no_x && (!q || !q_scale))))
    return fail(MOE_ERR_INVALID, "%s: null pointer", fn);
  if (!aligned(y, dt_bytes(ydt)) || !aligned(q_scale, 4) || !aligned(w_scale, 4))
    return fail(MOE_ERR_INVALID, "%s: pointer not aligned to its element type", fn);
  if (g->rows == 0) return MOE_OK;
  GroupArgs a = group_args(g, q, w, y, ydt);
  a.x_scale = q_scale, a.w_scale = w_scale;
  return launch_grouped(a, kOpY, kI8, nullptr, (hipStream_t)stream);
}

extern "C" int moe_quant_rows(const void* x, int xdt, int rows, int K, int act, const int32_t* n_rows, int8_t* q,
                              float* scale, void* stream) {
  const char* fn = "moe_quant_rows";
  if (!dtype_valid(xdt)) return fail(MOE_ERR_INVALID, "%s: bad dtype %d", fn, xdt);
  if (act != MOE_ACT_NONE && act != MOE_ACT_SWIGLU) return fail(MOE_ERR_INVALID, "%s: bad act %d", fn, act);
  if (rows < 0 || K < 1 || K > (1 << 20)) return fail(MOE_ERR_INVALID, "%s: rows=%d K=%d", fn, rows, K);
  if (rows == 0) return MOE_OK;
  if (!x || !q || !scale) return fail(MOE_ERR_INVALID, "%s: null pointer", fn);
  if (!aligned(x, dt_bytes(xdt)) || !aligned(scale, 4) || !aligned(n_rows, 4))
    return fail(MOE_ERR_INVALID, "%s: pointer not aligned to its element type", fn);
  return launch_quant_rows(x, xdt, rows, K, act, n_rows, q, scale, (hipStream_t)stream);
}

namespace {

int check_gate(const char* fn, const void* gu, int dt, int rows, int I, const int32_t* n_rows) {
  if (!dtype_valid(dt)) return fail(MOE_ERR_INVALID, "%s: bad dtype %d", fn, dt);
  if (rows < 0 || I < 1 || I > (1 << 20)) return fail(MOE_ERR_INVALID, "%s: rows=%d I=%d", fn, rows, I);
  if (rows > 0 && !gu) return fail(MOE_ERR_INVALID, "%s: null pointer", fn);
  if (!aligned(gu, dt_bytes(dt)) || !aligned(n_rows, 4))
    return fail(MOE_ERR_INVALID, "%s: pointer not aligned to its element type", fn);
  return MOE_OK;
}

}  // namespace

extern "C" int moe_swiglu(const void* gu, int dt, int rows, int I, const int32_t* n_rows, void* h, void* stream) {
  int rc = check_gate("moe_swiglu", gu, dt, rows, I, n_rows);
  if (rc != MOE_OK || rows == 0) return rc;
  if (!h || !aligned(h, dt_bytes(dt))) return fail(MOE_ERR_INVALID, "moe_swiglu: null or misaligned h");
  return launch_swiglu(gu, nullptr, dt, rows, I, n_rows, nullptr, h, (hipStream_t)stream);
}

extern "C" int moe_swiglu_grad(const void* gu, const void* dh, int dt, int rows, int I, const int32_t* n_rows,
                               void* dgu, void* h, void* stream) {
  int rc = check_gate("moe_swiglu_grad", gu, dt, rows, I, n_rows);
  if (rc != MOE_OK || rows == 0) return rc;
  const size_t b = dt_bytes(dt);
  if (!dh || !dgu || !aligned(dh, b) || !aligned(dgu, b) || !aligned(h, b))
    return fail(MOE_ERR_INVALID, "moe_swiglu_grad: null or misaligned pointer");
  return launch_swiglu(gu, dh, dt, rows, I, n_rows, dgu, h, (hipStream_t)stream);
}

extern "C" int moe_combine_grad(const void* dout, int odt, const float* y_perm, const float* topk_w,
                                const int32_t* inv_perm, int T, int k, int H, void* dy_perm, int ydt, float* dtopk_w,
                                const int32_t* topk_ids, int E, float* dlogits, void* stream) {
  const char* fn = "moe_combine_grad";
  if (!dtype_valid(odt) || !dtype_valid(ydt)) return fail(MOE_ERR_INVALID, "%s: bad dtype %d / %d", fn, odt, ydt);
  if (T < 0 || k < 1 || k > 16 || H < 1 || H > (1 << 20))
    return fail(MOE_ERR_INVALID, "%s: T=%d k=%d H=%d", fn, T, k, H);
  if ((long long)T * k > (1LL << 24)) return fail(MOE_ERR_INVALID, "%s: T*k too large", fn);
  if (dlogits && (E < 1 || E > 1024)) return fail(MOE_ERR_INVALID, "%s: E=%d out of 1..1024", fn, E);
  if (T == 0) return MOE_OK;
  if (!dout || !y_perm || !topk_w || !inv_perm || !dy_perm || !dtopk_w || (dlogits && !topk_ids))
    return fail(MOE_ERR_INVALID, "%s: null pointer", fn);
  if (!aligned(dout, dt_bytes(odt)) || !aligned(dy_perm, dt_bytes(ydt)) || !aligned(y_perm, 4) ||
      !aligned(topk_w, 4) || !aligned(inv_perm, 4) || !aligned(dtopk_w, 4) || !aligned(topk_ids, 4) ||
      !aligned(dlogits, 4))
    return fail(MOE_ERR_INVALID, "%s: pointer not aligned to its element type", fn);
  return launch_combine_grad(dout, odt, y_perm, topk_w, inv_perm, T, k, H, dy_perm, ydt, dtopk_w, topk_ids, E,
                             dlogits, (hipStream_t)stream);
}
