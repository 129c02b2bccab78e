// C-ABI entry points of the microscaled formats, the gated activation and the
// layer norm: argument validation, then kernel launches on the caller's
// stream.  No device allocation and no host synchronisation.
#include <stdint.h>

#include "../../include/fp8sg.h"
#include "launch_mx.hpp"

using namespace fp8sg;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool type_ok(int t) { return t == FP8SG_OUT_BF16 || t == FP8SG_OUT_F16 || t == FP8SG_OUT_F32; }
bool rule_ok(int r) { return r == FP8SG_MX_FLOOR || r == FP8SG_MX_FIT; }
uintptr_t esize(int t) { return t == FP8SG_OUT_F32 ? 4 : 2; }
fp8sg_status hip_status(hipError_t e) { return e == hipSuccess ? FP8SG_OK : FP8SG_ERR_HIP; }
hipStream_t S(fp8sg_stream s) { return reinterpret_cast<hipStream_t>(s); }

// rows x cols within FP8SG_MAX_DIM and FP8SG_MAX_ELEMS
bool mat_ok(int64_t r, int64_t c) {
  return r >= 0 && c >= 0 && r <= FP8SG_MAX_DIM && c <= FP8SG_MAX_DIM && (r == 0 || c <= FP8SG_MAX_ELEMS / r);
}

// A tensor of n elements of a type: NULL only when empty.
fp8sg_status check_tensor(const void* p, int64_t n, int type) {
  if (n > 0 && !p) return FP8SG_ERR_NULL;
  return aligned(p, esize(type)) ? FP8SG_OK : FP8SG_ERR_ALIGN;
}
// A pair of code and scale buffers over n elements.
template <class Pair>
fp8sg_status check_codes(const Pair& m, int64_t n) {
  if (n > 0 && (!m.q || !m.s)) return FP8SG_ERR_NULL;
  return aligned(m.q, 16) && aligned(m.s, 16) ? FP8SG_OK : FP8SG_ERR_ALIGN;
}
#define FP8SG_TRY(expr)                              \
  do {                                               \
    const fp8sg_status st_ = (expr);                 \
    if (st_ != FP8SG_OK) return st_;                 \
  } while (0)

// x's rows are ld elements apart
fp8sg_status check_rows(const void* p, int64_t ld, int64_t rows, int64_t cols, int type) {
  if (rows * cols > 0 && (ld < cols || !mat_ok(rows, ld))) return FP8SG_ERR_SHAPE;
  return check_tensor(p, rows * cols, type);
}

}  // namespace

extern "C" {

int64_t mxfp4_code_bytes(int64_t rows, int64_t k) { return mat_ok(rows, k) ? rows * mx_pitch(k) : -1; }

int64_t mxfp4_scale_bytes(int64_t rows, int64_t k) {
  return mat_ok(rows, k) ? (rows + 31) / 32 * mx_ktiles(k) * 256 : -1;
}

fp8sg_status mxfp4_quantize(const void* x, fp8sg_out type, int64_t rows, int64_t cols, fp8sg_mx_rule rule,
                            const mxfp4_operand* q, const mxfp4_operand* qT, fp8sg_stream stream) {
  if (!type_ok(type) || !rule_ok(rule)) return FP8SG_ERR_FORMAT;
  if (!mat_ok(rows, cols)) return FP8SG_ERR_SHAPE;
  if (!q && !qT) return FP8SG_ERR_NULL;
  FP8SG_TRY(check_tensor(x, rows * cols, type));
  MxQuantJob j{};
  j.x = x;
  j.rows = rows;
  j.cols = cols;
  if (q) {
    FP8SG_TRY(check_codes(*q, rows * cols));
    j.q = *q;
  }
  if (qT) {
    FP8SG_TRY(check_codes(*qT, rows * cols));
    j.t = *qT;
  }
  return hip_status(launch_mx_quantize(&j, 1, type, rule == FP8SG_MX_FIT, S(stream)));
}

fp8sg_status mxfp4_dequantize(const mxfp4_operand* m, int64_t rows, int64_t k, void* y, fp8sg_out type,
                              fp8sg_stream stream) {
  if (!m) return FP8SG_ERR_NULL;
  if (!type_ok(type)) return FP8SG_ERR_FORMAT;
  if (!mat_ok(rows, k)) return FP8SG_ERR_SHAPE;
  FP8SG_TRY(check_codes(*m, rows * k));
  FP8SG_TRY(check_tensor(y, rows * k, type));
  return hip_status(launch_mx_dequantize(*m, rows, k, y, type, S(stream)));
}

fp8sg_status mxfp4_gemm(const mxfp4_operand* A, const mxfp4_operand* B, void* C, fp8sg_out out, int64_t M,
                        int64_t N, int64_t Kc, fp8sg_stream stream) {
  if (!A || !B) return FP8SG_ERR_NULL;
  if (!type_ok(out)) return FP8SG_ERR_FORMAT;
  if (!mat_ok(M, Kc) || !mat_ok(N, Kc) || !mat_ok(M, N)) return FP8SG_ERR_SHAPE;
  FP8SG_TRY(check_codes(*A, M * Kc));
  FP8SG_TRY(check_codes(*B, N * Kc));
  FP8SG_TRY(check_tensor(C, M * N, out));
  return hip_status(launch_mx_gemm(MxGemmProblem{*A, *B, C, M, N, Kc}, out, S(stream)));
}

fp8sg_status mxfp4_linear_fwd(const void* x, const void* w, fp8sg_out type, int64_t M, int64_t N, int64_t K,
                              fp8sg_mx_rule rule, const mxfp4_linear_ws* ws, const mxfp4_linear_saved* saved,
                              void* y, fp8sg_out out, fp8sg_stream stream) {
  if (!ws) return FP8SG_ERR_NULL;
  if (!type_ok(type) || !type_ok(out) || !rule_ok(rule)) return FP8SG_ERR_FORMAT;
  if (!mat_ok(M, K) || !mat_ok(N, K) || !mat_ok(M, N)) return FP8SG_ERR_SHAPE;
  FP8SG_TRY(check_tensor(x, M * K, type));
  FP8SG_TRY(check_tensor(w, N * K, type));
  FP8SG_TRY(check_codes(ws->x_q, M * K));
  FP8SG_TRY(check_codes(ws->w_q, N * K));
  MxQuantJob j[2] = {{x, M, K, ws->x_q, {}}, {w, N, K, ws->w_q, {}}};
  if (saved) {
    FP8SG_TRY(check_codes(saved->x_qT, M * K));
    FP8SG_TRY(check_codes(saved->w_qT, N * K));
    j[0].t = saved->x_qT;
    j[1].t = saved->w_qT;
  }
  FP8SG_TRY(check_tensor(y, M * N, out));
  const hipError_t e = launch_mx_quantize(j, 2, type, rule == FP8SG_MX_FIT, S(stream));
  if (e != hipSuccess) return FP8SG_ERR_HIP;
  return hip_status(launch_mx_gemm(MxGemmProblem{ws->x_q, ws->w_q, y, M, N, K}, out, S(stream)));
}

fp8sg_status mxfp4_linear_bwd(const void* gy, fp8sg_out type, int64_t M, int64_t N, int64_t K, fp8sg_mx_rule rule,
                              const mxfp4_linear_ws* ws, const mxfp4_linear_saved* saved, void* gx, void* gw,
                              fp8sg_out out, fp8sg_stream stream) {
  if (!ws || !saved) return FP8SG_ERR_NULL;
  if (!type_ok(type) || !type_ok(out) || !rule_ok(rule)) return FP8SG_ERR_FORMAT;
  if (!mat_ok(M, K) || !mat_ok(N, K) || !mat_ok(M, N)) return FP8SG_ERR_SHAPE;
  if (!gx && !gw && M * K > 0 && N * K > 0) return FP8SG_ERR_NULL;  // (an empty gradient may be NULL)
  FP8SG_TRY(check_tensor(gy, M * N, type));
  MxQuantJob j{gy, M, N, {}, {}};
  if (gx) {
    FP8SG_TRY(check_codes(ws->gy_q, M * N));
    FP8SG_TRY(check_codes(saved->w_qT, N * K));
    FP8SG_TRY(check_tensor(gx, M * K, out));
    j.q = ws->gy_q;
  }
  if (gw) {
    FP8SG_TRY(check_codes(ws->gy_qT, M * N));
    FP8SG_TRY(check_codes(saved->x_qT, M * K));
    FP8SG_TRY(check_tensor(gw, N * K, out));
    j.t = ws->gy_qT;
  }
  if (!gx && !gw) return FP8SG_OK;  // what is wanted is empty
  hipError_t e = launch_mx_quantize(&j, 1, type, rule == FP8SG_MX_FIT, S(stream));
  if (e != hipSuccess) return FP8SG_ERR_HIP;
  const MxGemmProblem dgrad{ws->gy_q, saved->w_qT, gx, M, K, N}, wgrad{ws->gy_qT, saved->x_qT, gw, N, K, M};
  if (gx && gw) e = launch_mx_gemm_pair(dgrad, wgrad, out, S(stream));
  else e = launch_mx_gemm(gx ? dgrad : wgrad, out, S(stream));
  return hip_status(e);
}

fp8sg_status mxfp4_linear_apply(const void* x, fp8sg_out type, const mxfp4_operand* w, int64_t M, int64_t N,
                                int64_t K, fp8sg_mx_rule rule, const mxfp4_operand* x_ws, void* y, fp8sg_out out,
                                fp8sg_stream stream) {
  if (!w || !x_ws) return FP8SG_ERR_NULL;
  if (!type_ok(type) || !type_ok(out) || !rule_ok(rule)) return FP8SG_ERR_FORMAT;
  if (!mat_ok(M, K) || !mat_ok(N, K) || !mat_ok(M, N)) return FP8SG_ERR_SHAPE;
  FP8SG_TRY(check_tensor(x, M * K, type));
  FP8SG_TRY(check_codes(*w, N * K));
  FP8SG_TRY(check_codes(*x_ws, M * K));
  FP8SG_TRY(check_tensor(y, M * N, out));
  const MxQuantJob j{x, M, K, *x_ws, {}};
  return hip_status(launch_mx_apply(j, type, rule == FP8SG_MX_FIT, MxGemmProblem{*x_ws, *w, y, M, N, K}, out, S(stream)));
}

fp8sg_status act8_quantize(const void* x, fp8sg_out type, int64_t rows, int64_t cols, const fp8sg_act8* c,
                           fp8sg_stream stream) {
  if (!c) return FP8SG_ERR_NULL;
  if (!type_ok(type)) return FP8SG_ERR_FORMAT;
  if (!mat_ok(rows, cols)) return FP8SG_ERR_SHAPE;
  FP8SG_TRY(check_tensor(x, rows * cols, type));
  FP8SG_TRY(check_codes(*c, rows * cols));
  return hip_status(launch_act8_quantize(x, type, rows, cols, *c, S(stream)));
}

fp8sg_status act8_dequantize(const fp8sg_act8* c, int64_t rows, int64_t cols, void* y, fp8sg_out type,
                             fp8sg_stream stream) {
  if (!c) return FP8SG_ERR_NULL;
  if (!type_ok(type)) return FP8SG_ERR_FORMAT;
  if (!mat_ok(rows, cols)) return FP8SG_ERR_SHAPE;
  FP8SG_TRY(check_codes(*c, rows * cols));
  FP8SG_TRY(check_tensor(y, rows * cols, type));
  return hip_status(launch_act8_dequantize(*c, rows, cols, y, type, S(stream)));
}

fp8sg_status swiglu_fwd(const void* g, int64_t ldg, const void* u, int64_t ldu, fp8sg_out type, int64_t rows,
                        int64_t cols, void* a, const fp8sg_act8* cg, const fp8sg_act8* cu, fp8sg_stream stream) {
  if (!type_ok(type)) return FP8SG_ERR_FORMAT;
  if (!mat_ok(rows, cols)) return FP8SG_ERR_SHAPE;
  if (!cg != !cu) return FP8SG_ERR_NULL;
  FP8SG_TRY(check_rows(g, ldg, rows, cols, type));
  FP8SG_TRY(check_rows(u, ldu, rows, cols, type));
  FP8SG_TRY(check_tensor(a, rows * cols, type));
  SwigluArgs p{};
  if (cg) {
    FP8SG_TRY(check_codes(*cg, rows * cols));
    FP8SG_TRY(check_codes(*cu, rows * cols));
    p.cg = *cg;
    p.cu = *cu;
  }
  p.g = g;
  p.u = u;
  p.ldg = ldg;
  p.ldu = ldu;
  p.rows = rows;
  p.cols = cols;
  p.a = a;
  return hip_status(launch_swiglu_fwd(p, type, S(stream)));
}

fp8sg_status swiglu_bwd(const void* da, const void* g, int64_t ldg, const void* u, int64_t ldu, const fp8sg_act8* cg,
                        const fp8sg_act8* cu, fp8sg_out type, int64_t rows, int64_t cols, void* dg, int64_t lddg,
                        void* du, int64_t lddu, fp8sg_stream stream) {
  if (!type_ok(type)) return FP8SG_ERR_FORMAT;
  if (!mat_ok(rows, cols)) return FP8SG_ERR_SHAPE;
  if (!cg != !cu) return FP8SG_ERR_NULL;
  FP8SG_TRY(check_tensor(da, rows * cols, type));
  FP8SG_TRY(check_rows(dg, lddg, rows, cols, type));
  FP8SG_TRY(check_rows(du, lddu, rows, cols, type));
  SwigluArgs p{};
  if (cg) {
    FP8SG_TRY(check_codes(*cg, rows * cols));
    FP8SG_TRY(check_codes(*cu, rows * cols));
    p.cg = *cg;
    p.cu = *cu;
  } else {
    FP8SG_TRY(check_rows(g, ldg, rows, cols, type));
    FP8SG_TRY(check_rows(u, ldu, rows, cols, type));
    p.g = g;
    p.u = u;
    p.ldg = ldg;
    p.ldu = ldu;
  }
  p.da = da;
  p.rows = rows;
  p.cols = cols;
  p.dg = dg;
  p.du = du;
  p.lddg = lddg;
  p.lddu = lddu;
  return hip_status(launch_swiglu_bwd(p, type, S(stream)));
}

fp8sg_status layer_norm_fwd(const void* x, fp8sg_out type, const void* w, const void* b, fp8sg_out ptype,
                            int64_t rows, int64_t cols, float eps, void* y, float* mean, float* rstd,
                            const fp8sg_act8* ckpt, fp8sg_stream stream) {
  if (!type_ok(type) || (ptype != type && ptype != FP8SG_OUT_F32)) return FP8SG_ERR_FORMAT;
  if (!mat_ok(rows, cols) || (rows > 0 && cols == 0) || !(eps >= 0.f)) return FP8SG_ERR_SHAPE;
  FP8SG_TRY(check_tensor(x, rows * cols, type));
  FP8SG_TRY(check_tensor(y, rows * cols, type));
  if (!mean != !rstd && rows > 0) return FP8SG_ERR_NULL;
  if (!aligned(w, esize(ptype)) || !aligned(b, esize(ptype)) || !aligned(mean, 4) || !aligned(rstd, 4))
    return FP8SG_ERR_ALIGN;
  LayerNormArgs p{};
  if (ckpt) {
    FP8SG_TRY(check_codes(*ckpt, rows * cols));
    p.ckpt = *ckpt;
  }
  p.x = x;
  p.w = w;
  p.b = b;
  p.mean = mean;
  p.rstd = rstd;
  p.rows = rows;
  p.cols = cols;
  p.eps = eps;
  p.y = y;
  return hip_status(launch_layer_norm_fwd(p, type, ptype, S(stream)));
}

int64_t layer_norm_workspace_len(int64_t rows, int64_t cols) {
  return mat_ok(rows, cols) ? layer_norm_ws_len(rows, cols) : -1;
}

fp8sg_status layer_norm_bwd(const void* dy, const void* x, const fp8sg_act8* ckpt, fp8sg_out type, const void* w,
                            fp8sg_out ptype, const float* mean, const float* rstd, int64_t rows, int64_t cols,
                            void* dx, void* dw, void* db, float* ws, int64_t ws_len, fp8sg_stream stream) {
  if (!type_ok(type) || (ptype != type && ptype != FP8SG_OUT_F32)) return FP8SG_ERR_FORMAT;
  if (!mat_ok(rows, cols) || (rows > 0 && cols == 0)) return FP8SG_ERR_SHAPE;
  const int64_t n = rows * cols;
  FP8SG_TRY(check_tensor(dy, n, type));
  LayerNormArgs p{};
  if (ckpt) {
    if (x) return FP8SG_ERR_NULL;
    FP8SG_TRY(check_codes(*ckpt, n));
    p.ckpt = *ckpt;
  } else {
    FP8SG_TRY(check_tensor(x, n, type));
    p.x = x;
  }
  if (rows > 0 && (!mean || !rstd)) return FP8SG_ERR_NULL;
  if ((dw || db) && cols > 0) {
    if (!ws) return FP8SG_ERR_NULL;
    if (ws_len < layer_norm_ws_len(rows, cols)) return FP8SG_ERR_SHAPE;
  }
  if (!aligned(w, esize(ptype)) || !aligned(dx, esize(type)) || !aligned(dw, esize(ptype)) ||
      !aligned(db, esize(ptype)) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(ws, 16))
    return FP8SG_ERR_ALIGN;
  p.w = w;
  p.dy = dy;
  p.mean = const_cast<float*>(mean);
  p.rstd = const_cast<float*>(rstd);
  p.rows = rows;
  p.cols = cols;
  p.dx = dx;
  p.dw = dw;
  p.db = db;
  p.ws = ws;
  return hip_status(launch_layer_norm_bwd(p, type, ptype, S(stream)));
}

}  // extern "C"
