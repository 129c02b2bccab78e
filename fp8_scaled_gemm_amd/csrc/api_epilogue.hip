// C-ABI entry points of the products with an epilogue, their backward pass and
// dropout: argument validation, then kernel launches on the caller's stream.  No
// device allocation and no host synchronisation.
#include <stdint.h>

#include "../../include/fp8sg.h"
#include "launch_epilogue.hpp"

using namespace fp8sg;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool type_ok(int t) { return t == FP8SG_OUT_BF16 || t == FP8SG_OUT_F16 || t == FP8SG_OUT_F32; }
bool type16(int t) { return t == FP8SG_OUT_BF16 || t == FP8SG_OUT_F16; }
bool rule_ok(int r) { return r == FP8SG_MX_FLOOR || r == FP8SG_MX_FIT; }
uintptr_t esize(int t) { return t == FP8SG_OUT_F32 ? 4 : 2; }
bool p_ok(float p) { return p >= 0.f && p <= 1.f; }
fp8sg_status hip_status(hipError_t e) { return e == hipSuccess ? FP8SG_OK : FP8SG_ERR_HIP; }
hipStream_t S(fp8sg_stream s) { return reinterpret_cast<hipStream_t>(s); }

bool mat_ok(int64_t r, int64_t c) {
  return r >= 0 && c >= 0 && r <= FP8SG_MAX_DIM && c <= FP8SG_MAX_DIM && (r == 0 || c <= FP8SG_MAX_ELEMS / r);
}
bool gemm_ok(int64_t M, int64_t N, int64_t K) { return mat_ok(M, K) && mat_ok(N, K) && mat_ok(M, N); }
bool dims16(int64_t M, int64_t N, int64_t K) { return M % 16 == 0 && N % 16 == 0 && K % 16 == 0; }

#define FP8SG_TRY(expr)                              \
  do {                                               \
    const fp8sg_status st_ = (expr);                 \
    if (st_ != FP8SG_OK) return st_;                 \
  } while (0)

fp8sg_status check_tensor(const void* p, int64_t n, uintptr_t align) {
  if (n > 0 && !p) return FP8SG_ERR_NULL;
  return aligned(p, align) ? FP8SG_OK : FP8SG_ERR_ALIGN;
}
// A matrix whose rows are ld elements apart.
fp8sg_status check_rows(const void* p, int64_t ld, int64_t rows, int64_t cols, int type) {
  if (rows * cols > 0 && (ld < cols || !mat_ok(rows, ld))) return FP8SG_ERR_SHAPE;
  return check_tensor(p, rows * cols, esize(type));
}
template <class Pair>
fp8sg_status check_codes(const Pair& m, int64_t n) {
  if (n > 0 && (!m.q || !m.s)) return FP8SG_ERR_NULL;
  return aligned(m.q, 16) && aligned(m.s, 16) ? FP8SG_OK : FP8SG_ERR_ALIGN;
}
fp8sg_status check_saved(const fp8_linear_saved* s) {
  if (!s || !s->x_q || !s->w_q || !s->x_sc || !s->w_sc) return FP8SG_ERR_NULL;
  if (!aligned(s->x_q, 16) || !aligned(s->x_qT, 16) || !aligned(s->w_q, 16) || !aligned(s->w_qT, 16) ||
      !aligned(s->x_sc, 8) || !aligned(s->w_sc, 8))
    return FP8SG_ERR_ALIGN;
  return FP8SG_OK;
}

fp8sg_status check_drop(float p, const int64_t* rng, DropArgs& d) {
  if (!p_ok(p)) return FP8SG_ERR_SHAPE;  // (NaN too)
  d = drop_args(rng, p);
  if (d.t && !rng) return FP8SG_ERR_NULL;
  return !d.t || aligned(rng, 8) ? FP8SG_OK : FP8SG_ERR_ALIGN;
}

// A forward epilogue of an M x N result of `type` into C.
fp8sg_status check_epilogue(const fp8sg_epilogue* e, int64_t M, int64_t N, void* C, int type, EpilogueArgs& a) {
  if (!e) return FP8SG_ERR_NULL;
  if (!type_ok(type) || e->act < FP8SG_ACT_NONE || e->act > FP8SG_ACT_GELU_TANH) return FP8SG_ERR_FORMAT;
  if (e->bias && !type_ok(e->bias_type)) return FP8SG_ERR_FORMAT;
  FP8SG_TRY(check_rows(C, e->ld_out, M, N, type));
  if (e->residual) FP8SG_TRY(check_rows(e->residual, e->ld_residual, M, N, type));
  // a residual that is the output has its rows
  if (M > 1 && N > 0 && e->residual && e->residual == C && e->ld_residual != e->ld_out) return FP8SG_ERR_SHAPE;
  if (e->bias && !aligned(e->bias, esize(e->bias_type))) return FP8SG_ERR_ALIGN;
  if (!aligned(e->pre, esize(type))) return FP8SG_ERR_ALIGN;
  FP8SG_TRY(check_drop(e->p, e->rng, a.drop));
  a.bias = e->bias;
  a.residual = e->residual;
  a.pre = e->pre;
  a.C = C;
  a.M = M;
  a.N = N;
  a.ldr = e->ld_residual;
  a.ldc = e->ld_out;
  a.act = e->act;
  a.type = type;
  a.bias_type = e->bias_type;
  a.stream = M * N * (int64_t)esize(type) >= (64ll << 20);  // (kStreamOutBytes)
  return FP8SG_OK;
}

// The backward step; gh NULL stands for gy where that is what it would be.
fp8sg_status check_backward(const void* gy, int type, const fp8sg_epilogue* e, int64_t M, int64_t N, void* gh,
                            void* gb, float* ws, int64_t ws_len, uintptr_t align, EpilogueBwdArgs& a) {
  if (!e) return FP8SG_ERR_NULL;
  if (!type_ok(type) || e->act < FP8SG_ACT_NONE || e->act > FP8SG_ACT_GELU_TANH) return FP8SG_ERR_FORMAT;
  if (gb && e->bias_type != type && e->bias_type != FP8SG_OUT_F32) return FP8SG_ERR_FORMAT;
  if (!mat_ok(M, N)) return FP8SG_ERR_SHAPE;
  FP8SG_TRY(check_tensor(gy, M * N, align));
  if (!aligned(gh, align) || (gb && !aligned(gb, esize(e->bias_type)))) return FP8SG_ERR_ALIGN;
  if (e->act != FP8SG_ACT_NONE) FP8SG_TRY(check_tensor(e->pre, M * N, esize(type)));
  FP8SG_TRY(check_drop(e->p, e->rng, a.drop));
  if (gb) {
    const int64_t need = epilogue_ws_need(M, N);
    if (need > 0 && !ws) return FP8SG_ERR_NULL;
    if (need > ws_len) return FP8SG_ERR_SHAPE;
    if (!aligned(ws, 4)) return FP8SG_ERR_ALIGN;
  }
  a.gy = gy;
  a.pre = e->pre;
  a.gh = gh;
  a.gb = gb;
  a.part = ws;
  a.M = M;
  a.N = N;
  a.act = e->act;
  a.type = type;
  a.bias_type = e->bias_type;
  return FP8SG_OK;
}
// Whether gh is another tensor than gy.
bool changes(const EpilogueBwdArgs& a) { return a.act != FP8SG_ACT_NONE || a.drop.t != 0; }

fp8sg_status gemm_epilogue(const uint8_t* A, const uint8_t* B, const double* ia, const double* ib,
                           const fp8sg_epilogue* epi, void* C, fp8sg_out out, int64_t M, int64_t N, int64_t Kc,
                           bool rowwise, fp8sg_stream stream) {
  if (!dims16(M, N, Kc) || !gemm_ok(M, N, Kc)) return FP8SG_ERR_SHAPE;
  FP8SG_TRY(check_tensor(A, M * Kc, 16));
  FP8SG_TRY(check_tensor(B, N * Kc, 16));
  if (!ia || !ib) return FP8SG_ERR_NULL;
  if (!aligned(ia, 8) || !aligned(ib, 8)) return FP8SG_ERR_ALIGN;
  GemmEpiProblem p{GemmProblem{A, B, C, ia, ib, M, N, Kc}, {}};
  FP8SG_TRY(check_epilogue(epi, M, N, C, out, p.epi));
  return hip_status(launch_gemm_epilogue(p, rowwise, S(stream)));
}

}  // namespace

extern "C" {

fp8sg_status fp8_gemm_epilogue(const uint8_t* A, const uint8_t* B, const double* inv_a, const double* inv_b,
                               const fp8sg_epilogue* epi, void* C, fp8sg_out out, int64_t M, int64_t N, int64_t Kc,
                               fp8sg_stream stream) {
  return gemm_epilogue(A, B, inv_a, inv_b, epi, C, out, M, N, Kc, false, stream);
}

fp8sg_status fp8_gemm_rowwise_epilogue(const uint8_t* A, const uint8_t* B, const double* inv_a, const double* inv_b,
                                       const fp8sg_epilogue* epi, void* C, fp8sg_out out, int64_t M, int64_t N,
                                       int64_t Kc, fp8sg_stream stream) {
  return gemm_epilogue(A, B, inv_a, inv_b, epi, C, out, M, N, Kc, true, stream);
}

fp8sg_status fp8_scaled_linear_fwd_epilogue(const void* x, const void* w, fp8sg_out type, int64_t M, int64_t N,
                                            int64_t K, const fp8_linear_saved* saved, const fp8sg_epilogue* epi,
                                            void* y, fp8sg_out out, fp8sg_stream stream) {
  if (!x || !w || !y) return FP8SG_ERR_NULL;
  FP8SG_TRY(check_saved(saved));
  if (!type16(type)) return FP8SG_ERR_FORMAT;
  if (M <= 0 || N <= 0 || K <= 0 || !dims16(M, N, K) || !gemm_ok(M, N, K)) return FP8SG_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(w, 16)) return FP8SG_ERR_ALIGN;
  GemmEpiProblem p{GemmProblem{saved->x_q, saved->w_q, y, &saved->x_sc->inv, &saved->w_sc->inv, M, N, K}, {}};
  FP8SG_TRY(check_epilogue(epi, M, N, y, out, p.epi));
  if (epi->bias && epi->bias_type != type && epi->bias_type != FP8SG_OUT_F32) return FP8SG_ERR_FORMAT;
  const uint16_t *x16 = static_cast<const uint16_t*>(x), *w16 = static_cast<const uint16_t*>(w);
  const bool f16 = type == FP8SG_OUT_F16;
  const bool over = stored_over(p.epi, x, M * K * 2) || stored_over(p.epi, w, N * K * 2);
  if (!saved->x_qT && !saved->w_qT && small_layer_fits(M, N, K) && !over) {
    const SmallFwdEpiArgs a{x16, w16, p, saved->x_sc, saved->w_sc, saved->x_q, saved->w_q};
    return hip_status(launch_small_fwd_epilogue(a, f16, S(stream)));
  }
  const hipError_t e = launch_linear_casts(x16, w16, M, N, K, *saved, nullptr, nullptr, 0, f16, S(stream));
  return e != hipSuccess ? FP8SG_ERR_HIP : hip_status(launch_gemm_epilogue(p, false, S(stream)));
}

int64_t epilogue_workspace_len(int64_t M, int64_t N) { return mat_ok(M, N) ? epilogue_ws_len(M, N) : -1; }

fp8sg_status epilogue_bwd(const void* gy, fp8sg_out type, const fp8sg_epilogue* epi, int64_t M, int64_t N, void* gh,
                          void* gb, float* ws, int64_t ws_len, fp8sg_stream stream) {
  EpilogueBwdArgs a{};
  FP8SG_TRY(check_backward(gy, type, epi, M, N, gh, gb, ws, ws_len, type_ok(type) ? esize(type) : 2, a));
  if (!gh && !gb && M * N > 0) return FP8SG_ERR_NULL;
  return hip_status(launch_epilogue_bwd(a, S(stream)));
}

fp8sg_status fp8_scaled_linear_bwd_epilogue(const void* gy, fp8sg_out type, const fp8_linear_saved* saved, int64_t M,
                                            int64_t N, int64_t K, const fp8_linear_bwd_ws* ws,
                                            const fp8sg_epilogue* epi, void* gh, void* gb, float* ws_part,
                                            int64_t part_len, void* gx, void* gw, fp8sg_out out,
                                            fp8sg_stream stream) {
  if (!gy || !ws || !gx || !gw) return FP8SG_ERR_NULL;
  FP8SG_TRY(check_saved(saved));
  if (!ws->gy_q || !ws->gy_sc) return FP8SG_ERR_NULL;
  if (!type16(type) || !type_ok(out)) return FP8SG_ERR_FORMAT;
  if (M <= 0 || N <= 0 || K <= 0 || !dims16(M, N, K) || !gemm_ok(M, N, K)) return FP8SG_ERR_SHAPE;
  if (!aligned(gx, 16) || !aligned(gw, 16) || !aligned(ws->gy_q, 16) || !aligned(ws->gy_qT, 16) ||
      !aligned(ws->gy_sc, 8))
    return FP8SG_ERR_ALIGN;
  EpilogueBwdArgs a{};
  FP8SG_TRY(check_backward(gy, type, epi, M, N, gh, gb, ws_part, part_len, 16, a));
  if (changes(a) && !gh) return FP8SG_ERR_NULL;
  const bool step = changes(a) || gb;  // otherwise there is nothing to do before the cast
  // (a small layer's launch takes the maximum itself)
  const bool small = !saved->x_qT && !saved->w_qT && !ws->gy_qT && small_layer_fits(M, N, K);
  if (step) {
    a.rec = small ? nullptr : ws->gy_sc;
    if (!changes(a)) a.gh = nullptr;
    if (launch_epilogue_bwd(a, S(stream)) != hipSuccess) return FP8SG_ERR_HIP;
  }
  return hip_status(launch_linear_bwd(static_cast<const uint16_t*>(changes(a) ? gh : gy), *saved, M, N, K, *ws, nullptr,
                                      0, gx, gw, out, nullptr, nullptr, type == FP8SG_OUT_F16, step && !small,
                                      S(stream)));
}

fp8sg_status mxfp4_gemm_epilogue(const mxfp4_operand* A, const mxfp4_operand* B, const fp8sg_epilogue* epi, void* C,
                                 fp8sg_out out, int64_t M, int64_t N, int64_t Kc, fp8sg_stream stream) {
  if (!A || !B) return FP8SG_ERR_NULL;
  if (!gemm_ok(M, N, Kc)) return FP8SG_ERR_SHAPE;
  FP8SG_TRY(check_codes(*A, M * Kc));
  FP8SG_TRY(check_codes(*B, N * Kc));
  MxGemmEpiProblem p{MxGemmProblem{*A, *B, C, M, N, Kc}, {}};
  FP8SG_TRY(check_epilogue(epi, M, N, C, out, p.epi));
  return hip_status(launch_mx_gemm_epilogue(p, S(stream)));
}

fp8sg_status mxfp4_linear_fwd_epilogue(const void* x, const void* w, fp8sg_out type, int64_t M, int64_t N, int64_t K,
                                       fp8sg_mx_rule rule, const mxfp4_linear_ws* ws, const mxfp4_linear_saved* saved,
                                       const fp8sg_epilogue* epi, void* y, fp8sg_out out, fp8sg_stream stream) {
  if (!ws) return FP8SG_ERR_NULL;
  if (!type_ok(type) || !rule_ok(rule)) return FP8SG_ERR_FORMAT;
  if (!gemm_ok(M, N, K)) return FP8SG_ERR_SHAPE;
  FP8SG_TRY(check_tensor(x, M * K, esize(type)));
  FP8SG_TRY(check_tensor(w, N * K, esize(type)));
  FP8SG_TRY(check_codes(ws->x_q, M * K));
  FP8SG_TRY(check_codes(ws->w_q, N * K));
  MxQuantJob j[2] = {{x, M, K, ws->x_q, {}}, {w, N, K, ws->w_q, {}}};
  if (saved) {
    FP8SG_TRY(check_codes(saved->x_qT, M * K));
    FP8SG_TRY(check_codes(saved->w_qT, N * K));
    j[0].t = saved->x_qT;
    j[1].t = saved->w_qT;
  }
  MxGemmEpiProblem p{MxGemmProblem{ws->x_q, ws->w_q, y, M, N, K}, {}};
  FP8SG_TRY(check_epilogue(epi, M, N, y, out, p.epi));
  if (epi->bias && epi->bias_type != type && epi->bias_type != FP8SG_OUT_F32) return FP8SG_ERR_FORMAT;
  if (launch_mx_quantize(j, 2, type, rule == FP8SG_MX_FIT, S(stream)) != hipSuccess) return FP8SG_ERR_HIP;
  return hip_status(launch_mx_gemm_epilogue(p, S(stream)));
}

fp8sg_status mxfp4_linear_apply_epilogue(const void* x, fp8sg_out type, const mxfp4_operand* w, int64_t M, int64_t N,
                                         int64_t K, fp8sg_mx_rule rule, const mxfp4_operand* x_ws,
                                         const fp8sg_epilogue* epi, void* y, fp8sg_out out, fp8sg_stream stream) {
  if (!w || !x_ws) return FP8SG_ERR_NULL;
  if (!type_ok(type) || !rule_ok(rule)) return FP8SG_ERR_FORMAT;
  if (!gemm_ok(M, N, K)) return FP8SG_ERR_SHAPE;
  FP8SG_TRY(check_tensor(x, M * K, esize(type)));
  FP8SG_TRY(check_codes(*w, N * K));
  FP8SG_TRY(check_codes(*x_ws, M * K));
  MxGemmEpiProblem p{MxGemmProblem{*x_ws, *w, y, M, N, K}, {}};
  FP8SG_TRY(check_epilogue(epi, M, N, y, out, p.epi));
  if (epi->bias && epi->bias_type != type && epi->bias_type != FP8SG_OUT_F32) return FP8SG_ERR_FORMAT;
  const MxQuantJob j{x, M, K, *x_ws, {}};
  return hip_status(launch_mx_apply_epilogue(j, type, rule == FP8SG_MX_FIT, p, S(stream)));
}

fp8sg_status mxfp4_linear_bwd_epilogue(const void* gy, fp8sg_out type, int64_t M, int64_t N, int64_t K,
                                       fp8sg_mx_rule rule, const mxfp4_linear_ws* ws, const mxfp4_linear_saved* saved,
                                       const fp8sg_epilogue* epi, void* gh, void* gb, float* ws_part,
                                       int64_t part_len, void* gx, void* gw, fp8sg_out out, fp8sg_stream stream) {
  EpilogueBwdArgs a{};
  if (!gemm_ok(M, N, K)) return FP8SG_ERR_SHAPE;
  FP8SG_TRY(check_backward(gy, type, epi, M, N, gh, gb, ws_part, part_len, type_ok(type) ? esize(type) : 2, a));
  const bool products = gx || gw;
  if (changes(a) && products && !gh && M * N > 0) return FP8SG_ERR_NULL;
  if (!changes(a) || !products) a.gh = nullptr;
  // the products' own checks come before anything is enqueued
  if (!ws || !saved) return FP8SG_ERR_NULL;
  if (!type_ok(out) || !rule_ok(rule)) return FP8SG_ERR_FORMAT;
  if (gx) {
    FP8SG_TRY(check_codes(ws->gy_q, M * N));
    FP8SG_TRY(check_codes(saved->w_qT, N * K));
    FP8SG_TRY(check_tensor(gx, M * K, esize(out)));
  }
  if (gw) {
    FP8SG_TRY(check_codes(ws->gy_qT, M * N));
    FP8SG_TRY(check_codes(saved->x_qT, M * K));
    FP8SG_TRY(check_tensor(gw, N * K, esize(out)));
  }
  if (!products && !gb && M * K > 0 && N * K > 0) return FP8SG_ERR_NULL;
  const bool step = gb || (changes(a) && products);
  const int64_t parts = mx_epilogue_parts(M, N);
  // (few rows' sums need no workspace in the step alone: without one it is that)
  if (step && products && parts > 0 && (!gb || parts == 1 || (ws_part && part_len >= parts * N))) {
    const MxQuantJob j{gy, M, N, gx ? ws->gy_q : mxfp4_operand{}, gw ? ws->gy_qT : mxfp4_operand{}};
    if (launch_mx_quantize_epilogue(j, type, rule == FP8SG_MX_FIT, a, S(stream)) != hipSuccess) return FP8SG_ERR_HIP;
    const MxGemmProblem dgrad{ws->gy_q, saved->w_qT, gx, M, K, N}, wgrad{ws->gy_qT, saved->x_qT, gw, N, K, M};
    return hip_status(gx && gw ? launch_mx_gemm_pair(dgrad, wgrad, out, S(stream))
                               : launch_mx_gemm(gx ? dgrad : wgrad, out, S(stream)));
  }
  if (step && launch_epilogue_bwd(a, S(stream)) != hipSuccess) return FP8SG_ERR_HIP;
  if (!products) return FP8SG_OK;
  return mxfp4_linear_bwd(changes(a) ? gh : gy, type, M, N, K, rule, ws, saved, gx, gw, out, stream);
}

fp8sg_status dropout_fwd(const void* x, int64_t ldx, const void* residual, int64_t ldr, fp8sg_out type, int64_t rows,
                         int64_t cols, float p, const int64_t* rng, void* y, int64_t ldy, fp8sg_stream stream) {
  if (!type_ok(type)) return FP8SG_ERR_FORMAT;
  if (!mat_ok(rows, cols)) return FP8SG_ERR_SHAPE;
  DropoutArgs a{};
  FP8SG_TRY(check_rows(x, ldx, rows, cols, type));
  if (residual) FP8SG_TRY(check_rows(residual, ldr, rows, cols, type));
  FP8SG_TRY(check_rows(y, ldy, rows, cols, type));
  if (rows > 1 && cols > 0 && ((x == y && ldx != ldy) || (residual == y && residual && ldr != ldy)))
    return FP8SG_ERR_SHAPE;
  FP8SG_TRY(check_drop(p, rng, a.drop));
  a.x = x;
  a.residual = residual;
  a.y = y;
  a.rows = rows;
  a.cols = cols;
  a.ldx = ldx;
  a.ldr = ldr;
  a.ldy = ldy;
  a.type = type;
  return hip_status(launch_dropout(a, S(stream)));
}

fp8sg_status dropout_bwd(const void* gy, int64_t ldgy, fp8sg_out type, int64_t rows, int64_t cols, float p,
                         const int64_t* rng, void* gx, int64_t ldgx, fp8sg_stream stream) {
  return dropout_fwd(gy, ldgy, nullptr, 0, type, rows, cols, p, rng, gx, ldgx, stream);
}

}  // extern "C"
