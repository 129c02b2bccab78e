// Host-side launch interface of the products with an epilogue, their backward
// step and dropout (gemm_epilogue.hip, mx_gemm.hip, epilogue.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/fp8sg.h"
#include "launch.hpp"
#include "launch_mx.hpp"

namespace fp8sg {

// rng == nullptr: nothing is dropped.
struct DropArgs {
  const uint64_t* rng;
  uint32_t t;
  float scale;
};
// The rule for a probability p in [0, 1]: t = round(65536 p).  p below 2^-17 is none.
inline DropArgs drop_args(const int64_t* rng, float p) {
  const uint32_t t = (uint32_t)(65536.0 * (double)p + 0.5);
  if (t == 0) return DropArgs{nullptr, 0, 1.f};
  return DropArgs{reinterpret_cast<const uint64_t*>(rng), t, t < 65536 ? (float)(65536.0 / (65536.0 - t)) : 0.f};
}

// One product's epilogue; the types are fp8sg_out values.
struct EpilogueArgs {
  const void* bias;
  const void* residual;
  void* pre;
  void* C;
  int64_t M, N, ldr, ldc;
  DropArgs drop;
  int32_t act, type, bias_type;
  int32_t stream;  // results leave with non-temporal stores
};

// Whether y or pre lies over n bytes at in.
inline bool stored_over(const EpilogueArgs& e, const void* in, int64_t n) {
  const int64_t es = e.type == FP8SG_OUT_F32 ? 4 : 2;
  if (e.M == 0 || e.N == 0) return false;
  return shares(e.C, ((e.M - 1) * e.ldc + e.N) * es, in, n) || (e.pre && shares(e.pre, e.M * e.N * es, in, n));
}

struct GemmEpiProblem : GemmProblem {
  EpilogueArgs epi;
};
struct MxGemmEpiProblem : MxGemmProblem {
  EpilogueArgs epi;
};
// Both operands e4m3; per-tensor inverse scales, or vectors (rowwise).
hipError_t launch_gemm_epilogue(const GemmEpiProblem& p, bool rowwise, hipStream_t stream);
// A small layer's forward (small_layer_fits) in one launch.
struct SmallFwdEpiArgs {
  const uint16_t* x;
  const uint16_t* w;
  GemmEpiProblem p;
  fp8sg_scale_rec* x_sc;
  fp8sg_scale_rec* w_sc;
  uint8_t* x_q;
  uint8_t* w_q;
};
hipError_t launch_small_fwd_epilogue(const SmallFwdEpiArgs& a, bool f16, hipStream_t stream);
hipError_t launch_mx_gemm_epilogue(const MxGemmEpiProblem& p, hipStream_t stream);
hipError_t launch_mx_apply_epilogue(const MxQuantJob& j, int type, bool fit, const MxGemmEpiProblem& p,
                                    hipStream_t stream);

// The backward step: gh = drop(gy) act'(pre) of `type`, the bias's gradient gb
// (sums over rows, of bias_type) and per-block maxima of |gh| into rec, each
// optional.
struct EpilogueBwdArgs {
  const void *gy, *pre;
  void *gh, *gb;
  float* part;  // partial sums (epilogue_ws_len)
  fp8sg_scale_rec* rec;
  int64_t M, N;
  DropArgs drop;
  int32_t act, type, bias_type;
  // filled by the launcher
  int32_t lanes, parts;
  int64_t strips;
};
int64_t epilogue_ws_len(int64_t M, int64_t N);
// ... without which a call is refused: none where the step alone does with one part
int64_t epilogue_ws_need(int64_t M, int64_t N);
hipError_t launch_epilogue_bwd(EpilogueBwdArgs a, hipStream_t stream);
// gb from the a.parts rows of partial sums in a.part
hipError_t launch_bias_join(const EpilogueBwdArgs& a, hipStream_t stream);
// The backward step and gh's MXFP4 codes (of a job whose x is gy) in one pass, where
// M rows leave at most kMxEpiParts rows of partial sums, one for 64 rows (their join
// takes 7 of 82 us at 65536 x 512).  mx_epilogue_parts: how many, 0 where it does not apply.
constexpr int64_t kMxEpiParts = 1024;
int64_t mx_epilogue_parts(int64_t M, int64_t N);
hipError_t launch_mx_quantize_epilogue(const MxQuantJob& j, int type, bool fit, EpilogueBwdArgs e, hipStream_t stream);

// y = residual + drop(x) (residual may be nullptr), rows ldx, ldr and ldy apart
struct DropoutArgs {
  const void *x, *residual;
  void* y;
  int64_t rows, cols, ldx, ldr, ldy;
  DropArgs drop;
  int32_t type;
};
hipError_t launch_dropout(const DropoutArgs& a, hipStream_t stream);

}  // namespace fp8sg
