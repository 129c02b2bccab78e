// Host-side launch interface of the microscaled formats, the gated activation
// and the layer norm (mx_quantize.hip, mx_gemm.hip, swiglu.hip,
// layer_norm.hip).  Element types are fp8sg_out values.
#pragma once

#include <hip/hip_runtime.h>
#include <type_traits>
#include <stdint.h>

#include "../../include/fp8sg.h"

namespace fp8sg {

// ---- MXFP4 layout (mxfp4_operand)
__host__ __device__ inline int64_t mx_ktiles(int64_t k) { return (k + 255) >> 8; }
__host__ __device__ inline int64_t mx_pitch(int64_t k) { return mx_ktiles(k) * 128; }
// scale bytes: groups of 32 rows x 256 values, 256 bytes each
__host__ __device__ inline int64_t mx_scale_off(int64_t r, int64_t b, int64_t nk) {
  return ((r >> 5) * nk + (b >> 3)) * 256 + (((b & 7) >> 1) * 16 + (r & 15)) * 4 + ((r & 31) >> 4) * 2 + (b & 1);
}

// One matrix to quantise: x rows x cols; q and / or t may have null pointers.
struct MxQuantJob {
  const void* x;
  int64_t rows, cols;
  mxfp4_operand q;  // along cols
  mxfp4_operand t;  // transposed, along rows
};
// n <= 2 matrices of one element type.
hipError_t launch_mx_quantize(const MxQuantJob* j, int n, int type, bool fit, hipStream_t stream);
hipError_t launch_mx_dequantize(const mxfp4_operand& m, int64_t rows, int64_t k, void* y, int type,
                                hipStream_t stream);

struct MxGemmProblem {
  mxfp4_operand A, B;
  void* C;
  int64_t M, N, K;
};
hipError_t launch_mx_gemm(const MxGemmProblem& p, int out, hipStream_t stream);
// The two products of a linear layer's backward pass.
hipError_t launch_mx_gemm_pair(const MxGemmProblem& p0, const MxGemmProblem& p1, int out, hipStream_t stream);
// y = x W^T with x (j, quantised along K into p.A's buffers where that pays) and
// the packed weight p.B.
hipError_t launch_mx_apply(const MxQuantJob& j, int type, bool fit, const MxGemmProblem& p, int out,
                           hipStream_t stream);

// ---- 8-bit checkpoints, gated activation
__host__ __device__ inline int64_t act8_pitch(int64_t cols) { return (cols + 31) / 32 * 32; }
hipError_t launch_act8_quantize(const void* x, int type, int64_t rows, int64_t cols, fp8sg_act8 c,
                                hipStream_t stream);
hipError_t launch_act8_dequantize(fp8sg_act8 c, int64_t rows, int64_t cols, void* y, int type,
                                  hipStream_t stream);
struct SwigluArgs {
  const void *g, *u, *da;     // da: backward only
  int64_t ldg, ldu;
  int64_t rows, cols;
  void *a, *dg, *du;          // a: forward; dg, du: backward
  int64_t lddg, lddu;
  fp8sg_act8 cg, cu;          // null pointers: no checkpoints
};
hipError_t launch_swiglu_fwd(const SwigluArgs& a, int type, hipStream_t stream);
hipError_t launch_swiglu_bwd(const SwigluArgs& a, int type, hipStream_t stream);

// ---- layer norm
struct LayerNormArgs {
  const void *x, *w, *b, *dy;
  fp8sg_act8 ckpt;            // forward: written; backward: read instead of x
  float *mean, *rstd;
  int64_t rows, cols;
  float eps;
  void *y, *dx, *dw, *db;
  float* ws;
};
int64_t layer_norm_ws_len(int64_t rows, int64_t cols);
hipError_t launch_layer_norm_fwd(const LayerNormArgs& a, int type, int ptype, hipStream_t stream);
hipError_t launch_layer_norm_bwd(const LayerNormArgs& a, int type, int ptype, hipStream_t stream);

// Compute units of the current device (cached per device).
int device_cus();

// f(integral constant of the type) for a run-time element type
template <class F>
inline hipError_t by_type(int type, F f) {
  switch (type) {
    case FP8SG_OUT_BF16: return f(std::integral_constant<int, FP8SG_OUT_BF16>{});
    case FP8SG_OUT_F16: return f(std::integral_constant<int, FP8SG_OUT_F16>{});
    default: return f(std::integral_constant<int, FP8SG_OUT_F32>{});
  }
}

}  // namespace fp8sg
