// Scaled FP8 GEMM with an epilogue behind the product (bias, activation, dropout,
// residual: epilogue.hpp): the kernels of gemm_kernels.hpp instantiated for
// GemmEpiProblem, both operands e4m3 (the forward product) with per-tensor or
// row-wise scales.  The result's type is a run-time argument here: the product's
// arithmetic does not depend on it.
#include "gemm_kernels.hpp"

namespace fp8sg {
namespace {

template <bool RW, int BM>
hipError_t launch_big(const GemmEpiProblem& p, hipStream_t stream) {
  const unsigned nb = (unsigned)(((p.M + BM - 1) / BM) * ((p.N + 255) / 256));
  if (p.K % kBK == 0)
    hipLaunchKernelGGL((k_gemm_pingpong<0, 0, FP8SG_OUT_BF16, false, RW, BM, false, false, false, GemmEpiProblem>),
                       dim3(nb), dim3(512), 0, stream, p);
  else
    hipLaunchKernelGGL((k_gemm_pingpong<0, 0, FP8SG_OUT_BF16, true, RW, BM, false, false, false, GemmEpiProblem>),
                       dim3(nb), dim3(512), 0, stream, p);
  return hipGetLastError();
}

template <bool RW>
hipError_t launch_any(const GemmEpiProblem& p, hipStream_t stream) {
  if (p.M == 0 || p.N == 0) return hipSuccess;
  // the plain product's choice of tiles, without swapped roles
  if (big_tiles_wanted(p.M, p.N) && big_tiles_fit<false, false>(p))
    return big_tiling(p.M, p.N, device_cus(), false) == kTile224 ? launch_big<RW, 224>(p, stream)
                                                                 : launch_big<RW, 256>(p, stream);
  using Cfg = GemmCfg<128, 128, 2, 2>;
  static_assert(Cfg::kLdsBytes <= 64 * 1024, "no raised LDS limit");
  hipLaunchKernelGGL((k_gemm<128, 128, 2, 2, 0, 0, FP8SG_OUT_BF16, RW, false, false, GemmEpiProblem>),
                     dim3((unsigned)((p.N + 127) / 128), (unsigned)((p.M + 127) / 128)), dim3(Cfg::kThreads),
                     Cfg::kLdsBytes, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_epilogue(const GemmEpiProblem& p, bool rowwise, hipStream_t stream) {
  return rowwise ? launch_any<true>(p, stream) : launch_any<false>(p, stream);
}

}  // namespace fp8sg
