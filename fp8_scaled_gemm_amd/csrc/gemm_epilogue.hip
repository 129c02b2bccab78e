// Scaled FP8 GEMM with an epilogue behind the product (bias, activation, dropout,
// residual: epilogue.hpp): the kernels of gemm_kernels.hpp instantiated for
// GemmEpiProblem, both operands e4m3 (the forward product) with per-tensor or
// row-wise scales.  The result's type is a run-time argument; OUT only says whether
// it is fp32 or has 16 bits, which the activations' accuracy goes by.
#include "gemm_kernels.hpp"

namespace fp8sg {
namespace {

template <int OUT, bool RW, int BM>
hipError_t launch_big(const GemmEpiProblem& p, hipStream_t stream) {
  const unsigned nb = (unsigned)(((p.M + BM - 1) / BM) * ((p.N + 255) / 256));
  if (p.K % kBK == 0)
    hipLaunchKernelGGL((k_gemm_pingpong<0, 0, OUT, false, RW, BM, false, false, false, GemmEpiProblem>),
                       dim3(nb), dim3(512), 0, stream, p);
  else
    hipLaunchKernelGGL((k_gemm_pingpong<0, 0, OUT, true, RW, BM, false, false, false, GemmEpiProblem>),
                       dim3(nb), dim3(512), 0, stream, p);
  return hipGetLastError();
}

template <int OUT, int BM, int BN, int WM, int WN, bool RW>
hipError_t launch_small(const GemmEpiProblem& p, hipStream_t stream) {
  using Cfg = GemmCfg<BM, BN, WM, WN>;
  static_assert(Cfg::kLdsBytes <= 64 * 1024, "no raised LDS limit");
  hipLaunchKernelGGL((k_gemm<BM, BN, WM, WN, 0, 0, OUT, RW, false, false, GemmEpiProblem>),
                     dim3((unsigned)((p.N + BN - 1) / BN), (unsigned)((p.M + BM - 1) / BM)), dim3(Cfg::kThreads),
                     Cfg::kLdsBytes, stream, p);
  return hipGetLastError();
}

// Tiles of 64 x 64 in place of 128 x 128 while those would not go round all compute
// units: a wave's epilogue is a chain of instructions for each of its rows, which four
// times the waves share, and so do they the k-tiles' latency.  us, tiles of 128 / 64,
// with bias, then with gelu and h kept: 64 x 4096 x 4096 (32 tiles of 128) 32.5 / 17.4,
// 35.2 / 18.2; 1024^3 (64) 12.6 / 7.2, 15.8 / 8.0; 2048 x 3584 x 1024 (448) 17.8 / 19.6,
// 22.3 / 22.4.  At 256 of them, one for each unit, the small ones lose where little stands
// behind a long contraction: 2048 x 2048 with K = 512 10.5 / 9.5, 14.3 / 11.3, 2048
// 21.4 / 22.2, 25.3 / 23.4, 4096 35.8 / 39.0, 39.6 / 39.6.
bool small_tiles(const GemmEpiProblem& p) {
  return ((p.M + 127) / 128) * ((p.N + 127) / 128) <= device_cus();
}

template <int OUT, bool RW>
hipError_t launch_any(const GemmEpiProblem& p, hipStream_t stream) {
  if (p.M == 0 || p.N == 0) return hipSuccess;
  // the plain product's choice of tiles, without swapped roles
  if (big_tiles_wanted(p.M, p.N) && big_tiles_fit<false, false>(p))
    return big_tiling(p.M, p.N, device_cus(), false) == kTile224 ? launch_big<OUT, RW, 224>(p, stream)
                                                                 : launch_big<OUT, RW, 256>(p, stream);
  return small_tiles(p) ? launch_small<OUT, 64, 64, 4, 1, RW>(p, stream) : launch_small<OUT, 128, 128, 2, 2, RW>(p, stream);
}

}  // namespace

hipError_t launch_gemm_epilogue(const GemmEpiProblem& p, bool rowwise, hipStream_t stream) {
  if (p.epi.type == FP8SG_OUT_F32)
    return rowwise ? launch_any<FP8SG_OUT_F32, true>(p, stream) : launch_any<FP8SG_OUT_F32, false>(p, stream);
  return rowwise ? launch_any<FP8SG_OUT_BF16, true>(p, stream) : launch_any<FP8SG_OUT_BF16, false>(p, stream);
}

}  // namespace fp8sg
