// Product of two MXFP4 matrices on the matrix cores:
//   C[M,N] = out(sum_k A[m,k] * B[n,k])
// v_mfma_scale_f32_16x16x128_f8f6f4 with both operands e2m1: lane l holds row
// l % 16 of a fragment and the 32 consecutive k of block l / 16, and one scale
// byte for that block; products and the sums inside a block are exact, sums
// over blocks are fp32.
#include "mx.hpp"

namespace fp8sg {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

__device__ __forceinline__ v8i frag4(uint4 v) {
  return v8i{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
}

// One wave per 16 x 16 block of C, fragments straight from memory.
template <int OUT>
__global__ __launch_bounds__(64) void k_mx_gemm_plain(MxGemmProblem p) {
  const int lane = threadIdx.x, r = lane & 15, g = lane >> 4;
  const int64_t nk = mx_ktiles(p.K);
  const int64_t nbn = (p.N + 15) / 16;
  const int64_t bm = (int64_t)blockIdx.x / nbn * 16, bn = (int64_t)blockIdx.x % nbn * 16;
  const int64_t m = bm + r < p.M ? bm + r : p.M - 1, n = bn + r < p.N ? bn + r : p.N - 1;
  v4f acc = {0.f, 0.f, 0.f, 0.f};
  for (int64_t kt = 0; kt < nk; ++kt) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t b = kt * 8 + 2 * g + j;
      const uint4 a = *reinterpret_cast<const uint4*>(p.A.q + m * nk * 128 + b * 16);
      const uint4 w = *reinterpret_cast<const uint4*>(p.B.q + n * nk * 128 + b * 16);
      const int sa = p.A.s[mx_scale_off(m, b, nk)], sb = p.B.s[mx_scale_off(n, b, nk)];
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag4(w), frag4(a), acc, 4, 4, 0, sb, 0, sa);
    }
  }
  if (bm + r >= p.M) return;
  Elem<OUT>* c = reinterpret_cast<Elem<OUT>*>(p.C) + (bm + r) * p.N;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (bn + 4 * g + e < p.N) c[bn + 4 * g + e] = from_f32<OUT>(acc[e]);
}

}  // namespace

hipError_t launch_mx_gemm(const MxGemmProblem& p, int out, hipStream_t stream) {
  if (p.M == 0 || p.N == 0) return hipSuccess;
  return by_type(out, [&](auto t) {
    constexpr int T = decltype(t)::value;
    const int64_t nb = ((p.M + 15) / 16) * ((p.N + 15) / 16);
    hipLaunchKernelGGL((k_mx_gemm_plain<T>), dim3((unsigned)nb), dim3(64), 0, stream, p);
    return hipGetLastError();
  });
}

hipError_t launch_mx_gemm_pair(const MxGemmProblem& p0, const MxGemmProblem& p1, int out, hipStream_t stream) {
  const hipError_t e = launch_mx_gemm(p0, out, stream);
  return e != hipSuccess ? e : launch_mx_gemm(p1, out, stream);
}

hipError_t launch_mx_apply(const MxQuantJob& j, int type, bool fit, const MxGemmProblem& p, int out,
                           hipStream_t stream) {
  const hipError_t e = launch_mx_quantize(&j, 1, type, fit, stream);
  return e != hipSuccess ? e : launch_mx_gemm(p, out, stream);
}

}  // namespace fp8sg
