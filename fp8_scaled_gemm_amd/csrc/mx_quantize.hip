// MXFP4 quantisation along rows and / or columns, and the values of codes.
//
// For each block of 32 along the contraction: amax, its power-of-two scale,
// 32 codes of 4 bits.  Bound by memory: per element 2 bytes in (bf16) and
// 17/32 bytes out per direction.
#include "mx.hpp"

namespace fp8sg {
namespace {

// One thread per block of 32 along a row (blockIdx.y walks rows), padding
// blocks up to the last k-tile's end included.
template <int T>
__global__ __launch_bounds__(256) void k_mxq_rows(MxQuantJob j, bool fit) {
  const Elem<T>* x = reinterpret_cast<const Elem<T>*>(j.x);
  const int64_t nk = mx_ktiles(j.cols), nb = nk * 8, total = j.rows * nb;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / nb, b = i % nb;
    float v[32];
    uint32_t amax = 0;
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const int64_t c = b * 32 + e;
      v[e] = c < j.cols ? to_f32<T>(x[r * j.cols + c]) : 0.f;
      const uint32_t a = __float_as_uint(v[e]) & 0x7FFFFFFFu;
      amax = a > amax ? a : amax;
    }
    const uint32_t s = b * 32 < j.cols ? fp4_scale(amax, fit) : 127u;
    const float sc = s == 255u ? 1.f : scale_value(s);
    uint32_t w[4] = {0, 0, 0, 0};
    if (s != 255u) {
#pragma unroll
      for (int e = 0; e < 32; e += 2) w[e / 8] |= fp4_pair(v[e], v[e + 1], sc) << (8 * ((e / 2) % 4));
    }
    *reinterpret_cast<uint4*>(j.q.q + r * nk * 128 + b * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    j.q.s[mx_scale_off(r, b, nk)] = (uint8_t)s;
  }
}

// One thread per block of 32 along a column.
template <int T>
__global__ __launch_bounds__(256) void k_mxq_cols(MxQuantJob j, bool fit) {
  const Elem<T>* x = reinterpret_cast<const Elem<T>*>(j.x);
  const int64_t nk = mx_ktiles(j.rows), nb = nk * 8, total = j.cols * nb;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t b = i / j.cols, c = i % j.cols;
    float v[32];
    uint32_t amax = 0;
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const int64_t r = b * 32 + e;
      v[e] = r < j.rows ? to_f32<T>(x[r * j.cols + c]) : 0.f;
      const uint32_t a = __float_as_uint(v[e]) & 0x7FFFFFFFu;
      amax = a > amax ? a : amax;
    }
    const uint32_t s = b * 32 < j.rows ? fp4_scale(amax, fit) : 127u;
    const float sc = s == 255u ? 1.f : scale_value(s);
    uint32_t w[4] = {0, 0, 0, 0};
    if (s != 255u) {
#pragma unroll
      for (int e = 0; e < 32; e += 2) w[e / 8] |= fp4_pair(v[e], v[e + 1], sc) << (8 * ((e / 2) % 4));
    }
    *reinterpret_cast<uint4*>(j.t.q + c * nk * 128 + b * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    j.t.s[mx_scale_off(c, b, nk)] = (uint8_t)s;
  }
}

// One thread per byte of codes (two values).
template <int T>
__global__ __launch_bounds__(256) void k_mx_dequant(mxfp4_operand m, int64_t rows, int64_t k, Elem<T>* y) {
  const int64_t nk = mx_ktiles(k), pairs = (k + 1) / 2, total = rows * pairs;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / pairs, p = i % pairs;
    const float sc = scale_value(m.s[mx_scale_off(r, p / 16, nk)]);
    const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(m.q[r * nk * 128 + p], 1.f, 0);
    y[r * k + 2 * p] = from_f32<T>(v[0] * sc);
    if (2 * p + 1 < k) y[r * k + 2 * p + 1] = from_f32<T>(v[1] * sc);
  }
}

// Blocks of 256 threads for n items, each thread striding over the rest.
unsigned grid_for(int64_t n) {
  const int64_t b = (n + 255) / 256;
  return (unsigned)(b < (1 << 20) ? b : (1 << 20));
}

}  // namespace

hipError_t launch_mx_quantize(const MxQuantJob* jobs, int n, int type, bool fit, hipStream_t stream) {
  if (n > 1) {
    const hipError_t e = launch_mx_quantize(jobs + 1, n - 1, type, fit, stream);
    if (e != hipSuccess) return e;
  }
  const MxQuantJob& j = jobs[0];
  if (j.rows == 0 || j.cols == 0) return hipSuccess;
  return by_type(type, [&](auto t) {
    constexpr int T = decltype(t)::value;
    if (j.q.q)
      hipLaunchKernelGGL((k_mxq_rows<T>), dim3(grid_for(j.rows * mx_ktiles(j.cols) * 8)), dim3(256), 0, stream, j, fit);
    if (j.t.q)
      hipLaunchKernelGGL((k_mxq_cols<T>), dim3(grid_for(j.cols * mx_ktiles(j.rows) * 8)), dim3(256), 0, stream, j, fit);
    return hipGetLastError();
  });
}

hipError_t launch_mx_dequantize(const mxfp4_operand& m, int64_t rows, int64_t k, void* y, int type, hipStream_t stream) {
  if (rows == 0 || k == 0) return hipSuccess;
  return by_type(type, [&](auto t) {
    constexpr int T = decltype(t)::value;
    hipLaunchKernelGGL((k_mx_dequant<T>), dim3(grid_for(rows * ((k + 1) / 2))), dim3(256), 0, stream, m, rows, k,
                       reinterpret_cast<Elem<T>*>(y));
    return hipGetLastError();
  });
}

}  // namespace fp8sg
