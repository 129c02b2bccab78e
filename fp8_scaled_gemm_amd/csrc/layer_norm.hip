// Layer norm, forward and backward, with the reduction of the weight's and the
// bias's gradients over the rows.
#include "mx.hpp"

namespace fp8sg {
namespace {

template <int NT>
__device__ __forceinline__ float block_sum(float v) {
  __shared__ float red[NT / kWave];
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
  if ((threadIdx.x & (kWave - 1)) == 0) red[threadIdx.x / kWave] = v;
  __syncthreads();
  float r = 0.f;
#pragma unroll
  for (int w = 0; w < NT / kWave; ++w) r += red[w];
  __syncthreads();
  return r;
}

template <int P>
__device__ __forceinline__ float param(const void* w, int64_t c, float none) {
  return w ? to_f32<P>(reinterpret_cast<const Elem<P>*>(w)[c]) : none;
}

// One block per row (rows strided by the grid); the row is read once for the
// mean, once for the squared deviations, once for y.
template <int T, int P>
__global__ __launch_bounds__(256) void k_ln_fwd(LayerNormArgs p) {
  const float inv_n = 1.0f / (float)p.cols;
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const Elem<T>* x = reinterpret_cast<const Elem<T>*>(p.x) + r * p.cols;
    Elem<T>* y = reinterpret_cast<Elem<T>*>(p.y) + r * p.cols;
    float s = 0.f;
    for (int64_t c = threadIdx.x; c < p.cols; c += 256) s += to_f32<T>(x[c]);
    const float mean = block_sum<256>(s) * inv_n;
    s = 0.f;
    for (int64_t c = threadIdx.x; c < p.cols; c += 256) {
      const float d = to_f32<T>(x[c]) - mean;
      s += d * d;
    }
    const float rstd = 1.0f / sqrtf(block_sum<256>(s) * inv_n + p.eps);
    for (int64_t c = threadIdx.x; c < p.cols; c += 256)
      y[c] = from_f32<T>((to_f32<T>(x[c]) - mean) * rstd * param<P>(p.w, c, 1.f) + param<P>(p.b, c, 0.f));
    if (threadIdx.x == 0 && p.mean) {
      p.mean[r] = mean;
      p.rstd[r] = rstd;
    }
  }
}

// the forward's input, or its checkpoint's value
template <int T>
__device__ __forceinline__ float x_at(const LayerNormArgs& p, int64_t r, int64_t c) {
  if (p.x) return to_f32<T>(reinterpret_cast<const Elem<T>*>(p.x)[r * p.cols + c]);
  const int64_t at = r * act8_pitch(p.cols) + c;
  return __builtin_amdgcn_cvt_f32_fp8((int)p.ckpt.q[at], 0) * scale_value(p.ckpt.s[at >> 5]);
}

template <int T, int P>
__global__ __launch_bounds__(256) void k_ln_dx(LayerNormArgs p) {
  const float inv_n = 1.0f / (float)p.cols;
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const Elem<T>* dy = reinterpret_cast<const Elem<T>*>(p.dy) + r * p.cols;
    const float mean = p.mean[r], rstd = p.rstd[r];
    float s1 = 0.f, s2 = 0.f;
    for (int64_t c = threadIdx.x; c < p.cols; c += 256) {
      const float q = to_f32<T>(dy[c]) * param<P>(p.w, c, 1.f);
      s1 += q;
      s2 += q * ((x_at<T>(p, r, c) - mean) * rstd);
    }
    const float c1 = block_sum<256>(s1) * inv_n, c2 = block_sum<256>(s2) * inv_n;
    Elem<T>* dx = reinterpret_cast<Elem<T>*>(p.dx) + r * p.cols;
    for (int64_t c = threadIdx.x; c < p.cols; c += 256) {
      const float q = to_f32<T>(dy[c]) * param<P>(p.w, c, 1.f), xh = (x_at<T>(p, r, c) - mean) * rstd;
      dx[c] = from_f32<T>(rstd * (q - c1 - xh * c2));
    }
  }
}

constexpr int kParts = 64;  // row chunks of the weight gradient's reduction

// Column sums over one chunk of rows (blockIdx.y) into the workspace.
template <int T>
__global__ __launch_bounds__(256) void k_ln_dwb_part(LayerNormArgs p) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= p.cols) return;
  const int64_t per = (p.rows + kParts - 1) / kParts, r0 = blockIdx.y * per;
  const int64_t r1 = r0 + per < p.rows ? r0 + per : p.rows;
  float dw = 0.f, db = 0.f;
  for (int64_t r = r0; r < r1; ++r) {
    const float dy = to_f32<T>(reinterpret_cast<const Elem<T>*>(p.dy)[r * p.cols + c]);
    dw += dy * ((x_at<T>(p, r, c) - p.mean[r]) * p.rstd[r]);
    db += dy;
  }
  p.ws[(int64_t)blockIdx.y * 2 * p.cols + c] = dw;
  p.ws[(int64_t)blockIdx.y * 2 * p.cols + p.cols + c] = db;
}
template <int P>
__global__ __launch_bounds__(256) void k_ln_dwb_join(LayerNormArgs p) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= p.cols) return;
  float dw = 0.f, db = 0.f;
  for (int k = 0; k < kParts; ++k) {
    dw += p.ws[(int64_t)k * 2 * p.cols + c];
    db += p.ws[(int64_t)k * 2 * p.cols + p.cols + c];
  }
  if (p.dw) reinterpret_cast<Elem<P>*>(p.dw)[c] = from_f32<P>(dw);
  if (p.db) reinterpret_cast<Elem<P>*>(p.db)[c] = from_f32<P>(db);
}

unsigned row_blocks(int64_t rows) { return (unsigned)(rows < (1 << 20) ? rows : (1 << 20)); }

template <class F>
hipError_t by_types(int type, int ptype, F f) {
  return by_type(type, [&](auto t) {
    if (ptype == FP8SG_OUT_F32) f(t, std::integral_constant<int, FP8SG_OUT_F32>{});
    else f(t, t);
    return hipGetLastError();
  });
}

}  // namespace

int64_t layer_norm_ws_len(int64_t rows, int64_t cols) {
  (void)rows;
  return 2 * kParts * cols;
}

hipError_t launch_layer_norm_fwd(const LayerNormArgs& a, int type, int ptype, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  if (a.ckpt.q) {
    const hipError_t e = launch_act8_quantize(a.x, type, a.rows, a.cols, a.ckpt, stream);
    if (e != hipSuccess) return e;
  }
  return by_types(type, ptype, [&](auto t, auto p) {
    hipLaunchKernelGGL((k_ln_fwd<decltype(t)::value, decltype(p)::value>), dim3(row_blocks(a.rows)), dim3(256), 0,
                       stream, a);
  });
}

hipError_t launch_layer_norm_bwd(const LayerNormArgs& a, int type, int ptype, hipStream_t stream) {
  if (a.cols == 0) return hipSuccess;
  return by_types(type, ptype, [&](auto t, auto p) {
    constexpr int T = decltype(t)::value, P = decltype(p)::value;
    if (a.dx && a.rows > 0)
      hipLaunchKernelGGL((k_ln_dx<T, P>), dim3(row_blocks(a.rows)), dim3(256), 0, stream, a);
    if (a.dw || a.db) {
      const unsigned gx = (unsigned)((a.cols + 255) / 256);
      hipLaunchKernelGGL((k_ln_dwb_part<T>), dim3(gx, kParts), dim3(256), 0, stream, a);
      hipLaunchKernelGGL((k_ln_dwb_join<P>), dim3(gx), dim3(256), 0, stream, a);
    }
  });
}

}  // namespace fp8sg
