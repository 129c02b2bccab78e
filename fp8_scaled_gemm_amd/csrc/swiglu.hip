// Gated activation a = silu(g) u and its gradients, with g and u kept between
// the passes as they are or as 8-bit checkpoints, and the checkpoint cast on
// its own.
//
// Elementwise and bound by memory.  A thread takes 8 consecutive elements of a
// row, and four neighbouring lanes one block of 32, whose largest magnitude
// two DPP exchanges give all four; rows are cut into whole blocks, so four
// lanes never straddle two rows.  8192 x 14336 from a graph, with non-temporal
// accesses, which tensors past the caches take (a copy of 1 GiB reaches 5.2 TB/s, a
// streamed read and write 6.3):
//   bf16, checkpoints  forward 163 us, backward 149 us for 947 MB each (5.8, 6.4 TB/s)
//   bf16, without      116 us for 705 MB, 188 us for 1174 MB (6.1, 6.2)
//   fp16, checkpoints  157, 141 us
//   fp32, 4096 rows    checkpoints 154, 138 us for 826 MB; without 125 us for 705 MB, 214 us for 1174 MB
// The checkpoint alone: bf16 71 us for 356 MB (5.0), its values 55 us (6.5); fp32 99 us
// for 591 MB (6.0), its values 186 us (3.2).
// fp32's exponential costs its backward from checkpoints 5% (131 us with the
// hardware's), the rest nothing.
#include "mx.hpp"

namespace fp8sg {
namespace {

// Unit (8 elements) of this thread in group `blk` of 256: units are numbered row
// after row, `upr` a row.  One 64-bit division a block (uniform), one 32-bit
// division a thread.
struct Unit {
  int64_t row;
  int64_t u;
};
__device__ __forceinline__ Unit unit_of(int64_t blk, int64_t upr) {
  const int64_t i0 = blk * 256, r0 = i0 / upr;
  const int64_t t = i0 - r0 * upr + threadIdx.x;  // < upr + 256, and upr <= 2^26
  const uint32_t d = (uint32_t)t / (uint32_t)upr;
  return Unit{r0 + d, t - (int64_t)d * upr};
}

// Groups of 256 units of a rows x cols matrix, and the grid that walks them (a
// launch holds fewer than 2^32 threads).
__host__ __device__ inline int64_t groups_of(int64_t rows, int64_t cols) {
  return (rows * (act8_pitch(cols) / 8) + 255) / 256;
}
unsigned grid_of(int64_t rows, int64_t cols) {
  const int64_t n = groups_of(rows, cols);
  return (unsigned)(n < (1 << 22) ? n : (1 << 22));
}

// exp(-x) for x >= 0, within a step of fp32 and a little, subnormal results too: x
// log2 e = n + f with n whole and f in [-1/2, 1/2], log2 e in two parts, and 2^-f
// by the hardware.  (From 200 on the result is 0.)
__device__ __forceinline__ float exp_neg(float x) {
  constexpr float kHi = 1.44269502162933349609375f, kLo = 1.925963033500011e-8f;
  x = fminf(x, 200.f);
  const float n = __builtin_rintf(x * kHi);
  const float f = fmaf(x, kLo, fmaf(x, kHi, -n));
  return __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f(-f), -(int)n);
}
// Sigmoid of g and of -g (= 1 - sigmoid of g, without the subtraction's loss), from
// t = exp(-|g|), which cannot overflow: r = 1 / (1 + t) and t r.  fp32 takes the
// exponential above; the 16-bit types the hardware's alone, whose error grows to 2
// |g| half steps of fp32 (1e-5 of the value where fp32 ends, a twentieth of fp16's
// half step).  A NaN reaches the results through g itself.
struct Sigmoid {
  float at, neg;
};
template <int T>
__device__ __forceinline__ Sigmoid sigmoid(float g) {
  float t;
  if constexpr (T == FP8SG_OUT_F32) t = exp_neg(fabsf(g));
  else t = __expf(-fabsf(g));
  // (the divisor lies in [1, 2]: the hardware's reciprocal, a step off at most, and
  // one Newton step give the quotient within half a step and a little)
  const float d = 1.0f + t, q = __builtin_amdgcn_rcpf(d);
  const float r = fmaf(q, fmaf(-d, q, 1.0f), q), tr = t * r;
  return g < 0.f ? Sigmoid{tr, r} : Sigmoid{r, tr};
}

template <int T, bool S, bool CKPT>
__global__ __launch_bounds__(256) void k_swiglu_fwd(SwigluArgs p) {
  const int64_t pitch = act8_pitch(p.cols);
  for (int64_t blk = blockIdx.x; blk < groups_of(p.rows, p.cols); blk += gridDim.x) {
    const Unit w = unit_of(blk, pitch / 8);
    const bool in = w.row < p.rows;
    const int64_t c = w.u * 8;
    const int n = in && c < p.cols ? left8(p.cols, c) : 0;
    float g[8] = {}, u[8] = {}, a[8];
    if (n > 0) {
      load8<T, S>(reinterpret_cast<const Elem<T>*>(p.g) + w.row * p.ldg + c, n, g);
      load8<T, S>(reinterpret_cast<const Elem<T>*>(p.u) + w.row * p.ldu + c, n, u);
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] = g[e] * sigmoid<T>(g[e]).at * u[e];
      store8<T, S>(reinterpret_cast<Elem<T>*>(p.a) + w.row * p.cols + c, n, a);
    }
    if constexpr (CKPT) {
      const uint32_t sg = act8_scale(quad_amax(g)), su = act8_scale(quad_amax(u));
      if (in) {
        const int64_t at = w.row * pitch + c;
        st8<S>(p.cg.q + at, act8_codes(g, sg));
        st8<S>(p.cu.q + at, act8_codes(u, su));
        if ((w.u & 3) == 0) {
          p.cg.s[at >> 5] = (uint8_t)sg;
          p.cu.s[at >> 5] = (uint8_t)su;
        }
      }
    }
  }
}

template <int T, bool S, bool CKPT>
__global__ __launch_bounds__(256) void k_swiglu_bwd(SwigluArgs p) {
  const int64_t pitch = act8_pitch(p.cols);
  for (int64_t blk = blockIdx.x; blk < groups_of(p.rows, p.cols); blk += gridDim.x) {
    const Unit w = unit_of(blk, pitch / 8);
    const int64_t c = w.u * 8;
    if (w.row >= p.rows || c >= p.cols) continue;
    const int n = left8(p.cols, c);
    float g[8], u[8], da[8], dg[8], du[8];
    load8<T, S>(reinterpret_cast<const Elem<T>*>(p.da) + w.row * p.cols + c, n, da);
    if constexpr (CKPT) {
      const int64_t at = w.row * pitch + c;
      act8_values(*reinterpret_cast<const uint2*>(p.cg.q + at), p.cg.s[at >> 5], g);
      act8_values(*reinterpret_cast<const uint2*>(p.cu.q + at), p.cu.s[at >> 5], u);
    } else {
      load8<T, S>(reinterpret_cast<const Elem<T>*>(p.g) + w.row * p.ldg + c, n, g);
      load8<T, S>(reinterpret_cast<const Elem<T>*>(p.u) + w.row * p.ldu + c, n, u);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const Sigmoid sg = sigmoid<T>(g[e]);  // (da, often small, comes last: da sigmoid may lie below fp32's range)
      du[e] = da[e] * (g[e] * sg.at);
      dg[e] = da[e] * (u[e] * (sg.at * (1.0f + g[e] * sg.neg)));
    }
    store8<T, S>(reinterpret_cast<Elem<T>*>(p.dg) + w.row * p.lddg + c, n, dg);
    store8<T, S>(reinterpret_cast<Elem<T>*>(p.du) + w.row * p.lddu + c, n, du);
  }
}

template <int T, bool S>
__global__ __launch_bounds__(256) void k_act8_quant(const void* x, int64_t rows, int64_t cols, fp8sg_act8 q) {
  const int64_t pitch = act8_pitch(cols);
  for (int64_t blk = blockIdx.x; blk < groups_of(rows, cols); blk += gridDim.x) {
    const Unit w = unit_of(blk, pitch / 8);
    const bool in = w.row < rows;
    const int64_t c = w.u * 8;
    const int n = in && c < cols ? left8(cols, c) : 0;
    float v[8] = {};
    if (n > 0) load8<T, S>(reinterpret_cast<const Elem<T>*>(x) + w.row * cols + c, n, v);
    const uint32_t s = act8_scale(quad_amax(v));
    if (!in) continue;
    const int64_t at = w.row * pitch + c;
    st8<S>(q.q + at, act8_codes(v, s));
    if ((w.u & 3) == 0) q.s[at >> 5] = (uint8_t)s;
  }
}

template <int T, bool S>
__global__ __launch_bounds__(256) void k_act8_dequant(fp8sg_act8 q, int64_t rows, int64_t cols, void* y) {
  const int64_t pitch = act8_pitch(cols);
  for (int64_t blk = blockIdx.x; blk < groups_of(rows, cols); blk += gridDim.x) {
    const Unit w = unit_of(blk, pitch / 8);
    const int64_t c = w.u * 8;
    if (w.row >= rows || c >= cols) continue;
    const int n = left8(cols, c);
    const int64_t at = w.row * pitch + c;
    float v[8];
    act8_values(*reinterpret_cast<const uint2*>(q.q + at), q.s[at >> 5], v);
    store8<T, S>(reinterpret_cast<Elem<T>*>(y) + w.row * cols + c, n, v);
  }
}

int64_t esize(int type) { return type == FP8SG_OUT_F32 ? 4 : 2; }

// f(type, streaming) as compile-time constants
template <class F>
hipError_t pick(int type, bool stream, F f) {
  return by_type(type, [&](auto t) {
    if (stream) f(t, std::true_type{});
    else f(t, std::false_type{});
    return hipGetLastError();
  });
}

}  // namespace

hipError_t launch_swiglu_fwd(const SwigluArgs& a, int type, hipStream_t stream) {
  if (a.rows == 0 || a.cols == 0) return hipSuccess;
  const bool big = a.rows * a.cols * (3 * esize(type) + (a.cg.q ? 2 : 0)) >= kStreamBytes;
  const dim3 grid(grid_of(a.rows, a.cols));
  return pick(type, big, [&](auto t, auto s) {
    constexpr int T = decltype(t)::value;
    constexpr bool St = decltype(s)::value;
    if (a.cg.q) hipLaunchKernelGGL((k_swiglu_fwd<T, St, true>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((k_swiglu_fwd<T, St, false>), grid, dim3(256), 0, stream, a);
  });
}

hipError_t launch_swiglu_bwd(const SwigluArgs& a, int type, hipStream_t stream) {
  if (a.rows == 0 || a.cols == 0) return hipSuccess;
  const bool big = a.rows * a.cols * (3 * esize(type) + 2 * (a.cg.q ? 1 : esize(type))) >= kStreamBytes;
  const dim3 grid(grid_of(a.rows, a.cols));
  return pick(type, big, [&](auto t, auto s) {
    constexpr int T = decltype(t)::value;
    constexpr bool St = decltype(s)::value;
    if (a.cg.q) hipLaunchKernelGGL((k_swiglu_bwd<T, St, true>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((k_swiglu_bwd<T, St, false>), grid, dim3(256), 0, stream, a);
  });
}

hipError_t launch_act8_quantize(const void* x, int type, int64_t rows, int64_t cols, fp8sg_act8 c, hipStream_t stream) {
  if (rows == 0 || cols == 0) return hipSuccess;
  const bool big = rows * cols * (esize(type) + 1) >= kStreamBytes;
  return pick(type, big, [&](auto t, auto s) {
    hipLaunchKernelGGL((k_act8_quant<decltype(t)::value, decltype(s)::value>),
                       dim3(grid_of(rows, cols)), dim3(256), 0, stream, x, rows, cols, c);
  });
}

hipError_t launch_act8_dequantize(fp8sg_act8 c, int64_t rows, int64_t cols, void* y, int type, hipStream_t stream) {
  if (rows == 0 || cols == 0) return hipSuccess;
  const bool big = rows * cols * (esize(type) + 1) >= kStreamBytes;
  return pick(type, big, [&](auto t, auto s) {
    hipLaunchKernelGGL((k_act8_dequant<decltype(t)::value, decltype(s)::value>),
                       dim3(grid_of(rows, cols)), dim3(256), 0, stream, c, rows, cols, y);
  });
}

}  // namespace fp8sg
