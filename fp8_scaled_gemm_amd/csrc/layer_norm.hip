// Layer norm, forward and backward, with the reduction of the weight's and the
// bias's gradients over the rows.
//
// Bound by memory: the forward reads a row once and writes it once, the
// backward reads dy and x (or x's 8-bit checkpoint) once and writes dx.  A row
// stays in registers between the passes over it (mean, squared deviations,
// result), 8 to 32 elements a thread, so a row takes 1 to 16 waves by its
// length; rows past kMaxCols are re-read instead (k_*_long).
//
// Gradients of the weight and the bias: each block walks its share of the rows
// with its columns' sums in registers and leaves one partial row of each in
// the workspace; a second kernel adds the partial rows.  Every sum's order
// follows from the sizes alone, so results repeat bit for bit.
//
// Measured: 8192 x 4096 bf16 forward 24 us from a graph (5.6 TB/s), with the checkpoint
// 30 there and 32 alone (5.3 TB/s), backward from the checkpoint 35 us and the join
// 5; fp32 44 and 82 us (6.0, 4.9 TB/s).  1000 x 14336 fp16 forward 15 us, backward 23 us
// and the join 7: there the 250 partial rows are as many bytes as dx.  Past kMaxCols,
// 4096 x 20480 bf16: forward 101 us (3.3 TB/s), backward 192 (2.6).
#include "mx.hpp"

namespace fp8sg {
namespace {

constexpr int64_t kMaxCols = 16384;  // 16 waves x 64 lanes x 16 elements

template <int CTRL>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xF, 0xF, false));
}
// Sum over groups of N neighbouring lanes (N a power of two up to 64), the same in
// each of them: quads, then mirrored halves and rows of 16, then rows and halves
// of the wave swapped.  All on the vector unit; all lanes active.
template <int N>
__device__ __forceinline__ float lane_sum(float v) {
  if constexpr (N > 1) v = add_dpp<0xB1>(v);   // quad_perm 1 0 3 2
  if constexpr (N > 2) v = add_dpp<0x4E>(v);   // quad_perm 2 3 0 1
  if constexpr (N > 4) v = add_dpp<0x141>(v);  // row_half_mirror
  if constexpr (N > 8) v = add_dpp<0x140>(v);  // row_mirror
  if constexpr (N > 16) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  if constexpr (N > 32) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  return v;
}
__device__ __forceinline__ float wave_sum(float v) { return lane_sum<kWave>(v); }
// Sum over the NW waves of a row, the same in every lane.  `red`: NW floats of
// the row's own, not in use before the last barrier; buffers alternate between
// consecutive calls, so one barrier a call is enough.
template <int NW>
__device__ __forceinline__ float row_sum(float v, float* red, int wave) {
  v = wave_sum(v);
  if constexpr (NW == 1) return v;
  red[wave] = v;  // every lane holds the sum: a write of one value to one address
  __syncthreads();
  return lane_sum<NW>(red[threadIdx.x & (NW - 1)]);
}
// The same for two sums at once; `red`: 2 NW floats.
template <int NW>
__device__ __forceinline__ void row_sum2(float& a, float& b, float* red, int wave) {
  a = wave_sum(a);
  b = wave_sum(b);
  if constexpr (NW > 1) {
    red[wave] = a;
    red[NW + wave] = b;
    __syncthreads();
    a = lane_sum<NW>(red[threadIdx.x & (NW - 1)]);
    b = lane_sum<NW>(red[NW + (threadIdx.x & (NW - 1))]);
  }
}

// s / n as the product with the rounded 1 / n and one correction: within half a
// step and a little, and exact where n divides s.  (The product alone gives a row
// of n values 1000 a mean one step off.)
struct Count {
  float n, inv;
  __device__ __forceinline__ explicit Count(int64_t cols) : n((float)cols), inv(1.0f / n) {}
  __device__ __forceinline__ float mean(float s) const {
    const float q = s * inv;
    return fmaf(fmaf(-q, n, s), inv, q);
  }
};

// 1 / sqrt(v): the library's estimate (a step or two off) and one Newton step, about
// a step off at most; as it is for 0, infinity and NaN.
__device__ __forceinline__ float inv_sqrt(float v) {
  const float r = rsqrtf(v);
  return v > 0.f && v < __builtin_inff() ? fmaf(0.5f * r, fmaf(-v * r, r, 1.0f), r) : r;
}

// A row's statistics from a first mean m0 and the sums s1, s2 of the deviations
// from it and of their squares: the mean is m0 + shift, the variance s2 / n -
// shift^2.  A row of one value has deviations of one value, a few steps, whose
// sum is exact: a variance of exactly 0, however its own sum rounded; and
// deviations keep their own precision where the mean is far from zero.  The third
// sum is paid for by adding over lanes on the vector unit (8192 x 4096 bf16 23.7
// us, 23.9 without it and through LDS permutes; 130000 x 256 36.5 and 35.7).
struct RowStats {
  float shift, rstd;
};
__device__ __forceinline__ RowStats row_stats(float s1, float s2, const Count& n, float eps) {
  const float shift = n.mean(s1), var = fmaf(-shift, shift, n.mean(s2));
  return RowStats{shift, inv_sqrt((var < 0.f ? 0.f : var) + eps)};
}

template <int P>
__device__ __forceinline__ void load_params(const void* w, int64_t c, int n, float none, float (&v)[8]) {
  if (w && n > 0) {
    load8<P, false>(reinterpret_cast<const Elem<P>*>(w) + c, n, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = none;
  }
}

// A row per NW waves, R rows a block; V groups of 8 elements a thread: group k
// of a row's thread t is elements 8 (t + 64 NW k) .. + 7.  With two groups the next
// row's loads are issued before this row's sums (4000 x 14336 bf16 with checkpoint:
// 67 us, 92 us a row at a time; 8192 x 8192: 50, 62 us; 16384 x 1024: 13.6, 17.2); with
// one, the waves that the registers for it would cost do more (8192 x 2048: 16.3
// us, without 15.4).
template <int T, int P, int NW, int V>
__global__ __launch_bounds__(NW == 1 ? 256 : 64 * NW) void k_ln_fwd(LayerNormArgs p) {
  constexpr int R = NW == 1 ? 4 : 1;
  __shared__ float red[3 * NW];
  const int lane = threadIdx.x & 63, wave = NW == 1 ? 0 : threadIdx.x >> 6;
  const int t = wave * 64 + lane;
  const Count count(p.cols);
  float w[V][8], b[V][8];
  int64_t c[V];
  int n[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    c[k] = 8 * (t + 64 * NW * k);
    n[k] = left8(p.cols, c[k]);
    load_params<P>(p.w, c[k], n[k], 1.f, w[k]);
    load_params<P>(p.b, c[k], n[k], 0.f, b[k]);
  }
  const int64_t pitch = act8_pitch(p.cols);
  const Elem<T>* xp = reinterpret_cast<const Elem<T>*>(p.x);
  Row8<T> next[V];
  auto fetch = [&](int64_t r) {
    if (r >= p.rows) return;
#pragma unroll
    for (int k = 0; k < V; ++k) next[k] = load_row8<T, false>(xp + r * p.cols + c[k], n[k]);
  };
  const int64_t step = (int64_t)gridDim.x * R;
  int64_t r = (int64_t)blockIdx.x * R + (NW == 1 ? threadIdx.x >> 6 : 0);
  constexpr bool kAhead = V > 1;
  const bool ragged = (p.cols & 7) != 0;  // (uniform)
  if constexpr (kAhead) fetch(r);
#pragma unroll 1
  for (; r < p.rows; r += step) {
    float v[V][8], s = 0.f;
    if constexpr (!kAhead) fetch(r);
#pragma unroll
    for (int k = 0; k < V; ++k) next[k].values(v[k]);
    if constexpr (kAhead) fetch(r + step);
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += v[k][e];
    if (p.ckpt.q) {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const uint32_t sc = act8_scale(quad_amax(v[k]));
        if (c[k] < pitch) {
          *reinterpret_cast<uint2*>(p.ckpt.q + r * pitch + c[k]) = act8_codes(v[k], sc);
          if ((lane & 3) == 0) p.ckpt.s[(r * pitch + c[k]) >> 5] = (uint8_t)sc;
        }
      }
    }
    const float m0 = count.mean(row_sum<NW>(s, red, wave));
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const float m = n[k] > 0 ? m0 : 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[k][e] -= m;
      if (ragged) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[k][e] = e < n[k] ? v[k][e] : 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s1 += v[k][e];
        s2 = fmaf(v[k][e], v[k][e], s2);
      }
    }
    row_sum2<NW>(s1, s2, red + NW, wave);
    const RowStats st = row_stats(s1, s2, count, p.eps);
    Elem<T>* y = reinterpret_cast<Elem<T>*>(p.y) + r * p.cols;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = fmaf((v[k][e] - st.shift) * st.rstd, w[k][e], b[k][e]);
      store8<T, false>(y + c[k], n[k], o);
    }
    if (t == 0 && p.mean) {
      p.mean[r] = m0 + st.shift;
      p.rstd[r] = st.rstd;
    }
  }
}

// The backward's x: 8 elements of the input, or of its checkpoint.
template <int T, bool CKPT>
struct XRow {
  Row8<T> x;
  __device__ __forceinline__ void load(const LayerNormArgs& p, int64_t r, int64_t c, int n) {
    x = load_row8<T, false>(reinterpret_cast<const Elem<T>*>(p.x) + r * p.cols + c, n);
  }
  __device__ __forceinline__ void values(float (&v)[8]) const { x.values(v); }
};
template <int T>
struct XRow<T, true> {
  uint2 q;
  uint32_t s;
  __device__ __forceinline__ void load(const LayerNormArgs& p, int64_t r, int64_t c, int n) {
    q = make_uint2(0, 0);
    s = 127u;
    if (n > 0) {
      const int64_t at = r * act8_pitch(p.cols) + c;
      q = *reinterpret_cast<const uint2*>(p.ckpt.q + at);
      s = p.ckpt.s[at >> 5];
    }
  }
  __device__ __forceinline__ void values(float (&v)[8]) const { act8_values(q, s, v); }
};

// dx of a row, and the block's partial rows of dw and db.  The next row's loads
// are issued before this row's sums, whose barrier they then hide behind.
template <int T, int P, int NW, int V, bool CKPT>
__global__ __launch_bounds__(NW == 1 ? 256 : 64 * NW) void k_ln_bwd(LayerNormArgs p, int direct) {
  constexpr int R = NW == 1 ? 4 : 1;
  __shared__ float red[2][2 * NW];
  extern __shared__ float part[];  // NW == 1: three waves' partial rows
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, rw = NW == 1 ? 0 : wave;
  const int t = rw * 64 + lane;
  const Count count(p.cols);
  float w[V][8], dw[V][8], db[V][8];
  int64_t c[V];
  int n[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    c[k] = 8 * (t + 64 * NW * k);
    n[k] = left8(p.cols, c[k]);
    load_params<P>(p.w, c[k], n[k], 1.f, w[k]);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[k][e] = db[k][e] = 0.f;
  }
  const Elem<T>* dyp = reinterpret_cast<const Elem<T>*>(p.dy);
  Row8<T> ndy[V];
  XRow<T, CKPT> nx[V];
  float nmean = 0.f, nrstd = 0.f;
  auto fetch = [&](int64_t r) {
    if (r >= p.rows) return;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      ndy[k] = load_row8<T, false>(dyp + r * p.cols + c[k], n[k]);
      nx[k].load(p, r, c[k], n[k]);
    }
    nmean = p.mean[r];
    nrstd = p.rstd[r];
  };
  const int64_t step = (int64_t)gridDim.x * R;
  int64_t r = (int64_t)blockIdx.x * R + (NW == 1 ? wave : 0);
  constexpr bool kAhead = !(T == FP8SG_OUT_F32 && V == 4);  // (there the registers are all in use)
  if constexpr (kAhead) fetch(r);
#pragma unroll 1
  for (int it = 0; r < p.rows; r += step, it ^= 1) {
    float dy[V][8], xh[V][8];
    if constexpr (!kAhead) fetch(r);
    const float mean = nmean, rstd = nrstd;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      ndy[k].values(dy[k]);
      nx[k].values(xh[k]);
    }
    if constexpr (kAhead) fetch(r + step);
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        xh[k][e] = (xh[k][e] - mean) * rstd;
        dw[k][e] += dy[k][e] * xh[k][e];  // (elements past the row's end have dy = 0)
        db[k][e] += dy[k][e];
        dy[k][e] *= w[k][e];
        s1 += dy[k][e];
        s2 += dy[k][e] * xh[k][e];
      }
    if (p.dx) {
      s1 = wave_sum(s1);
      s2 = wave_sum(s2);
      if constexpr (NW > 1) {
        float* buf = red[it];
        buf[rw] = s1;
        buf[NW + rw] = s2;
        __syncthreads();
        s1 = buf[0];
        s2 = buf[NW];
#pragma unroll
        for (int i = 1; i < NW; ++i) {
          s1 += buf[i];
          s2 += buf[NW + i];
        }
      }
      const float c1 = count.mean(s1), c2 = count.mean(s2);
      Elem<T>* dx = reinterpret_cast<Elem<T>*>(p.dx) + r * p.cols;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = rstd * (dy[k][e] - c1 - xh[k][e] * c2);
        store8<T, false>(dx + c[k], n[k], o);
      }
    }
  }
  if (!p.dw && !p.db) return;
  if constexpr (NW == 1) {  // the block's four waves hold the same columns
    if (wave > 0) {
#pragma unroll
      for (int k = 0; k < V; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          part[((wave - 1) * 2 * V + k) * 512 + 64 * e + lane] = dw[k][e];
          part[((wave - 1) * 2 * V + V + k) * 512 + 64 * e + lane] = db[k][e];
        }
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dw[k][e] += part[(i * 2 * V + k) * 512 + 64 * e + lane];
          db[k][e] += part[(i * 2 * V + V + k) * 512 + 64 * e + lane];
        }
  }
#pragma unroll
  for (int k = 0; k < V; ++k) {
    if (direct) {  // one block: these are the gradients
      if (p.dw) store8<P, false>(reinterpret_cast<Elem<P>*>(p.dw) + c[k], n[k], dw[k]);
      if (p.db) store8<P, false>(reinterpret_cast<Elem<P>*>(p.db) + c[k], n[k], db[k]);
    } else {
      float* o = p.ws + (int64_t)blockIdx.x * 2 * p.cols + c[k];
      store8<FP8SG_OUT_F32, false>(o, n[k], dw[k]);
      store8<FP8SG_OUT_F32, false>(o + p.cols, n[k], db[k]);
    }
  }
}

// The sum of `parts` partial rows: 32 columns at a time, 32 threads down each
// column with eight loads under way each (one at a time: 8192 x 1024, backward 19.9
// us, so 16.6), then a tree.
template <int P>
__global__ __launch_bounds__(1024) void k_ln_join(LayerNormArgs p, int parts) {
  __shared__ float red[32][33];
  const int cl = threadIdx.x & 31, k = threadIdx.x >> 5;
  const bool bias = blockIdx.y != 0;
  void* out = bias ? p.db : p.dw;
  if (!out) return;
  for (int64_t c0 = (int64_t)blockIdx.x * 32; c0 < p.cols; c0 += (int64_t)gridDim.x * 32) {
    const int64_t c = c0 + cl;
    float s = 0.f;
    if (c < p.cols) {
      const float* at = p.ws + (int64_t)bias * p.cols + c;
      for (int i = k; i < parts; i += 256) {
        float v[8];
#pragma unroll
        for (int h = 0; h < 8; ++h) v[h] = i + 32 * h < parts ? at[(int64_t)(i + 32 * h) * 2 * p.cols] : 0.f;
#pragma unroll
        for (int h = 0; h < 8; ++h) s += v[h];
      }
    }
    red[k][cl] = s;
    __syncthreads();
#pragma unroll
    for (int h = 16; h > 0; h >>= 1) {
      if (k < h) red[k][cl] += red[k + h][cl];
      __syncthreads();
    }
    if (k == 0 && c < p.cols) reinterpret_cast<Elem<P>*>(out)[c] = from_f32<P>(red[0][cl]);
    __syncthreads();
  }
}

// ---- rows past kMaxCols: the same sums, the row read again for each
template <int T, int P>
__global__ __launch_bounds__(1024) void k_ln_fwd_long(LayerNormArgs p) {
  __shared__ float red[3 * 16];
  const int wave = threadIdx.x >> 6;
  const Count count(p.cols);
  const int64_t pitch = act8_pitch(p.cols);
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const Elem<T>* x = reinterpret_cast<const Elem<T>*>(p.x) + r * p.cols;
    Elem<T>* y = reinterpret_cast<Elem<T>*>(p.y) + r * p.cols;
    float s = 0.f, v[8];
    for (int64_t c = 8 * (int64_t)threadIdx.x; c < p.cols; c += 8192) {
      load8<T, false>(x + c, left8(p.cols, c), v);
#pragma unroll
      for (int e = 0; e < 8; ++e) s += v[e];
    }
    const float m0 = count.mean(row_sum<16>(s, red, wave));
    float s1 = 0.f, s2 = 0.f;
    for (int64_t c = 8 * (int64_t)threadIdx.x; c < p.cols; c += 8192) {
      const int n = left8(p.cols, c);
      load8<T, false>(x + c, n, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = e < n ? v[e] - m0 : 0.f;
        s1 += d;
        s2 = fmaf(d, d, s2);
      }
    }
    row_sum2<16>(s1, s2, red + 16, wave);
    const RowStats st = row_stats(s1, s2, count, p.eps);
    // whole waves walk the last round: the checkpoint's blocks span lanes
    for (int64_t c0 = 0; c0 < p.cols; c0 += 8192) {
      const int64_t c = c0 + 8 * (int64_t)threadIdx.x;
      const int n = left8(p.cols, c);
      load8<T, false>(x + c, n, v);
      if (p.ckpt.q) {
        const uint32_t sc = act8_scale(quad_amax(v));
        if (c < pitch) {
          *reinterpret_cast<uint2*>(p.ckpt.q + r * pitch + c) = act8_codes(v, sc);
          if ((threadIdx.x & 3) == 0) p.ckpt.s[(r * pitch + c) >> 5] = (uint8_t)sc;
        }
      }
      float w[8], b[8];
      load_params<P>(p.w, c, n, 1.f, w);
      load_params<P>(p.b, c, n, 0.f, b);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = fmaf(((v[e] - m0) - st.shift) * st.rstd, w[e], b[e]);
      store8<T, false>(y + c, n, v);
    }
    if (threadIdx.x == 0 && p.mean) {
      p.mean[r] = m0 + st.shift;
      p.rstd[r] = st.rstd;
    }
  }
}

template <int T, int P, bool CKPT>
__global__ __launch_bounds__(1024) void k_ln_dx_long(LayerNormArgs p) {
  __shared__ float red[2][2][16];
  const int wave = threadIdx.x >> 6;
  const Count count(p.cols);
  int it = 0;
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x, it ^= 1) {
    const Elem<T>* dy = reinterpret_cast<const Elem<T>*>(p.dy) + r * p.cols;
    const float mean = p.mean[r], rstd = p.rstd[r];
    float s1 = 0.f, s2 = 0.f, q[8], xh[8], w[8];
    auto load = [&](int64_t c, int n) {
      XRow<T, CKPT> x;
      x.load(p, r, c, n);
      x.values(xh);
      load8<T, false>(dy + c, n, q);
      load_params<P>(p.w, c, n, 1.f, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        xh[e] = (xh[e] - mean) * rstd;
        q[e] *= w[e];
      }
    };
    for (int64_t c = 8 * (int64_t)threadIdx.x; c < p.cols; c += 8192) {
      load(c, left8(p.cols, c));
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s1 += q[e];
        s2 += q[e] * xh[e];
      }
    }
    const float c1 = count.mean(row_sum<16>(s1, red[it][0], wave)), c2 = count.mean(row_sum<16>(s2, red[it][1], wave));
    Elem<T>* dx = reinterpret_cast<Elem<T>*>(p.dx) + r * p.cols;
    for (int64_t c = 8 * (int64_t)threadIdx.x; c < p.cols; c += 8192) {
      const int n = left8(p.cols, c);
      load(c, n);
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = rstd * (q[e] - c1 - xh[e] * c2);
      store8<T, false>(dx + c, n, q);
    }
  }
}

// Partial rows of dw and db: 8 columns a thread, the rows of chunk blockIdx.y.
template <int T, bool CKPT>
__global__ __launch_bounds__(64) void k_ln_dwb_long(LayerNormArgs p) {
  const int64_t c = ((int64_t)blockIdx.x * 64 + threadIdx.x) * 8;
  if (c >= p.cols) return;
  const int n = left8(p.cols, c);
  const int64_t per = (p.rows + gridDim.y - 1) / gridDim.y, r0 = blockIdx.y * per;
  const int64_t r1 = r0 + per < p.rows ? r0 + per : p.rows;
  float dw[8] = {}, db[8] = {}, x[8], dy[8];
  for (int64_t r = r0; r < r1; ++r) {
    XRow<T, CKPT> xr;
    xr.load(p, r, c, n);
    xr.values(x);
    load8<T, false>(reinterpret_cast<const Elem<T>*>(p.dy) + r * p.cols + c, n, dy);
    const float mean = p.mean[r], rstd = p.rstd[r];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      dw[e] += dy[e] * ((x[e] - mean) * rstd);
      db[e] += dy[e];
    }
  }
  float* o = p.ws + (int64_t)blockIdx.y * 2 * p.cols + c;
  store8<FP8SG_OUT_F32, false>(o, n, dw);
  store8<FP8SG_OUT_F32, false>(o + p.cols, n, db);
}

template <class F>
hipError_t by_types(int type, int ptype, F f) {
  return by_type(type, [&](auto t) {
    if (ptype == FP8SG_OUT_F32) f(t, std::integral_constant<int, FP8SG_OUT_F32>{});
    else f(t, t);
    return hipGetLastError();
  });
}
// f(waves per row, groups of 8 per thread) for a row of up to kMaxCols.  The
// backward keeps five fp32 values an element: past 8192 columns 8 waves x 4 groups
// take all 256 registers a thread, and in the 16-bit types 10 more, saved before
// the loop over the rows and read back after it (40 bytes a thread, 4.9 MiB of
// writes at 1000 x 14336).  16 waves x 2 groups would have 128 registers for the 139 -
// 150 that two groups take at 4 waves, inside that loop.
template <bool BWD, class F>
void by_width(int64_t cols, F f) {
  typedef std::integral_constant<int, 1> C1;
  typedef std::integral_constant<int, 2> C2;
  if (cols <= 512) f(C1{}, C1{});
  else if (cols <= 1024) f(C1{}, C2{});
  else if (cols <= 2048) f(std::integral_constant<int, 4>{}, C1{});
  else if (cols <= 4096) f(std::integral_constant<int, 4>{}, C2{});
  else if (cols <= 8192) f(std::integral_constant<int, 8>{}, C2{});
  else if constexpr (BWD) f(std::integral_constant<int, 8>{}, std::integral_constant<int, 4>{});
  else f(std::integral_constant<int, 16>{}, C2{});
}

// Partial rows of the weight gradients: a block each, enough of them to fill
// the chip, few enough that writing and adding them stays small next to the
// rows themselves (8 bytes a column and part against 4 to 12 a column and
// row).  At most 512 of up to 4096 columns, 256 of more, and 4 rows a block (a
// wave, where a row takes one) at least.  Backward from a graph, us:
//   parts            128    256    512   1024
//   65536 x 512       82     45     37     39
//   16384 x 1000      47     29     24     27
//   16384 x 2048     103     56     39     39
//   4000 x 4096       40     26     25     31
//   8192 x 4096 ckpt  77     44     36     41
//   4000 x 5000       49     32     38     48
//   16384 x 8192     198    167    175    186
//   4000 x 14336      95     81     92    120
//   least rows         2      4      8
//   1000 x 4096     18.3   15.4   16.9
//   1000 x 2048     12.5   11.4   13.3
//   1000 x 14336    30.1   30.3   34.1
//   256 x 1000       9.7   11.7   16.4   (few rows of up to 2048 columns: 2 would be better)
// One, when the rows are few: the block then writes the gradients.
constexpr int64_t kDirectRows = 8;
int64_t parts_of(int64_t rows, int64_t cols) {
  if (cols > kMaxCols) {
    const int64_t n = (rows + 7) / 8;
    return n < 1 ? 1 : n < 64 ? n : 64;
  }
  const int64_t per_block = cols <= 1024 ? 4 : 1;
  if (rows <= kDirectRows * per_block) return 1;
  const int64_t n = (rows + 4 * per_block - 1) / (4 * per_block);
  const int64_t most = cols > 4096 ? 256 : 512;
  return n < most ? n : most;
}

unsigned cap(int64_t n, int64_t most) { return (unsigned)(n < most ? n : most); }

}  // namespace

int64_t layer_norm_ws_len(int64_t rows, int64_t cols) { return 2 * parts_of(rows, cols) * cols; }

hipError_t launch_layer_norm_fwd(const LayerNormArgs& a, int type, int ptype, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  return by_types(type, ptype, [&](auto t, auto p) {
    constexpr int T = decltype(t)::value, P = decltype(p)::value;
    if (a.cols > kMaxCols) {
      hipLaunchKernelGGL((k_ln_fwd_long<T, P>), dim3(cap(a.rows, 1 << 16)), dim3(1024), 0, stream, a);
      return;
    }
    by_width<false>(a.cols, [&](auto nw, auto v) {
      constexpr int NW = decltype(nw)::value, V = decltype(v)::value, R = NW == 1 ? 4 : 1;
      // Several rows a block, so that the parameters are loaded once for them:
      // with the next row's loads ahead, as many blocks as are resident (16 waves
      // a compute unit); else enough to cover each other's loads.
      const int64_t most = V > 1 ? (int64_t)device_cus() * 16 / (NW == 1 ? 4 : NW) : 4096;
      const unsigned grid = cap((a.rows + R - 1) / R, most);
      hipLaunchKernelGGL((k_ln_fwd<T, P, NW, V>), dim3(grid), dim3(NW == 1 ? 256 : 64 * NW), 0, stream, a);
    });
  });
}

hipError_t launch_layer_norm_bwd(const LayerNormArgs& a, int type, int ptype, hipStream_t stream) {
  if (a.cols == 0 || (a.rows == 0 && !a.dw && !a.db)) return hipSuccess;
  const int parts = (int)parts_of(a.rows, a.cols);
  const bool wb = a.dw || a.db;
  return by_types(type, ptype, [&](auto t, auto p) {
    constexpr int T = decltype(t)::value, P = decltype(p)::value;
    auto run = [&](auto ck) {
      constexpr bool CK = decltype(ck)::value;
      if (a.cols > kMaxCols) {
        if (a.dx && a.rows > 0)
          hipLaunchKernelGGL((k_ln_dx_long<T, P, CK>), dim3(cap(a.rows, 1 << 16)), dim3(1024), 0, stream, a);
        if (wb)
          hipLaunchKernelGGL((k_ln_dwb_long<T, CK>), dim3((unsigned)((a.cols + 511) / 512), parts), dim3(64), 0, stream, a);
        return;
      }
      by_width<true>(a.cols, [&](auto nw, auto v) {
        constexpr int NW = decltype(nw)::value, V = decltype(v)::value, R = NW == 1 ? 4 : 1;
        const unsigned grid = wb ? (unsigned)parts : cap((a.rows + R - 1) / R, 2048);
        const size_t lds = NW == 1 ? 3 * 2 * V * 512 * sizeof(float) : 0;
        hipLaunchKernelGGL((k_ln_bwd<T, P, NW, V, CK>), dim3(grid), dim3(NW == 1 ? 256 : 64 * NW), lds, stream, a,
                           parts == 1 ? 1 : 0);
      });
    };
    if (a.ckpt.q) run(std::true_type{});
    else run(std::false_type{});
    if (wb && (a.cols > kMaxCols || parts > 1))
      hipLaunchKernelGGL((k_ln_join<P>), dim3(cap((a.cols + 31) / 32, 1 << 16), 2), dim3(1024), 0, stream, a, parts);
  });
}

}  // namespace fp8sg
