// What stands behind a linear layer's product, in the product's own epilogue and
// in kernels of its own:
//   h = acc + bias[n],  y = residual + drop(act(h)),
// and, for the backward pass, gh = drop'(gy) act'(h).  Everything is computed in
// fp32 from the fp32 accumulator and rounded once, to y (and to the kept h).
#pragma once

#include "launch_epilogue.hpp"
#include "mx.hpp"

namespace fp8sg {

typedef float v4f __attribute__((ext_vector_type(4)));

// ---- dropout: a counter-based generator, so the mask is computed again wherever
// it is needed and never stored.  Philox 4x32 with 10 rounds (Salmon, Moraes,
// Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011).  One call
// gives 128 bits, 16 for each of eight consecutive columns: p is a multiple of
// 2^-16, and the 20 products of a call, which the vector unit takes at a quarter
// of its rate, are shared by eight elements.  (Dropout of 8192 x 4096 bf16, us, in a
// graph: 27; with 32 bits an element, so two calls a group, 31.)
__device__ __forceinline__ uint4 philox(uint64_t n, uint64_t offset, uint64_t key) {
  uint32_t c0 = (uint32_t)n, c1 = (uint32_t)(n >> 32), c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
  uint32_t k0 = (uint32_t)key, k1 = (uint32_t)(key >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c1 = (uint32_t)b;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// The generator's state and the rule of one call.
struct Drop {
  uint64_t key, offset;
  uint32_t t;   // an element is kept where its 16 bits are at least this
  float scale;  // 65536 / (65536 - t); 0 where nothing is kept
};
__device__ __forceinline__ Drop drop_of(const DropArgs& a) {
  return a.rng ? Drop{a.rng[0], a.rng[1], a.t, a.scale} : Drop{0, 0, 0, 1.f};
}
// v[i] (column 8 g + FIRST + i of a row whose groups start at `group`) dropped or
// scaled; a dropped element is 0 whatever it held.
template <int N>
__device__ __forceinline__ void drop_n(const Drop& d, uint64_t group, int first, float (&v)[N]) {
  const uint4 r = philox(group, d.offset, d.key);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  if constexpr (N == 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (w[i / 2] >> (16 * (i & 1)) & 0xFFFFu) >= d.t ? v[i] * d.scale : 0.f;
  } else if constexpr (N == 4) {
    const uint32_t a = first ? w[2] : w[0], b = first ? w[3] : w[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = ((i < 2 ? a : b) >> (16 * (i & 1)) & 0xFFFFu) >= d.t ? v[i] * d.scale : 0.f;
  } else {
    static_assert(N == 1, "1, 4 or 8 columns");
    const uint32_t lo = first & 2 ? w[1] : w[0], hi = first & 2 ? w[3] : w[2];
    v[0] = ((first & 4 ? hi : lo) >> (16 * (first & 1)) & 0xFFFFu) >= d.t ? v[0] * d.scale : 0.f;
  }
}

// ---- activations.  FAST: for results of 16 bits, exponentials by the hardware's
// 2^x alone (within 2 |x| half steps of fp32) and a shorter series for the normal
// distribution; otherwise within about a step of fp32.
// exp(-x), x >= 0
template <bool FAST>
__device__ __forceinline__ float exp_minus(float x) {
  constexpr float kHi = 1.44269502162933349609375f, kLo = 1.925963033500011e-8f;  // log2 e in two parts
  if constexpr (FAST) {
    return __builtin_amdgcn_exp2f(x * -kHi);
  } else {
    // 2^-(n + f), n whole: the hardware's 2^-f, f in [-1/2, 1/2]
    x = fminf(x, 200.f);
    const float n = __builtin_rintf(x * kHi);
    const float f = fmaf(x, kLo, fmaf(x, kHi, -n));
    return __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f(-f), -(int)n);
  }
}
// 1 / d, d in [1, 2] or larger
template <bool FAST>
__device__ __forceinline__ float recip(float d) {
  const float q = __builtin_amdgcn_rcpf(d);
  return FAST ? q : fmaf(q, fmaf(-d, q, 1.0f), q);
}
// The sigmoid of g and 1 minus it, from t = exp(-|g|).
struct Sigm {
  float at, neg;
};
__device__ __forceinline__ Sigm sigm(float g) {
  const float t = exp_minus<false>(fabsf(g)), r = recip<false>(1.0f + t), tr = t * r;
  return g < 0.f ? Sigm{tr, r} : Sigm{r, tr};
}
// 1 / (1 + 2^x), which is what 2^x's overflow makes of it, 0, for large x
__device__ __forceinline__ float inv_1p_exp2(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x));
}
// The normal distribution's upper tail Q(z) = erfc(z / sqrt 2) / 2 and exp(-z^2 / 2)
// for z >= 0: Q = exp(-z^2 / 2) m(z), where m falls slowly from 1/2 like 1 / z, so
// m = t P(t) with t = 1 / (1 + c z) and P a polynomial fitted to m for the least
// relative error on [0, 16] (with the constants as rounded to fp32 8.6e-6 with six
// terms, 1.06e-7 with nine).  The tail keeps
// its relative precision, which 1 - erf would lose.
struct Tail {
  float t, p, e;  // Q = t p e
};
template <bool FAST>
__device__ __forceinline__ Tail tail(float z) {
  if constexpr (FAST) {
    const float t = __builtin_amdgcn_rcpf(fmaf(0.46f, z, 1.0f));
    const float e = __builtin_amdgcn_exp2f(z * z * -0.72134752044448170367f);
    float p = fmaf(0.0722274631f, t, -0.236543089f);
    p = fmaf(p, t, 0.177799612f);
    p = fmaf(p, t, 0.116107389f);
    p = fmaf(p, t, 0.18706657f);
    p = fmaf(p, t, 0.183346346f);
    return Tail{t, p, e};
  } else {
    const float t = recip<false>(fmaf(0.26f, z, 1.0f));
    const float s = z * z, lo = fmaf(z, z, -s);  // z^2 in two parts
    const float e0 = exp_minus<false>(0.5f * s), e = fmaf(e0, -0.5f * lo, e0);
    float p = fmaf(0.0294354856f, t, -0.147663906f);
    p = fmaf(p, t, 0.240891442f);
    p = fmaf(p, t, -0.138905317f);
    p = fmaf(p, t, 0.152682543f);
    p = fmaf(p, t, 0.0545273423f);
    p = fmaf(p, t, 0.102139488f);
    p = fmaf(p, t, 0.103141129f);
    p = fmaf(p, t, 0.103751779f);
    return Tail{t, p, e};
  }
}
constexpr float kPhi0 = 0.3989422804014327f;  // 1 / sqrt(2 pi)
constexpr float kTanhA = 1.5957691216057308f, kTanhB = 0.044715f;  // 2 sqrt(2 / pi)
constexpr float kLog2E = 1.4426950408889634f;

// act(h) and act'(h).  Every one has its limit at h = -inf (0) instead of the
// formula's NaN: where an exponential has gone to 0 the factor beside it is bounded.
// A NaN stays (it reaches the result through the exponential, or through h).
template <int ACT, bool FAST>
__device__ __forceinline__ float act_of(float h) {
  if constexpr (ACT == FP8SG_ACT_RELU) {
    return h <= 0.f ? 0.f : h;
  } else if constexpr (ACT == FP8SG_ACT_SILU) {
    if constexpr (FAST) return fmaxf(h, -150.f) * inv_1p_exp2(h * -kLog2E);
    return (h < -150.f ? -150.f : h) * sigm(h).at;
  } else if constexpr (ACT == FP8SG_ACT_GELU) {  // max(h, 0) - |h| Q(|h|)
    if constexpr (FAST) {
      const float z = fabsf(h);
      const Tail q = tail<true>(z);
      return fmaf(-(fminf(z, 16.f) * q.t), q.p * q.e, fmaxf(h, 0.f));
    }
    const float z = fminf(fabsf(h), 16.f);
    const Tail q = tail<false>(z);
    const float zq = z * (q.p * q.t * q.e);
    return h <= 0.f ? -zq : h - zq;
  } else if constexpr (ACT == FP8SG_ACT_GELU_TANH) {
    if constexpr (FAST)
      return fmaxf(h, -16.f) * inv_1p_exp2(h * fmaf(h * h, -kLog2E * kTanhA * kTanhB, -kLog2E * kTanhA));
    const float c = h < -16.f ? -16.f : h;
    return c * sigm(kTanhA * fmaf(kTanhB * c * c, c, c)).at;
  } else {
    return h;
  }
}
template <int ACT, bool FAST>
__device__ __forceinline__ float slope_of(float h) {
  if constexpr (ACT == FP8SG_ACT_SILU) {  // s (1 + h (1 - s))
    const float c = __builtin_amdgcn_fmed3f(h, -150.f, 150.f);
    if constexpr (FAST) {
      const float s = inv_1p_exp2(h * -kLog2E);
      return s * fmaf(c, 1.0f - s, 1.0f);
    }
    const Sigm s = sigm(c);
    return h != h ? h : s.at * fmaf(c, s.neg, 1.0f);
  } else if constexpr (ACT == FP8SG_ACT_GELU) {  // Q(z) - z phi(z) at -z, 1 minus it at z
    if constexpr (FAST) {
      const float z = fabsf(h);
      const Tail q = tail<true>(z);
      const float d = q.e * fmaf(q.t, q.p, -kPhi0 * fminf(z, 16.f));
      return h <= 0.f ? d : 1.0f - d;
    }
    const float z = fminf(fabsf(h), 16.f);
    const Tail q = tail<false>(z);
    const float d = q.e * fmaf(q.t, q.p, -kPhi0 * z);
    return h != h ? h : h <= 0.f ? d : 1.0f - d;
  } else if constexpr (ACT == FP8SG_ACT_GELU_TANH) {  // s (1 + h (1 - s) 2 u'(h))
    const float c = __builtin_amdgcn_fmed3f(h, -16.f, 16.f), cc = c * c;
    if constexpr (FAST) {
      const float s = inv_1p_exp2(h * fmaf(h * h, -kLog2E * kTanhA * kTanhB, -kLog2E * kTanhA));
      return s * fmaf(c * (1.0f - s), fmaf(cc, 3.f * kTanhA * kTanhB, kTanhA), 1.0f);
    }
    const Sigm s = sigm(kTanhA * fmaf(kTanhB * cc, c, c));
    return h != h ? h : s.at * fmaf(s.neg * kTanhA * c, fmaf(3.f * kTanhB, cc, 1.0f), 1.0f);
  } else {
    return 1.0f;
  }
}
// The gradient g behind act at h.  relu selects: an inactive unit passes exactly 0,
// where a product would make a NaN of an infinity.
template <int ACT, bool FAST>
__device__ __forceinline__ float through(float g, float h) {
  if constexpr (ACT == FP8SG_ACT_RELU) return h <= 0.f ? 0.f : g;
  return g * slope_of<ACT, FAST>(h);
}
// f(integral constant of the activation): one branch for a whole group of values
template <class F>
__device__ __forceinline__ void by_act(int act, F f) {
  switch (act) {
    case FP8SG_ACT_RELU: f(std::integral_constant<int, FP8SG_ACT_RELU>{}); break;
    case FP8SG_ACT_SILU: f(std::integral_constant<int, FP8SG_ACT_SILU>{}); break;
    case FP8SG_ACT_GELU: f(std::integral_constant<int, FP8SG_ACT_GELU>{}); break;
    case FP8SG_ACT_GELU_TANH: f(std::integral_constant<int, FP8SG_ACT_GELU_TANH>{}); break;
    default: break;
  }
}

// ---- elements of a type known at run time (one branch a group), at a byte address
__device__ __forceinline__ int esize(int type) { return type == FP8SG_OUT_F32 ? 4 : 2; }
template <int N>
struct Raw {  // N elements as loaded: N dwords of fp32, N / 2 of 16 bits
  uint32_t w[N];
};
// Elements past `n` read as 0.
template <int N>
__device__ __forceinline__ Raw<N> load_raw(const uint8_t* p, int n, int type) {
  Raw<N> r;
#pragma unroll
  for (int i = 0; i < N; ++i) r.w[i] = 0u;
  if (type == FP8SG_OUT_F32) {
    const float* q = reinterpret_cast<const float*>(p);
    if constexpr (N == 8) {
      if (n >= 8) {
        const u32x4 a = ld_any<false>(q), b = ld_any<false>(q + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[i] = a[i], r.w[4 + i] = b[i];
        return r;
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) r.w[i] = __float_as_uint(q[i]);
  } else {
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
    if constexpr (N == 8) {
      if (n >= 8) {
        const u32x4 a = ld_any<false>(q);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[i] = a[i];
        return r;
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) r.w[i / 2] |= (uint32_t)q[i] << (16 * (i & 1));
  }
  return r;
}
template <int N>
__device__ __forceinline__ void raw_values(const Raw<N>& r, int type, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (type == FP8SG_OUT_F32) v[i] = __uint_as_float(r.w[i]);
    else if (type == FP8SG_OUT_F16) v[i] = (i & 1) ? in_hi<true>(r.w[i / 2]) : in_lo<true>(r.w[i / 2]);
    else v[i] = (i & 1) ? in_hi<false>(r.w[i / 2]) : in_lo<false>(r.w[i / 2]);
  }
}
template <int N, int T, bool S>
__device__ __forceinline__ void store_t(uint8_t* p, int n, const float (&v)[N]) {
  Elem<T>* q = reinterpret_cast<Elem<T>*>(p);
  if constexpr (N == 8) {
    store8<T, S>(q, n, v);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) q[i] = from_f32<T>(v[i]);
  }
}
// S: non-temporal
template <int N, bool S>
__device__ __forceinline__ void store_n(uint8_t* p, int n, int type, const float (&v)[N]) {
  if (type == FP8SG_OUT_BF16) store_t<N, FP8SG_OUT_BF16, S>(p, n, v);
  else if (type == FP8SG_OUT_F16) store_t<N, FP8SG_OUT_F16, S>(p, n, v);
  else store_t<N, FP8SG_OUT_F32, S>(p, n, v);
}

// What a kernel's epilogue may meet, so that small kernels carry no code for the
// rest.  FAST: see above; TAIL: rows that end inside a group of columns; NT: results
// that leave with non-temporal stores.
template <bool FAST_, bool TAIL_, bool NT_>
struct EpiMode {
  static constexpr bool FAST = FAST_, TAIL = TAIL_, NT = NT_;
};

// Where a lane's N columns of a row lie in each matrix, and in the generator's
// sequence; from row to row by additions (products of 64 bits run at a quarter of the
// vector rate, and took as long as the activation).
struct EpiAt {
  uint8_t *c, *pre;
  const uint8_t* res;
  uint64_t group;
  __device__ __forceinline__ EpiAt(const EpilogueArgs& e, int64_t m, int64_t n) {
    const int es = esize(e.type);
    c = reinterpret_cast<uint8_t*>(e.C) + (m * e.ldc + n) * es;
    pre = reinterpret_cast<uint8_t*>(e.pre) + (m * e.N + n) * es;
    res = reinterpret_cast<const uint8_t*>(e.residual) + (m * e.ldr + n) * es;
    group = (uint64_t)m * (uint64_t)((e.N + 7) >> 3) + (uint64_t)(n >> 3);
  }
  __device__ __forceinline__ void down(const EpilogueArgs& e, int rows) {
    const int es = esize(e.type) * rows;
    c += e.ldc * es;
    pre += e.N * es;
    res += e.ldr * es;
    group += (uint64_t)rows * (uint64_t)((e.N + 7) >> 3);
  }
};

// The epilogue of U rows, 8 apart, of N columns: accumulators and their factor alpha,
// the columns' bias and the residual as loaded.  `first`: the first column mod 8;
// `cnt`: columns that exist; `rows`: of the U, those with 8 u < rows exist.
template <int U, int N, class Mode>
__device__ __forceinline__ void epilogue_rows(const EpilogueArgs& e, const Drop& d, float (&v)[U][N], float alpha,
                                              const float (&bias)[N], const Raw<N> (&res)[U], const EpiAt& at,
                                              int first, int cnt, int rows) {
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < N; ++i) v[u][i] = fmaf(v[u][i], alpha, bias[i]);
  const int es8 = 8 * esize(e.type);
  if (e.pre) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (8 * u >= rows) break;
      uint8_t* to = at.pre + u * (e.N * es8);
      if (Mode::NT && e.stream) store_n<N, true>(to, cnt, e.type, v[u]);
      else store_n<N, false>(to, cnt, e.type, v[u]);
    }
  }
  by_act(e.act, [&](auto a) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < N; ++i) v[u][i] = act_of<decltype(a)::value, Mode::FAST>(v[u][i]);
  });
  if (e.drop.rng) {
    const uint64_t step = 8 * (uint64_t)((e.N + 7) >> 3);
#pragma unroll
    for (int u = 0; u < U; ++u) drop_n<N>(d, at.group + u * step, first, v[u]);
  }
  if (e.residual) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float r[N];
      raw_values(res[u], e.type, r);
#pragma unroll
      for (int i = 0; i < N; ++i) v[u][i] += r[i];
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (8 * u >= rows) break;
    uint8_t* to = at.c + u * (e.ldc * es8);
    if (Mode::NT && e.stream) store_n<N, true>(to, cnt, e.type, v[u]);
    else store_n<N, false>(to, cnt, e.type, v[u]);
  }
}
template <int N, bool TAIL = true>
__device__ __forceinline__ void load_bias(const EpilogueArgs& e, int64_t n, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
  if (e.bias && n < e.N)
    raw_values(load_raw<N>(reinterpret_cast<const uint8_t*>(e.bias) + n * esize(e.bias_type),
                           TAIL && e.N - n < N ? (int)(e.N - n) : N, e.bias_type),
               e.bias_type, v);
}
// N columns whose inputs were not loaded ahead
template <int N, bool FAST>
__device__ __forceinline__ void epilogue_at(const EpilogueArgs& e, float (&v)[N], int64_t m, int64_t n) {
  if (m >= e.M || n >= e.N) return;
  const int cnt = e.N - n < N ? (int)(e.N - n) : N;
  const EpiAt at(e, m, n);
  float b[N], w[1][N];
  load_bias<N>(e, n, b);
  Raw<N> res[1] = {};
  if (e.residual) res[0] = load_raw<N>(at.res, cnt, e.type);
#pragma unroll
  for (int i = 0; i < N; ++i) w[0][i] = v[i];
  epilogue_rows<1, N, EpiMode<FAST, true, false>>(e, drop_of(e.drop), w, 1.0f, b, res, at, (int)(n & 7), cnt, 1);
}

// The lane's number, taken behind the main loop: nothing for that to keep.
__device__ __forceinline__ int lane_anew() {
  int lane = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
  asm volatile("" : "+v"(lane));
  return lane;
}

// The epilogue of a wave's 16 TM x 64 sub-tile with origin (m0, n0), held as 16 x 16
// blocks of the matrix instruction's layout (lane: row lane % 16, columns 4 (lane /
// 16) .. + 3 of a block).  The accumulators go through 16 KB of LDS that belong to
// the wave alone, 64 rows at a time in fp32, so no wave waits for another, and a
// lane gets eight consecutive columns of a row: residual and results then move 16
// bytes a lane in whole 128-byte lines (in the blocks' own layout a lane's four
// columns would be 8 bytes of a line that 16 rows share), the generator's eight
// elements are one lane's, and the activation is code for 8 values in a loop, not
// for the tile's 128 a lane.  The next row group's residual is loaded ahead.  us of an
// FP8 product of 8192 x 14336 x 4096, 335 without an epilogue: bias 341, relu 344, silu
// 357, gelu 384, gelu and h kept 406, residual 418, residual and dropout 438: in each
// of its seven rounds of tiles all units come here together, and what the memory and
// the vector unit then take no product hides.
// bias: of the lane's columns (load_bias<8> of n0 + 8 (lane % 8)); alpha: the
// product's factor; scale(c, i, j): other factors on block (i, j).
constexpr int kWaveEpilogueLds = 64 * 64 * 4;  // (with fewer than 64 rows, 256 bytes a row)
template <int TM, class Mode, int kU, class Scale>
__device__ __forceinline__ void wave_epilogue(const EpilogueArgs& e, v4f (&acc)[TM][4], uint8_t* lds, int64_t m0,
                                              int64_t n0, const float (&bias)[8], float alpha, Scale scale) {
  const int lane = lane_anew();
  const int cc = lane & 7, lr = lane >> 3;
  const int64_t n = n0 + 8 * cc;
  const int cnt = n >= e.N ? 0 : Mode::TAIL && e.N - n < 8 ? (int)(e.N - n) : 8;
  // rows of the sub-tile that exist, counted from the lane's first
  const int left = (int)(e.M - m0 < 16 * TM ? e.M - m0 : 16 * TM) - lr;
  float* tile = reinterpret_cast<float*>(lds);
  // 16-byte chunk c of row r at c ^ r % 16: the 16 rows that a store writes, and the
  // even chunks of two rows that a load reads, fall on different banks
  auto place = [&](int r, int c) { return tile + r * 64 + ((c ^ (r & 15)) << 2); };
  const Drop d = drop_of(e.drop);
  EpiAt at(e, m0 + lr, n);
  Raw<8> res[kU] = {};
  auto load_res = [&](int r0) {  // of rows r0 + 8 u, seen from `at`
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (e.residual && cnt > 0 && r0 + 8 * u < left)
        res[u] = load_raw<8>(at.res + u * (e.ldr * 8 * esize(e.type)), Mode::TAIL ? cnt : 8, e.type);
  };
  load_res(0);
  static_for<(TM + 3) / 4>([&](auto half) {
    constexpr int h = 4 * decltype(half)::value;
#pragma unroll
    for (int i = h; i < TM && i < h + 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v4f c = acc[i][j];
        scale(c, i, j);
        *reinterpret_cast<v4f*>(place(16 * (i - h) + (lane & 15), 4 * j + (lane >> 4))) = c;
      }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    // (the last half of a 7-block tile has 48 rows; what LDS holds behind them is not stored)
#pragma unroll 1
    for (int r0 = 0; r0 < (TM < 4 ? 16 * TM : 64); r0 += 8 * kU) {
      float v[kU][8];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int r = r0 + 8 * u + lr;
        const v4f a = *reinterpret_cast<const v4f*>(place(r, 2 * cc));
        const v4f b = *reinterpret_cast<const v4f*>(place(r, 2 * cc + 1));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[u][i] = a[i], v[u][4 + i] = b[i];
      }
      const int row = 16 * h + r0;
      if (cnt > 0)
        epilogue_rows<kU, 8, Mode>(e, d, v, alpha, bias, res, at, 0, Mode::TAIL ? cnt : 8, left - row);
      at.down(e, 8 * kU);
      load_res(row + 8 * kU);  // the next rows' residual, while they are read and computed
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  });
}

}  // namespace fp8sg
