// MXFP4 quantisation along rows and / or columns, and the values of codes.
//
// For each block of 32 along the contraction: amax, its power-of-two scale,
// 32 codes of 4 bits.  Bound by memory: per element 2 bytes in (bf16) and
// 17/32 bytes out per direction.
#include "mx.hpp"

namespace fp8sg {
namespace {

// Running largest magnitudes as bit patterns: two 16-bit ones a dword, or fp32.
template <int T>
__device__ __forceinline__ uint32_t mag_max(uint32_t m, uint32_t w) {
  if constexpr (T == FP8SG_OUT_F32) {
    w &= 0x7FFFFFFFu;
    return w > m ? w : m;
  } else {
    return pmax(m, w & 0x7FFF7FFFu);
  }
}
// A 16-bit magnitude's fp32 bits (inf and NaN stay above every finite value).
template <int T>
__device__ __forceinline__ uint32_t mag_bits(uint32_t code) {
  if constexpr (T == FP8SG_OUT_BF16) return code << 16;
  else if constexpr (T == FP8SG_OUT_F16) return __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)code));
  else return code;
}
// Two elements to the byte SEL of a dword of codes.
template <int T, int SEL>
__device__ __forceinline__ uint32_t put_pair(uint32_t d, uint32_t pair, float scale) {
  typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
  typedef _Float16 h2 __attribute__((ext_vector_type(2)));
  if constexpr (T == FP8SG_OUT_BF16)
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(d, __builtin_bit_cast(bf2, pair), scale, SEL);
  else
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(d, __builtin_bit_cast(h2, pair), scale, SEL);
}
template <int SEL>
__device__ __forceinline__ uint32_t put_pair32(uint32_t d, uint32_t a, uint32_t b, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, __uint_as_float(a), __uint_as_float(b), scale, SEL);
}
// Eight elements of a row to a dword of codes.
template <int T>
__device__ __forceinline__ uint32_t row_codes(const Row8<T>& r, uint32_t s) {
  const float sc = scale_value(s);
  uint32_t d = 0;
  if constexpr (T == FP8SG_OUT_F32) {
    d = put_pair32<0>(d, r.w[0], r.w[1], sc);
    d = put_pair32<1>(d, r.w[2], r.w[3], sc);
    d = put_pair32<2>(d, r.w[4], r.w[5], sc);
    d = put_pair32<3>(d, r.w[6], r.w[7], sc);
  } else {
    d = put_pair<T, 0>(d, r.w[0], sc);
    d = put_pair<T, 1>(d, r.w[1], sc);
    d = put_pair<T, 2>(d, r.w[2], sc);
    d = put_pair<T, 3>(d, r.w[3], sc);
  }
  return s == 255u ? 0u : d;
}
// Column J of rows R .. R + 2 L - 1 to L bytes of codes (L = 2 or 4).
template <int T, int J, int R, int L, int N>
__device__ __forceinline__ uint32_t col_codes(const Row8<T> (&v)[N], float sc) {
  uint32_t d = 0;
  static_for<L>([&](auto bc) {
    constexpr int B = decltype(bc)::value, r = R + 2 * B;
    if constexpr (T == FP8SG_OUT_F32) {
      d = put_pair32<B>(d, v[r].w[J], v[r + 1].w[J], sc);
    } else {
      constexpr uint32_t sel = (J & 1) ? 0x07060302u : 0x05040100u;  // the column's half of two rows
      d = put_pair<T, B>(d, __builtin_amdgcn_perm(v[r + 1].w[J / 2], v[r].w[J / 2], sel), sc);
    }
  });
  return d;
}

struct MxQuantArgs {
  MxQuantJob job[2];
  uint32_t blocks0;  // blocks of job 0
  int32_t fit;
};

// A block quantises 32 G rows x 256 columns, read once: a wave holds 32 rows x
// 8 C columns, C = 2 RL lanes across, each with RL rows x 8 columns (RL = 16: one
// wave spans the 256 columns; RL = 4: four do).  Then
//   - a block along a row lies in four neighbouring lanes (two DPP steps give
//     its amax) and 32 lanes write a row's 128 bytes of codes;
//   - a block along a column lies in lanes C apart; a lane's codes go through
//     LDS, so that the columns' codes leave in runs of 16 G bytes.
// Scales of both directions are gathered in LDS in their stored order.
// Memory bound (both ways, bf16: 8192 x 14336 71 - 75 us, 4.8 - 5.1 TB/s; 14336 x 4096
// 45 - 52 us; 8192 x 4096 25 us; fp32, whose 128 elements a lane leave half the
// waves: 147 us, 4.05 TB/s; 80 us; 38 us).  G = 8, RL = 16 writes whole 128-byte lines
// with the fewest instructions; G = 2, RL = 4 gives small matrices four times the
// blocks and 16 times the waves (37 x 1001 fp32, both ways: 9.2 us with RL = 16; so,
// less than the call's 6.1 us on the host).
template <int T, int G, int RL, bool S>
__global__ __launch_bounds__(64 * G * (16 / RL), T == FP8SG_OUT_F32 && RL == 16 ? 2 : 4) void k_mxq(MxQuantArgs args) {
  constexpr int kRows = 32 * G, C = 2 * RL, kAcross = 32 / C, kThreads = 64 * G * kAcross;
  // column c's codes start at tcol(c); the 16-byte pieces (G = 8) or the
  // columns (G = 2) are shifted so that lanes 8 columns apart write to
  // different banks
  auto tcol = [](int c) { return G == 8 ? c * 128 : c * 32 + (c >> 3) * 16; };
  __shared__ __attribute__((aligned(16))) uint8_t tq[G == 8 ? 256 * 128 : 256 * 32 + 32 * 16];
  __shared__ __attribute__((aligned(16))) uint8_t rs[G * 256];  // row scales: G groups of 256 bytes
  __shared__ __attribute__((aligned(16))) uint8_t ts[G * 256];  // column scales: 8 groups of 32 G bytes

  const bool second = blockIdx.x >= args.blocks0;
  const MxQuantJob& j = args.job[second];
  const uint32_t blk = blockIdx.x - (second ? args.blocks0 : 0u);
  const int64_t nkc = mx_ktiles(j.cols), nkr = mx_ktiles(j.rows);
  const int64_t rt = blk / (uint32_t)nkc, ct = blk % (uint32_t)nkc;  // tile
  const int64_t r0 = rt * kRows, c0 = ct * 256;
  const bool fit = args.fit != 0;

  // group wg of 32 rows; rows RL rg .. of it; columns 8 cc .. of the tile
  const int tid = threadIdx.x, lane = tid & 63, wg = (tid >> 6) / kAcross, rg = lane / C;
  const int cc = (tid >> 6) % kAcross * C + lane % C;
  const int64_t c = c0 + 8 * cc, rw = r0 + 32 * wg + RL * rg;
  const Elem<T>* x = reinterpret_cast<const Elem<T>*>(j.x);
  Row8<T> v[RL];
#pragma unroll
  for (int i = 0; i < RL; ++i) {
    if (rw + i < j.rows && c < j.cols) {
      v[i] = load_row8<T, S>(x + (rw + i) * j.cols + c, left8(j.cols, c));
    } else {
      v[i].zero();
    }
  }

  if (j.q.q) {
    const bool blk_in = (c & ~31) < j.cols;  // this lane's block of 32 exists
#pragma unroll
    for (int i = 0; i < RL; ++i) {
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < Row8<T>::kW; ++e) m = mag_max<T>(m, v[i].w[e]);
      if constexpr (T != FP8SG_OUT_F32) m = (m & 0xFFFFu) > (m >> 16) ? (m & 0xFFFFu) : (m >> 16);
      m = quad_max(m);
      const uint32_t s = blk_in ? fp4_scale(mag_bits<T>(m), fit) : 127u;
      if (rw + i < j.rows) *reinterpret_cast<uint32_t*>(j.q.q + ((rw + i) * nkc + ct) * 128 + 4 * cc) = row_codes<T>(v[i], s);
      const int row = RL * rg + i;  // of the group
      if ((lane & 3) == 0)          // block cc / 4
        rs[wg * 256 + ((cc >> 3) * 16 + (row & 15)) * 4 + (row >> 4) * 2 + ((cc >> 2) & 1)] = (uint8_t)s;
    }
  }
  if (j.t.q) {
    constexpr int kM = Row8<T>::kW;
    uint32_t m[kM];
#pragma unroll
    for (int e = 0; e < kM; ++e) m[e] = 0u;
#pragma unroll
    for (int i = 0; i < RL; ++i)
#pragma unroll
      for (int e = 0; e < kM; ++e) m[e] = mag_max<T>(m[e], v[i].w[e]);
#pragma unroll
    for (int d = C; d < 64; d *= 2)
#pragma unroll
      for (int e = 0; e < kM; ++e) m[e] = mag_max<T>(m[e], (uint32_t)__shfl_xor((int)m[e], d, kWave));
    const bool blk_in = r0 + 32 * wg < j.rows;
    static_for<8>([&](auto jc) {
      constexpr int J = decltype(jc)::value;
      const uint32_t code = T == FP8SG_OUT_F32 ? m[J % kM] : ((J & 1) ? m[J / 2] >> 16 : m[J / 2] & 0xFFFFu);
      const uint32_t s = blk_in ? fp4_scale(mag_bits<T>(code), fit) : 127u;
      const float sc = scale_value(s);
      const int cl = 8 * cc + J;
      const int piece = G == 8 ? (wg ^ (cc & 7)) : wg;
      uint8_t* at = tq + tcol(cl) + piece * 16 + rg * (RL / 2);
      if constexpr (RL == 16) {
        const uint2 d = make_uint2(col_codes<T, J, 0, 4>(v, sc), col_codes<T, J, 8, 4>(v, sc));
        *reinterpret_cast<uint2*>(at) = s == 255u ? make_uint2(0, 0) : d;
      } else {
        *reinterpret_cast<uint16_t*>(at) = s == 255u ? (uint16_t)0 : (uint16_t)col_codes<T, J, 0, 2>(v, sc);
      }
      if (rg == 0)  // block wg of column cl: the tile's blocks are pairs 0 .. G / 2 - 1 here
        ts[(cl >> 5) * (G * 32) + ((wg >> 1) * 16 + (cl & 15)) * 4 + ((cl & 31) >> 4) * 2 + (wg & 1)] = (uint8_t)s;
    });
  }
  __syncthreads();
  if (j.q.q && tid < 16 * G && r0 + (tid >> 4) * 32 < j.rows)
    *reinterpret_cast<uint4*>(j.q.s + ((r0 / 32 + (tid >> 4)) * nkc + ct) * 256 + (tid & 15) * 16) =
        *reinterpret_cast<const uint4*>(rs + tid * 16);
  if (j.t.q) {
    // k-tile r0 / 256 of the transposed matrix, from byte (r0 % 256) / 2 on
    const int64_t kt = r0 >> 8, sub = (r0 & 255) >> 1;
#pragma unroll
    for (int p = 0; p < 256 * G / kThreads; ++p) {  // 256 columns x G pieces of 16 bytes
      const int id = p * kThreads + tid, cl = id / G, k = id % G;
      const int piece = G == 8 ? (k ^ ((cl >> 3) & 7)) : k;
      if (c0 + cl < j.cols)
        st16<S>(j.t.q + ((c0 + cl) * nkr + kt) * 128 + sub + k * 16, *reinterpret_cast<const uint4*>(tq + tcol(cl) + piece * 16));
    }
    // 8 groups of 32 columns, of each the bytes of the tile's block pairs
    if (tid < 16 * G) {
      const int grp = tid / (2 * G), w = tid % (2 * G);
      if (c0 + grp * 32 < j.cols)
        *reinterpret_cast<uint4*>(j.t.s + (((c0 >> 5) + grp) * nkr + kt) * 256 + ((r0 & 255) >> 6) * 64 + w * 16) =
            *reinterpret_cast<const uint4*>(ts + tid * 16);
    }
  }
}

// Rows only, for matrices too small for k_mxq's wide tiles to fill the chip: 8
// elements a thread, 8 rows x 256 columns a block (16 x 4096: 6.1 us in tiles of
// 16 rows a lane, 2.4 us so).
template <int T>
__global__ __launch_bounds__(256) void k_mxq_rows(MxQuantArgs args) {
  const MxQuantJob& j = args.job[0];
  const int64_t nk = mx_ktiles(j.cols);
  const int64_t r = (blockIdx.x / (uint32_t)nk) * 8ll + (threadIdx.x >> 5), ct = blockIdx.x % (uint32_t)nk;
  if (r >= j.rows) return;  // a half wave: its lanes' groups of four stay whole
  const int cc = threadIdx.x & 31;
  const int64_t c = ct * 256 + 8 * cc;
  const Row8<T> v = load_row8<T, false>(reinterpret_cast<const Elem<T>*>(j.x) + r * j.cols + c, left8(j.cols, c));
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < Row8<T>::kW; ++e) m = mag_max<T>(m, v.w[e]);
  if constexpr (T != FP8SG_OUT_F32) m = (m & 0xFFFFu) > (m >> 16) ? (m & 0xFFFFu) : (m >> 16);
  m = quad_max(m);
  const uint32_t s = (c & ~31) < j.cols ? fp4_scale(mag_bits<T>(m), args.fit != 0) : 127u;
  *reinterpret_cast<uint32_t*>(j.q.q + (r * nk + ct) * 128 + 4 * cc) = row_codes<T>(v, s);
  if ((cc & 3) == 0) j.q.s[mx_scale_off(r, ct * 8 + (cc >> 2), nk)] = (uint8_t)s;
}

// One thread per 8 values: 4 bytes of codes, their block's scale.  Bound by the
// values' writes (14336 x 4096 to bf16: 26.5 - 28.6 us, 5.2 - 5.6 TB/s; to fp32 48 us,
// 5.5; 8192 x 14336: 68 us, 4.3 TB/s, to fp32 111, 4.8).
template <int T>
__global__ __launch_bounds__(256) void k_mx_dequant(mxfp4_operand m, int64_t rows, int64_t k, Elem<T>* y) {
  const int64_t nk = mx_ktiles(k), upr = (k + 7) / 8, total = rows * upr;
  for (int64_t i0 = (int64_t)blockIdx.x * 256; i0 < total; i0 += (int64_t)gridDim.x * 256) {
    const int64_t rb = i0 / upr;  // uniform
    const uint32_t t = (uint32_t)(i0 - rb * upr) + threadIdx.x, dr = t / (uint32_t)upr;
    const int64_t r = rb + dr, u = t - dr * (uint32_t)upr;
    if (r >= rows) continue;
    const float sc = scale_value(m.s[mx_scale_off(r, u / 4, nk)]);
    const uint32_t q = *reinterpret_cast<const uint32_t*>(m.q + r * nk * 128 + 4 * u);
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 1);
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 3);
    const float v[8] = {a[0] * sc, a[1] * sc, b[0] * sc, b[1] * sc, c[0] * sc, c[1] * sc, d[0] * sc, d[1] * sc};
    store8<T, false>(y + r * k + 8 * u, left8(k, 8 * u), v);
  }
}

// Blocks of 256 threads for n items, each thread striding over the rest.
unsigned grid_for(int64_t n) {
  const int64_t b = (n + 255) / 256;
  return (unsigned)(b < (1 << 20) ? b : (1 << 20));
}
// Tiles of a job: column tiles cover the padded columns; the row tiles the
// rows, and with a transposed copy the padding of its last k-tile too.
template <int G>
int64_t tiles_of(const MxQuantJob& j) {
  if (j.rows == 0 || j.cols == 0 || (!j.q.q && !j.t.q)) return 0;
  const int64_t rt = j.t.q ? mx_ktiles(j.rows) * (8 / G) : (j.rows + 32 * G - 1) / (32 * G);
  return rt * mx_ktiles(j.cols);
}

}  // namespace

hipError_t launch_mx_quantize(const MxQuantJob* jobs, int n, int type, bool fit, hipStream_t stream) {
  MxQuantArgs a{};
  int64_t bytes = 0, wide = 0;
  for (int i = 0; i < n; ++i) {
    a.job[i] = jobs[i];
    wide += tiles_of<8>(jobs[i]);
    bytes += jobs[i].rows * jobs[i].cols * (type == FP8SG_OUT_F32 ? 5 : 3);
  }
  a.fit = fit;
  const int cus = device_cus();
  return by_type(type, [&](auto t) {
    constexpr int T = decltype(t)::value;
    auto launch = [&](auto gc, auto rl, auto st) {
      constexpr int G = decltype(gc)::value, RL = decltype(rl)::value;
      const int64_t b0 = tiles_of<G>(a.job[0]), b1 = n > 1 ? tiles_of<G>(a.job[1]) : 0;
      if (b0 + b1 == 0) return hipSuccess;
      a.blocks0 = (uint32_t)b0;
      hipLaunchKernelGGL((k_mxq<T, G, RL, decltype(st)::value>), dim3((unsigned)(b0 + b1)), dim3(64 * G * (16 / RL)), 0,
                         stream, a);
      return hipGetLastError();
    };
    if (wide < cus && n == 1 && !a.job[0].t.q) {
      const int64_t blocks = (a.job[0].rows + 7) / 8 * mx_ktiles(a.job[0].cols);
      if (blocks == 0 || !a.job[0].q.q) return hipSuccess;
      hipLaunchKernelGGL((k_mxq_rows<T>), dim3((unsigned)blocks), dim3(256), 0, stream, a);
      return hipGetLastError();
    }
    // a wide tile per compute unit, or the narrow ones
    typedef std::integral_constant<int, 16> C16;
    typedef std::integral_constant<int, 8> C8;
    if (wide < cus) return launch(std::integral_constant<int, 2>{}, std::integral_constant<int, 4>{}, std::false_type{});
    if (bytes >= kStreamBytes) return launch(C8{}, C16{}, std::true_type{});
    return launch(C8{}, C16{}, std::false_type{});
  });
}

hipError_t launch_mx_dequantize(const mxfp4_operand& m, int64_t rows, int64_t k, void* y, int type, hipStream_t stream) {
  if (rows == 0 || k == 0) return hipSuccess;
  return by_type(type, [&](auto t) {
    constexpr int T = decltype(t)::value;
    const dim3 grid(grid_for(rows * ((k + 7) / 8)));
    hipLaunchKernelGGL((k_mx_dequant<T>), grid, dim3(256), 0, stream, m, rows, k, reinterpret_cast<Elem<T>*>(y));
    return hipGetLastError();
  });
}

}  // namespace fp8sg
