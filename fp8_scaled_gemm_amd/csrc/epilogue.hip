// The backward step of a product's epilogue (gh = drop(gy) act'(pre), the bias's
// gradient, the largest |gh|), and dropout on its own.  Elementwise and bound by
// memory.
#include "epilogue.hpp"

namespace fp8sg {
namespace {

constexpr int kBlock = 256;  // threads of a block; of the backward step's:
constexpr int kBwd = 512;
constexpr int kRows = 2;  // rows a thread of the backward step has in flight (fp32: one)

// ---- backward.  A block owns a strip of 8 L columns (a thread 8 of them); the
// blocks of a strip, its parts, take its rows in turns of kRows rows for each of their
// 512 / L row groups, so that all blocks in flight read one short run of rows (each a
// run of its own: 8192 x 4096, bf16, 54 -> 46 us).  Each thread adds up its columns
// in fp32, lanes and waves join at the end, and with several parts each leaves a row
// of partial sums that k_bias_join adds in a fixed order (no atomics: a repeated call
// gives the same bits).  Two blocks fit a compute unit (87 registers: five waves a
// SIMD; three of fp32's 72), so 512 of a launch's at most 1024 (a record's slots) are
// in flight, the first half of the parts and then the second.  us for 8192 x 14336 bf16 with gelu and gb, 705 MB,
// past the caches: 132 (5.3 TB/s; a copy 5.2), of which gelu 7, gb 2; 4 rows and 256
// threads a block 136; cached accesses 146.  fp32 takes cached ones at any size: its
// lanes' 16-byte halves of 32 bytes meet in the caches (4096 x 14336 142, non-temporal 153).
template <int T, bool S>
__global__ __launch_bounds__(kBwd, 2) void k_epilogue_bwd(EpilogueBwdArgs p) {
  constexpr bool kFast = T != FP8SG_OUT_F32;
  constexpr int kU = kFast ? kRows : kRows / 2;
  __shared__ float red[kBwd / kWave][8 * kWave];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int L = p.lanes, R = kBwd / L, cl = tid & (L - 1), rl = tid / L;
  const Drop d = drop_of(p.drop);
  const uint64_t groups = (uint64_t)((p.N + 7) >> 3);
  uint32_t amax = 0;  // packed 16-bit magnitudes
  for (int64_t task = blockIdx.x; task < p.strips * p.parts; task += gridDim.x) {
    const int64_t part = task / p.strips, strip = task - part * p.strips;
    const int64_t c = (strip * L + cl) * 8;
    const int n = c < p.N ? left8(p.N, c) : 0;
    float sum[8] = {};
    if (n > 0) {
      for (int64_t r0 = part * kU * R + rl; r0 < p.M; r0 += (int64_t)p.parts * kU * R) {
        Row8<T> g[kU], h[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int64_t r = r0 + u * R;
          g[u].zero();
          h[u].zero();
          if (r < p.M) {
            g[u] = load_row8<T, S>(reinterpret_cast<const Elem<T>*>(p.gy) + r * p.N + c, n);
            if (p.act != FP8SG_ACT_NONE)
              h[u] = load_row8<T, S>(reinterpret_cast<const Elem<T>*>(p.pre) + r * p.N + c, n);
          }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int64_t r = r0 + u * R;
          if (r >= p.M) break;
          float v[8], x[8];
          g[u].values(v);
          by_act(p.act, [&](auto a) {
            h[u].values(x);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = through<decltype(a)::value, kFast>(v[i], x[i]);
          });
          if (p.drop.rng) drop_n<8>(d, (uint64_t)r * groups + (uint64_t)(c >> 3), 0, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[i] += v[i];
          if constexpr (T == FP8SG_OUT_F32) {
            if (p.gh) store8<T, S>(reinterpret_cast<Elem<T>*>(p.gh) + r * p.N + c, n, v);
          } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              w[i] = (uint32_t)from_f32<T>(v[2 * i]) | ((uint32_t)from_f32<T>(v[2 * i + 1]) << 16);
              amax = pmax(amax, w[i] & 0x7FFF7FFFu);
            }
            if (p.gh) {
              uint16_t* to = reinterpret_cast<uint16_t*>(p.gh) + r * p.N + c;
              if (n >= 8) {
                st_any<S>(to, u32x4{w[0], w[1], w[2], w[3]});
              } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  if (i < n) to[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
              }
            }
          }
        }
      }
    }
    if (p.gb) {
      for (int o = L; o < kWave; o *= 2)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += __shfl_xor(sum[i], o, kWave);
      __syncthreads();  // red may hold an earlier strip's sums
      if (lane < L)
#pragma unroll
        for (int i = 0; i < 8; ++i) red[wave][8 * lane + i] = sum[i];
      __syncthreads();
      for (int i = tid; i < 8 * L; i += kBwd) {
        const int64_t col = strip * L * 8 + i;
        if (col >= p.N) continue;
        const float v = ((red[0][i] + red[1][i]) + (red[2][i] + red[3][i])) +
                        ((red[4][i] + red[5][i]) + (red[6][i] + red[7][i]));
        if (p.parts > 1) {
          p.part[part * p.N + col] = v;
        } else {
          const float one[1] = {v};
          store_n<1, false>(reinterpret_cast<uint8_t*>(p.gb) + col * esize(p.bias_type), 1, p.bias_type, one);
        }
      }
    }
  }
  if (p.rec) {  // this block's slot of the record, as the amax kernel leaves it
    const uint32_t bits = block_max_u32<kBwd>(absmax_bits<T == FP8SG_OUT_F16>(amax));
    if (tid == 0) {
      p.rec->_part[blockIdx.x] = bits;
      if (blockIdx.x == 0) p.rec->_nparts = gridDim.x;
    }
    if (blockIdx.x == 0)
      for (int i = gridDim.x + tid; i < FP8SG_AMAX_PARTS; i += kBwd) p.rec->_part[i] = 0;
  }
}

// gb[n] = the sum of `parts` partial rows: 16 columns a block, a sixteenth of the
// rows for each of 16 threads a column (with 64 columns a block too few blocks share
// the loads' latency: 4096 x 4096 with gb 24.8 -> 24.4 us).
constexpr int kJoin = 16;
__global__ __launch_bounds__(kBlock) void k_bias_join(const float* part, int parts, int64_t N, void* gb, int type) {
  __shared__ float red[kBlock / kJoin][kJoin];
  const int c = threadIdx.x % kJoin, g = threadIdx.x / kJoin;
  const int64_t n = (int64_t)blockIdx.x * kJoin + c;
  float s = 0.f;
  if (n < N)
#pragma unroll 8
    for (int r = g; r < parts; r += kBlock / kJoin) s += part[r * N + n];
  red[g][c] = s;
  __syncthreads();
  if (g == 0 && n < N) {
    float one[1] = {0.f};
#pragma unroll
    for (int i = 0; i < kBlock / kJoin; ++i) one[0] += red[i][c];
    store_n<1, false>(reinterpret_cast<uint8_t*>(gb) + n * esize(type), 1, type, one);
  }
}

// Strips and parts of an M x N gradient.
struct Split {
  int lanes;
  int64_t strips, parts;
};
Split split_of(int64_t M, int64_t N) {
  Split s{1, 0, 1};
  // few rows: strips of 64 columns (128 bytes of 16-bit values), whose 64 row groups
  // take all rows, so nothing is left to join (64 x 256 with gb 7.5 -> 5.0 us)
  const bool few = M <= 256;
  while (s.lanes < (few ? 8 : kWave) && 8 * s.lanes < N) s.lanes *= 2;
  s.strips = (N + 8 * s.lanes - 1) / (8 * s.lanes);
  const int64_t turn = (int64_t)(kBwd / s.lanes) * kRows, turns = (M + turn - 1) / turn;
  // at most as many blocks as a record has slots
  if (s.strips && !few) s.parts = FP8SG_AMAX_PARTS / s.strips;
  if (s.parts > turns) s.parts = turns;
  if (s.parts < 1) s.parts = 1;
  return s;
}

// ---- dropout: a thread takes one group of eight columns, the generator's unit.
template <int T, bool S>
__global__ __launch_bounds__(kBlock) void k_dropout(DropoutArgs p) {
  const int64_t upr = (p.cols + 7) >> 3, units = p.rows * upr;
  const Drop d = drop_of(p.drop);
  for (int64_t blk = blockIdx.x; blk * kBlock < units; blk += gridDim.x) {
    // one 64-bit division a block, one 32-bit division a thread
    const int64_t i0 = blk * kBlock, r0 = i0 / upr;
    const uint32_t t = (uint32_t)(i0 - r0 * upr) + threadIdx.x, q = t / (uint32_t)upr;
    const int64_t row = r0 + q, c = (int64_t)(t - q * (uint32_t)upr) * 8;
    if (row >= p.rows) continue;
    const int n = left8(p.cols, c);
    float v[8];
    const Row8<T> x = load_row8<T, S>(reinterpret_cast<const Elem<T>*>(p.x) + row * p.ldx + c, n);
    Row8<T> r;
    if (p.residual) r = load_row8<T, S>(reinterpret_cast<const Elem<T>*>(p.residual) + row * p.ldr + c, n);
    x.values(v);
    if (p.drop.rng) drop_n<8>(d, (uint64_t)(i0 + threadIdx.x), 0, v);
    if (p.residual) {
      float a[8];
      r.values(a);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += a[i];
    }
    store8<T, S>(reinterpret_cast<Elem<T>*>(p.y) + row * p.ldy + c, n, v);
  }
}

}  // namespace

int64_t epilogue_ws_len(int64_t M, int64_t N) {
  // (of either form: with MXFP4 the step is part of the quantising pass)
  const int64_t a = split_of(M, N).parts, b = mx_epilogue_parts(M, N), parts = a > b ? a : b;
  return parts > 1 ? parts * N : 0;
}
int64_t epilogue_ws_need(int64_t M, int64_t N) { return split_of(M, N).parts > 1 ? epilogue_ws_len(M, N) : 0; }

hipError_t launch_epilogue_bwd(EpilogueBwdArgs a, hipStream_t stream) {
  if (a.N == 0) return hipSuccess;
  const Split s = split_of(a.M, a.N);
  a.lanes = s.lanes;
  a.parts = (int32_t)s.parts;
  a.strips = s.strips;
  const int64_t tasks = s.strips * s.parts;
  const dim3 grid((unsigned)(tasks < FP8SG_AMAX_PARTS ? tasks : FP8SG_AMAX_PARTS));
  const bool st = a.M * a.N * 6 >= kStreamBytes;
  hipError_t err = by_type(a.type, [&](auto t) {
    constexpr int T = decltype(t)::value;
    if constexpr (T != FP8SG_OUT_F32) {
      if (st) {
        hipLaunchKernelGGL((k_epilogue_bwd<T, true>), grid, dim3(kBwd), 0, stream, a);
        return hipGetLastError();
      }
    }
    hipLaunchKernelGGL((k_epilogue_bwd<T, false>), grid, dim3(kBwd), 0, stream, a);
    return hipGetLastError();
  });
  return err != hipSuccess || !a.gb || s.parts == 1 ? err : launch_bias_join(a, stream);
}

hipError_t launch_bias_join(const EpilogueBwdArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(k_bias_join, dim3((unsigned)((a.N + kJoin - 1) / kJoin)), dim3(kBlock), 0, stream, a.part,
                     a.parts, a.N, a.gb, a.bias_type);
  return hipGetLastError();
}

hipError_t launch_dropout(const DropoutArgs& a, hipStream_t stream) {
  const int64_t units = a.rows * ((a.cols + 7) / 8), e = a.type == FP8SG_OUT_F32 ? 4 : 2;
  if (units == 0) return hipSuccess;
  const int64_t blocks = (units + kBlock - 1) / kBlock;
  const dim3 grid((unsigned)(blocks < (1 << 22) ? blocks : (1 << 22)));
  const bool st = a.rows * a.cols * e * (a.residual ? 3 : 2) >= kStreamBytes;
  return by_type(a.type, [&](auto t) {
    constexpr int T = decltype(t)::value;
    if (st) hipLaunchKernelGGL((k_dropout<T, true>), grid, dim3(kBlock), 0, stream, a);
    else hipLaunchKernelGGL((k_dropout<T, false>), grid, dim3(kBlock), 0, stream, a);
    return hipGetLastError();
  });
}

}  // namespace fp8sg
