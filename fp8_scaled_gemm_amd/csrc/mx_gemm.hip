// Product of two MXFP4 matrices on the matrix cores:
//   C[M,N] = out(sum_k A[m,k] * B[n,k])
// v_mfma_scale_f32_16x16x128_f8f6f4 with both operands e2m1: lane l holds row
// l % 16 of a fragment and the 32 consecutive k of block l / 16, and one scale
// byte for that block; products and the sums inside a block are exact, sums
// over blocks are fp32.
#include <algorithm>
#include <atomic>

#include "epilogue.hpp"
#include "gemm_kernels.hpp"  // LDS staging, tile order
#include "mx.hpp"

namespace fp8sg {
namespace {

// A problem with an epilogue behind the product (epilogue.hpp) has its result's
// type at run time; OUT then only says whether it is fp32 or has 16 bits.
template <class Prob>
constexpr bool kEpi = std::is_same_v<Prob, MxGemmEpiProblem>;
template <int OUT>
constexpr bool kFast = OUT != FP8SG_OUT_F32;

// One 16 x 16 x 128 product of e2m1 fragments; SA / SB: which byte of sa / sb is
// the lane's scale.  The first operand's rows become the lane's four
// accumulators, so it is the one whose rows are C's columns.
template <int SB, int SA>
__device__ __forceinline__ v4f mfma4(uint4 b, uint4 a, v4f c, uint32_t sb, uint32_t sa) {
  const v8i vb = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  const v8i va = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(vb, va, c, 4, 4, SB, (int)sb, SA, (int)sa);
}

// Four consecutive outputs of a row of N columns from column n on, at whatever
// address the row has (the hardware takes any; unless FOURS, N % 4 == 0, the
// row's end goes by element: 1000 x 1032 x 2085 8.9 us with FOURS, 9.8 without).
template <int OUT, bool FOURS>
__device__ __forceinline__ void put4(Elem<OUT>* row, int64_t n, int64_t N, v4f v) {
  if (FOURS ? n < N : n + 4 <= N) {
    if constexpr (OUT == FP8SG_OUT_F32) {
      st_any<false>(row + n, __builtin_bit_cast(u32x4, v));
    } else {
      typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
      *reinterpret_cast<u32x2_any*>(row + n) =
          u32x2_any{(uint32_t)from_f32<OUT>(v[0]) | ((uint32_t)from_f32<OUT>(v[1]) << 16),
                    (uint32_t)from_f32<OUT>(v[2]) | ((uint32_t)from_f32<OUT>(v[3]) << 16)};
    }
  } else if constexpr (!FOURS) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < N) row[n + e] = from_f32<OUT>(v[e]);
  }
}

// One wave per 16 x 16 block of C, fragments straight from memory, in 64-bit
// addresses: for contractions of 2^24 values or more, too long for the other
// kernels' offsets.  Kept simple: such a matrix has at most 2048 rows.
template <int OUT, class Prob = MxGemmProblem>
__global__ __launch_bounds__(64) void k_mx_gemm_plain(Prob p) {
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
      const uint32_t sa = p.A.s[mx_scale_off(m, b, nk)], sb = p.B.s[mx_scale_off(n, b, nk)];
      acc = mfma4<0, 0>(w, a, acc, sb, sa);
    }
  }
  if (bm + r >= p.M) return;
  if constexpr (kEpi<Prob>) {
    float v[4] = {acc[0], acc[1], acc[2], acc[3]};
    epilogue_at<4, kFast<OUT>>(p.epi, v, bm + r, bn + 4 * g);
    return;
  }
  put4<OUT, false>(reinterpret_cast<Elem<OUT>*>(p.C) + (bm + r) * p.N, bn + 4 * g, p.N, acc);
}

// Large-tile kernel: a 256 x 256 tile of C per workgroup, K consumed 256 values
// (128 bytes) at a time, 8 waves in two groups of four, one wave of each group
// per SIMD.  Group g owns rows [128 g, 128 g + 128), wave q of a group columns
// [64 q, 64 q + 64): 8 x 4 blocks of 16 x 16.
//
// The groups run half a k-tile apart and alternate, meeting at a barrier at
// every swap, between
//   - a memory phase: all fragments of the next k-tile from LDS (8 A, 4 B, two
//     128-deep halves each: 96 VGPRs) and their scales (6 VGPRs), and
//   - a compute phase: 64 products of 16 cycles on registers only.
// In phases of half a k-tile, group 0 reads tile t in phase 2 t and computes in
// 2 t + 1, group 1 a phase later.
//
// LDS (136 KB): two slots of A and of B (32 KB each) and of their scales (2 KB
// each).  In its memory phase for t,
//   - group 0 loads B and all scales of t + 1: that slot's t - 1 was last read
//     in phase 2 t - 1, by group 1;
//   - group 1 loads its own half of A of t + 1, whose slot it last read in phase
//     2 t - 1, and group 0's half of A of t + 2, whose slot (that of t) group 0
//     last read in phase 2 t.
// Each has two phases or more to land; the wave that issued a load waits for it
// before the swap ahead of its first read.
//
// 8192 x 14336 x 4096 230 - 255 us (3.8 - 4.2 PFLOP/s), 8192 x 4096 x 14336 194 - 213
// us (4.5 - 4.96), 14336 x 4096 x 8192 212 - 245 us, 4096^3 35 - 37 us; the same
// instructions alone reach 6.3 - 6.8 PFLOP/s, at the 1.5 - 1.8 GHz that such
// products leave.  The matrix cores are busy 51, 63 and 53 % of the first three's
// cycles.  Of the first's 64 thousand cycles a tile, 34 are products (16 k-tiles of
// 2150), 8 the swaps and the phases' unequal lengths (a k-tile takes about 2650),
// and some 20 the tile's start and its stores: one workgroup fills a unit and all
// tiles are alike, so all units store at once while none multiplies.  256 x 256:
// halving either side doubles the LDS reads per product (see k_mx_mid).
template <int OUT, class Prob = MxGemmProblem>
__global__ __launch_bounds__(512) void k_mx_pingpong(Prob p) {
  constexpr int BM = 256, BN = 256, kTM = 8, kTN = 4;
  __shared__ __attribute__((aligned(1024))) uint8_t sA0[256 * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t sA1[256 * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t sB0[256 * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t sB1[256 * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t sS[4 * 2048];  // scales: A0, A1, B0, B1

  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int grp = wave >> 2, wq = wave & 3;
  const int64_t M = p.M, N = p.N;
  const int nk = (int)mx_ktiles(p.K);
  const int pitch = nk * 128;
  const int nbm = (int)((M + BM - 1) / BM), nbn = (int)((N + BN - 1) / BN);
  int tm, tn;
  tile_of(nbm, nbn, tm, tn);
  const int64_t bm = (int64_t)tm * BM, bn = (int64_t)tn * BN;

  // This group's operand: group 0 stages B, group 1 stages A.  The descriptors
  // span the rows (and 32-row scale groups) that exist: the rest reads as zero.
  const int64_t row0 = grp ? bm : bn, rows = (grp ? M : N) - row0;
  const i32x4 rq = make_rsrc((grp ? p.A.q : p.B.q) + row0 * pitch, (rows < 256 ? rows : 256) * (int64_t)pitch);
  // scales, by group 0: A's by waves 0 and 1, B's by waves 2 and 3, four groups
  // of 32 rows (256 bytes each) a wave
  const bool of_a = wq < 2;
  const int64_t srow = of_a ? bm : bn, sleft = (of_a ? M : N) - srow;
  const i32x4 rs = make_rsrc((of_a ? p.A.s : p.B.s) + (srow >> 5) * (int64_t)nk * 256,
                             (sleft < 256 ? (sleft + 31) / 32 : 8) * (int64_t)nk * 256);
  const uint32_t vos = (uint32_t)((4 * (wq & 1) + (lane >> 4)) * nk * 256 + (lane & 15) * 16);
  // A load moves 8 rows, one 16-byte chunk a lane; the row's swizzle takes two
  // values, for even and odd multiples of 8.  Wave q starts at row 64 q of B's
  // 256, or at row 32 q of each half of A.
  const int lr = lane >> 3, r0 = (grp ? 32 : 64) * wq + lr;
  const uint32_t vo0 = (uint32_t)(r0 * pitch + 16 * ((lane & 7) ^ swz16(lr)));
  const uint32_t vo1 = (uint32_t)(r0 * pitch + 16 * ((lane & 7) ^ swz16(8 + lr)));
  // rows from 8 i (+ 128 h): loads [wave][i] of a slot; past the last k-tile, zeros
  auto issue = [&](int i, int h, int kt, uint32_t dst) {
    const uint32_t sb = kt < nk ? (uint32_t)((8 * i + 128 * h) * pitch + kt * 128) : kOob;
    lds_dma16_split(dst, (i & 1) ? vo1 : vo0, sb, rq);
  };
  auto issue_b = [&](int kt, uint32_t slot) {
#pragma unroll
    for (int i = 0; i < 8; ++i) issue(i, 0, kt, slot + (wq * 8 + i) * 1024);
  };
  auto issue_a = [&](int h, int kt, uint32_t slot) {
#pragma unroll
    for (int i = 0; i < 4; ++i) issue(i, h, kt, slot + (16 * h + wq * 4 + i) * 1024);
  };
  auto issue_scales = [&](int kt, int slot) {  // sS: A0, A1, B0, B1
    lds_dma16_split(lds_u32(sS) + (of_a ? 0 : 4096) + slot * 2048 + (wq & 1) * 1024, vos,
                    kt < nk ? (uint32_t)kt * 256 : kOob, rs);
  };
  auto barrier = [&]() {
    __builtin_amdgcn_s_barrier();
    compiler_fence();
  };

  v4f acc[kTM][kTN];
#pragma unroll
  for (int i = 0; i < kTM; ++i)
#pragma unroll
    for (int j = 0; j < kTN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  uint4 af[kTM][2], bf[kTN][2];
  uint32_t sa[4], sb[2];

  if (grp == 0) {
    issue_b(0, lds_u32(sB0));
    issue_scales(0, 0);
  } else {
    issue_a(0, 0, lds_u32(sA0));
    issue_a(1, 0, lds_u32(sA0));
    issue_a(0, 1, lds_u32(sA1));
  }
  wait_vmcnt<0>();
  barrier();
  if (grp == 1) barrier();  // group 1 starts half a k-tile later

  const int frow = lane & 15, fchunk = 2 * (lane >> 4);
  auto step = [&](auto pc, int t) {
    constexpr int P = decltype(pc)::value;  // t % 2
    const uint8_t* a = P ? sA1 : sA0;
    const uint8_t* b = P ? sB1 : sB0;
    if (grp == 0) {
      issue_b(t + 1, lds_u32(P ? sB0 : sB1));
      issue_scales(t + 1, 1 - P);
    } else {
      issue_a(1, t + 1, lds_u32(P ? sA0 : sA1));
      issue_a(0, t + 2, lds_u32(P ? sA1 : sA0));
    }
#pragma unroll
    for (int j = 0; j < kTN; ++j) {
      const int r = 16 * (4 * wq + j) + frow;
      bf[j][0] = *reinterpret_cast<const uint4*>(b + lds_off2(r, fchunk));
      bf[j][1] = *reinterpret_cast<const uint4*>(b + lds_off2(r, fchunk + 1));
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) sb[j] = *reinterpret_cast<const uint32_t*>(sS + 4096 + 2048 * P + 256 * (2 * wq + j) + 4 * lane);
#pragma unroll
    for (int i = 0; i < 4; ++i) sa[i] = *reinterpret_cast<const uint32_t*>(sS + 2048 * P + 256 * (4 * grp + i) + 4 * lane);
#pragma unroll
    for (int i = 0; i < kTM; ++i) {
      const int r = 16 * (8 * grp + i) + frow;
      af[i][0] = *reinterpret_cast<const uint4*>(a + lds_off2(r, fchunk));
      af[i][1] = *reinterpret_cast<const uint4*>(a + lds_off2(r, fchunk + 1));
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    if (grp == 1) wait_vmcnt<8>();       // group 0's half of A of t + 1 has landed
    barrier();
    __builtin_amdgcn_sched_barrier(0);
    static_for<2>([&](auto kk) {
      constexpr int KK = decltype(kk)::value;
      static_for<kTM>([&](auto ic) {
        constexpr int I = decltype(ic)::value;
        static_for<kTN>([&](auto jc) {
          constexpr int J = decltype(jc)::value;
          acc[I][J] = mfma4<(J & 1) * 2 + KK, (I & 1) * 2 + KK>(bf[J][KK], af[I][KK], acc[I][J], sb[J / 2], sa[I / 2]);
        });
      });
    });
    // The products stay in this phase: without this use of their results (no
    // instruction) the compiler sank them past the swap below, where both
    // groups then computed at once.
#pragma unroll
    for (int i = 0; i < kTM; ++i)
      asm volatile("" : "+v"(acc[i][0]), "+v"(acc[i][1]), "+v"(acc[i][2]), "+v"(acc[i][3]));
    __builtin_amdgcn_sched_barrier(0);
    if (grp == 0) wait_vmcnt<0>();  // B and the scales of t + 1 have landed
    else wait_vmcnt<4>();           // so has group 1's half of A of t + 1
    barrier();
  };
  for (int t = 0;;) {
    step(std::integral_constant<int, 0>{}, t);
    if (++t >= nk) break;
    step(std::integral_constant<int, 1>{}, t);
    if (++t >= nk) break;
  }
  if (grp == 0) barrier();

  // Lane: rows wr0 + 16 i + lane % 16, columns wc0 + 16 j + 4 (lane / 16) .. + 3.
  const int wr0 = grp * 128 + (lane & 15), wc0 = wq * 64 + 4 * (lane >> 4);
  if constexpr (kEpi<Prob>) {
    __builtin_amdgcn_s_waitcnt(0);  // no load may still be writing a slot
    float bias[8];
    load_bias<8>(p.epi, bn + wq * 64 + 8 * (lane_anew() & 7), bias);
    barrier();
    static_assert(2 * kWaveEpilogueLds == sizeof(sA0), "two waves a slot");
    uint8_t* slot = wave < 2 ? sA0 : wave < 4 ? sA1 : wave < 6 ? sB0 : sB1;
    wave_epilogue<kTM, EpiMode<kFast<OUT>, true, true>, 2>(p.epi, acc, slot + (wave & 1) * kWaveEpilogueLds, bm + grp * 128, bn + wq * 64,
                                      bias, 1.0f, [](v4f&, int, int) {});
  } else if constexpr (OUT == FP8SG_OUT_F32) {
    float* C = reinterpret_cast<float*>(p.C);
#pragma unroll
    for (int i = 0; i < kTM; ++i) {
      const int64_t m = bm + wr0 + 16 * i;
      if (m >= M) continue;
#pragma unroll
      for (int j = 0; j < kTN; ++j) put4<OUT, false>(C + m * N, bn + wc0 + 16 * j, N, acc[i][j]);
    }
  } else {
    // the tile through LDS (64 rows of 512 bytes per slot), out in 16-byte chunks
    auto crow = [&](int r) -> uint8_t* {
      uint8_t* base = r < 64 ? sA0 : r < 128 ? sA1 : r < 192 ? sB0 : sB1;
      return base + (r & 63) * 512;
    };
    __builtin_amdgcn_s_waitcnt(0);  // no load may still be writing a slot
    barrier();
#pragma unroll
    for (int i = 0; i < kTM; ++i)
#pragma unroll
      for (int j = 0; j < kTN; ++j) {
        const int r = wr0 + 16 * i, col = wc0 + 16 * j;
        store4<OUT>(crow(r) + ((((col >> 3) ^ (r & 31)) << 4) + (col & 7) * 2), 0, acc[i][j]);
      }
    __builtin_amdgcn_s_waitcnt(0xC07F);
    barrier();
    uint16_t* C = reinterpret_cast<uint16_t*>(p.C);
    auto write_tile = [&](auto nt) {
#pragma unroll 4
      for (int pass = 0; pass < 16; ++pass) {
        const int id = pass * 512 + (int)threadIdx.x, r = id >> 5, cc = id & 31;
        const uint4 v = *reinterpret_cast<const uint4*>(crow(r) + ((cc ^ (r & 31)) << 4));
        const int64_t m = bm + r, n = bn + 8 * cc;
        if (m >= M || n >= N) continue;
        if (n + 8 <= N) {  // (C's rows may start anywhere)
          st_any<decltype(nt)::value>(C + m * N + n, u32x4{v.x, v.y, v.z, v.w});
        } else {
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (n + e < N) C[m * N + n + e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
        }
      }
    };
    if (2 * M * N >= kStreamOutBytes) write_tile(std::true_type{});
    else write_tile(std::false_type{});
  }
}


// Medium kernel: a 128 x 128 tile per workgroup of four waves (64 x 64 each), two
// LDS stages of 256 values of K (34 KB each with the scales), so that two
// workgroups share a compute unit and cover each other's barriers.  Its LDS
// reads (8 fragments per 16 products) bound it at about half the matrix rate
// (2048 x 2048 x 4096 16 us, 2.1 PFLOP/s; 256 x 14336 x 4096 15.5 us, 1.9), so it is
// for products that the large tiles would leave compute units idle for.
template <int OUT, class Prob = MxGemmProblem>
__global__ __launch_bounds__(256, 2) void k_mx_mid(Prob p) {
  constexpr int kStage = 2 * 128 * 128 + 2048;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kStage];  // A, B, scales of A, of B
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave >> 1, wn = wave & 1;
  const int64_t M = p.M, N = p.N;
  const int nk = (int)mx_ktiles(p.K), pitch = nk * 128;
  const int nbm = (int)((M + 127) / 128), nbn = (int)((N + 127) / 128);
  int tm, tn;
  tile_of(nbm, nbn, tm, tn);
  const int64_t bm = (int64_t)tm * 128, bn = (int64_t)tn * 128;
  const i32x4 ra = make_rsrc(p.A.q + bm * pitch, (M - bm < 128 ? M - bm : 128) * (int64_t)pitch);
  const i32x4 rb = make_rsrc(p.B.q + bn * pitch, (N - bn < 128 ? N - bn : 128) * (int64_t)pitch);
  // scales: wave 0 A's, wave 1 B's, four groups of 32 rows (those that exist)
  const int64_t left = wave ? N - bn : M - bm;
  const i32x4 rs = make_rsrc(wave ? p.B.s + (bn >> 5) * nk * 256 : p.A.s + (bm >> 5) * nk * 256,
                             (left < 128 ? (left + 31) / 32 : 4) * (int64_t)nk * 256);
  const uint32_t vos = (uint32_t)((lane >> 4) * nk * 256 + (lane & 15) * 16);
  // load i of a wave: rows 32 wave + 8 i + lane / 8 of either operand
  const int lr = lane >> 3;
  const uint32_t vo0 = (uint32_t)((32 * wave + lr) * pitch + 16 * ((lane & 7) ^ swz16(lr)));
  const uint32_t vo1 = (uint32_t)((32 * wave + lr) * pitch + 16 * ((lane & 7) ^ swz16(8 + lr)));
  auto issue = [&](int kt) {
    const uint32_t d = lds_u32(lds) + (kt & 1) * kStage + wave * 4096;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t sb = (uint32_t)(8 * i * pitch + kt * 128);
      lds_dma16_split(d + i * 1024, (i & 1) ? vo1 : vo0, sb, ra);
      lds_dma16_split(d + 16384 + i * 1024, (i & 1) ? vo1 : vo0, sb, rb);
    }
    if (wave < 2)
      lds_dma16_split(lds_u32(lds) + (kt & 1) * kStage + 32768 + wave * 1024, vos, (uint32_t)kt * 256, rs);
  };
  v4f acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  const int frow = lane & 15, fchunk = 2 * (lane >> 4);
  float bias[8];
  if constexpr (kEpi<Prob>) {
    load_bias<8>(p.epi, bn + 64 * wn + 8 * (lane & 7), bias);
  }
  issue(0);
  for (int t = 0; t < nk; ++t) {
    if (t + 1 < nk) {
      issue(t + 1);
      if (wave < 2) wait_vmcnt<9>();
      else wait_vmcnt<8>();
    } else {
      wait_vmcnt<0>();
    }
    __builtin_amdgcn_s_barrier();
    compiler_fence();
    const uint8_t* a = lds + (t & 1) * kStage;
    const uint8_t* b = a + 16384;
    uint32_t sav[2], sbv[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sav[i] = *reinterpret_cast<const uint32_t*>(a + 32768 + 256 * (2 * wm + i) + 4 * lane);
      sbv[i] = *reinterpret_cast<const uint32_t*>(a + 33792 + 256 * (2 * wn + i) + 4 * lane);
    }
    auto half = [&](auto kk, int chunk) {
      constexpr int KK = decltype(kk)::value;
      uint4 af[4], bf[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        af[i] = *reinterpret_cast<const uint4*>(a + lds_off2(64 * wm + 16 * i + frow, chunk));
        bf[i] = *reinterpret_cast<const uint4*>(b + lds_off2(64 * wn + 16 * i + frow, chunk));
      }
      static_for<4>([&](auto ic) {
        constexpr int I = decltype(ic)::value;
        static_for<4>([&](auto jc) {
          constexpr int J = decltype(jc)::value;
          acc[I][J] = mfma4<(J & 1) * 2 + KK, (I & 1) * 2 + KK>(bf[J], af[I], acc[I][J], sbv[J / 2], sav[I / 2]);
        });
      });
    };
    if constexpr (kEpi<Prob>) {
      // one product per accumulator in the loop's body (see few_tile): with two, the
      // registers that the epilogue needs led to products that do not add in place
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        half(std::integral_constant<int, 0>{}, fchunk + h);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          sav[i] >>= 8;
          sbv[i] >>= 8;
        }
      }
    } else {
      half(std::integral_constant<int, 0>{}, fchunk);
      half(std::integral_constant<int, 1>{}, fchunk + 1);
    }
    // this stage is loaded again two k-tiles on: every wave has read it by then
    __builtin_amdgcn_s_waitcnt(0xC07F);
    __builtin_amdgcn_s_barrier();
    compiler_fence();
  }
  if constexpr (kEpi<Prob>) {  // (every load has landed, every wave has read its last stage)
    static_assert(4 * kWaveEpilogueLds <= sizeof(lds), "wave sub-tiles");
    wave_epilogue<4, EpiMode<kFast<OUT>, true, false>, 4>(p.epi, acc, lds + wave * kWaveEpilogueLds, bm + 64 * wm, bn + 64 * wn, bias,
                                    1.0f, [](v4f&, int, int) {});
    return;
  }
  Elem<OUT>* C = reinterpret_cast<Elem<OUT>*>(p.C);
  auto write = [&](auto fours) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t m = bm + 64 * wm + 16 * i + frow;
      if (m >= M) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        put4<OUT, decltype(fours)::value>(C + m * N, bn + 64 * wn + 16 * j + 4 * (lane >> 4), N, acc[i][j]);
    }
  };
  if (N % 4 == 0)
    write(std::true_type{});
  else
    write(std::false_type{});
}

// 4 bytes per lane from buffer offset `voff` into LDS at lds + 4 * lane (as
// lds_dma16).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void lds_dma4(uint32_t lds, uint32_t voff, i32x4 rsrc) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 1\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(rsrc)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// Few rows or few tiles: a 16 TM x 16 TN tile per workgroup, whose waves split K
// (wave w takes k-tiles w, w + W, ...) and join their sums through LDS.  Each
// wave streams its k-tiles of both operands into LDS stages of its own, two in
// flight, so nothing waits for another wave before the join.  (Fragments loaded
// straight into registers put 16 rows in 16 neighbouring lanes, which the
// address coalescer takes one at a time: 24 tokens, 4096 x 14336, 12.8 us; with
// 8 lanes a row through LDS 7.9 us.)  Bound by the weight's bytes and the time to
// get them moving: one token, 14336 x 4096, 31 MB, 6.9 us (4.5 TB/s), of which the
// launch and the join are about 2 us.
// FT >= 0: operand A is not quantised yet (its up to kFusedRows rows, of element
// type FT, are x): a wave first quantises what its k-tiles need of x into LDS.
// Consecutive tiles go to one XCD: two of them may share a row group's scales.
constexpr int kFusedRows = 4, kFusedTiles = 8;  // rows of x, k-tiles a wave
struct MxApply {
  const void* x;
  int32_t fit;
};
// Bytes of a wave's stage: codes of TM + TN fragments, the 32-row groups' scales.
constexpr int few_stage(int tm, int tn, bool fused) {
  return (fused ? 0 : tm * 2048 + (tm + 1) / 2 * 256) + tn * 2048 + (tn + 1) / 2 * 256;
}
constexpr int few_own(bool fused) { return fused ? kFusedTiles * kFusedRows * 136 : 0; }

constexpr int64_t kLds = 160 * 1024;  // of a compute unit
constexpr int few_wave_bytes(int tm, int tn, bool fused) { return 2 * few_stage(tm, tn, fused) + few_own(fused); }
// Waves a workgroup can have: what LDS holds.
constexpr int few_waves(int tm, int tn, bool fused) {
  return (int)kLds / few_wave_bytes(tm, tn, fused) < 16 ? (int)kLds / few_wave_bytes(tm, tn, fused) : 16;
}

// Columns a thread takes in a join with an epilogue: more share a call of the
// generator, fewer are done sooner.  us with 1 / 4 / 8, bias and gelu, then silu with
// dropout, residual and h kept: one token 14336 x 4096 (tiles 16 x 32) 7.1 / 7.7 / 8.0;
// tiles 16 x 16, 300 x 2000 x 1000, fp32 8.2 / 9.6 / 11.2, 10.0 / 11.9 / 13.1; 16 x 32,
// 1000 x 1031 x 2085, 13.7 / 12.0 / 13.8, 18.4 / 14.9 / 16.2; 32 x 32 (8) 11.1, 13.1.
constexpr int few_share(int tm, int tn, bool fused) { return fused || tm * tn == 1 ? 1 : tm * tn == 2 ? 4 : 8; }

// blk of blocks: this workgroup's place among the problem's.
template <int TM, int TN, int OUT, int FT, class Prob>
__device__ __forceinline__ void few_tile(const Prob& p, const MxApply& ap, int64_t blk, int64_t blocks) {
  constexpr bool kFused = FT >= 0;
  constexpr int kStage = few_stage(TM, TN, kFused), kOwn = few_own(kFused);
  // loads of a stage (a wave's count of vmcnt)
  constexpr int kLoads = (kFused ? 0 : 2 * TM + (TM + 1) / 2) + 2 * TN + (TN + 1) / 2;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int lane = threadIdx.x & (kWave - 1), r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), W = blockDim.x / kWave;
  const int64_t M = p.M, N = p.N;
  const int nk = (int)mx_ktiles(p.K), pitch = nk * 128;
  const int64_t nbm = (M + 16 * TM - 1) / (16 * TM);
  const int64_t b = xcd_contiguous(blk, blocks);
  const int64_t bm = b % nbm * (16 * TM), bn = b / nbm * (16 * TN);
  uint8_t* my = lds + wave * (2 * kStage + kOwn);

  // descriptors over the tile's rows (and 32-row scale groups) that exist
  const int64_t lm = M - bm < 16 * TM ? M - bm : 16 * TM, ln = N - bn < 16 * TN ? N - bn : 16 * TN;
  const i32x4 ra = make_rsrc(p.A.q + bm * pitch, kFused ? 0 : lm * pitch);
  const i32x4 rb = make_rsrc(p.B.q + bn * pitch, ln * pitch);
  auto groups = [&](int64_t row0, int64_t rows) { return ((row0 + rows + 31) >> 5) - (row0 >> 5); };
  const i32x4 sa = make_rsrc(p.A.s + (bm >> 5) * (int64_t)nk * 256, kFused ? 0 : groups(bm, lm) * nk * 256);
  const i32x4 sb = make_rsrc(p.B.s + (bn >> 5) * (int64_t)nk * 256, groups(bn, ln) * nk * 256);
  // a load: 8 rows of 128 bytes, 8 lanes a row, chunks swizzled by the row
  const int lr = lane >> 3;
  const uint32_t vo0 = (uint32_t)(lr * pitch + 16 * ((lane & 7) ^ swz16(lr)));
  const uint32_t vo1 = (uint32_t)((8 + lr) * pitch + 16 * ((lane & 7) ^ swz16(8 + lr)));
  auto issue = [&](int kt, uint32_t dst) {
    const uint32_t k0 = (uint32_t)kt * 128, s0 = (uint32_t)kt * 256 + 4 * lane;
    if constexpr (!kFused) {
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        lds_dma16_split(dst + i * 2048, vo0, k0 + 16 * i * pitch, ra);
        lds_dma16_split(dst + i * 2048 + 1024, vo1, k0 + 16 * i * pitch, ra);
      }
      dst += TM * 2048;
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      lds_dma16_split(dst + j * 2048, vo0, k0 + 16 * j * pitch, rb);
      lds_dma16_split(dst + j * 2048 + 1024, vo1, k0 + 16 * j * pitch, rb);
    }
    dst += TN * 2048;
    if constexpr (!kFused) {
#pragma unroll
      for (int i = 0; i < (TM + 1) / 2; ++i) lds_dma4(dst + i * 256, s0 + i * nk * 256, sa);
      dst += (TM + 1) / 2 * 256;
    }
#pragma unroll
    for (int j = 0; j < (TN + 1) / 2; ++j) lds_dma4(dst + j * 256, s0 + j * nk * 256, sb);
  };
  v4f acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  // a 16-row tile starts in the middle of its 32-row scale group where its
  // first row is odd in 16s
  const int odd_a = TM == 1 ? (int)(bm >> 4) & 1 : 0, odd_b = TN == 1 ? (int)(bn >> 4) & 1 : 0;

  const uint32_t d0 = lds_u32(my), d1 = d0 + kStage;
  if (wave < nk) issue(wave, d0);
  if (wave + W < nk) issue(wave + W, d1);
  // x to codes: k-tile kt of row m at own + ((kt - wave) / W * kFusedRows + m) * 136
  if constexpr (kFused) {
    const int cc = lane & 31;
    int t = 0;
    for (int kt = wave; kt < nk; kt += W, ++t) {
      const int64_t c = (int64_t)kt * 256 + 8 * cc;
#pragma unroll
      for (int i = 0; i < kFusedRows / 2; ++i) {
        const int m = 2 * i + (lane >> 5);
        float v[8];
        load8<FT, false>(reinterpret_cast<const Elem<FT>*>(ap.x) + (m < M ? m : 0) * p.K + c, left8(p.K, c), v);
        const uint32_t sc = fp4_scale(quad_amax(v), ap.fit != 0);
        const float f = scale_value(sc);
        uint32_t d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0], v[1], f, 0);
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[2], v[3], f, 1);
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[4], v[5], f, 2);
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[6], v[7], f, 3);
        uint8_t* row = my + 2 * kStage + (t * kFusedRows + m) * 136;
        *reinterpret_cast<uint32_t*>(row + 4 * cc) = sc == 255u ? 0u : d;
        if ((lane & 3) == 0) row[128 + (cc >> 2)] = (uint8_t)sc;
      }
    }
  }

  int t = 0;
#pragma unroll 1
  for (int kt = wave; kt < nk; kt += W, ++t) {
    const uint8_t* st = my + (t & 1) * kStage;
    if (kt + W < nk) wait_vmcnt<kLoads>();
    else wait_vmcnt<0>();
    compiler_fence();
    uint4 a[TM][2], w[TN][2];
    uint32_t ua[TM], ub[TN];
    const uint8_t* q = st;
    if constexpr (kFused) {  // rows past M repeat the last one
      const uint8_t* row = my + 2 * kStage + (t * kFusedRows + (r < M ? r : (int)M - 1)) * 136;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint2 lo = *reinterpret_cast<const uint2*>(row + 32 * g + 16 * h);
        const uint2 hi = *reinterpret_cast<const uint2*>(row + 32 * g + 16 * h + 8);
        a[0][h] = make_uint4(lo.x, lo.y, hi.x, hi.y);
      }
      ua[0] = *reinterpret_cast<const uint16_t*>(row + 128 + 2 * g);
    } else {
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) a[i][h] = *reinterpret_cast<const uint4*>(q + i * 2048 + lds_off2(r, 2 * g + h));
      q += TM * 2048;
    }
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) w[j][h] = *reinterpret_cast<const uint4*>(q + j * 2048 + lds_off2(r, 2 * g + h));
    q += TN * 2048;
    if constexpr (!kFused) {
#pragma unroll
      for (int i = 0; i < TM; ++i) ua[i] = *reinterpret_cast<const uint32_t*>(q + i / 2 * 256 + 4 * lane) >> (16 * (TM == 1 ? odd_a : i & 1));
      q += (TM + 1) / 2 * 256;
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) ub[j] = *reinterpret_cast<const uint32_t*>(q + j / 2 * 256 + 4 * lane) >> (16 * (TN == 1 ? odd_b : j & 1));
    __builtin_amdgcn_s_waitcnt(0xC07F);  // the stage is in registers: load it again
    compiler_fence();
    if (kt + 2 * W < nk) issue(kt + 2 * W, (t & 1) ? d1 : d0);
    // One product per accumulator in the loop's body, so that each is updated
    // in place: otherwise the compiler (clang 22 of ROCm 7.2) once gave a
    // product's result registers that still held another accumulator.  The
    // build checks that every product's result and addend are the same
    // registers.
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = mfma4<0, 0>(w[j][0], a[i][0], acc[i][j], ub[j], ua[i]);
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        keep_loaded(a[i][0]);
        a[i][0] = a[i][1];
        ua[i] >>= 8;
      }
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        keep_loaded(w[j][0]);
        w[j][0] = w[j][1];
        ub[j] >>= 8;
      }
    }
  }

  Elem<OUT>* C = reinterpret_cast<Elem<OUT>*>(p.C);
  if (!kEpi<Prob> && W == 1) {  // nothing to join (an epilogue takes the join's order all the same)
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int64_t m = bm + 16 * i + r;
      if (m >= M) continue;
#pragma unroll
      for (int j = 0; j < TN; ++j) put4<OUT, false>(C + m * N, bn + 16 * j + 4 * g, N, acc[i][j]);
    }
    return;
  }
  float* red = reinterpret_cast<float*>(lds);
  if constexpr (kEpi<Prob>) {
    // join with an epilogue: all blocks at once, [wave][i][j][lane] in LDS, then NV
    // neighbouring columns a thread, which share a call of the generator
    constexpr int NV = few_share(TM, TN, kFused);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
        *reinterpret_cast<v4f*>(red + (((wave * TM + i) * TN + j) * 64 + lane) * 4) = acc[i][j];
    __syncthreads();
    for (int u = threadIdx.x; u < 256 / NV * TM * TN; u += blockDim.x) {
      const int ml = u / (16 / NV * TN), c = u % (16 / NV * TN) * NV;
      if (bm + ml >= M) continue;
      const float* src = red + (((ml >> 4) * TN + (c >> 4)) * 64 + (c & 15) / 4 * 16 + (ml & 15)) * 4 + (c & 3);
      float v[NV];
#pragma unroll
      for (int e = 0; e < NV; ++e) v[e] = 0.f;
      for (int w = 0; w < W; ++w)
#pragma unroll
        for (int e = 0; e < NV; ++e) v[e] += src[w * TM * TN * 256 + e / 4 * 64 + e % 4];
      epilogue_at<NV, kFast<OUT>>(p.epi, v, bm + ml, bn + c);
    }
    return;
  }
  // join: a row of blocks at a time, [wave][j][lane] in LDS
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < TN; ++j) *reinterpret_cast<v4f*>(red + ((wave * TN + j) * 64 + lane) * 4) = acc[i][j];
    __syncthreads();
    for (int e = threadIdx.x; e < 256 * TN; e += blockDim.x) {
      const int ml = e / (16 * TN), nl = e % (16 * TN);
      const int64_t m = bm + 16 * i + ml, n = bn + nl;
      if (m >= M || n >= N) continue;
      const float* src = red + ((nl >> 4) * 64 + ((nl & 15) >> 2) * 16 + ml) * 4 + (nl & 3);
      float v = 0.f;
      for (int w = 0; w < W; ++w) v += src[w * TN * 256];
      C[m * N + n] = from_f32<OUT>(v);
    }
  }
}

template <int TM, int TN, int OUT, int FT, class Prob>
__global__ __launch_bounds__(64 * few_waves(TM, TN, (FT >= 0))) void k_mx_few(Prob p, MxApply ap) {
  few_tile<TM, TN, OUT, FT>(p, ap, blockIdx.x, gridDim.x);
}
// Two small products in one launch: the first `blocks0` workgroups' and the rest's.
template <int OUT>
__global__ __launch_bounds__(64 * few_waves(1, 1, false)) void k_mx_few_pair(MxGemmProblem p0, MxGemmProblem p1, int blocks0) {
  const bool second = (int)blockIdx.x >= blocks0;
  const MxGemmProblem p = second ? p1 : p0;
  few_tile<1, 1, OUT, -1>(p, MxApply{}, second ? blockIdx.x - blocks0 : blockIdx.x,
                                 second ? gridDim.x - blocks0 : blocks0);
}

// A kernel's dynamic LDS limit, raised once per device.
template <class K>
hipError_t allow_lds(K kern, std::atomic<uint64_t>& done) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
  e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)kLds);
  if (e == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Waves that split nk k-tiles: as many (at most `most`) as give each the same
// number of them, and few enough that all workgroups are resident at once.
int split_waves(int64_t nk, int64_t blocks, int64_t per_wave, int64_t most) {
  if (nk < 1) return 1;
  const int64_t room = (int64_t)device_cus() * kLds / (blocks * per_wave);
  if (room < most) most = room < 4 ? 4 : room;
  const int64_t per = (nk + most - 1) / most;
  return (int)((nk + per - 1) / per);
}
template <int TM, int TN, int OUT, int FT, class Prob>
hipError_t launch_few(const Prob& p, const MxApply& ap, hipStream_t stream) {
  auto kern = k_mx_few<TM, TN, OUT, FT, Prob>;
  static std::atomic<uint64_t> done{0};
  const hipError_t attr = allow_lds(kern, done);
  if (attr != hipSuccess) return attr;
  constexpr int64_t kWaveBytes = few_wave_bytes(TM, TN, FT >= 0);
  static_assert(kWaveBytes >= TM * TN * 1024, "the join fits a wave's stages");
  const int64_t blocks = ((p.M + 16 * TM - 1) / (16 * TM)) * ((p.N + 16 * TN - 1) / (16 * TN));
  const int W = split_waves(mx_ktiles(p.K), blocks, kWaveBytes, few_waves(TM, TN, FT >= 0));
  hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(64 * W), W * kWaveBytes, stream, p, ap);
  return hipGetLastError();
}
// Estimated time (us) of a product in workgroup tiles of 16 TM x 16 TN whose
// waves split K: rounds of resident workgroups, each a fixed part (start, join,
// stores) and one part per k-tile of a wave; or the fixed part and the operands'
// way through L2, or from memory.  The constants are fits to products of 1 to
// 1600 rows, 8 to 14336 columns and K of 500 to 14336 in every tile shape (us,
// measured: 200 x 200 x 14336, tiles of 16 5.5, 32 8.0, 64 19.1, 128 37.7; 128 x
// 4096 x 14336: 22.8, 15.0, 20.5, 38.8; 1600 x 1600 x 6000: 68, 34, 39.5, 20.1; one
// token, 14336 x 4096: 7.3, 7.7, 9.2, 12.5).
struct FewCost {
  double fixed, step;
};
double few_cost(const MxGemmProblem& p, int tm, int tn, FewCost c, int cus) {
  const int64_t nk = mx_ktiles(p.K), per_wave = few_wave_bytes(tm, tn, false);
  const int64_t bm = (p.M + 16 * tm - 1) / (16 * tm), bn = (p.N + 16 * tn - 1) / (16 * tn), blocks = bm * bn;
  const int64_t W = split_waves(nk, blocks, per_wave, few_waves(tm, tn, false)), per = (nk + W - 1) / W;
  const int64_t resident = kLds / (W * per_wave) * cus, rounds = (blocks + resident - 1) / resident;
  const double row = (double)nk * 136;  // bytes of an operand's row: codes and scales
  const double l2 = (double)blocks * 16 * (tm + tn) * row / 20e6, hbm = (double)(p.M + p.N) * row / 5.2e6;
  const double work = rounds * (c.fixed + per * c.step) - c.fixed;
  return c.fixed + (work > l2 ? (work > hbm ? work : hbm) : (l2 > hbm ? l2 : hbm));
}
// ... and in tiles of 128 x 128, one or two workgroups a compute unit.
double mid_cost(const MxGemmProblem& p, int cus) {
  const int64_t nk = mx_ktiles(p.K), tiles = ((p.M + 127) / 128) * ((p.N + 127) / 128);
  if (tiles <= cus) return 2.8 + nk * (0.62 + 0.2 * tiles / cus);
  return 2.8 + nk * 1.35 * ((tiles + 2 * cus - 1) / (2 * cus));
}

// What an epilogue adds to those times.  Vector operations an element (activation: 20
// for 16-bit results, 40 for fp32; a call of the generator 200, shared), at 64 a cycle
// and unit where a tile's waves share them; in tiles of 128 one wave of 64 elements a
// lane works on its own (us, 1000 x 1031 x 2085 fp32, without / gelu / silu with dropout,
// residual and h kept: tiles of 128 10.0, 16.3, 22.9, of 32 10.5, 11.1, 13.1).
double epilogue_slots(const EpilogueArgs& e, int share) {
  const double act = e.act == FP8SG_ACT_NONE ? 0 : e.type == FP8SG_OUT_F32 ? 40 : 20;
  return 10 + act + (e.drop.rng ? 200.0 / share : 0) + (e.pre ? 5 : 0) + (e.residual ? 5 : 0);
}
double few_epilogue(const MxGemmProblem&, int, int, int) { return 0; }
double few_epilogue(const MxGemmEpiProblem& p, int tm, int tn, int cus) {
  return (double)p.M * p.N * epilogue_slots(p.epi, few_share(tm, tn, false)) / (64 * 2400.0 * cus);
}
// (2048 x 2048 x 512 in tiles of 128, one round: bf16 6.5 without an epilogue, 8.0 with
// a bias, 10 slots, 10.0 with gelu, 30, 16.7 with silu, dropout, residual and h kept, 65;
// fp32 7.5, 9.7, 13.7 with 50, 21.1 with 85: 0.14 us a slot.)
double mid_epilogue(const MxGemmProblem&, int) { return 0; }
double mid_epilogue(const MxGemmEpiProblem& p, int cus) {
  const int64_t tiles = ((p.M + 127) / 128) * ((p.N + 127) / 128);
  return 0.14 * epilogue_slots(p.epi, 8) * ((tiles + 2 * cus - 1) / (2 * cus));
}

// A product with or without an epilogue.
template <int T, class Prob>
hipError_t launch_product(const Prob& p, hipStream_t stream) {
  auto tiles = [&](int64_t e) { return ((p.M + e - 1) / e) * ((p.N + e - 1) / e); };
  // The tiled kernels' 32-bit offsets span 256 rows: K below 2^24.
  if (mx_pitch(p.K) * 256 >= (1ll << 31) - 256) {
    hipLaunchKernelGGL((k_mx_gemm_plain<T, Prob>), dim3((unsigned)tiles(16)), dim3(64), 0, stream, p);
    return hipGetLastError();
  }
  const MxApply none{};
  // Nothing to add up: zeros, in the fewest workgroups of those kernels that
  // take an empty contraction.
  if (p.K == 0) return launch_few<4, 4, T, -1>(p, none, stream);
  const int cus = device_cus();
  // The large tiles where they occupy most of the chip (2048 x 4096 x 4096, 128
  // tiles on 256 units: 33.9 us, 24.4 us in tiles of 128; 4096^3, 256 tiles:
  // 37.1 against 43.3 us).
  if (tiles(256) * 8 >= 5 * cus) {
    hipLaunchKernelGGL((k_mx_pingpong<T, Prob>), dim3((unsigned)tiles(256)), dim3(512), 0, stream, p);
    return hipGetLastError();
  }
  // (64 x 64 tiles have two microseconds less of fixed time with an epilogue, which joins
  // all blocks at once instead of row by row: plain and with a bias 512 x 512 x 4096 11.4,
  // 9.3, 1024 x 1024 x 4096 11.7, 9.6)
  auto cost = [&](int tm, int tn, FewCost c) { return few_cost(p, tm, tn, c, cus) + few_epilogue(p, tm, tn, cus); };
  const double c11 = cost(1, 1, FewCost{2.0, 0.7}), c12 = cost(1, 2, FewCost{2.4, 0.7});
  const double c22 = cost(2, 2, FewCost{3.5, 0.6}), c44 = cost(4, 4, FewCost{kEpi<Prob> ? 6.8 : 8.8, 0.7});
  const double few = std::min(std::min(c11, c12), std::min(c22, c44));
  if (mid_cost(p, cus) + mid_epilogue(p, cus) < few) {
    hipLaunchKernelGGL((k_mx_mid<T, Prob>), dim3((unsigned)tiles(128)), dim3(256), 0, stream, p);
    return hipGetLastError();
  }
  if (few == c11) return launch_few<1, 1, T, -1>(p, none, stream);
  if (few == c12) return launch_few<1, 2, T, -1>(p, none, stream);
  if (few == c22) return launch_few<2, 2, T, -1>(p, none, stream);
  return launch_few<4, 4, T, -1>(p, none, stream);
}

}  // namespace

hipError_t launch_mx_gemm(const MxGemmProblem& p, int out, hipStream_t stream) {
  if (p.M == 0 || p.N == 0) return hipSuccess;
  return by_type(out, [&](auto t) { return launch_product<decltype(t)::value>(p, stream); });
}

hipError_t launch_mx_gemm_epilogue(const MxGemmEpiProblem& p, hipStream_t stream) {
  if (p.M == 0 || p.N == 0) return hipSuccess;
  return p.epi.type == FP8SG_OUT_F32 ? launch_product<FP8SG_OUT_F32>(p, stream)
                                     : launch_product<FP8SG_OUT_BF16>(p, stream);
}

hipError_t launch_mx_gemm_pair(const MxGemmProblem& p0, const MxGemmProblem& p1, int out, hipStream_t stream) {
  // Where launches dominate (few tiles of 16, short contractions), both in one
  // launch, in tiles of 16; as two, each takes the tiles that suit it.  The whole
  // backward call from a graph, M x N x K, as two / in one (us): 16 x 64 x 64 8.4 / 6.5,
  // 64 x 256 x 128 9.3 / 7.2, 256^3 9.5 / 7.5, 64 x 1024 x 128 10.0 / 8.2, 2048 x 2048 x 32
  // (8 k-tiles) 15.0 / 12.8.  The gain ends between 1000 and 4000 tiles: 64 x 2048 x 128
  // (1056) 10.6 / 10.8, 512^3 (2048) 11.6 / 9.4, 2048 x 2048 x 256 (4096) 21.7 / 27.3.
  auto tiles = [](const MxGemmProblem& p) { return ((p.M + 15) / 16) * ((p.N + 15) / 16); };
  constexpr int64_t kTiles = 512, kLong = 8;
  const int64_t b0 = tiles(p0), b1 = tiles(p1), n0 = mx_ktiles(p0.K), n1 = mx_ktiles(p1.K);
  if (b0 > 0 && b1 > 0 && b0 + b1 <= kTiles && n0 <= kLong && n1 <= kLong)
    return by_type(out, [&](auto t) {
      auto kern = k_mx_few_pair<decltype(t)::value>;
      static std::atomic<uint64_t> done{0};
      const hipError_t attr = allow_lds(kern, done);
      if (attr != hipSuccess) return attr;
      const int64_t W = n0 > n1 ? n0 : n1;
      static_assert(kLong <= few_waves(1, 1, false), "a wave a k-tile");
      hipLaunchKernelGGL(kern, dim3((unsigned)(b0 + b1)), dim3(64 * (unsigned)(W > 0 ? W : 1)),
                         (W > 0 ? W : 1) * few_wave_bytes(1, 1, false), stream, p0, p1, (int)b0);
      return hipGetLastError();
    });
  const hipError_t e = launch_mx_gemm(p0, out, stream);
  return e != hipSuccess ? e : launch_mx_gemm(p1, out, stream);
}

namespace {

// Every workgroup quantises x again, so in the product's own launch only for
// a few rows, only k-tiles that fit its LDS, and not where results lie over x (`over`).
bool apply_fused(const MxGemmProblem& p, bool over) {
  return p.M <= kFusedRows && p.K > 0 && mx_ktiles(p.K) <= 4 * kFusedTiles && !over;
}
int64_t bytes_of(int64_t n, int type) { return n * (type == FP8SG_OUT_F32 ? 4 : 2); }
template <int T, class Prob>
hipError_t launch_apply_fused(const MxQuantJob& j, int type, bool fit, const Prob& p, hipStream_t stream) {
  return by_type(type, [&](auto f) {
    constexpr int X = decltype(f)::value;
    const MxApply ap{j.x, fit};
    return (p.N + 31) / 32 >= device_cus() ? launch_few<1, 2, T, X>(p, ap, stream)
                                           : launch_few<1, 1, T, X>(p, ap, stream);
  });
}

}  // namespace

hipError_t launch_mx_apply(const MxQuantJob& j, int type, bool fit, const MxGemmProblem& p, int out,
                           hipStream_t stream) {
  if (p.M == 0 || p.N == 0) return hipSuccess;
  if (apply_fused(p, shares(p.C, bytes_of(p.M * p.N, out), j.x, bytes_of(p.M * p.K, type))))
    return by_type(out, [&](auto t) { return launch_apply_fused<decltype(t)::value>(j, type, fit, p, stream); });
  const hipError_t e = launch_mx_quantize(&j, 1, type, fit, stream);
  return e != hipSuccess ? e : launch_mx_gemm(p, out, stream);
}

hipError_t launch_mx_apply_epilogue(const MxQuantJob& j, int type, bool fit, const MxGemmEpiProblem& p,
                                    hipStream_t stream) {
  if (p.M == 0 || p.N == 0) return hipSuccess;
  if (apply_fused(p, stored_over(p.epi, j.x, bytes_of(p.M * p.K, type))))
    return p.epi.type == FP8SG_OUT_F32 ? launch_apply_fused<FP8SG_OUT_F32>(j, type, fit, p, stream)
                                       : launch_apply_fused<FP8SG_OUT_BF16>(j, type, fit, p, stream);
  const hipError_t e = launch_mx_quantize(&j, 1, type, fit, stream);
  return e != hipSuccess ? e : launch_mx_gemm_epilogue(p, stream);
}

}  // namespace fp8sg
