// int8_gemm.hpp -- C = diag(s_a) (A B^T) diag(s_b) of two int8 operands
// (format: int8.hpp) on gfx950's int8 matrix instructions.
//
// Products are summed exactly in int32 (K <= kI8MaxK keeps |sum| <= 127^2 K
// below 2^31, so any split of K gives the same sum); an output is
// RN(RN(RN(sum) s_a) s_b) in binary32, rounded once more for bf16.
#pragma once

#include <type_traits>

#include "gemm_common.hpp"

namespace metis {

constexpr int64_t kI8MaxK = 133056;  // multiple of 128; 127^2 * 133056 < 2^31

struct I8GemmParams {
  int64_t M, N, pitch;     // pitch: K rounded up to 128, zeros behind K
  const int8_t* a;         // [M][pitch]
  const int8_t* b;         // [N][pitch]
  const float* sa;         // [M]
  const float* sb;         // [N]
  void* C;
  int64_t ldc;
  int bf16;                // C is bf16 (else fp32)
};

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

__device__ inline uint16_t i8_bf16(float v) {  // nearest, ties to even; v is finite or infinite
  const uint32_t u = __float_as_uint(v);
  return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}

// 256 threads as WM x WN waves, each TM x TN tiles of 32 x 32.  The codes
// travel global -> LDS by DMA into a two-slot ring, one K-stage of 128 bytes
// ahead, in the swizzled image of the FP4 kernels: a row's 128 bytes as
// 16-byte chunks, chunk c of row R at ((R / 8) * 64 + (R % 8) * 8 +
// (c ^ (R % 8))) * 16.  The instruction's lane l takes 16 K-consecutive bytes
// of row l % 32; lane half h of sub-step kk reads chunk 2 kk + h of both
// operands, so the order along K is the same on both sides.  Rows past M / N
// repeat the last row (never stored).
template <int WM, int WN, int TM, int TN>
__global__ __launch_bounds__(WM * WN * 64) void i8_gemm_kernel(I8GemmParams p) {
  constexpr int NW = WM * WN, BM = WM * TM * 32, BN = WN * TN * 32;
  constexpr int A_BYTES = BM * 128, STAGE = A_BYTES + BN * 128;
  constexpr int PA = BM / 8 / NW, PB = BN / 8 / NW;
  static_assert(PA * 8 * NW == BM && PB * 8 * NW == BN, "DMA split");
  __shared__ __attribute__((aligned(16))) uint8_t st0[STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t st1[STAGE];
  using S0 = std::integral_constant<int, 0>;
  using S1 = std::integral_constant<int, 1>;
  auto slot = [&](auto s) -> uint8_t* {
    if constexpr (decltype(s)::value == 0) return st0;
    else return st1;
  };

  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int wm = wave / WN, wn = wave % WN;
  const int64_t tiles_m = ceil_div<int64_t>(p.M, BM), tiles_n = ceil_div<int64_t>(p.N, BN);
  const int64_t tile = remap_tile(blockIdx.x, tiles_m, tiles_n);
  const int64_t m0 = (tile / tiles_n) * BM, n0 = (tile % tiles_n) * BN;
  const int64_t nk = p.pitch >> 7;

  i32x16_t acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = i32x16_t{};

  // a DMA moves 8 rows; its lanes' offsets from the tile's first row fit 32
  // bits (256 rows of at most 133056 bytes)
  const int dr = lane >> 3, dc = (lane & 7) ^ dr;
  const int8_t* ga = p.a + m0 * p.pitch;
  const int8_t* gb = p.b + n0 * p.pitch;
  uint32_t oa[PA], ob[PB];
#pragma unroll
  for (int d = 0; d < PA; ++d)
    oa[d] = (uint32_t)(min((int64_t)((wave + d * NW) * 8 + dr), p.M - 1 - m0) * p.pitch) + 16 * dc;
#pragma unroll
  for (int d = 0; d < PB; ++d)
    ob[d] = (uint32_t)(min((int64_t)((wave + d * NW) * 8 + dr), p.N - 1 - n0) * p.pitch) + 16 * dc;
  auto issue = [&](int64_t kt, auto s) {
#pragma unroll
    for (int d = 0; d < PA; ++d) dma16(ga + kt * 128 + oa[d], slot(s) + (wave + d * NW) * 1024);
#pragma unroll
    for (int d = 0; d < PB; ++d) dma16(gb + kt * 128 + ob[d], slot(s) + A_BYTES + (wave + d * NW) * 1024);
  };

  const int hh = lane >> 5, li = lane & 31, lr8 = li & 7;
  auto stage = [&](auto s) {
    i32x4_t fa[2][TM], fb[2][TN];
    auto read = [&](int kk, int buf) {
      const int sw = ((2 * kk + hh) ^ lr8) * 16 + lr8 * 128;
#pragma unroll
      for (int i = 0; i < TM; ++i)
        fa[buf][i] = *(const i32x4_t*)(slot(s) + ((wm * TM + i) * 32 + li) / 8 * 1024 + sw);
#pragma unroll
      for (int j = 0; j < TN; ++j)
        fb[buf][j] = *(const i32x4_t*)(slot(s) + A_BYTES + ((wn * TN + j) * 32 + li) / 8 * 1024 + sw);
    };
    read(0, 0);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const int cur = kk & 1;
      if (kk < 3) read(kk + 1, cur ^ 1);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[cur][i], fb[cur][j], acc[i][j], 0, 0, 0);
#pragma unroll
      for (int t = 0; t < TM * TN; ++t) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
        if (kk < 3 && t < TM + TN) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // LDS read
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  issue(0, S0{});
  ring_barrier();
  for (int64_t kt = 0; kt < nk; kt += 2) {
    // past the last stage the DMAs repeat data into a slot never read again
    issue(kt + 1 < nk ? kt + 1 : kt, S1{});
    stage(S0{});
    ring_barrier();
    if (kt + 1 < nk) {
      issue(kt + 2 < nk ? kt + 2 : kt, S0{});
      stage(S1{});
      ring_barrier();
    }
  }

  // epilogue: lane holds column lane % 32 and rows 8 (v / 4) + 4 (lane / 32) + v % 4
  float sb[TN];
#pragma unroll
  for (int j = 0; j < TN; ++j) sb[j] = p.sb[min(n0 + (wn * TN + j) * 32 + li, p.N - 1)];
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int64_t row = m0 + (wm * TM + i) * 32 + 8 * (v >> 2) + 4 * hh + (v & 3);
      if (row >= p.M) continue;
      const float sa = p.sa[row];
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int64_t col = n0 + (wn * TN + j) * 32 + li;
        if (col >= p.N) continue;
        const float c = (float)acc[i][j][v] * sa * sb[j];
        if (p.bf16) ((uint16_t*)p.C)[row * p.ldc + col] = i8_bf16(c);
        else __builtin_nontemporal_store(c, (float*)p.C + row * p.ldc + col);
      }
    }
  }
}

// Few rows of A (tokens): one workgroup of NW waves per 16 rows of B, the
// waves taking turns along K in steps of U x 64 bytes, so that a wave keeps
// U loads of B in flight; the partial sums meet in LDS.  The instruction is
// 16 x 16 x 64: lane l takes 16 bytes of row l % 16 at 16 (l / 16).  TM tiles
// of 16 tokens.
template <int NW, int TM, int U>
__global__ __launch_bounds__(64 * NW) void i8_gemm_skinny_kernel(I8GemmParams p) {
  __shared__ i32x4_t red[NW > 1 ? NW - 1 : 1][TM][64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int li = lane & 15, hq = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * (16 * TM);
  const int8_t* b = p.b + min(n0 + li, p.N - 1) * p.pitch + 16 * hq;
  const int8_t* a[TM];
#pragma unroll
  for (int i = 0; i < TM; ++i) a[i] = p.a + min(m0 + 16 * i + li, p.M - 1) * p.pitch + 16 * hq;
  i32x4_t acc[TM];
#pragma unroll
  for (int i = 0; i < TM; ++i) acc[i] = i32x4_t{};
  const int64_t steps = p.pitch >> 6;  // even
  for (int64_t s0 = (int64_t)wave * U; s0 < steps; s0 += NW * U) {
    i32x4_t fb[U], fa[U][TM];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t s = s0 + u;
      fb[u] = s < steps ? *(const i32x4_t*)(b + s * 64) : i32x4_t{};
#pragma unroll
      for (int i = 0; i < TM; ++i) fa[u][i] = s < steps ? *(const i32x4_t*)(a[i] + s * 64) : i32x4_t{};
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < TM; ++i) acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fa[u][i], fb[u], acc[i], 0, 0, 0);
  }
  if (wave > 0) {
#pragma unroll
    for (int i = 0; i < TM; ++i) red[wave - 1][i][lane] = acc[i];
  }
  __syncthreads();
  if (wave > 0) return;
  // lane holds column lane % 16 and rows 4 (lane / 16) + v
  const int64_t col = n0 + li;
  if (col >= p.N) return;
  const float sb = p.sb[col];
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int w = 0; w < NW - 1; ++w) acc[i] += red[w][i][lane];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int64_t row = m0 + 16 * i + 4 * hq + v;
      if (row >= p.M) continue;
      const float c = (float)acc[i][v] * p.sa[row] * sb;
      if (p.bf16) ((uint16_t*)p.C)[row * p.ldc + col] = i8_bf16(c);
      else ((float*)p.C)[row * p.ldc + col] = c;
    }
  }
}

}  // namespace metis
