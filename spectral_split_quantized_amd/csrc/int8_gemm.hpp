// int8_gemm.hpp -- C = diag(s_a) (A B^T) diag(s_b) of two int8 operands
// (format: int8.hpp) on gfx950's int8 matrix instructions.
//
// Products are summed exactly in int32 (K <= kI8MaxK keeps |sum| <= 128^2 K
// below 2^31, so any split of K gives the same sum); an output is
// RN(RN(RN(sum) s_a) s_b) in binary32, rounded once more for bf16.
#pragma once

#include <algorithm>
#include <type_traits>

#include "gemm_common.hpp"

namespace metis {

constexpr int64_t kI8MaxK = 131071;

struct I8GemmParams {
  int64_t M, N, pitch;     // pitch: K rounded up to 128, zeros behind K
  const int8_t* a;         // [M][pitch]
  const int8_t* b;         // [N][pitch]
  const float* sa;         // [M]
  const float* sb;         // [N]
  void* C;
  int64_t ldc;
  int bf16;                // C is bf16 (else fp32)
  int splits;              // K is cut into this many runs of
  int run;                 // `run` stages of 128 (the last may be shorter)
  int32_t* part;           // [splits][M][N] partial sums, or null with one run
};

// Which kernel a product takes, and its cut of K.  Times in us.
struct I8Plan {
  int tile;    // rows of A a workgroup: 256 (x 256), 128 or 64 (x 128), 16 (x 16, few tokens)
  int slots;   // of the ring
  int splits, run;
};

// (weights from HBM; M x N x K)
inline I8Plan i8_plan(int64_t M, int64_t N, int64_t pitch) {
  const int stages = (int)(pitch >> 7);
  auto tiles = [&](int m, int n) { return ceil_div<int64_t>(M, m) * ceil_div<int64_t>(N, n); };
  if (M <= 16) return {16, 0, 1, stages};
  // the largest tile that still gives every CU one (4096^3: 60 against 69 with
  // 128 x 128; 2048 x 4096 x 4096: 48 against 36)
  if (tiles(256, 256) >= 256) return {256, 2, 1, stages};
  if (tiles(128, 128) >= 256) return {128, 2, 1, stages};  // 300 x 14336 x 4096: 30, 35 with 64 rows
  // K is cut where the tiles leave half the CUs idle, in runs long enough that
  // they outweigh their sums, 8 bytes an output each (37 x 4096 x 14336, 32
  // tiles: 52 whole, 18 in 8 runs, 22 in 16; 64 x 14336 x 4096, 112 tiles: 21
  // whole, 20 in 2, 24 in 4; 200 x 4096 x 4096, 128 tiles: 15 whole, 16 in 2)
  const int64_t t = tiles(64, 128);
  const int64_t s = t < 128 ? std::min<int64_t>({256 / t, stages / (M <= 128 ? 8 : 16), 8}) : 1;
  I8Plan pl{64, 2, 1, stages};
  if (s > 1) {
    pl.run = (int)ceil_div<int64_t>(stages, s);
    pl.splits = (int)ceil_div<int64_t>(stages, pl.run);
  }
  // a third slot hides more latency (200 x 4096 x 4096: 15 against 19), two
  // start sooner where K is short (1000 x 2304 x 768: 8 against 9)
  if (stages >= 16) pl.slots = 3;
  return pl;
}

enum I8Out { kOutF32, kOutBF16, kOutPart };

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

__device__ inline uint16_t i8_bf16(float v) {  // nearest, ties to even; v is finite or infinite
  const uint32_t u = __float_as_uint(v);
  return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}

// Global -> LDS load of 16 bytes a lane to LDS address lds + 16 lane (base and
// lds wave-uniform).  As assembly, so that the compiler does not wait for the
// loads in flight before every LDS read: it cannot tell the ring's slots
// apart.  The ring's own waits order them.  A wait state stands between the
// write of M0 and its use, and five before the first use of a base, which a
// vector instruction just before may have written.
template <bool FIRST>
__device__ __forceinline__ void dma16_async(const int8_t* base, uint32_t off, uint32_t lds) {
  if constexpr (FIRST)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base)
                 : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base)
                 : "memory", "m0");
}

__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// LDS operations of one wave complete in order; this keeps the compiler's order
__device__ __forceinline__ void wave_fence() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
}

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// WM x WN waves of TM x 2 tiles of 32 x 32, one workgroup for many tiles of
// C.  The codes travel global -> LDS by DMA into a ring of NS slots, each one
// K-stage of 128 bytes; a row's 16-byte chunk c lies at R * 128 +
// (c ^ (R / 2 % 8)) * 16, so that the 16 lanes that read LDS together hit all
// 64 banks once.  The instruction's lane l takes 16 K-consecutive bytes of row
// l % 32; lane half h of sub-step kk reads chunk 2 kk + h of both operands.
// B is the instruction's first operand, so a lane ends up with one row of C
// and runs of four consecutive columns.
//
// A stage is four sub-steps; each reads the next sub-step's fragments from
// LDS under its matrix instructions.  In the last one every wave holds the
// stage's fragments, so its slot takes the stage NS ahead, and the first
// fragments of the next stage (landed by then) are read.  The stages of one
// tile follow those of the one before without a gap: the loads run NS stages
// ahead of the products, across tiles, and the epilogue, which has LDS of its
// own (ER rows a wave), stands between two matrix instructions.
//
// 16384 x 14336 x 4096 to bf16, 256 x 256 tiles of 8 waves: 766 us, 2.5 POP/s.
// The matrix cores are busy 66% of the cycles, at a clock of 1.66 GHz (both
// under counters), and LDS is active 28% of them; four waves of 128 x 128 read
// less of it but leave a SIMD one wave, whose waits nothing fills (1320 us
// against 1110 at that stage).
//
// Rows past M / N repeat the last row (never stored).
template <int WM, int WN, int TM, int NS, int ER, I8Out OUT>
__global__ __launch_bounds__(WM * WN * 64, 2) void i8_gemm_kernel(I8GemmParams p) {
  constexpr int TN = 2;
  constexpr int NW = WM * WN, BM = WM * TM * 32, BN = WN * TN * 32;
  constexpr int A_BYTES = BM * 128, STAGE = A_BYTES + BN * 128;
  constexpr int PA = BM / 8 / NW, PB = BN / 8 / NW;
  static_assert(PA * 8 * NW == BM && PB * 8 * NW == BN && (NS - 1) * (PA + PB) < 64, "DMA split");
  __shared__ __attribute__((aligned(16))) uint8_t ring[NS * STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t ep[NW * ER * 128];

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wm = wave / WN, wn = wave % WN;
  // (fewer than 2^31 units: 32-bit divisions)
  const uint32_t tiles_m = (uint32_t)ceil_div<int64_t>(p.M, BM), tiles_n = (uint32_t)ceil_div<int64_t>(p.N, BN);
  const uint32_t total = tiles_m * tiles_n * p.splits, chunk = (total + 7) / 8;
  const int stages = (int)(p.pitch >> 7);

  // Workgroups go round the 8 XCDs; each XCD takes a contiguous run of tiles,
  // in groups of 8 tile rows, so that its CUs share rows of both operands in
  // its L2; the runs of K of one tile follow each other.  Sequence number q ->
  // first row and column and the run, or none.
  auto locate = [&](uint32_t q, int64_t& m0, int64_t& n0, int& split) {
    const uint32_t ts = (q & 7) * chunk + (q >> 3);
    if ((q >> 3) >= chunk || ts >= total) return false;
    const uint32_t t = p.splits == 1 ? ts : ts / p.splits;
    split = (int)(ts - t * p.splits);
    const uint32_t g = t / (8 * tiles_n), in = t - g * 8 * tiles_n, rows = min(tiles_m - g * 8, 8u);
    const uint32_t col = in / rows;
    m0 = (int64_t)(g * 8 + in - col * rows) * BM;
    n0 = (int64_t)col * BN;
    return true;
  };
  uint32_t q = blockIdx.x, qi = q;  // of the products, of the loads
  int64_t m0, n0;
  int split;
  if (!locate(q, m0, n0, split)) return;

  // the loads: a DMA moves 8 rows, its lanes' offsets from the tile's first
  // row fit 32 bits (256 rows of at most 131072 bytes)
  const int8_t *ga, *gb;
  uint32_t oa[PA], ob[PB];
  int left;  // stages of the tile still to load
  auto source = [&](int64_t m, int64_t n, int s) {
    ga = p.a + m * p.pitch + (int64_t)s * p.run * 128;
    gb = p.b + n * p.pitch + (int64_t)s * p.run * 128;
    left = min(p.run, stages - s * p.run);
    const int last_a = (int)min(p.M - 1 - m, (int64_t)BM), last_b = (int)min(p.N - 1 - n, (int64_t)BN);
#pragma unroll
    for (int d = 0; d < PA; ++d) {
      const int r = (wave + d * NW) * 8 + (lane >> 3);
      oa[d] = (uint32_t)min(r, last_a) * (uint32_t)p.pitch + 16 * ((lane & 7) ^ ((r >> 1) & 7));
    }
#pragma unroll
    for (int d = 0; d < PB; ++d) {
      const int r = (wave + d * NW) * 8 + (lane >> 3);
      ob[d] = (uint32_t)min(r, last_b) * (uint32_t)p.pitch + 16 * ((lane & 7) ^ ((r >> 1) & 7));
    }
  };
  const uint32_t base = lds_offset(ring) + wave * 1024;
  auto issue = [&](int slot) {
    if (left == 0) {  // on to the next tile, or, behind the last one, the same once more
      int64_t m = m0, n = n0;
      int s = split;
      qi += gridDim.x;
      locate(qi, m, n, s);
      source(m, n, s);
    }
    const uint32_t at = base + slot * STAGE;
    dma16_async<true>(ga, oa[0], at);
#pragma unroll
    for (int d = 1; d < PA; ++d) dma16_async<false>(ga, oa[d], at + d * NW * 1024);
    dma16_async<true>(gb, ob[0], at + A_BYTES);
#pragma unroll
    for (int d = 1; d < PB; ++d) dma16_async<false>(gb, ob[d], at + A_BYTES + d * NW * 1024);
    ga += 128;
    gb += 128;
    --left;
  };

  const int hh = lane >> 5, li = lane & 31, sx = (li >> 1) & 7;
  i32x16_t acc[TM][TN];
  i32x4_t fa[2][TM], fb[2][TN];
  auto read = [&](int slot, int kk) {
    const uint8_t* const st = ring + slot * STAGE + li * 128 + ((2 * kk + hh) ^ sx) * 16;
#pragma unroll
    for (int i = 0; i < TM; ++i) fa[kk & 1][i] = *(const i32x4_t*)(st + (wm * TM + i) * 4096);
#pragma unroll
    for (int j = 0; j < TN; ++j) fb[kk & 1][j] = *(const i32x4_t*)(st + A_BYTES + (wn * TN + j) * 4096);
  };
  auto multiply = [&](int kk) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[kk & 1][j], fa[kk & 1][i], acc[i][j], 0, 0, 0);
    // one LDS read after each of the first matrix instructions
#pragma unroll
    for (int t = 0; t < TM * TN; ++t) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (t < TM + TN) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // this wave's LDS reads are done and at most N of its loads in flight: with
  // the barrier, a stage has landed and the one before it is read out
  auto landed = [&](auto in_flight) {
    constexpr int N = decltype(in_flight)::value;
    __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4 << 14) | (7 << 4) | (0 << 8));  // vmcnt(N) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  using First = std::integral_constant<int, (NS - 1) * (PA + PB)>;
  using Left = std::integral_constant<int, (NS - 2) * (PA + PB)>;

  source(m0, n0, split);
#pragma unroll
  for (int s = 0; s < NS; ++s) issue(s);
  landed(First{});
  read(0, 0);
  int slot = 0;
  const bool vec = ((uintptr_t)p.C & 15) == 0 && (p.ldc * (OUT == kOutBF16 ? 2 : 4)) % 16 == 0;
  for (bool more = true; more;) {
    const int nk = min(p.run, stages - split * p.run);
    const int64_t row0 = m0 + wm * TM * 32, col0 = n0 + wn * TN * 32;
    float sa[TM], sb = 0.0f;
    if constexpr (OUT != kOutPart) {
#pragma unroll
      for (int i = 0; i < TM; ++i) sa[i] = p.sa[min(row0 + i * 32 + li, p.M - 1)];
      sb = p.sb[min(col0 + lane, p.N - 1)];
    }
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = i32x16_t{};
    for (int kt = 0; kt < nk; ++kt) {
#pragma unroll
      for (int kk = 0; kk < 3; ++kk) {
        read(slot, kk + 1);
        multiply(kk);
      }
      landed(Left{});
      issue(slot);
      slot = slot + 1 == NS ? 0 : slot + 1;
      read(slot, 0);
      multiply(3);
    }

    // epilogue: the lane holds row li of each tile and columns 8 g + 4 hh + v.
    // Its lane indices are taken anew, so that the addresses made of them do
    // not occupy registers all through the main loop.
    int el = lane;
    asm volatile("" : "+v"(el));
    const int li = el & 31, hh = el >> 5, sx = (li >> 1) & 7;
    uint8_t* const my = ep + wave * (ER * 128);
    float4 sc[TN][4];
    if constexpr (OUT != kOutPart) {
      *(float*)(my + el * 4) = sb;
      wave_fence();
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) sc[j][g] = *(const float4*)(my + (j * 32 + 8 * g + 4 * hh) * 4);
      wave_fence();
    }
    const int rr = el >> 3, rc = el & 7;  // read back: 8 rows of 8 chunks
    auto value = [&](int i, int j, int g, float (&c)[4]) {
      const float s[4] = {sc[j][g].x, sc[j][g].y, sc[j][g].z, sc[j][g].w};
#pragma unroll
      for (int v = 0; v < 4; ++v)
        c[v] = OUT == kOutPart ? __int_as_float(acc[i][j][4 * g + v]) : (float)acc[i][j][4 * g + v] * sa[i] * s[v];
    };
    // bf16: 32 rows of 64 columns a tile row, in chunks of 8 values; else 32
    // rows of 32 columns, chunks of 4
    constexpr int COLS = OUT == kOutBF16 ? 64 : 32, PER = COLS / 8;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
      for (int j0 = 0; j0 < TN; j0 += COLS / 32) {
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += ER) {
          if (ER == 32 || li / ER == r0 / ER) {
#pragma unroll
            for (int j = j0; j < j0 + COLS / 32; ++j)
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                float c[4];
                value(i, j, g, c);
                uint8_t* const row = my + (li % ER) * 128;
                if constexpr (OUT == kOutBF16)
                  *(uint2*)(row + ((j * 4 + g) ^ sx) * 16 + hh * 8) =
                      make_uint2(i8_bf16(c[0]) | (uint32_t)i8_bf16(c[1]) << 16, i8_bf16(c[2]) | (uint32_t)i8_bf16(c[3]) << 16);
                else
                  *(float4*)(row + ((2 * g + hh) ^ sx) * 16) = make_float4(c[0], c[1], c[2], c[3]);
              }
          }
          wave_fence();
          const int64_t split0 = OUT == kOutPart ? split * p.M * p.ldc : 0;
          if (vec) {
#pragma unroll
            for (int k = 0; k < ER / 8; ++k) {
              const int r = k * 8 + rr;
              const u32x4_t w = *(const u32x4_t*)(my + r * 128 + (rc ^ ((r >> 1) & 7)) * 16);
              const int64_t row = row0 + i * 32 + r0 + r, col = col0 + j0 * 32 + rc * PER;
              if (row >= p.M) continue;
              const int64_t at = split0 + row * p.ldc + col;
              if (col + PER <= p.N) {
                u32x4_t* const to = OUT == kOutBF16 ? (u32x4_t*)((uint16_t*)p.C + at) : (u32x4_t*)((float*)p.C + at);
                __builtin_nontemporal_store(w, to);
              } else {
#pragma unroll
                for (int e = 0; e < PER; ++e) {
                  if (col + e >= p.N) break;
                  if constexpr (OUT == kOutBF16) ((uint16_t*)p.C)[at + e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
                  else ((float*)p.C)[at + e] = __uint_as_float(w[e]);
                }
              }
            }
          } else {
            // rows of any alignment: neighbouring lanes write neighbouring
            // values (4096 x 4095 x 4096 to fp32: 72 us; 86 with four values a lane)
            constexpr int RS = 64 / COLS;  // rows a store
            const int c = el & (COLS - 1);
            const int64_t col = col0 + j0 * 32 + c;
#pragma unroll
            for (int k = 0; k < ER / RS; ++k) {
              const int r = k * RS + el / COLS;
              const uint8_t* const from = my + r * 128 + ((c / PER) ^ ((r >> 1) & 7)) * 16;
              const int64_t row = row0 + i * 32 + r0 + r;
              if (row >= p.M || col >= p.N) continue;
              const int64_t at = split0 + row * p.ldc + col;
              if constexpr (OUT == kOutBF16) ((uint16_t*)p.C)[at] = *((const uint16_t*)from + c % PER);
              else ((float*)p.C)[at] = *((const float*)from + c % PER);
            }
          }
          wave_fence();
        }
      }
    }
    q += gridDim.x;
    more = locate(q, m0, n0, split);
  }
  // no load may land in LDS that a later workgroup owns
  __builtin_amdgcn_s_waitcnt((0 & 15) | (7 << 4) | (15 << 8));
}

// C from the partial sums of the runs of K: 4 values a thread, eight runs in
// flight (37 x 4096 of 8 runs: 3.9 us, latency; 8.9 with four in flight and
// larger workgroups).
template <bool BF16>
__global__ __launch_bounds__(64) void i8_join_kernel(I8GemmParams p) {
  const int64_t per_row = (p.N + 3) >> 2, id = (int64_t)blockIdx.x * 64 + threadIdx.x;
  if (id >= p.M * per_row) return;
  const int64_t row = id / per_row, col = (id - row * per_row) * 4;
  const int n = (int)min((int64_t)4, p.N - col);
  const int32_t* at = p.part + row * p.N + col;
  int sum[4] = {0, 0, 0, 0};
  const bool vec = n == 4 && (p.N & 3) == 0;
  for (int s = 0; s < p.splits; s += 8) {  // eight loads in flight
    i32x4_t v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[k] = i32x4_t{};
      if (s + k < p.splits) {
        const int32_t* from = at + (int64_t)(s + k) * p.M * p.N;
        if (vec) {
          v[k] = *(const i32x4_t*)from;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (e < n) v[k][e] = from[e];
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] += v[k][e];
  }
  const float sa = p.sa[row];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (e >= n) break;
    const float c = (float)sum[e] * sa * p.sb[col + e];
    if constexpr (BF16) ((uint16_t*)p.C)[row * p.ldc + col + e] = i8_bf16(c);
    else ((float*)p.C)[row * p.ldc + col + e] = c;
  }
}

// At most 16 rows of A (tokens): one workgroup of NW waves per 16 rows of B,
// the waves taking turns along K in steps of U x 64 bytes, so that a wave
// keeps U loads of B in flight; the partial sums meet in LDS.  The
// instruction is 16 x 16 x 64: lane l takes 16 bytes of row l % 16 at
// 16 (l / 16).  Bound by B's bytes (1 x 14336 x 4096: 12.1 us, 4.9 TB/s) and,
// towards 16 tokens, by fetching A again for every 16 rows of B (17.8 us).
template <int NW, int U>
__global__ __launch_bounds__(64 * NW) void i8_gemm_skinny_kernel(I8GemmParams p) {
  __shared__ i32x4_t red[NW - 1][64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int li = lane & 15, hq = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int8_t* b = p.b + min(n0 + li, p.N - 1) * p.pitch + 16 * hq;
  const bool have = li < p.M;  // lanes without a token fetch nothing
  const int8_t* a = p.a + min((int64_t)li, p.M - 1) * p.pitch + 16 * hq;
  i32x4_t acc{};
  const int64_t steps = p.pitch >> 6;
  for (int64_t s0 = (int64_t)wave * U; s0 < steps; s0 += NW * U) {
    i32x4_t fb[U], fa[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t s = s0 + u;
      fb[u] = s < steps ? *(const i32x4_t*)(b + s * 64) : i32x4_t{};
      fa[u] = s < steps && have ? *(const i32x4_t*)(a + s * 64) : i32x4_t{};
    }
#pragma unroll
    for (int u = 0; u < U; ++u) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(fa[u], fb[u], acc, 0, 0, 0);
  }
  if (wave > 0) red[wave - 1][lane] = acc;
  __syncthreads();
  if (wave > 0) return;
  // lane holds column lane % 16 and rows 4 (lane / 16) + v
  const int64_t col = n0 + li;
  if (col >= p.N) return;
  const float sb = p.sb[col];
#pragma unroll
  for (int w = 0; w < NW - 1; ++w) acc += red[w][lane];
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int64_t row = 4 * hq + v;
    if (row >= p.M) continue;
    const float c = (float)acc[v] * p.sa[row] * sb;
    if (p.bf16) ((uint16_t*)p.C)[row * p.ldc + col] = i8_bf16(c);
    else ((float*)p.C)[row * p.ldc + col] = c;
  }
}

}  // namespace metis
