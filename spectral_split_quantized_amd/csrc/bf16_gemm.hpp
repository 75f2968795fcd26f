// bf16_gemm.hpp -- A B^T of 16-bit operands on gfx950's matrix instructions,
// with the epilogues of the loss over a vocabulary.
//
// An operand lies with K along the row, at a pitch that is a multiple of 64
// values, zeros behind K; or transposed, with K down the columns (rows of k,
// each readable up to a multiple of 8 values).  Its values are bf16 as a user
// has them, or binary16 planes made of them: x 2^s, with s such that the
// operand's largest finite value lies in [2^14, 2^15).  One plane holds a bf16
// operand (exactly, down to 2^-29 of the largest value); a binary32 operand is
// a pair of planes, hi = x 2^s rounded and lo = the rest rounded, off by 2^-22 of x and
// 2^-40 of the largest value at most.  (bf16 planes would be off by 2^-16.)  The
// product is the sum of up to three products of planes (hi hi, hi lo, lo hi;
// lo lo is no larger than the planes' own error), which simply follow each
// other along K; the epilogue takes the scales off.  Products of 16-bit values
// are exact, sums are binary32.
#pragma once

#include <algorithm>
#include <type_traits>

#include "rows.hpp"

namespace metis {

enum BfOut : int {
  kBfStats,  // softmax statistics of the rows
  kBfProb,   // scaled probabilities minus one at the target, binary16 planes
  kBfF32,    // C, binary32, stored or added; with splits one C for each
  kBfBF16    // C, bf16
};

struct BfGemmParams {
  int64_t M, N;
  const uint8_t *a, *b;
  int64_t pitch_a, pitch_b;   // bytes between rows, multiples of 128
  int64_t rows_a, rows_b;     // of a transposed operand: rows of K (the last repeats up to a whole stage)
  int runs, run_stages;       // K: `runs` products of planes of run_stages stages of 64 each
  int64_t at_a[3], at_b[3];   // where the planes of a run begin, bytes
  const int *shift_a, *shift_b;  // the operands' s (null: 0)
  int splits, split_stages;   // all stages cut into splits of split_stages (the last may be shorter)
  // kBfF32, kBfBF16
  void* C;
  int64_t ldc;
  int64_t split_ld;           // values between the C of two splits
  int add;                    // kBfF32: C += (else C =)
  // kBfStats, kBfProb: row i is token i, column j word v0 + j
  int64_t v0;
  const void* targets;        // [M]
  int targets64;
  int64_t vocab, ignore;
  float2* stat;               // [ceil(N / 64) of all words][M]: largest logit, sum of exponentials
  float* target_logit;        // [M]
  uint32_t* done;             // kBfStats: set to zero
  const float* lse;           // [M]
  const float* grad;          // [M], or one with `count`
  const float* count;         // tokens that the loss is the mean over, or null
  int grad_each;              // grad has a value for each token, by which also P's s goes (dx: it is taken off row i)
  const int* shift_p;         // P's s, where grad has one value (else 0)
  uint16_t* prob;             // [M rounded up to 64][ldp], and lo_plane values behind it the low plane
  int64_t ldp, lo_plane;      // lo_plane 0: none
};

typedef __bf16 bf16x8v_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8v_t __attribute__((ext_vector_type(8)));
typedef float f32x4v_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4v_t __attribute__((ext_vector_type(4)));

constexpr float kLog2E = 1.4426950408889634f;

// Global -> LDS load of 16 bytes a lane to LDS address lds + 16 lane (base and
// lds wave-uniform), as assembly so that the compiler does not wait for the
// loads in flight before every LDS read.  A wait state stands between the
// write of M0 and its use.  (The base comes from scalar arithmetic: no vector
// instruction writes it just before.)
__device__ __forceinline__ void bf_dma16(const uint8_t* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base)
               : "memory", "m0");
}

// two values rounded to binary16 (nearest even), a in the low half
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{a, b}), f16x2_t));
}

__device__ __forceinline__ float unpack_f16(uint32_t w, int i) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)(i & 1 ? w >> 16 : w));
}

// the rest of x behind its rounded value; none behind an infinity
__device__ __forceinline__ float rest_f16(float x, float rounded) { return fabsf(rounded) <= 65504.0f ? x - rounded : 0.0f; }

// the word of token `row`, or -1 where it has no part in the loss
__device__ __forceinline__ int64_t target_of(const void* targets, int targets64, int64_t ignore, int64_t vocab, int64_t row) {
  const int64_t t = targets64 ? ((const int64_t*)targets)[row] : (int64_t)((const int32_t*)targets)[row];
  return t == ignore || t < 0 || t >= vocab ? -1 : t;
}

// The gradient of token `row`'s loss.
__device__ __forceinline__ float loss_gradient(const float* grad, const float* count, int each, int64_t row) {
  const float g = grad[each ? row : 0];
  return count ? g / count[0] : g;
}

// The s of the probabilities of a token with a gradient of its own: g 2^s lies
// in [2^14, 2^15) in size (15 where g is 0 or not finite).
__device__ __forceinline__ int gradient_shift(float g) { return 15 - __builtin_amdgcn_frexp_expf(g); }

// Four rows of K by sixteen columns of a transposed operand, from LDS rows of
// bf16: of each sixteen lanes, lane 4 r + c names the columns 4 c .. 4 c + 3 of
// row r, and lane i receives column i of the four rows.
typedef short s16x4v_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4v_t lds_s16x4_t;

__device__ __forceinline__ bf16x8v_t read_transposed(uint32_t at, uint32_t row4) {
  const s16x4v_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(uintptr_t)at);
  const s16x4v_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(uintptr_t)(at + row4));
  return __builtin_bit_cast(bf16x8v_t, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// WM x WN waves of TM x 4 tiles of 16 x 16, one workgroup for many tiles of C.
// K-stages of 128 bytes (64 values) travel global -> LDS by DMA into a ring of
// NS slots; a row's 16-byte chunk c lies at R * 128 + (c ^ (R / 2 % 8)) * 16, so
// that the 16 lanes that read together hit all banks once.  The matrix
// instruction is 16 x 16 x 32 (lane l takes 8 K-consecutive values of row
// l % 16 at 8 (l / 16)): the card's power holds random operands to 1.83 PFLOP/s
// with it and to 1.30 with 32 x 32 x 16, in loops of nothing else.  B is its
// first operand: a lane ends up with row lane % 16 of a tile of C and columns
// 4 (lane / 16) + v.
//
// A stage is two sub-steps of 32 values; each reads the next one's fragments
// under its matrix instructions.  In the second one every wave holds the
// stage's fragments, so its slot takes the stage NS ahead; the loads run NS
// stages ahead of the products, across tiles.
//
// TA, TB: that operand is transposed.  Its stage is 64 rows of K with the
// tile's columns, and the fragments are read by the transposing LDS read, two
// for eight values of K.  32 lanes read 32 bytes of each of eight rows at a
// time, k .. k + 3 and k + 8 .. k + 11; chunk c of row k lies at
// c ^ (4 (k % 4) + 2 (k / 8 % 2)) (rows of 128 bytes: c ^ (4 (k / 2 % 2) + 2 (k /
// 8 % 2))), which puts them on different banks.
//
// Bound by what the matrix instructions draw and by the stages' loads from
// memory, which run little more than a stage ahead (two stages of 64 KB fill the
// LDS): 8192 x 16384 x 4096 with statistics 756 us, 1.45 PFLOP/s, both operands
// in the cache behind the memory; 8192 x 128256 x 4096 6.1 ms, 1.42; the
// epilogues' stores of P take 8192 x 32768 x 4096 to 1.71 ms, 1.29.  (Cards
// differ by a few percent: 770 us, 6.2 and 1.75 ms on another, 711 us, 5.95 and
// 1.67 ms where the choices below were measured.)
//
// HALF: the operands are binary16 planes, else bf16.  (A product of random
// operands takes 2 to 3 % longer with binary16, which draws more power.)
//
// Rows past M / N repeat the last row (never stored).
template <int WM, int WN, int TM, int NS, int ER, BfOut OUT, bool TA, bool TB, bool HALF>
__global__ __launch_bounds__(WM * WN * 64, 2) void bf_gemm_kernel(BfGemmParams p) {
  constexpr int TN = 4;
  constexpr int NW = WM * WN, BM = WM * TM * 16, BN = WN * TN * 16;
  constexpr int A_BYTES = BM * 128, STAGE = A_BYTES + BN * 128;
  constexpr int PA = BM / 8 / NW, PB = BN / 8 / NW;
  static_assert(PA * 8 * NW == BM && PB * 8 * NW == BN && (NS - 1) * (PA + PB) < 64, "DMA split");
  static_assert(ER % 16 == 0 && (TM * 16) % ER == 0, "epilogue rows");
  __shared__ __attribute__((aligned(16))) uint8_t ring[NS * STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t ep[NW * ER * 128];

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wm = wave / WN, wn = wave % WN;
  const uint32_t tiles_m = (uint32_t)ceil_div<int64_t>(p.M, BM), tiles_n = (uint32_t)ceil_div<int64_t>(p.N, BN);
  const uint32_t total = tiles_m * tiles_n * p.splits, chunk = (total + 7) / 8;
  const int stages = p.runs * p.run_stages;

  // Workgroups go round the 8 XCDs; each XCD takes a contiguous run of tiles,
  // in groups of GR tile rows, so that its CUs share rows of both operands in
  // its L2; the splits of one tile follow each other.  (us with groups of 4, 8
  // and 16: statistics of 8192 x 128256 x 4096 5949, 5995, 6268; 32768 x 4096 x
  // 8192, both transposed, 1582, 1675, 1792; probabilities of 8192 x 21760 x 768
  // 317, 312, 338; 8192 x 4096 x 32768, one transposed, 1612, 1598, 1626.)
  // Sequence number q -> first row and column and the split, or none.
  constexpr uint32_t GR = TA || OUT == kBfStats ? 4 : 8;
  auto locate = [&](uint32_t q, int64_t& m0, int64_t& n0, int& split) {
    const uint32_t ts = (q & 7) * chunk + (q >> 3);
    if ((q >> 3) >= chunk || ts >= total) return false;
    const uint32_t t = p.splits == 1 ? ts : ts / p.splits;
    split = (int)(ts - t * p.splits);
    const uint32_t g = t / (GR * tiles_n), in = t - g * GR * tiles_n, rows = min(tiles_m - g * GR, GR);
    const uint32_t col = in / rows;
    m0 = (int64_t)(g * GR + in - col * rows) * BM;
    n0 = (int64_t)col * BN;
    return true;
  };
  uint32_t q = blockIdx.x, qi = q;  // of the products, of the loads
  int64_t m0, n0;
  int split;
  if (!locate(q, m0, n0, split)) return;

  // the loads: a DMA moves 8 rows, its lanes' offsets from the tile's first
  // row fit 32 bits (256 rows at a pitch below 2^24 bytes)
  const uint8_t *ga, *gb, *ra, *rb;  // at the next stage; of the tile's rows
  uint32_t oa[PA], ob[PB];
  int left, run, run_left;  // stages of the tile still to load; the run of planes and its stages left
  // bytes of a stage along K
  const int64_t step_a = TA ? 64 * p.pitch_a : 128, step_b = TB ? 64 * p.pitch_b : 128;
  auto begin_run = [&](int skip) {
    ga = ra + p.at_a[run] + skip * step_a;
    gb = rb + p.at_b[run] + skip * step_b;
    run_left = p.run_stages - skip;
  };
  // lane's row and chunk of the d-th DMA: K along the row, 8 rows of 8 chunks;
  // transposed, rows of K of B / 8 chunks
  auto row_of = [&](bool t, int B, int d) { return (wave + d * NW) * (t ? 512 / B : 8) + (t ? lane / (B / 8) : lane >> 3); };
  auto offset = [&](bool t, int B, int d, int64_t pitch, int last) {
    const int r = row_of(t, B, d);
    if (!t) return (uint32_t)min(r, last) * (uint32_t)pitch + 16 * ((lane & 7) ^ ((r >> 1) & 7));
    const int c = (lane & (B / 8 - 1)) ^ ((B >= 128 ? 4 * (r & 3) : 4 * ((r >> 1) & 1)) + 2 * ((r >> 3) & 1));
    return (uint32_t)r * (uint32_t)pitch + 16 * min(c, last);
  };
  int last_a, last_b;
  auto offsets = [&] {
#pragma unroll
    for (int d = 0; d < PA; ++d) oa[d] = offset(TA, BM, d, p.pitch_a, last_a);
#pragma unroll
    for (int d = 0; d < PB; ++d) ob[d] = offset(TB, BN, d, p.pitch_b, last_b);
  };
  auto source = [&](int64_t m, int64_t n, int s) {
    ra = p.a + (TA ? m * 2 : m * p.pitch_a);
    rb = p.b + (TB ? n * 2 : n * p.pitch_b);
    const int first = s * p.split_stages;
    left = min(p.split_stages, stages - first);
    run = first / p.run_stages;
    begin_run(first - run * p.run_stages);
    // the tile's last row, or last chunk of a transposed operand's rows
    last_a = (int)min(TA ? (p.M - 1 - m) >> 3 : p.M - 1 - m, (int64_t)BM);
    last_b = (int)min(TB ? (p.N - 1 - n) >> 3 : p.N - 1 - n, (int64_t)BN);
    offsets();
  };
  const uint32_t base = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)ring + wave * 1024;
  // begin: on to the loads of the next stage; rows past a transposed operand's last one repeat it, which only
  // a run's last stage has.
  auto repeat_last = [&](int B, int n, uint32_t* o, int64_t pitch, int last) {
    if (last >= 63) return;
#pragma unroll
    for (int d = 0; d < n; ++d) o[d] -= (uint32_t)max(row_of(true, B, d) - last, 0) * (uint32_t)pitch;
  };
  auto begin = [&] {
    if (left == 0) {  // on to the next tile, or, behind the last one, the same once more
      int64_t m = m0, n = n0;
      int s = split;
      qi += gridDim.x;
      locate(qi, m, n, s);
      source(m, n, s);
    } else if (run_left == 0) {
      ++run;
      offsets();
      begin_run(0);
    }
    if ((TA || TB) && run_left == 1) {
      const int k0 = (p.run_stages - 1) * 64;
      if (TA) repeat_last(BM, PA, oa, p.pitch_a, (int)(p.rows_a - 1 - k0));
      if (TB) repeat_last(BN, PB, ob, p.pitch_b, (int)(p.rows_b - 1 - k0));
    }
  };
  // load d of the stage into a slot: A's, then B's
  auto load = [&](int slot, int d) {
    const uint32_t at = base + slot * STAGE;
    if (d < PA) bf_dma16(ga, oa[d < PA ? d : 0], at + d * NW * 1024);
    else bf_dma16(gb, ob[d < PA ? 0 : d - PA], at + A_BYTES + (d - PA) * NW * 1024);
    if (d == PA + PB - 1) {
      ga += step_a;
      gb += step_b;
      --left;
      --run_left;
    }
  };

  const int lq = lane >> 4, li = lane & 15, sx = (li >> 1) & 7;
  f32x4v_t acc[TM][TN];
  bf16x8v_t fa[2][TM], fb[2][TN];
  // transposed: the lane's place of the first four rows of K, before the
  // fragment's 32 bytes of columns, which its row's swizzle picks
  const int tr = (lane & 15) >> 2;
  auto place = [&](int B) { return (uint32_t)((8 * lq + tr) * (B * 2) + (lane & 3) * 8); };
  const int pick_a = (BM >= 128 ? 2 * tr : 2 * (tr >> 1)) + (lq & 1), pick_b = (BN >= 128 ? 2 * tr : 2 * (tr >> 1)) + (lq & 1);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)ring;
  auto read_a = [&](int slot, int kk, int i) {
    if constexpr (TA) {
      const uint32_t at = lds0 + slot * STAGE + place(BM) + kk * 32 * (BM * 2);
      fa[kk][i] = read_transposed(at + (((wm * TM + i) ^ pick_a) * 32), 4 * (BM * 2));
    } else {
      fa[kk][i] = *(const bf16x8v_t*)(ring + slot * STAGE + li * 128 + ((4 * kk + lq) ^ sx) * 16 + (wm * TM + i) * 2048);
    }
  };
  auto read_b = [&](int slot, int kk, int j) {
    if constexpr (TB) {
      const uint32_t at = lds0 + slot * STAGE + A_BYTES + place(BN) + kk * 32 * (BN * 2);
      fb[kk][j] = read_transposed(at + (((wn * TN + j) ^ pick_b) * 32), 4 * (BN * 2));
    } else {
      fb[kk][j] = *(const bf16x8v_t*)(ring + slot * STAGE + A_BYTES + li * 128 + ((4 * kk + lq) ^ sx) * 16 + (wn * TN + j) * 2048);
    }
  };
  // the fragments in the order of their use
  auto read = [&](int slot, int kk, int f) {
    if (f < TN) read_b(slot, kk, f);
    else read_a(slot, kk, f - TN);
  };
  // Sub-step kk: its matrix instructions, and between them the LDS reads of the
  // next one (of slot `from`) and, in the second, the loads of a stage (into
  // slot `to`), one at a time: the loads of all waves at once would fill the
  // memory pipe's queue and hold the matrix instructions behind them.
  auto step = [&](int kk, int from, int to) {
    // (us with the loads over the whole sub-step, its first half and its first
    // quarter: 32768 x 4096 x 8192, both transposed, 1674, 1717, 1728;
    // statistics of 8192 x 128256 x 4096 6098, 5980, 6040; probabilities of 8192
    // x 32768 x 4096 1784, 1744, 1690; 8192 x 4096 x 32768, one transposed,
    // 1628, 1610, 1595)
    constexpr int T = TM * TN, R = TM + TN, D = PA + PB, SOON = TA ? 1 : OUT == kBfStats ? 2 : 4;
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const int i = t / TN, j = t % TN;
      if constexpr (HALF)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8v_t, fb[kk][j]),
                                                           __builtin_bit_cast(f16x8v_t, fa[kk][i]), acc[i][j], 0, 0, 0);
      else
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[kk][j], fa[kk][i], acc[i][j], 0, 0, 0);
      // reads over the first three quarters
#pragma unroll
      for (int f = t * R * 4 / (3 * T); f < (t + 1) * R * 4 / (3 * T) && f < R; ++f) read(from, kk ^ 1, f);
      if (kk == 1) {
#pragma unroll
        for (int d = t * D * SOON / T; d < (t + 1) * D * SOON / T && d < D; ++d) load(to, d);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // this wave's LDS reads are done and at most N of its loads in flight: with
  // the barrier, a stage has landed and the one before it is read out
  auto landed = [&](auto in_flight) {
    constexpr int N = decltype(in_flight)::value;
    __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4 << 14) | (7 << 4) | (0 << 8));  // vmcnt(N) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  // LDS operations of one wave complete in order; this keeps the compiler's order
  auto wave_fence = [] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
  };
  using First = std::integral_constant<int, (NS - 1) * (PA + PB)>;
  using Left = std::integral_constant<int, (NS - 2) * (PA + PB)>;

  source(m0, n0, split);
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    begin();
#pragma unroll
    for (int d = 0; d < PA + PB; ++d) load(s, d);
  }
  landed(First{});
#pragma unroll
  for (int f = 0; f < TM + TN; ++f) read(0, 0, f);
  int slot = 0;
  for (bool more = true; more;) {
    const int nk = min(p.split_stages, stages - split * p.split_stages);
    const int64_t row0 = m0 + wm * TM * 16, col0 = n0 + wn * TN * 16;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = f32x4v_t{};
    for (int kt = 0; kt < nk; ++kt) {
      step(0, slot, 0);
      landed(Left{});
      const int free_slot = slot;
      slot = slot + 1 == NS ? 0 : slot + 1;
      begin();
      step(1, slot, free_slot);
    }

    // the lane indices taken anew, so that what is made of them does not
    // occupy registers all through the main loop
    int el = lane;
    asm volatile("" : "+v"(el));
    const int li = el & 15, lq = el >> 4;
    // and the arguments read anew, so that they do not occupy scalar registers
    auto args = (const __attribute__((address_space(4))) BfGemmParams*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(args));
    const __attribute__((address_space(4))) BfGemmParams& p = *args;
    // C = acc 2^down; as a factor of logits, kept above 0 (and -inf -inf)
    const int down = HALF ? -(p.shift_a[0] + p.shift_b[0]) : 0;
    const float unit = HALF ? __builtin_ldexpf(1.0f, max(down, -126)) : 1.0f, log2e = unit * kLog2E;

    if constexpr (OUT == kBfStats) {
      if (blockIdx.x == 0 && threadIdx.x == 0) *p.done = 0;
      // a row's 64 columns lie in four lanes, 16 values each
      if (col0 < p.N) {
        const int cols = (int)min((int64_t)64, p.N - col0);
        auto column = [&](int j, int v) { return j * 16 + 4 * lq + v; };
        int64_t word[TM];  // all rows' loads in flight at once
#pragma unroll
        for (int i = 0; i < TM; ++i) word[i] = target_of(p.targets, p.targets64, p.ignore, p.vocab, min(row0 + i * 16 + li, p.M - 1));
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          const int64_t row = row0 + i * 16 + li, t = word[i] - p.v0 - col0;
          const int at = row < p.M && word[i] >= 0 && t >= 0 && t < 64 ? (int)t : -1;
          if (cols < 64) {
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
              for (int v = 0; v < 4; ++v)
                if (column(j, v) >= cols) acc[i][j][v] = -__builtin_inff();
          }
          float m = -__builtin_inff();
#pragma unroll
          for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) m = fmaxf(m, acc[i][j][v]);
          const auto m1 = __builtin_amdgcn_permlane32_swap(__float_as_uint(m), __float_as_uint(m), false, false);
          m = fmaxf(__uint_as_float(m1[0]), __uint_as_float(m1[1]));
          const auto m2 = __builtin_amdgcn_permlane16_swap(__float_as_uint(m), __float_as_uint(m), false, false);
          m = fmaxf(__uint_as_float(m2[0]), __uint_as_float(m2[1]));
          const float off = m == -__builtin_inff() ? 0.0f : -m * log2e;
          float s = 0.0f;
#pragma unroll
          for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) s += __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][v], log2e, off));
          const auto s1 = __builtin_amdgcn_permlane32_swap(__float_as_uint(s), __float_as_uint(s), false, false);
          s = __uint_as_float(s1[0]) + __uint_as_float(s1[1]);
          const auto s2 = __builtin_amdgcn_permlane16_swap(__float_as_uint(s), __float_as_uint(s), false, false);
          s = __uint_as_float(s2[0]) + __uint_as_float(s2[1]);
          if (lq == 0 && row < p.M) p.stat[((p.v0 + col0) >> 6) * p.M + row] = make_float2(m * unit, s);
          if (__ballot(at >= 0)) {
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
              for (int v = 0; v < 4; ++v)
                if (column(j, v) == at) p.target_logit[row] = acc[i][j][v] * unit;
          }
        }
      }
    } else {
      constexpr bool BF = OUT != kBfF32;
      uint8_t* const my = ep + wave * (ER * 128);
      const int rr = el >> 3, rc = el & 7;  // read back: 8 rows of 8 chunks
      // bf16: ER rows of 64 columns at a time, in chunks of 8 values; else ER
      // rows of 32 columns, chunks of 4
      constexpr int COLS = BF ? 64 : 32, PER = COLS / 8;
      const bool lo_too = OUT == kBfProb && p.lo_plane != 0;
      // P has rows up to a multiple of 64, zeros behind M
      const int64_t M = OUT == kBfProb ? (p.M + 63) & ~(int64_t)63 : p.M;
      const int64_t N = OUT == kBfProb ? p.ldp : p.N, ld = OUT == kBfProb ? p.ldp : p.ldc;
      uint16_t* const c16 = OUT == kBfProb ? p.prob : (uint16_t*)p.C;
      const bool vec = OUT == kBfProb || (((uintptr_t)p.C & 15) == 0 && (p.ldc * (BF ? 2 : 4)) % 16 == 0);
#pragma unroll
      for (int i0 = 0; i0 < TM; i0 += ER / 16) {
        if constexpr (OUT == kBfProb) {
          const int cols = (int)max((int64_t)0, min((int64_t)64, p.N - col0));
          const int up = p.shift_p[0];
          float each = 0.0f;
          if (!p.grad_each) each = loss_gradient(p.grad, p.count, 0, 0);
          auto column = [&](int j, int v) { return j * 16 + 4 * lq + v; };
#pragma unroll
          for (int i = i0; i < i0 + ER / 16; ++i) {
            const int64_t r = row0 + i * 16 + li, row = min(r, p.M - 1);
            const int64_t word = r < p.M ? target_of(p.targets, p.targets64, p.ignore, p.vocab, row) : -1;
            const int64_t t = word - p.v0 - col0;
            const int at = word >= 0 && t >= 0 && t < 64 ? (int)t : -1;
            float g = each;
            if (p.grad_each) g = loss_gradient(p.grad, p.count, 1, row);
            const float off = -p.lse[row] * kLog2E;
            g = __builtin_ldexpf(g, p.grad_each ? gradient_shift(g) : up);
            const bool some = word >= 0 && g != 0.0f;  // a token without a part: zeros, whatever its logits
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
              for (int v = 0; v < 4; ++v) {
                const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][v], log2e, off)) * g;
                acc[i][j][v] = some ? x : 0.0f;
              }
            if (__ballot(some && at >= 0)) {
#pragma unroll
              for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                  if (some && column(j, v) == at) acc[i][j][v] -= g;
            }
            if (cols < 64) {
#pragma unroll
              for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                  if (column(j, v) >= cols) acc[i][j][v] = 0.0f;
            }
          }
        }
#pragma unroll
        for (int j0 = 0; j0 < TN; j0 += COLS / 16) {
          for (int plane = 0; plane < 1 + (int)lo_too; ++plane) {
#pragma unroll
            for (int i = i0; i < i0 + ER / 16; ++i) {
              const int r = (i - i0) * 16 + li;
              uint8_t* const row = my + r * 128;
              int here = down;
              if constexpr (OUT != kBfProb && !TA) {
                if (p.grad_each) here -= gradient_shift(loss_gradient(p.grad, p.count, 1, min(row0 + i * 16 + li, p.M - 1)));
              }
#pragma unroll
              for (int j = j0; j < j0 + COLS / 16; ++j) {
                f32x4v_t c = acc[i][j];
                if constexpr (OUT != kBfProb) {
#pragma unroll
                  for (int v = 0; v < 4; ++v) c[v] = __builtin_ldexpf(c[v], here);
                }
                if constexpr (BF) {
                  uint2 w;
                  if constexpr (OUT == kBfProb) {
                    w = make_uint2(pack_f16(c[0], c[1]), pack_f16(c[2], c[3]));
                    if (plane) {
                      auto rest = [&](int v) { return rest_f16(c[v], unpack_f16(v < 2 ? w.x : w.y, v)); };
                      w = make_uint2(pack_f16(rest(0), rest(1)), pack_f16(rest(2), rest(3)));
                    }
                  } else {
                    w = make_uint2(pack_bf16(c[0], c[1]), pack_bf16(c[2], c[3]));
                  }
                  *(uint2*)(row + ((2 * j + (lq >> 1)) ^ ((r >> 1) & 7)) * 16 + (lq & 1) * 8) = w;
                } else {
                  *(f32x4v_t*)(row + ((4 * (j - j0) + lq) ^ ((r >> 1) & 7)) * 16) = c;
                }
              }
            }
            wave_fence();
            const int64_t offset = OUT == kBfProb ? plane * p.lo_plane : split * p.split_ld;
            if (vec) {
#pragma unroll
              for (int k = 0; k < ER / 8; ++k) {
                const int r = k * 8 + rr;
                u32x4v_t w = *(const u32x4v_t*)(my + r * 128 + (rc ^ ((r >> 1) & 7)) * 16);
                const int64_t row = row0 + i0 * 16 + r, col = col0 + j0 * 16 + rc * PER;
                if (row >= M) continue;
                const int64_t at = offset + row * ld + col;
                if (col + PER <= N) {
                  u32x4v_t* const to = BF ? (u32x4v_t*)(c16 + at) : (u32x4v_t*)((float*)p.C + at);
                  if constexpr (!BF) {
                    if (p.add) {
                      const u32x4v_t o = *to;
#pragma unroll
                      for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) + __uint_as_float(o[e]));
                    }
                  }
                  // P and gradients go past the caches, which the operands need (a
                  // backward pass in us without and with it, two runs of each: 8192 x
                  // 50257 x 768 2150 and 2150, 2111 and 2109; 4096 x 32000 x 2048 1458
                  // and 1458, 1448 and 1448; 8192 x 128256 x 4096 20938 and 20894, 20799
                  // and 20910, no difference; 1024 x 50257 x 768 368 and 368, 372 and
                  // 372; binary32 sums, read again at once, gain nothing)
                  if constexpr (BF) __builtin_nontemporal_store(w, to);
                  else *to = w;
                } else {
#pragma unroll
                  for (int e = 0; e < PER; ++e) {
                    if (col + e >= N) break;
                    if constexpr (BF) {
                      c16[at + e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
                    } else {
                      float* const to = (float*)p.C + at + e;
                      *to = __uint_as_float(w[e]) + (p.add ? *to : 0.0f);
                    }
                  }
                }
              }
            } else {
              // rows of any alignment: neighbouring lanes write neighbouring values
              constexpr int RS = 64 / COLS;  // rows a store
              const int c = el & (COLS - 1);
              const int64_t col = col0 + j0 * 16 + c;
#pragma unroll
              for (int k = 0; k < ER / RS; ++k) {
                const int r = k * RS + el / COLS;
                const uint8_t* const from = my + r * 128 + ((c / PER) ^ ((r >> 1) & 7)) * 16;
                const int64_t row = row0 + i0 * 16 + r;
                if (row >= M || col >= N) continue;
                const int64_t at = offset + row * ld + col;
                if constexpr (BF) {
                  c16[at] = *((const uint16_t*)from + c % PER);
                } else {
                  float* const to = (float*)p.C + at;
                  *to = *((const float*)from + c % PER) + (p.add ? *to : 0.0f);
                }
              }
            }
            wave_fence();
          }
        }
      }
    }
    q += gridDim.x;
    more = locate(q, m0, n0, split);
    // read again: their registers served the epilogue
#pragma unroll
    for (int f = 0; f < TM + TN; ++f) read(slot, 0, f);
  }
  // no load may land in LDS that a later workgroup owns
  __builtin_amdgcn_s_waitcnt((0 & 15) | (7 << 4) | (15 << 8));
}

}  // namespace metis
