// int8.hpp -- int8 quantiser with one scale per line (token or channel).
//
// A line is a row of M (K along the row, axis 1) or a column (K down the
// column, axis 0: the codes are the quantised transpose).  With a its largest
// magnitude, in binary32 steps (RN: rounded to nearest):
//   s = max(RN(a / 127), 2^-126),  inv = RN(1 / s),  y = RN(x inv),
//   code = rint(y), or floor(y) + [u < y - floor(y)] stochastically,
// clamped to +-127.  |y| <= 127 (1 + 3 2^-24), so the clamp only meets a
// rounding of the extremes.  The floor 2^-126 keeps s and inv normal (an
// all-zero line has codes 0).  u = h 2^-16 with h the 16-bit Philox draw of
// the element's row-major position in M, the same for both orientations.
// Code rows have a pitch of K rounded up to 128 bytes with zeros behind K, so
// the product's K loop has no tail.
//
// Columns, or both orientations together, take one sweep for the maxima and
// one for the codes.  Rows alone take one sweep: a row stays in registers
// between its maximum and its codes.
#pragma once

#include "quant.hpp"
#include "int8_gemm.hpp"
#include "quant_fast.hpp"

namespace metis {

constexpr int kI8Pitch = 128;

__host__ __device__ inline int64_t i8_pitch(int64_t k) { return (k + kI8Pitch - 1) / kI8Pitch * kI8Pitch; }

struct I8QuantParams {
  const void* src;
  int dtype;
  int64_t rows, cols, ld;
  int64_t row0;      // first row of this launch (rows alone)
  bool vec;          // rows start 16-byte aligned and ld keeps them so
  int8_t* codes0;    // [cols][i8_pitch(rows)] or null
  int8_t* codes1;    // [rows][i8_pitch(cols)] or null
  float* scales0;    // [cols]
  float* scales1;    // [rows]
  float* part0;      // [row tiles][cols] column maxima of a tile
  float* part1;      // [column tiles][rows] row maxima of a tile, or null
  int amax_rows;     // rows of a wave in the first sweep
  int sr;
  uint64_t seed;
  uint32_t tag, step;
  const int64_t* step_count;  // the step in device memory where not negative, or null

  __device__ uint32_t step_now() const {
    const int64_t count = step_count ? *step_count : -1;
    return count < 0 ? step : (uint32_t)count;
  }
};

__device__ inline float i8_scale(float amax) { return fmaxf(__fdiv_rn(amax, 127.0f), 0x1p-126f); }
__device__ inline float i8_inverse(float scale) { return __fdiv_rn(1.0f, scale); }

// The code, in the low byte of the result.  To nearest: y kept within +-127
// (an integer, so before the rounding as well as after it) plus 1.5 2^23,
// whose unit is 1: the sum's rounding to nearest even leaves the integer in
// its low bits.  SR: u is the draw times 2^-16; v_fract_f32 is y - floor(y)
// rounded to binary32 but kept below 1, where u < 1 decides the same.
template <bool SR>
__device__ inline int i8_code(float x, float inv, float u) {
  const float y = x * inv;
  if constexpr (SR) {
    int c;  // floor(y) in one instruction
    asm("v_cvt_flr_i32_f32 %0, %1" : "=v"(c) : "v"(y));
    c += u < __builtin_amdgcn_fractf(y) ? 1 : 0;
    return max(-127, min(127, c));
  } else {
    return __float_as_int(__builtin_amdgcn_fmed3f(y, -127.0f, 127.0f) + 12582912.0f);
  }
}

// low bytes of four codes
__device__ inline uint32_t pack4(int a, int b, int c, int d) {
  const uint32_t lo = __builtin_amdgcn_perm((uint32_t)b, (uint32_t)a, 0x0C0C0400u);
  const uint32_t hi = __builtin_amdgcn_perm((uint32_t)d, (uint32_t)c, 0x04000C0Cu);
  return lo | hi;
}

// eight consecutive elements at an address that 16 divides
__device__ inline void i8_load8_vec(const void* at, int dtype, float (&x)[8]) {
  if (dtype == 0) {
    const uint4 q = *(const uint4*)at;
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const float4 a = *(const float4*)at, b = *((const float4*)at + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
}

// eight consecutive elements of a row from column c (n of them exist)
__device__ inline void i8_load8(const I8QuantParams& p, int64_t row, int64_t c, int n, float (&x)[8]) {
  const int64_t at = row * p.ld + c;
  if (n == 8 && p.vec) {
    i8_load8_vec((const char*)p.src + (at << (p.dtype ? 2 : 1)), p.dtype, x);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = i < n ? load_as_float(p.src, p.dtype, at + i) : 0.0f;
}

// the same eight elements as they lie in memory
template <bool BF16>
struct I8Raw8 {
  uint32_t w[BF16 ? 4 : 8];

  __device__ void load_vec(const void* at) {
    const uint4 a = *(const uint4*)at;
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    if constexpr (!BF16) {
      const uint4 b = *((const uint4*)at + 1);
      w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    }
  }
  __device__ void load(const I8QuantParams& p, int64_t row, int64_t c, int n) {
    const int64_t at = row * p.ld + c;
    if (n == 8 && p.vec) {
      load_vec((const char*)p.src + at * (BF16 ? 2 : 4));
      return;
    }
#pragma unroll
    for (int i = 0; i < (BF16 ? 4 : 8); ++i) {
      if constexpr (BF16) {
        const uint32_t lo = 2 * i < n ? ((const uint16_t*)p.src)[at + 2 * i] : 0;
        w[i] = lo | (2 * i + 1 < n ? (uint32_t)((const uint16_t*)p.src)[at + 2 * i + 1] << 16 : 0);
      } else {
        w[i] = i < n ? ((const uint32_t*)p.src)[at + i] : 0;
      }
    }
  }
  __device__ float operator[](int i) const {
    if constexpr (BF16) return __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
    else return __uint_as_float(w[i]);
  }
};

// draws (times 2^-16) of the row-major positions e .. e + 7: the halves of one
// Philox block, or of two where e is no multiple of 8
__device__ inline void i8_draws8(const I8QuantParams& p, uint32_t step, uint64_t e, float (&u)[8]) {
  const Philox4 b0 = philox_block(e >> 3, p.tag, step, p.seed);
  const uint32_t o = (uint32_t)(e & 7);
  if (o == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = (float)philox_half_of(b0, i) * 0x1p-16f;
    return;
  }
  const Philox4 b1 = philox_block((e >> 3) + 1, p.tag, step, p.seed);
  uint32_t h[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = philox_half_of(b0, i), h[8 + i] = philox_half_of(b1, i);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t v = 0;
#pragma unroll
    for (int j = 1; j < 8; ++j) v = o == (uint32_t)j ? h[i + j] : v;
    u[i] = (float)v * 0x1p-16f;
  }
}

__device__ inline float i8_absmax8(const float (&x)[8], float m, bool& bad) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = fabsf(x[i]);
    bad |= !(a <= 3.402823466e38f);
    m = fmaxf(m, a);
  }
  return m;
}

// ------------------------------------------------------------ rows alone --
//
// One workgroup of 64 W threads per row; each thread holds CH chunks of eight
// elements (chunk t + 64 W j).  Longer rows are read a second time (from L2).
// Bound by HBM to nearest (16384 x 4096 bf16: 32 us, 201 MB) and by the vector
// units stochastically (48 us: ten Philox rounds for eight elements); W CH 512
// elements cover the row with as few idle threads as the sizes allow (4096
// columns: 4 waves of two chunks 32 us, 8 waves half idle 42).
template <int W, int CH, bool SR>
__global__ __launch_bounds__(64 * W) void i8_quant_rows_kernel(I8QuantParams p) {
  constexpr int T = 64 * W;
  __shared__ float red[W];
  const int64_t row = p.row0 + blockIdx.x;
  const int64_t chunks = i8_pitch(p.cols) >> 3;  // the zero padding included
  float x[CH][8];
  float m = 0.0f;
  bool bad = false;
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int64_t c = ((int64_t)threadIdx.x + T * j) * 8;
    const int n = (int)min((int64_t)8, max((int64_t)0, p.cols - c));
    i8_load8(p, row, c, n, x[j]);
  }
#pragma unroll
  for (int j = 0; j < CH; ++j) m = i8_absmax8(x[j], m, bad);
  for (int64_t ch = (int64_t)threadIdx.x + T * CH; ch < chunks; ch += T) {
    float y[8];
    i8_load8(p, row, ch * 8, (int)min((int64_t)8, max((int64_t)0, p.cols - ch * 8)), y);
    m = i8_absmax8(y, m, bad);
  }
  m = wave_max(m);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    m = red[0];
#pragma unroll
    for (int w = 1; w < W; ++w) m = fmaxf(m, red[w]);
  }
  if (bad) raise_status(kStatusNonFinite);
  const float s = i8_scale(m), inv = i8_inverse(s);
  if (threadIdx.x == 0) p.scales1[row] = s;
  const uint32_t step = SR ? p.step_now() : 0;
  auto put = [&](int64_t ch, const float (&y)[8]) {
    float u[8];
    if constexpr (SR) i8_draws8(p, step, (uint64_t)row * p.cols + ch * 8, u);
    int q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = i8_code<SR>(y[i], inv, SR ? u[i] : 0.0f);
    *(uint2*)(p.codes1 + row * (chunks << 3) + ch * 8) =
        make_uint2(pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]));
  };
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int64_t ch = (int64_t)threadIdx.x + T * j;
    if (ch < chunks) put(ch, x[j]);
  }
  for (int64_t ch = (int64_t)threadIdx.x + T * CH; ch < chunks; ch += T) {
    float y[8];
    i8_load8(p, row, ch * 8, (int)min((int64_t)8, max((int64_t)0, p.cols - ch * 8)), y);
    put(ch, y);
  }
}

// ------------------------------------------------- columns, or both sides --
//
// Two sweeps.  The first leaves, for tiles of 4 R rows x 512 columns, each
// column's and row's largest magnitude in the tile; a wave covers 512 columns
// of R rows, lane l the columns 8 l .. + 7.  The second sweep joins the
// maxima of its own 128 rows and columns into scales (the first workgroups
// along each side store them) and writes the codes, the transposed ones
// through LDS: 256 threads on 128 x 128, thread t the column chunk
// 8 (t % 16) .. + 7 of rows 4 (t / 16) .. + 3 and of the rows 64 further down,
// so that both orientations are written in whole 128-byte lines.
// 16384 x 4096 bf16, both orientations: the first sweep 23 us (134 MB, the
// second reading of them comes partly from the last-level cache), the second
// 52 us to nearest (268 MB, the rate of a copy) and 73 us stochastically
// (vector units: Philox and two roundings an element).  Every tile joins the
// maxima of its lines, 68 KB here and more with every row: 131072 rows take
// 995 us, 13.6 times as long.  Scales joined in a
// kernel of their own cost 39 us at one thread a line.
constexpr int kI8Tile = 128;
constexpr int kI8AmaxCols = 512;

// rows of a wave in the first sweep: long runs leave few maxima to join, short
// ones fill the chip
inline int i8_amax_rows(int64_t rows, int64_t cols) {
  const int64_t wide = (cols + kI8AmaxCols - 1) / kI8AmaxCols;
  int r = 64;
  while (r > 8 && (rows + 4 * r - 1) / (4 * r) * wide < 1024) r >>= 1;
  return r;
}

__global__ __launch_bounds__(256) void i8_amax_kernel(I8QuantParams p) {
  __shared__ uint32_t cmax[4][kI8AmaxCols];
  const int64_t tiles_n = ceil_div<int64_t>(p.cols, kI8AmaxCols);
  const int64_t tm = blockIdx.x / tiles_n, tn = blockIdx.x % tiles_n;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t c = tn * kI8AmaxCols + lane * 8;
  const int n = (int)min((int64_t)8, max((int64_t)0, p.cols - c));
  const int64_t row0 = (tm * 4 + wave) * p.amax_rows;
  uint32_t cm[8] = {0, 0, 0, 0, 0, 0, 0, 0}, mine = 0, top = 0;
  for (int r0 = 0; r0 < p.amax_rows; r0 += 8) {
    float x[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t row = row0 + r0 + i;
      i8_load8(p, min(row, p.rows - 1), c, row < p.rows ? n : 0, x[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t rm = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {  // magnitudes order like their bits, NaN above all
        const uint32_t a = __float_as_uint(x[i][j]) & 0x7FFFFFFFu;
        cm[j] = max(cm[j], a);
        rm = max(rm, a);
      }
      if (p.part1) {
        rm = wave_max_u32(rm);
        mine = lane == r0 + i ? rm : mine;
      }
    }
  }
  if (p.part1 && lane < p.amax_rows && row0 + lane < p.rows) p.part1[tn * p.rows + row0 + lane] = __uint_as_float(mine);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    cmax[wave][lane * 8 + j] = cm[j];
    top = max(top, cm[j]);
  }
  if (top >= 0x7F800000u) raise_status(kStatusNonFinite);
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kI8AmaxCols; k += 256) {
    const int i = k + threadIdx.x;
    const int64_t col = tn * kI8AmaxCols + i;
    if (col < p.cols)
      p.part0[tm * p.cols + col] = __uint_as_float(max(max(cmax[0][i], cmax[1][i]), max(cmax[2][i], cmax[3][i])));
  }
}

template <bool SR, bool BF16>
__global__ __launch_bounds__(256) void i8_quant_tile_kernel(I8QuantParams p) {
  // transposed codes: column c at words c * kPitch .. + 31 (four rows a word)
  constexpr int kPitch = 33;
  __shared__ uint32_t tr[kI8Tile * kPitch];
  __shared__ float inv[2][kI8Tile];  // columns, rows
  const int64_t pitch0 = i8_pitch(p.rows), pitch1 = i8_pitch(p.cols);
  const uint32_t tiles_n = (uint32_t)(pitch1 / kI8Tile);
  const uint32_t tm = blockIdx.x / tiles_n, tn = blockIdx.x - tm * tiles_n;
  const int64_t r0 = (int64_t)tm * kI8Tile, c0 = (int64_t)tn * kI8Tile;
  const int cc = threadIdx.x & 15, rg = threadIdx.x >> 4;
  // a whole tile addresses its elements by a uniform base and a 32-bit offset
  const bool whole = r0 + kI8Tile <= p.rows && c0 + kI8Tile <= p.cols;
  I8Raw8<BF16> x[8];  // unpacked where they are used: 8 of 16 bytes or 8 of 32 a thread
  if (whole && p.vec && p.ld < (1 << 22)) {
    constexpr int sh = BF16 ? 1 : 2;
    const uint32_t off = ((uint32_t)(rg * 4) * (uint32_t)p.ld + cc * 8) << sh;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const char* base = (const char*)p.src + (((r0 + (i & 3) + (i >> 2) * 64) * p.ld + c0) << sh);
      x[i].load_vec(base + off);
    }
  } else {
    const int n = (int)min((int64_t)8, max((int64_t)0, p.cols - c0 - cc * 8));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t row = r0 + rg * 4 + (i & 3) + (i >> 2) * 64;
      x[i].load(p, min(row, p.rows - 1), c0 + cc * 8, row < p.rows ? n : 0);
    }
  }
  {  // the 128 columns' and rows' scales: two threads a line, of different waves, join its maxima
    const int i = threadIdx.x & (kI8Tile - 1), odd = __builtin_amdgcn_readfirstlane(threadIdx.x >> 7);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const float* part = side ? p.part1 : p.part0;
      const int64_t first = side ? r0 : c0, lines = side ? p.rows : p.cols;
      const int tiles = (int)(side ? ceil_div<int64_t>(p.cols, kI8AmaxCols) : ceil_div<int64_t>(p.rows, 4 * p.amax_rows));
      const bool have = part && first + i < lines;
      const uint32_t at = have ? i : 0;
      float m = 0.0f;
      if (part) {
        for (int t = odd; t < tiles; t += 16) {
          float v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = (part + first + (int64_t)min(t + 2 * k, tiles - 1) * lines)[at];
#pragma unroll
          for (int k = 0; k < 8; ++k) m = fmaxf(m, v[k]);
        }
      }
      if (odd) inv[side][i] = m;
      __syncthreads();
      if (!odd) {
        const float s = i8_scale(fmaxf(m, inv[side][i]));
        inv[side][i] = i8_inverse(s);
        if (have && (side ? tn == 0 : tm == 0)) (side ? p.scales1 : p.scales0)[first + i] = s;
      }
    }
  }
  __syncthreads();
  float inv0[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) inv0[j] = inv[0][cc * 8 + j];
  const int64_t off1 = rg * 4 * pitch1 + cc * 8;
  uint64_t e = (uint64_t)(r0 + rg * 4) * p.cols + c0 + cc * 8;
  const uint32_t step = SR ? p.step_now() : 0;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    int w[8][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = half * 64 + rg * 4 + i;
      const I8Raw8<BF16>& v = x[half * 4 + i];
      float u[8];
      if constexpr (SR) {
        i8_draws8(p, step, e, u);
        e += i < 3 ? p.cols : 61 * p.cols;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j][i] = i8_code<SR>(v[j], inv0[j], SR ? u[j] : 0.0f);
      if (p.codes1 && (whole || r0 + r < p.rows)) {
        const float inv1 = inv[1][r];
        int q[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = i8_code<SR>(v[j], inv1, SR ? u[j] : 0.0f);
        int8_t* base = p.codes1 + (r0 + half * 64 + i) * pitch1 + c0;
        *(uint2*)(base + off1) = make_uint2(pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]));
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      tr[(cc * 8 + j) * kPitch + half * 16 + rg] = pack4(w[j][0], w[j][1], w[j][2], w[j][3]);
  }
  __syncthreads();
  // 8 threads write a column's 128 bytes
  const int ci = threadIdx.x >> 3, part = threadIdx.x & 7;
  int8_t* const out = p.codes0 + c0 * pitch0 + r0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int col = ci + 32 * k;
    const uint32_t* t = tr + col * kPitch + part * 4;
    if (whole || c0 + col < p.cols)
      *(uint4*)(out + col * pitch0 + part * 16) = make_uint4(t[0], t[1], t[2], t[3]);
  }
}

// ------------------------------------------------- serving, single token --
//
// y = x W-hat in one launch: one workgroup of NW waves per 16 output
// channels, the waves taking turns along K in steps of U x 64 bytes.  The
// workgroup sends off its loads of the token, then each wave its first loads
// of W (16 rows); loads return in order, so the token is quantised into LDS,
// as the row quantiser does it, while W is under way.  The instruction is
// 16 x 16 x 64: lane l takes 16 bytes of row l % 16 at 16 (l / 16); the
// token is the only row of the first operand that is not zero.
// CH: chunks of eight elements a thread holds of the token.
// Bound by the weight's bytes: 4096 -> 14336 in 13.4 us (58.7 MB, 4.4 TB/s);
// quantiser and product as two launches 16.7.
constexpr int64_t kI8TokenPitch = 16384;  // longest token: 512 threads of 4 chunks

struct I8TokenParams {
  I8QuantParams x;  // src, dtype, rows = 1, cols = K, ld, vec
  int64_t N, pitch;
  const int8_t* w;  // [N][pitch]
  const float* sw;  // [N]
  void* y;
  int bf16;         // y is bf16 (else fp32)
};

template <int NW, int U, int CH>
__global__ __launch_bounds__(64 * NW, 4) void i8_linear_token_kernel(I8TokenParams p) {
  constexpr int T = 64 * NW;
  __shared__ __attribute__((aligned(16))) int8_t codes[T * CH * 8];
  __shared__ float red[NW];
  __shared__ int sum[NW][16];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int li = lane & 15, hq = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int steps = (int)(p.pitch >> 6);
  float x[CH][8];
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int64_t c = ((int64_t)threadIdx.x + T * j) * 8;
    i8_load8(p.x, 0, c, (int)min((int64_t)8, max((int64_t)0, p.x.cols - c)), x[j]);
  }
  const int8_t* const w = p.w + min(n0 + li, p.N - 1) * p.pitch + 16 * hq;
  i32x4_t fw[U];
  auto fetch = [&](int s0) {
#pragma unroll
    for (int u = 0; u < U; ++u) fw[u] = s0 + u < steps ? *(const i32x4_t*)(w + (int64_t)(s0 + u) * 64) : i32x4_t{};
  };
  fetch(wave * U);

  float top = 0.0f;
  bool bad = false;
#pragma unroll
  for (int j = 0; j < CH; ++j) top = i8_absmax8(x[j], top, bad);
  top = wave_max(top);
  if (lane == 0) red[wave] = top;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < NW; ++k) top = fmaxf(top, red[k]);
  if (bad) raise_status(kStatusNonFinite);
  const float s = i8_scale(top), inv = i8_inverse(s);
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    int q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = i8_code<false>(x[j][i], inv, 0.0f);
    *(uint2*)(codes + (threadIdx.x + T * j) * 8) = make_uint2(pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]));
  }
  __syncthreads();

  i32x4_t acc{};
  for (int s0 = wave * U; s0 < steps; s0 += NW * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const i32x4_t fx = li == 0 && s0 + u < steps ? *(const i32x4_t*)(codes + (s0 + u) * 64 + 16 * hq) : i32x4_t{};
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(fx, fw[u], acc, 0, 0, 0);
    }
    if (s0 + NW * U < steps) fetch(s0 + NW * U);
  }
  // the token's sums: first value of the first 16 lanes, one a column
  if (lane < 16) sum[wave][lane] = acc[0];
  __syncthreads();
  const int64_t col = n0 + threadIdx.x;
  if (threadIdx.x >= 16 || col >= p.N) return;
  int total = 0;
#pragma unroll
  for (int k = 0; k < NW; ++k) total += sum[k][threadIdx.x];
  const float c = (float)total * s * p.sw[col];
  if (p.bf16) ((uint16_t*)p.y)[col] = i8_bf16(c);
  else ((float*)p.y)[col] = c;
}

}  // namespace metis
