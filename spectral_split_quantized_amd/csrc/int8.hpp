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
// Code rows have a pitch of K rounded up to 256 bytes with zeros behind K, so
// the product's K loop has no tail.
//
// Both orientations together take one sweep for the row and column maxima and
// one for the codes.  Rows alone take one sweep: a row stays in registers
// between its maximum and its codes.
#pragma once

#include "quant.hpp"

namespace metis {

constexpr int kI8Pitch = 256;

__host__ __device__ inline int64_t i8_pitch(int64_t k) { return (k + kI8Pitch - 1) / kI8Pitch * kI8Pitch; }

struct I8QuantParams {
  const void* src;
  int dtype;
  int64_t rows, cols, ld;
  bool vec;          // rows start 16-byte aligned and ld keeps them so
  int8_t* codes0;    // [cols][i8_pitch(rows)] or null
  int8_t* codes1;    // [rows][i8_pitch(cols)] or null
  float* scales0;    // [cols]
  float* scales1;    // [rows]
  float* part0;      // [row tiles][cols] column maxima of a tile
  float* part1;      // [column tiles][rows] row maxima of a tile
  int sr;
  uint64_t seed;
  uint32_t tag, step;
};

__device__ inline float i8_scale(float amax) { return fmaxf(__fdiv_rn(amax, 127.0f), 0x1p-126f); }
__device__ inline float i8_inverse(float scale) { return __fdiv_rn(1.0f, scale); }

// u: the draw times 2^-16, or a negative value to round to nearest
template <bool SR>
__device__ inline int i8_code(float x, float inv, float u) {
  const float y = x * inv;
  float c;
  if constexpr (SR) {
    const float k = floorf(y);
    c = k + (u < y - k ? 1.0f : 0.0f);
  } else {
    c = rintf(y);
  }
  return (int)fminf(fmaxf(c, -127.0f), 127.0f);
}

__device__ inline uint32_t pack4(int a, int b, int c, int d) {
  return (uint32_t)(a & 255) | (uint32_t)(b & 255) << 8 | (uint32_t)(c & 255) << 16 | (uint32_t)(d & 255) << 24;
}

// eight consecutive elements of a row from column c (n of them exist)
__device__ inline void i8_load8(const I8QuantParams& p, int64_t row, int64_t c, int n, float (&x)[8]) {
  const int64_t at = row * p.ld + c;
  if (n == 8 && p.vec) {
    if (p.dtype == 0) {
      const uint4 q = *(const uint4*)((const uint16_t*)p.src + at);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
      const float4 a = *(const float4*)((const float*)p.src + at), b = *(const float4*)((const float*)p.src + at + 4);
      x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
      x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = i < n ? load_as_float(p.src, p.dtype, at + i) : 0.0f;
}

// draws (times 2^-16) of the row-major positions e .. e + 7
__device__ inline void i8_draws8(const I8QuantParams& p, uint64_t e, float (&u)[8]) {
  const Philox4 b0 = philox_block(e >> 3, p.tag, p.step, p.seed);
  const uint32_t o = (uint32_t)(e & 7);
  if (o == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = (float)philox_half_of(b0, i) * 0x1p-16f;
    return;
  }
  const Philox4 b1 = philox_block((e >> 3) + 1, p.tag, p.step, p.seed);
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
template <int W, int CH, bool SR>
__global__ __launch_bounds__(64 * W) void i8_quant_rows_kernel(I8QuantParams p) {
  constexpr int T = 64 * W;
  __shared__ float red[W];
  const int64_t row = blockIdx.x;
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
  auto put = [&](int64_t ch, const float (&y)[8]) {
    float u[8];
    if constexpr (SR) i8_draws8(p, (uint64_t)row * p.cols + ch * 8, u);
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
// Tiles of 128 rows x 128 columns, 256 threads: thread t holds the column
// chunk 8 (t % 16) .. + 7 of rows 4 (t / 16) .. + 3 and of the 64 rows further
// down.  The first sweep leaves each tile's row and column maxima, a small
// kernel joins them into scales, and the second sweep writes the codes, the
// transposed ones through LDS.
constexpr int kI8Tile = 128;

__global__ __launch_bounds__(256) void i8_amax_kernel(I8QuantParams p) {
  __shared__ float cmax[16][kI8Tile];
  const int64_t tiles_n = ceil_div<int64_t>(p.cols, kI8Tile);
  const int64_t tm = blockIdx.x / tiles_n, tn = blockIdx.x % tiles_n;
  const int cc = threadIdx.x & 15, rg = threadIdx.x >> 4;
  const int64_t c = tn * kI8Tile + cc * 8;
  const int n = (int)min((int64_t)8, max((int64_t)0, p.cols - c));
  float x[8][8], cm[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = tm * kI8Tile + rg * 4 + (i & 3) + (i >> 2) * 64;
    i8_load8(p, min(row, p.rows - 1), c, row < p.rows ? n : 0, x[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = tm * kI8Tile + rg * 4 + (i & 3) + (i >> 2) * 64;
    float rm = i8_absmax8(x[i], 0.0f, bad);
#pragma unroll
    for (int j = 0; j < 8; ++j) cm[j] = fmaxf(cm[j], fabsf(x[i][j]));
    if (p.part1) {
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) rm = fmaxf(rm, __shfl_xor(rm, o, 64));
      if (cc == 0 && row < p.rows) p.part1[tn * p.rows + row] = rm;
    }
  }
  if (bad) raise_status(kStatusNonFinite);
#pragma unroll
  for (int j = 0; j < 8; ++j) cmax[rg][cc * 8 + j] = cm[j];
  __syncthreads();
  if (threadIdx.x < kI8Tile && tn * kI8Tile + threadIdx.x < p.cols) {
    float m = 0.0f;
#pragma unroll
    for (int r = 0; r < 16; ++r) m = fmaxf(m, cmax[r][threadIdx.x]);
    p.part0[tm * p.cols + tn * kI8Tile + threadIdx.x] = m;
  }
}

// scales of the columns (first n0 threads), then of the rows
__global__ __launch_bounds__(256) void i8_scales_kernel(I8QuantParams p) {
  const int64_t n1 = p.part1 ? p.rows : 0;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= p.cols + n1) return;
  const bool col = id < p.cols;
  const int64_t i = col ? id : id - p.cols, n = col ? p.cols : p.rows;
  const int64_t tiles = ceil_div<int64_t>(col ? p.rows : p.cols, kI8Tile);
  const float* part = col ? p.part0 : p.part1;
  float m = 0.0f;
  for (int64_t t = 0; t < tiles; ++t) m = fmaxf(m, part[t * n + i]);
  (col ? p.scales0 : p.scales1)[i] = i8_scale(m);
}

template <bool SR>
__global__ __launch_bounds__(256) void i8_quant_tile_kernel(I8QuantParams p) {
  // transposed codes: column c at words c * kPitch .. + 31 (four rows a word)
  constexpr int kPitch = 33;
  __shared__ uint32_t tr[kI8Tile * kPitch];
  const int64_t pitch0 = i8_pitch(p.rows), pitch1 = i8_pitch(p.cols);
  const int64_t tiles_n = pitch1 / kI8Tile;
  const int64_t tm = blockIdx.x / tiles_n, tn = blockIdx.x % tiles_n;
  const int cc = threadIdx.x & 15, rg = threadIdx.x >> 4;
  const int64_t c = tn * kI8Tile + cc * 8;
  const int n = (int)min((int64_t)8, max((int64_t)0, p.cols - c));
  float inv0[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) inv0[j] = j < n ? i8_inverse(p.scales0[c + j]) : 0.0f;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float x[4][8];
    uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = tm * kI8Tile + half * 64 + rg * 4 + i;
      i8_load8(p, min(row, p.rows - 1), c, row < p.rows ? n : 0, x[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = tm * kI8Tile + half * 64 + rg * 4 + i;
      float u[8];
      if constexpr (SR) i8_draws8(p, (uint64_t)row * p.cols + c, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] |= (uint32_t)(i8_code<SR>(x[i][j], inv0[j], SR ? u[j] : 0.0f) & 255) << (8 * i);
      if (p.codes1 && row < p.rows) {
        const float inv = i8_inverse(p.scales1[row]);
        int q[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = i8_code<SR>(x[i][j], inv, SR ? u[j] : 0.0f);
        *(uint2*)(p.codes1 + row * pitch1 + c) =
            make_uint2(pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]));
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) tr[(cc * 8 + j) * kPitch + half * 16 + rg] = w[j];
  }
  __syncthreads();
  // 8 threads write a column's 128 bytes
  const int ci = threadIdx.x >> 3, part = threadIdx.x & 7;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t col = tn * kI8Tile + ci + 32 * k;
    const uint32_t* t = tr + (ci + 32 * k) * kPitch + part * 4;
    if (col < p.cols)
      *(uint4*)(p.codes0 + col * pitch0 + tm * kI8Tile + part * 16) = make_uint4(t[0], t[1], t[2], t[3]);
  }
}

}  // namespace metis
