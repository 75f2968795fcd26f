// norm.hpp -- layer norm of rows, forward and backward.
//
//   mu = mean_j x_ij,  r = 1 / sqrt(mean_j (x_ij - mu)^2 + eps),
//   h_ij = (x_ij - mu) r,  y_ij = h_ij w_j + b_j;
// with g = dy w:
//   dx_ij = r (g_ij - mean_j g_ij - h_ij mean_j (g_ij h_ij)),
//   dw_j = sum_i dy_ij h_ij,  db_j = sum_i dy_ij.
// Bound by memory: 16384 x 4096 bf16 forward 47 to 50 us (5.4 to 5.7 TB/s),
// backward 83 to 87 + 5 (4.6 to 4.8 TB/s), the card's copy rate being 4.7 to 5.1.
// Rows that 16 bytes do not divide go a value at a time: 16384 x 4095 bf16
// forward 67 us, backward with the sums 122; of 4097, where a thread has twice
// the columns and half of them are none, 121 and 277; binary32 8192 x 769 as
// fast as x 768 (14 and 21).
//
// Sums in binary32; the variance is that of the centred values, never a
// difference of sums.  Only y and dx (and dw, db of bf16 weights) are rounded
// to fewer bits, once.
//
// T threads share a row and hold it in registers, so that x is read once: a
// wave up to 2048 columns, workgroups of 256 and 512 threads up to 8192 and
// 16384.  Each thread keeps its columns of w and b (and of the sums dw, db)
// for all rows that it takes.  The sums of dw and db end in a row of partial
// sums for each workgroup, added by a second kernel in the order of the
// workgroups, so that equal calls give equal bits.  Longer rows are read from
// memory again for each sum.
#pragma once

#include <type_traits>

#include "rows.hpp"

namespace metis {

constexpr int kNormThreads = 1024;     // of a long row
constexpr int kNormCols = 16384;       // longest row in registers
constexpr int kNormSumRows = 64;       // rows of one partial sum of a long row's dw, db

struct NormParams {
  int64_t rows;
  int cols;
  const void *x, *w, *b;   // w, b or null
  int64_t ldx;
  int x_bf16, w_bf16, y_bf16;
  float eps, inv;          // inv = 1 / cols
  void* y;
  int64_t ldy;
  float *mean, *rstd;      // written forward (or null), read backward
  // backward
  const void* dy;          // y's type
  int64_t lddy;
  void* dx;                // x's type, or null
  int64_t lddx;
  float* part;             // [workgroups][2][cols], or null
};

// The columns of one thread: NV groups of VEC consecutive ones, the groups of
// neighbouring threads next to each other.
template <int VEC, int T, int NV>
struct NormCols {
  static constexpr int E = VEC * NV;
  static __device__ __forceinline__ int first(int t, int k) { return (t + T * k) * VEC; }

  static __device__ __forceinline__ void load(const void* p, int bf16, int64_t row, int cols, int t, float other, float* v) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = first(t, k);
      if (VEC == 8 && c + 8 <= cols) {
        load8(p, bf16, row + c, v + 8 * k);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[VEC * k + e] = c + e < cols ? load1(p, bf16, row + c + e) : other;
      }
    }
  }
  static __device__ __forceinline__ void store(void* p, int bf16, int64_t row, int cols, int t, const float* v) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = first(t, k);
      if (VEC == 8 && c + 8 <= cols) {
        store8(p, bf16, row + c, v + 8 * k);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (c + e < cols) store1(p, bf16, row + c + e, v[VEC * k + e]);
      }
    }
  }
};

// A row's values of one thread as they lie in memory, so that the next row's
// loads are in flight while a row is worked on: two 16-byte words a group of
// eight (bf16 fills the first), or a value a group of one.
template <int VEC, int T, int NV>
struct NormRaw {
  uint4 q[VEC == 8 ? 2 * NV : 1];
  uint32_t w[VEC == 8 ? 1 : NV];

  __device__ __forceinline__ void load(const void* p, int bf16, int64_t row, int cols, int t) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = NormCols<VEC, T, NV>::first(t, k), n = cols - c;
      if constexpr (VEC == 1) {
        w[k] = n <= 0 ? 0 : bf16 ? ((const uint16_t*)p)[row + c] : ((const uint32_t*)p)[row + c];
      } else if (bf16) {
        const uint16_t* const at = (const uint16_t*)p + row + c;
        if (n >= 8) {
          q[2 * k] = *(const uint4*)at;
        } else {
          auto two = [&](int i) { return (i < n ? at[i] : 0) | (uint32_t)(i + 1 < n ? at[i + 1] : 0) << 16; };
          q[2 * k] = make_uint4(two(0), two(2), two(4), two(6));
        }
      } else {
        const uint32_t* const at = (const uint32_t*)p + row + c;
        if (n >= 8) {
          q[2 * k] = *(const uint4*)at;
          q[2 * k + 1] = *((const uint4*)at + 1);
        } else {
          auto one = [&](int i) { return i < n ? at[i] : 0; };
          q[2 * k] = make_uint4(one(0), one(1), one(2), one(3));
          q[2 * k + 1] = make_uint4(one(4), one(5), one(6), one(7));
        }
      }
    }
  }

  // the values, zeros behind the row
  __device__ __forceinline__ void get(int bf16, float* v) const {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if constexpr (VEC == 1) {
        v[k] = __uint_as_float(bf16 ? w[k] << 16 : w[k]);
      } else {
        const uint4 a = q[2 * k], b = q[2 * k + 1];
        const uint32_t lo[4] = {a.x, a.y, a.z, a.w}, hi[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) v[8 * k + e] = bf16 ? unpack_bf16(lo[e >> 1], e) : __uint_as_float(e < 4 ? lo[e & 3] : hi[e & 3]);
      }
    }
  }
};

// The next row's loads go ahead where a thread has registers for them.
constexpr bool norm_ahead(int VEC, int NV) { return VEC * NV <= 16; }

// threads of a workgroup
constexpr int norm_block(int T) { return T < 256 ? 256 : T; }

template <int VEC, int T, int NV>
__global__ __launch_bounds__(norm_block(T)) void norm_fwd_kernel(NormParams p) {
  using C = NormCols<VEC, T, NV>;
  constexpr int E = C::E, G = norm_block(T) / T;  // G rows at a time
  __shared__ float red[2][T / 64];
  const int t = threadIdx.x & (T - 1);
  const int64_t step = (int64_t)gridDim.x * G;
  int64_t row = (int64_t)blockIdx.x * G + threadIdx.x / T;
  NormRaw<VEC, T, NV> raw;
  constexpr bool AHEAD = norm_ahead(VEC, NV);
  if (AHEAD && row < p.rows) raw.load(p.x, p.x_bf16, row * p.ldx, p.cols, t);
  float w[E], b[E];
#pragma unroll
  for (int e = 0; e < E; ++e) w[e] = 1.0f, b[e] = 0.0f;
  if (p.w) C::load(p.w, p.w_bf16, 0, p.cols, t, 0.0f, w);
  if (p.b) C::load(p.b, p.w_bf16, 0, p.cols, t, 0.0f, b);
  for (; row < p.rows; row += step) {
    float x[E], s = 0.0f;
    if (!AHEAD) raw.load(p.x, p.x_bf16, row * p.ldx, p.cols, t);
    raw.get(p.x_bf16, x);
    if (AHEAD && row + step < p.rows) raw.load(p.x, p.x_bf16, (row + step) * p.ldx, p.cols, t);
#pragma unroll
    for (int e = 0; e < E; ++e) s += x[e];
    const float mu = row_sum<T>(s, red[0]) * p.inv;
    s = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      x[e] -= mu;
      s += C::first(t, e / VEC) + e % VEC < p.cols ? x[e] * x[e] : 0.0f;
    }
    const float r = 1.0f / sqrtf(row_sum<T>(s, red[1]) * p.inv + p.eps);
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = x[e] * r * w[e] + b[e];
    C::store(p.y, p.y_bf16, row * p.ldy, p.cols, t, x);
    if (p.mean && t == 0) {
      p.mean[row] = mu;
      p.rstd[row] = r;
    }
  }
}

template <int VEC, int T, int NV>
__global__ __launch_bounds__(norm_block(T)) void norm_bwd_kernel(NormParams p) {
  using C = NormCols<VEC, T, NV>;
  constexpr int E = C::E, G = norm_block(T) / T;  // G rows at a time
  __shared__ float red[2][2][T / 64];
  const int t = threadIdx.x & (T - 1);
  const int64_t step = (int64_t)gridDim.x * G;
  int64_t row = (int64_t)blockIdx.x * G + threadIdx.x / T;
  NormRaw<VEC, T, NV> xr, gr;
  float mu = 0.0f, r = 0.0f;
  auto fetch = [&](int64_t i) {
    xr.load(p.x, p.x_bf16, i * p.ldx, p.cols, t);
    gr.load(p.dy, p.y_bf16, i * p.lddy, p.cols, t);
    mu = p.mean[i];
    r = p.rstd[i];
  };
  constexpr bool AHEAD = norm_ahead(VEC, NV);
  if (AHEAD && row < p.rows) fetch(row);
  float w[E], dw[E], db[E];
#pragma unroll
  for (int e = 0; e < E; ++e) w[e] = 1.0f, dw[e] = db[e] = 0.0f;
  if (p.w) C::load(p.w, p.w_bf16, 0, p.cols, t, 0.0f, w);
  int odd = 0;
  for (; row < p.rows; row += step, odd ^= 1) {
    float h[E], g[E], s = 0.0f, q = 0.0f;
    if (!AHEAD) fetch(row);
    const float m0 = mu, r0 = r;
    xr.get(p.x_bf16, h);
    gr.get(p.y_bf16, g);
    if (AHEAD && row + step < p.rows) fetch(row + step);
#pragma unroll
    for (int e = 0; e < E; ++e) {  // (g is 0 behind the row)
      h[e] = (h[e] - m0) * r0;
      dw[e] += g[e] * h[e];
      db[e] += g[e];
      g[e] *= w[e];
      s += g[e];
      q += g[e] * h[e];
    }
    if (!p.dx) continue;
    // both sums with one barrier; the arrays alternate
    s = wave_sum(s);
    q = wave_sum(q);
    if constexpr (T > 64) {
      if ((threadIdx.x & 63) == 0) red[odd][0][threadIdx.x >> 6] = s, red[odd][1][threadIdx.x >> 6] = q;
      __syncthreads();
      s = q = 0.0f;
#pragma unroll
      for (int k = 0; k < T / 64; ++k) s += red[odd][0][k], q += red[odd][1][k];
    }
    s *= p.inv;
    q *= p.inv;
#pragma unroll
    for (int e = 0; e < E; ++e) g[e] = r0 * (g[e] - s - h[e] * q);
    C::store(p.dx, p.x_bf16, row * p.lddx, p.cols, t, g);
  }
  if (!p.part) return;
  float* const to = p.part + (int64_t)blockIdx.x * 2 * p.cols;
  if constexpr (G > 1) {  // the waves of a workgroup one after the other
    __shared__ float sums[2][64 * E];
    for (int i = 0; i < G; ++i) {
      if (threadIdx.x / T == i) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          float* const a = &sums[0][e * 64 + t];
          float* const c = &sums[1][e * 64 + t];
          *a = dw[e] += i ? *a : 0.0f;
          *c = db[e] += i ? *c : 0.0f;
        }
      }
      __syncthreads();
    }
    if (threadIdx.x / T != G - 1) return;
  }
  C::store(to, 0, 0, p.cols, t, dw);
  C::store(to + p.cols, 0, 0, p.cols, t, db);
}

// sum of f(column) over a row by all threads of a long row's workgroup
// (columns as unsigned numbers: they run past 2^31 in a last step)
template <typename F>
__device__ inline float long_row_sum(uint32_t cols, float* red, F f) {
  float s = 0.0f;
  for (uint32_t c = threadIdx.x; c < cols; c += kNormThreads) s += f(c);
  __syncthreads();  // the array's last use
  return row_sum<kNormThreads>(s, red);
}

__global__ __launch_bounds__(kNormThreads) void norm_fwd_long_kernel(NormParams p) {
  __shared__ float red[kNormThreads / 64];
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    auto x = [&](uint32_t c) { return load1(p.x, p.x_bf16, row * p.ldx + c); };
    const float mu = long_row_sum(p.cols, red, x) * p.inv;
    auto square = [&](uint32_t c) {
      const float d = x(c) - mu;
      return d * d;
    };
    const float r = 1.0f / sqrtf(long_row_sum(p.cols, red, square) * p.inv + p.eps);
    for (uint32_t c = threadIdx.x; c < (uint32_t)p.cols; c += kNormThreads) {
      const float w = p.w ? load1(p.w, p.w_bf16, c) : 1.0f, b = p.b ? load1(p.b, p.w_bf16, c) : 0.0f;
      store1(p.y, p.y_bf16, row * p.ldy + c, (x(c) - mu) * r * w + b);
    }
    if (p.mean && threadIdx.x == 0) {
      p.mean[row] = mu;
      p.rstd[row] = r;
    }
  }
}

__global__ __launch_bounds__(kNormThreads) void norm_dx_long_kernel(NormParams p) {
  __shared__ float red[kNormThreads / 64];
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const float mu = p.mean[row], r = p.rstd[row];
    auto h = [&](uint32_t c) { return (load1(p.x, p.x_bf16, row * p.ldx + c) - mu) * r; };
    auto g = [&](uint32_t c) { return load1(p.dy, p.y_bf16, row * p.lddy + c) * (p.w ? load1(p.w, p.w_bf16, c) : 1.0f); };
    const float s = long_row_sum(p.cols, red, g) * p.inv;
    const float q = long_row_sum(p.cols, red, [&](uint32_t c) { return g(c) * h(c); }) * p.inv;
    for (uint32_t c = threadIdx.x; c < (uint32_t)p.cols; c += kNormThreads)
      store1(p.dx, p.x_bf16, row * p.lddx + c, r * (g(c) - s - h(c) * q));
  }
}

// partial sums of dw and db over kNormSumRows rows, a column a thread
__global__ __launch_bounds__(256) void norm_dw_long_kernel(NormParams p) {
  const int c = (int)(blockIdx.x * 256 + threadIdx.x);
  if (c >= p.cols) return;
  for (int64_t group = blockIdx.y; group * kNormSumRows < p.rows; group += gridDim.y) {
    float dw = 0.0f, db = 0.0f;
    const int64_t end = min((group + 1) * kNormSumRows, p.rows);
    for (int64_t row = group * kNormSumRows; row < end; ++row) {
      const float dy = load1(p.dy, p.y_bf16, row * p.lddy + c);
      dw += dy * ((load1(p.x, p.x_bf16, row * p.ldx + c) - p.mean[row]) * p.rstd[row]);
      db += dy;
    }
    p.part[group * 2 * p.cols + c] = dw;
    p.part[(group * 2 + 1) * p.cols + c] = db;
  }
}

// dw (blockIdx.y 0) and db (1) from the partial sums: 64 columns a workgroup
// at a time, its 16 waves take every sixteenth partial sum, in order, and their
// sums are added in order.
__global__ __launch_bounds__(1024) void norm_sum_kernel(const float* part, int64_t groups, int64_t cols, void* dw, void* db,
                                                        int w_bf16) {
  __shared__ float red[16][64];
  void* const to = blockIdx.y ? db : dw;
  if (!to) return;
  const int wave = threadIdx.x >> 6;
  for (int64_t c0 = (int64_t)blockIdx.x * 64; c0 < cols; c0 += (int64_t)gridDim.x * 64) {
    const int64_t c = c0 + (threadIdx.x & 63);
    float s = 0.0f;
    if (c < cols) {
      const float* at = part + (int64_t)blockIdx.y * cols + c;
      int64_t i = wave;
      for (; i + 112 < groups; i += 128) {  // eight in flight
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = at[(i + 16 * k) * 2 * cols];
#pragma unroll
        for (int k = 0; k < 8; ++k) s += v[k];
      }
      for (; i < groups; i += 16) s += at[i * 2 * cols];
    }
    red[wave][threadIdx.x & 63] = s;
    __syncthreads();
    if (!wave && c < cols) {
      s = 0.0f;
#pragma unroll
      for (int k = 0; k < 16; ++k) s += red[k][threadIdx.x];
      store1(to, w_bf16, c, s);
    }
    __syncthreads();  // the array's next use
  }
}

}  // namespace metis
