// dropout.hpp -- dropout from a counter-based generator, with an optional
// residual added; the mask is never stored.
//
// Element e (its row-major position) of the matrix takes the 16-bit Philox
// draw h(e) of (seed, tag with role 8, step), the stream that stochastic
// rounding draws from; with t = 65536 p rounded to an integer,
//   y = [h >= t] (x s) + residual,  s = 65536 / (65536 - t),
// so a value is kept with probability exactly 1 / s and the mean is x.  A
// dropped value counts as zero whatever it is (infinite and NaN too).  The
// backward pass is the same call on dy without a residual.
//
// One Philox block serves eight elements, which a thread loads as 16 bytes
// (bf16) or 32.  Bound by memory, the ten Philox rounds hidden behind it: 16384
// x 4096 bf16, forward with a residual and backward 122 to 130 us, 5.2 to 5.5
// TB/s.
#pragma once

#include "rows.hpp"

namespace metis {

constexpr uint32_t kRoleDropout = 8;

struct DropoutParams {
  const void *x, *res;  // res or null
  void* y;
  int64_t rows, cols, ldx, ldr, ldy;
  int bf16;
  uint32_t t;           // dropped below, of 65536
  float scale;
  uint64_t seed;
  uint32_t tag, step;   // tag with the role
  const int64_t* step_count;
};

// FLAT: rows without gaps, 16-byte aligned (cols = all elements).  Otherwise
// the eight elements of a block lie anywhere.
template <bool FLAT>
__global__ __launch_bounds__(256) void dropout_kernel(DropoutParams p) {
  const int64_t n = FLAT ? p.cols : p.rows * p.cols, blocks = (n + 7) >> 3;
  const int64_t count = p.step_count ? *p.step_count : -1;
  const uint32_t step = count < 0 ? p.step : (uint32_t)count;
  for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < blocks; q += (int64_t)gridDim.x * 256) {
    const int64_t e0 = q * 8;
    const int m = (int)min((int64_t)8, n - e0);
    if (FLAT && m == 8) {
      float x[8], r[8];
      load8(p.x, p.bf16, e0, x);
      if (p.res) load8(p.res, p.bf16, e0, r);
      const Philox4 h = philox_block((uint64_t)q, p.tag, step, p.seed);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = philox_half_of(h, e) >= p.t ? x[e] * p.scale : 0.0f;
        if (p.res) x[e] += r[e];
      }
      store8(p.y, p.bf16, e0, x);
    } else {
      const Philox4 h = philox_block((uint64_t)q, p.tag, step, p.seed);
      int64_t row = FLAT ? 0 : e0 / p.cols, col = e0 - row * p.cols;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e < m) {
          float v = philox_half_of(h, e) >= p.t ? load1(p.x, p.bf16, row * p.ldx + col) * p.scale : 0.0f;
          if (p.res) v += load1(p.res, p.bf16, row * p.ldr + col);
          store1(p.y, p.bf16, row * p.ldy + col, v);
          if (++col == p.cols && !FLAT) {
            col = 0;
            ++row;
          }
        }
      }
    }
  }
}

}  // namespace metis
