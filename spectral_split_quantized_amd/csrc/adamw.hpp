// adamw.hpp -- AdamW over many tensors in one launch, states in binary32 or in
// 8 bits, and the global gradient norm that clips it.
//
// Per element, every operation rounded to binary32 on its own (g already
// times the clip coefficient):
//   m' = b1 m + (1 - b1) g,   v' = b2 v + ((1 - b2) g) g,   r' = sqrt(v'),
//   p' = p (1 - lr wd) - (lr / (1 - b1^t)) m' / (r' / sqrt(1 - b2^t) + eps).
// An element whose m', v' or p' is not finite keeps p, m and v and raises the
// numeric flag.  8-bit moments are kept as values, which are encoded again: the
// block has one scale, and its other elements move it.  A stored 8-bit moment
// that is itself not finite stays NaN and has no part in its block's scale.
//
// 8-bit states: E4M3 codes of m and of r = sqrt(v) (the square root halves
// the exponent range that v needs) in blocks of 256 consecutive elements,
// each with a power-of-two scale 2^(floor(log2 amax) - 7), at least 2^-126:
// scaling is exact and the largest element lies in [128, 256), inside the
// format even after rounding up.  Codes are rounded to nearest even or
// stochastically with 16-bit draws (the low half of the element's 32-bit
// Philox draw for m, the high half for r): a step changes v by a thousandth,
// far less than E4M3's spacing of an eighth, so to nearest a state would not
// move at all; stochastically it moves by the right amount on average.  A
// positive r never becomes zero, which would turn m / r into m / eps.
//
// A wave takes four state blocks, a lane four consecutive elements of each, so
// a block's maxima are joined inside the wave and every load of the wave is in
// flight at once.  Bound by HBM: 176 M binary32 elements in 827-915 us with
// 32-bit states (28 bytes an element, 5.4-6.0 TB/s between cards) and in 536 us
// with 8-bit states rounded stochastically (16.06 bytes, 5.3 TB/s); a copy runs
// at 5.1.  bf16 parameters and gradients with 32-bit states: 783 us (24 bytes,
// 5.4 TB/s).  With 8 bits the vector units are close behind: 95 instructions an
// element.
#pragma once

#include "common.hpp"
#include "quant_fast.hpp"
#include "status.hpp"

namespace metis {

constexpr int kStateBlock = 256;
constexpr uint32_t kRoleMoments = 6, kRoleParam = 7;

// E4M3 code of y in [0, 256): nearest even, or the dropped bits decided by
// the 16-bit draw h (up with probability floor(d / 16) / 65536, d the 20
// dropped bits).  Below 2^-6 the grid is 2^-9: y + 2^-6 has that spacing.
template <bool SR>
__host__ __device__ inline uint32_t state_encode(float y, uint32_t h) {
  const bool low = y < 0x1p-6f;
  const uint32_t b = __builtin_bit_cast(uint32_t, low ? y + 0x1p-6f : y);
  const uint32_t i = (b + (SR ? h << 4 : 0x7FFFFu + ((b >> 20) & 1u))) >> 20;
  return i - (low ? 968u : 960u);
}

// exponent (unbiased) of a block's scale from the bits of its largest magnitude
__host__ __device__ inline int state_exponent(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23) - 127 - 7;
  return e < -126 ? -126 : e;
}

// A launch's table of tensors travels as its kernel argument, at most 4 KB:
// nothing to copy or to keep, and a capture records it by value.
constexpr int kAdamWork = 4096;     // elements of one workgroup: 4 waves of 4 state blocks
constexpr int kNormTensors = 192;
constexpr int kNormWork = 16384;

template <bool EIGHT>
struct AdamTable {
  static constexpr int kTensors = EIGHT ? 60 : 80, kScales = EIGHT ? kTensors : 1;
  int count, p_bf16, g_bf16;
  float b1, c1, b2, c2, eps, decay;  // c1 = 1 - b1, c2 = 1 - b2, decay = 1 - lr wd
  float step_size, inv_c2;           // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  double lr, db1, db2;               // for a step count in device memory
  const int64_t* step_count;         // or null: the host's t
  const float* clip;                 // gradient factor, or null
  uint64_t seed;
  uint32_t step;
  uint32_t first[kTensors];          // first workgroup of each tensor
  uint32_t tag[kTensors];
  void* p[kTensors];
  const void* g[kTensors];
  void* m[kTensors];
  void* v[kTensors];
  float* ms[kScales];
  float* vs[kScales];
  int64_t n[kTensors];
};
static_assert(sizeof(AdamTable<true>) <= 4096 && sizeof(AdamTable<false>) <= 4096, "kernel arguments");

struct NormTable {
  int count, g_bf16;
  int64_t base;                      // first partial of this launch
  double* part;
  uint32_t first[kNormTensors];
  const void* g[kNormTensors];
  int64_t n[kNormTensors];
};
static_assert(sizeof(NormTable) <= 4096, "kernel arguments");

// the tensor of a workgroup: the last one that starts at or before it (the
// lanes compare all starts at once; tensors without elements start where
// their successor does and are never the last)
template <int CAP>
__device__ inline int table_index(const uint32_t* first, int count, uint32_t bid) {
  int found = 0;
#pragma unroll
  for (int o = 0; o < CAP; o += 64) {
    const int i = o + (int)(threadIdx.x & 63);
    const bool in = i < count && i < CAP && first[min(i, CAP - 1)] <= bid;
    found += __popcll(__ballot(in));
  }
  return __builtin_amdgcn_readfirstlane(found - 1);
}

// neither NaN nor infinite: one class compare
__device__ inline bool is_finite_class(float x) { return __builtin_amdgcn_classf(x, 0x1F8); }

// E4M3 byte I of a word
template <int I>
__device__ inline float state_decode(uint32_t w) {
  return __builtin_amdgcn_cvt_f32_fp8((int)w, I);
}

// four consecutive values from element e (n of them exist)
__device__ inline void load4(const void* base, bool bf16, int64_t e, int n, bool vec, float (&x)[4]) {
  if (n == 4 && vec) {
    if (bf16) {
      const uint2 q = *(const uint2*)((const uint16_t*)base + e);
      x[0] = __uint_as_float(q.x << 16), x[1] = __uint_as_float(q.x & 0xFFFF0000u);
      x[2] = __uint_as_float(q.y << 16), x[3] = __uint_as_float(q.y & 0xFFFF0000u);
    } else {
      const float4 q = *(const float4*)((const float*)base + e);
      x[0] = q.x, x[1] = q.y, x[2] = q.z, x[3] = q.w;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = i < n ? load_as_float(base, bf16 ? 0 : 1, e + i) : 0.0f;
}

__device__ inline void store4(float* base, int64_t e, int n, bool vec, const float (&x)[4]) {
  if (n == 4 && vec) {
    *(float4*)(base + e) = make_float4(x[0], x[1], x[2], x[3]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) base[e + i] = x[i];
}

__device__ inline uint32_t load_codes4(const uint8_t* base, int64_t e, int n, bool vec) {
  if (n == 4 && vec) return *(const uint32_t*)(base + e);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) w |= (uint32_t)base[e + i] << (8 * i);
  return w;
}

__device__ inline void store_codes4(uint8_t* base, int64_t e, int n, bool vec, uint32_t w) {
  if (n == 4 && vec) {
    *(uint32_t*)(base + e) = w;
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) base[e + i] = (uint8_t)(w >> (8 * i));
}

__device__ inline float pow2_float(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126..127

template <bool EIGHT, bool SR>
__global__ __launch_bounds__(256) void adamw_kernel(AdamTable<EIGHT> t) {
  constexpr int NB = 4;  // state blocks a wave
  const int ti = table_index<AdamTable<EIGHT>::kTensors>(t.first, t.count, blockIdx.x);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t n = t.n[ti];
  const int64_t block0 = (int64_t)(blockIdx.x - t.first[ti]) * (kAdamWork / kStateBlock) + wave * NB;
  if (block0 * kStateBlock >= n) return;
  void* const pp = t.p[ti];
  const void* const gp = t.g[ti];
  void* const mp = t.m[ti];
  void* const vp = t.v[ti];
  const bool vec = (((uintptr_t)pp | (uintptr_t)gp | (EIGHT ? 0 : (uintptr_t)mp | (uintptr_t)vp)) & 15) == 0 &&
                   (((uintptr_t)mp | (uintptr_t)vp) & 3) == 0;
  const float gs = t.clip ? *t.clip : 1.0f;
  float step_size = t.step_size, inv_c2 = t.inv_c2;
  uint32_t step = t.step;
  if (t.step_count) {  // b^t by squaring, in binary64
    const int64_t s = *t.step_count;
    double x1 = t.db1, x2 = t.db2, y1 = 1.0, y2 = 1.0;
    for (uint64_t q = (uint64_t)s; q; q >>= 1) {
      if (q & 1) y1 *= x1, y2 *= x2;
      x1 *= x1, x2 *= x2;
    }
    step_size = (float)(t.lr / (1.0 - y1));
    inv_c2 = (float)(1.0 / sqrt(1.0 - y2));
    step = (uint32_t)s;
  }

  float p[NB][4], g[NB][4], m[NB][4], v[NB][4];
  uint32_t mc[NB], vc[NB];
  float ms[NB], vs[NB];
  int cnt[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int64_t e = (block0 + b) * kStateBlock + lane * 4;
    cnt[b] = (int)min((int64_t)4, max((int64_t)0, n - e));
    load4(pp, t.p_bf16, e, cnt[b], vec, p[b]);
    load4(gp, t.g_bf16, e, cnt[b], vec, g[b]);
    if constexpr (EIGHT) {
      mc[b] = load_codes4((const uint8_t*)mp, e, cnt[b], vec);
      vc[b] = load_codes4((const uint8_t*)vp, e, cnt[b], vec);
      const bool have = (block0 + b) * kStateBlock < n;
      ms[b] = have ? t.ms[ti][block0 + b] : 0.0f;
      vs[b] = have ? t.vs[ti][block0 + b] : 0.0f;
    } else {
      load4(mp, false, e, cnt[b], vec, m[b]);
      load4(vp, false, e, cnt[b], vec, v[b]);
    }
  }
  bool bad = false;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int64_t e = (block0 + b) * kStateBlock + lane * 4;
    if ((block0 + b) * kStateBlock >= n) break;
    float r[4], m1[4], v1[4], r1[4], p1[4];
    if constexpr (EIGHT) {
      m[b][0] = state_decode<0>(mc[b]), m[b][1] = state_decode<1>(mc[b]);
      m[b][2] = state_decode<2>(mc[b]), m[b][3] = state_decode<3>(mc[b]);
      r[0] = state_decode<0>(vc[b]), r[1] = state_decode<1>(vc[b]);
      r[2] = state_decode<2>(vc[b]), r[3] = state_decode<3>(vc[b]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m[b][i] *= ms[b];
        r[i] *= vs[b];
        v[b][i] = r[i] * r[i];
      }
    }
    bool ok = true;
    uint32_t nan_m = 0, nan_r = 0;  // codes of moments that stay NaN
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float gr = t.clip ? g[b][i] * gs : g[b][i];
      m1[i] = t.b1 * m[b][i] + t.c1 * gr;
      v1[i] = t.b2 * v[b][i] + t.c2 * gr * gr;
      r1[i] = sqrtf(v1[i]);
      // the hardware reciprocal is within one unit in the last place, far
      // below what the parameter's own rounding leaves of the step
      const float upd = m1[i] * __builtin_amdgcn_rcpf(r1[i] * inv_c2 + t.eps);
      p1[i] = p[b][i] * t.decay - step_size * upd;
      // an m' that is not finite makes p' so, unless v' is not finite either
      ok &= is_finite_class(v1[i]) && is_finite_class(p1[i]);
    }
    if (!__all(ok)) {  // rare: such elements keep what they had (places behind the end do not count)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (is_finite_class(v1[i]) && is_finite_class(p1[i])) continue;
        bad |= i < cnt[b];
        m1[i] = m[b][i];
        v1[i] = v[b][i];
        r1[i] = EIGHT ? fabsf(r[i]) : 0.0f;
        p1[i] = p[b][i];
        if constexpr (EIGHT) {  // as zeros they leave the block's maxima to the others
          if (!is_finite_class(m1[i])) m1[i] = 0.0f, nan_m |= 0x7Fu << (8 * i);
          if (!is_finite_class(r1[i])) r1[i] = 0.0f, nan_r |= 0x7Fu << (8 * i);
        }
      }
    }
    uint32_t am = 0, ar = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[b][i] = m1[i];
      v[b][i] = v1[i];
      r[i] = r1[i];
      p[b][i] = p1[i];
      if constexpr (EIGHT) {
        am = max(am, __float_as_uint(m1[i]) & 0x7FFFFFFFu);
        ar = max(ar, __float_as_uint(r1[i]));
      }
    }
    if (t.p_bf16) {
      uint32_t h[4] = {0, 0, 0, 0};
      if constexpr (SR) {
        const Philox4 d = philox_block((uint64_t)e >> 2, tag_with_role(t.tag[ti], kRoleParam), step, t.seed);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = d.v[i] & 0xFFFFu;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t u = __float_as_uint(p[b][i]);
        if (i < cnt[b]) ((uint16_t*)pp)[e + i] = (uint16_t)((u + (SR ? h[i] : 0x7FFFu + ((u >> 16) & 1u))) >> 16);
      }
    } else {
      store4((float*)pp, e, cnt[b], vec, p[b]);
    }
    if constexpr (EIGHT) {
      const int em = state_exponent(wave_max_u32(am)), er = state_exponent(wave_max_u32(ar));
      const float im = pow2_float(-em), ir = pow2_float(-er);
      Philox4 d{};
      if constexpr (SR) d = philox_block((uint64_t)e >> 2, tag_with_role(t.tag[ti], kRoleMoments), step, t.seed);
      uint32_t wm = 0, wr = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t u = __float_as_uint(m[b][i]);
        const uint32_t cm = state_encode<SR>(__uint_as_float(u & 0x7FFFFFFFu) * im, d.v[i] & 0xFFFFu);
        uint32_t cr = state_encode<SR>(r[i] * ir, d.v[i] >> 16);
        cr = cr == 0 && r[i] != 0.0f ? 1u : cr;
        wm |= (cm | (m[b][i] < 0.0f ? 0x80u : 0u)) << (8 * i);
        wr |= cr << (8 * i);
      }
      store_codes4((uint8_t*)mp, e, cnt[b], vec, wm | nan_m);
      store_codes4((uint8_t*)vp, e, cnt[b], vec, wr | nan_r);
      if (lane == 0) {
        t.ms[ti][block0 + b] = pow2_float(em);
        t.vs[ti][block0 + b] = pow2_float(er);
      }
    } else {
      store4((float*)mp, e, cnt[b], vec, m[b]);
      store4((float*)vp, e, cnt[b], vec, v[b]);
    }
  }
  if (bad) raise_status(kStatusNonFinite);
}

// ------------------------------------------------------------ global norm --
//
// Squares are exact in binary64 and summed there, in an order that the sizes
// alone fix, so the norm does not depend on how the work is spread.  One read
// of the gradients (148 tensors, 57 MB: 12 us), then a workgroup that joins the
// partial sums (4 us, latency).
__global__ __launch_bounds__(256) void grad_norm_kernel(NormTable t) {
  __shared__ double red[4];
  const int ti = table_index<kNormTensors>(t.first, t.count, blockIdx.x);
  const int64_t n = t.n[ti];
  const void* const gp = t.g[ti];
  const int64_t e0 = (int64_t)(blockIdx.x - t.first[ti]) * kNormWork;
  const bool vec = ((uintptr_t)gp & 15) == 0;
  double s = 0.0;
#pragma unroll 4
  for (int k = 0; k < kNormWork / 1024; ++k) {
    const int64_t e = e0 + k * 1024 + threadIdx.x * 4;
    float x[4];
    load4(gp, t.g_bf16, e, (int)min((int64_t)4, max((int64_t)0, n - e)), vec, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) s += (double)x[i] * (double)x[i];
  }
  s = wave_sum_d(s);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) t.part[t.base + blockIdx.x] = (red[0] + red[1]) + (red[2] + red[3]);
}

__global__ __launch_bounds__(1024) void grad_norm_final_kernel(const double* part, int64_t n, double max_norm,
                                                               float* out) {
  __shared__ double red[16];
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += 1024) s += part[i];
  s = wave_sum_d(s);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double v = 0.0;
    for (int i = 0; i < 16; ++i) v += red[i];
    const double norm = sqrt(v), c = max_norm / (norm + 1e-6);
    out[0] = (float)norm;
    out[1] = norm != norm ? (float)norm : (float)(c < 1.0 ? c : 1.0);  // NaN stays NaN
  }
}

}  // namespace metis
