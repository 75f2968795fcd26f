// loss.hpp -- softmax cross entropy over a vocabulary of the logits x W^T, in
// pieces of the vocabulary: the logits exist in the matrix cores' accumulators
// only (bf16_gemm.hpp), never in memory.
//
//   l_iv = x_i . w_v,  lse_i = log sum_v exp l_iv,  loss_i = lse_i - l_it(i);
// with G_i the gradient of loss_i:
//   P_iv = G_i (exp(l_iv - lse_i) - [v = t(i)]),  dx = P W,  dW = P^T x.
// Forward: a product whose epilogue leaves, for each token and 64 words, the
// largest logit and the sum of exponentials below it; they are joined here in
// a fixed order.  Backward, for a piece of words at a time: the product again,
// whose epilogue forms P (rounded to binary16, or to a pair of planes where a
// gradient is binary32), then the two products of the gradients.  So the
// backward pass spends 8 operations where keeping all logits would spend 6,
// and its memory does not grow with the vocabulary.  Bound by the products:
// 8192 tokens of 128256 words x 4096 bf16, forward 6.1 ms, backward 20.0, of
// which the logits again 6.7, dx 6.3, dw 6.3, planes and largest values 0.7 (3 %
// more on another card); a large library product of that shape takes 5.8.
// (8192 x 50257 x 768: bf16 0.55 and 2.1 ms, bf16 tokens with a binary32 weight
// 1.14 and 3.2, binary32 1.63 and 5.7.)
//
// dx and dw are products of binary16 because P in bf16, rounded by 2^-8 of
// itself, left a bf16 dx off by 0.0025 of its norm where its own rounding gives
// 0.0017; with binary16 (2^-11) it is 0.0017, for 4 % of the time.
//
// A token whose target is ignore_index, or not a word (which raises the status
// flag), has loss 0 and gradients 0, whatever its x holds.
#pragma once

#include "bf16_gemm.hpp"

namespace metis {

// What the products take of rows that they cannot take as they lie in memory:
// planes[row][pitch], zeros behind cols, in the rows behind `rows` up to
// out_rows, and, masked, in the rows of tokens without a part in the loss.
// `shift` null: bf16 rows copied.  Else the binary16 planes that the product's
// file describes, whose scale comes from the largest finite value: one launch
// takes the largest values (each workgroup leaves its own, so that nothing has
// to be cleared before), the next joins them, leaves the s in `shift` and makes
// the planes.  Both are bound by memory; a piece of a bf16 weight that
// 8192 tokens or more meet is small enough to stay in the cache behind the
// memory (256 MB) between them, at up to 4096 features.
struct PlanesJob {
  const void* src;  // null: no planes, just the s (of the gradients of the losses)
  int64_t rows, cols, ld;
  int bf16, masked;
  uint16_t* dst;
  int64_t out_rows, pitch, plane;  // pitch and plane in values; plane 0: one plane
  int* shift;
  uint32_t* top;       // [kTopBlocks] largest values of the workgroups, their bits
  const void* values;  // what `top` is taken of (src, or the gradients)
  const float* count;  // null, or what the gradients are divided by
  const float* weigh;  // null, or a gradient for each row: the rows for P^T x, see below
  int top_blocks, blocks;
  int flat;  // the values of all rows follow each other
};

// Where each token has a gradient g_i of its own, its row of P has an s_i of its
// own, by which the row of dx is scaled back; in P^T x the tokens are summed, so
// there the rows are x_i 2^-s_i (2^s with the s of them all), and a row counts as
// much as its gradient lets it.  `top` holds exponents of them then, from 1 on:
// their range is wider than binary32's.  A token with a gradient of 0 has no
// part.
constexpr int kTopBlocks = 1024, kPlaneJobs = 3, kWeighedZero = 512;

struct PlanesParams {
  PlanesJob job[kPlaneJobs];
  const void* targets;
  int targets64;
  int64_t vocab, ignore;
  int* zero;  // null, or set to zero
};

// eight consecutive values at any address of theirs
template <bool BF>
__device__ __forceinline__ void load8_anywhere(const void* p, int64_t at, float* v) {
  typedef uint32_t u32x4_2_t __attribute__((ext_vector_type(4), aligned(2)));
  typedef uint32_t u32x4_4_t __attribute__((ext_vector_type(4), aligned(4)));
  if constexpr (BF) {
    const u32x4_2_t q = *(const u32x4_2_t*)((const uint16_t*)p + at);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = unpack_bf16(q[i >> 1], i);
  } else {
    const u32x4_4_t a = *(const u32x4_4_t*)((const float*)p + at), b = *(const u32x4_4_t*)((const float*)p + at + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(i < 4 ? a[i & 3] : b[i & 3]);
  }
}

// Calls f(row, column, v) for blocks of eight values of the rows up to out_rows
// of `pitch` columns (a multiple of 8), zeros where there is no value: all
// workgroups of a job share them, four loads in flight a thread.
template <bool WEIGH, bool BF, class F>
__device__ __forceinline__ void each8(const PlanesJob& j, const PlanesParams& p, int64_t out_rows, int64_t pitch, int block,
                                      int blocks, const void* from, F f) {
  constexpr int K = 4;
  const int64_t per = pitch >> 3, total = out_rows * per;
  const int64_t stride = (int64_t)blocks * 256;
  for (int64_t id0 = (int64_t)block * 256 + threadIdx.x; id0 < total; id0 += K * stride) {
    float v[K][8];
    int64_t row[K];
    int col[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t id = id0 + k * stride;
      row[k] = total <= UINT32_MAX ? (int64_t)((uint32_t)id / (uint32_t)per) : id / per;
      const int64_t c = (id - row[k] * per) * 8;
      if (id >= total) row[k] = -1;
      col[k] = (int)c;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[k][e] = 0.0f;
      if (row[k] < 0 || row[k] >= j.rows) continue;
      if (j.masked && target_of(p.targets, p.targets64, p.ignore, p.vocab, row[k]) < 0) continue;
      if (WEIGH && j.weigh && loss_gradient(j.weigh, j.count, 1, row[k]) == 0.0f) continue;
      const int64_t at = row[k] * j.ld + c;
      if (c + 8 <= j.cols) {
        load8_anywhere<BF>(from, at, v[k]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e < j.cols) v[k][e] = load1(from, BF, at + e);
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (row[k] >= 0) f(row[k], col[k], v[k]);
  }
}

__device__ __forceinline__ uint32_t top_of_workgroup(uint32_t top, uint32_t* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
  __syncthreads();
  return max(max(red[0], red[1]), max(red[2], red[3]));
}

// the job of a workgroup and its number there
__device__ __forceinline__ int job_of(const int* blocks, int& block) {
  int j = 0;
  block = blockIdx.x;
  while (j + 1 < kPlaneJobs && block >= blocks[j]) block -= blocks[j++];
  return j;
}

// WEIGH: a job has rows weighed by gradients (a training pass of 1001 x 10007 x
// 1001 binary32 without such: 378.5 us, with one kernel for both cases 380.5).
template <bool WEIGH>
__global__ __launch_bounds__(256) void top_kernel(PlanesParams p) {
  __shared__ uint32_t red[4];
  const int blocks[kPlaneJobs] = {p.job[0].top_blocks, p.job[1].top_blocks, p.job[2].top_blocks};
  int block;
  PlanesJob j = p.job[job_of(blocks, block)];
  if (j.flat) j.cols *= j.rows, j.rows = 1;
  uint32_t top = 0;  // of values of one sign, larger bits are larger values
  auto take = [&](int64_t row, int, const float* v) {
    uint32_t here = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t b = __float_as_uint(v[e]) & 0x7FFFFFFFu;
      if (b < 0x7F800000u) here = max(here, b);
    }
    if (WEIGH && j.weigh && here) here = (here >> 23) + kWeighedZero - gradient_shift(loss_gradient(j.weigh, j.count, 1, row));
    top = max(top, here);
  };
  const int64_t pitch = (j.cols + 7) & ~(int64_t)7;
  if (j.bf16) each8<WEIGH, true>(j, p, j.rows, pitch, block, j.top_blocks, j.values, take);
  else each8<WEIGH, false>(j, p, j.rows, pitch, block, j.top_blocks, j.values, take);
  top = top_of_workgroup(top, red);
  if (threadIdx.x == 0) j.top[block] = top;
}

template <bool WEIGH>
__global__ __launch_bounds__(256) void planes_kernel(PlanesParams p) {
  __shared__ uint32_t red[4];
  const int blocks[kPlaneJobs] = {p.job[0].blocks, p.job[1].blocks, p.job[2].blocks};
  int block;
  const PlanesJob j = p.job[job_of(blocks, block)];
  if (p.zero && blockIdx.x == 0 && threadIdx.x == 0) *p.zero = 0;
  float scale = 1.0f;
  int s = 0;
  if (j.shift) {
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < kTopBlocks / 256; ++k)
      if (k * 256 + (int)threadIdx.x < j.top_blocks) top = max(top, j.top[k * 256 + threadIdx.x]);
    top = top_of_workgroup(top, red);
    if (WEIGH && j.weigh) {
      s = top == 0 ? 14 : 14 - ((int)top - kWeighedZero - 127);
    } else {
      if (j.count) top = __float_as_uint(__uint_as_float(top) / j.count[0]);
      // (2^126 is the largest power of two whose inverse is no subnormal; no
      // value but 0, or no finite quotient: 14)
      s = top == 0 || top >= 0x7F800000u ? 14 : min(14 - ((int)(top >> 23) - 127), 126);
      scale = __builtin_ldexpf(1.0f, s);
    }
    if (block == 0 && threadIdx.x == 0) *j.shift = s;
  }
  if (!j.src) return;
  auto store = [&](int64_t row, int col, const float* v) {
    uint32_t h[4], l[4];
    const int weight = WEIGH && j.weigh && row < j.rows ? s - gradient_shift(loss_gradient(j.weigh, j.count, 1, row)) : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = WEIGH && j.weigh ? __builtin_ldexpf(v[2 * i], weight) : v[2 * i] * scale;
      const float b = WEIGH && j.weigh ? __builtin_ldexpf(v[2 * i + 1], weight) : v[2 * i + 1] * scale;
      h[i] = j.shift ? pack_f16(a, b) : pack_bf16(a, b);
      if (j.plane) l[i] = pack_f16(rest_f16(a, unpack_f16(h[i], 0)), rest_f16(b, unpack_f16(h[i], 1)));
    }
    uint16_t* const to = j.dst + row * j.pitch + col;
    *(uint4*)to = make_uint4(h[0], h[1], h[2], h[3]);
    if (j.plane) *(uint4*)(to + j.plane) = make_uint4(l[0], l[1], l[2], l[3]);
  };
  if (j.bf16) each8<WEIGH, true>(j, p, j.out_rows, j.pitch, block, j.blocks, j.src, store);
  else each8<WEIGH, false>(j, p, j.out_rows, j.pitch, block, j.blocks, j.src, store);
}

// Loss and log-sum-exp of each token from its statistics, 16 tokens a
// workgroup: 64 threads share a token, each takes every 64th block in order,
// and their results are joined in order.  The last workgroup to end (a counter
// in the workspace, zeroed by the product's launch before) adds the losses:
// total[0] their sum, or their mean over the tokens that have one (0 where
// none has), total[1] the number of those tokens, in binary64 and in an order
// that does not depend on which workgroup it is.
struct LossJoinParams {
  const float2* stat;  // [blocks][tokens]
  int64_t blocks, tokens;
  const float* target_logit;
  const void* targets;
  int targets64;
  int64_t vocab, ignore;
  float *losses, *lse;
  int mean;
  float* total;        // or null
  uint32_t* done;
  int* status;
};

__global__ __launch_bounds__(1024) void loss_join_kernel(LossJoinParams p) {
  __shared__ float2 red[64][16];
  __shared__ bool last;
  const int token = threadIdx.x & 15, part = threadIdx.x >> 4;
  const int64_t row = (int64_t)blockIdx.x * 16 + token;
  float m = -__builtin_inff(), s = 0.0f;
  auto join = [&](float m2, float s2) {
    const float top = fmaxf(m, m2), at = top == -__builtin_inff() ? 0.0f : top;
    // (max leaves out a NaN; it comes back through the sum)
    s = s * __builtin_amdgcn_exp2f((m - at) * kLog2E) + s2 * __builtin_amdgcn_exp2f((m2 - at) * kLog2E);
    m = top;
  };
  if (row < p.tokens) {
    int64_t b = part;
    for (; b + 448 < p.blocks; b += 512) {  // eight loads in flight
      float2 v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = p.stat[(b + 64 * k) * p.tokens + row];
#pragma unroll
      for (int k = 0; k < 8; ++k) join(v[k].x, v[k].y);
    }
    for (; b < p.blocks; b += 64) {
      const float2 v = p.stat[b * p.tokens + row];
      join(v.x, v.y);
    }
  }
  red[part][token] = make_float2(m, s);
  __syncthreads();
#pragma unroll
  for (int half = 32; half > 0; half >>= 1) {
    if (part < half) {
      const float2 o = red[part + half][token];
      join(o.x, o.y);
      red[part][token] = make_float2(m, s);
    }
    __syncthreads();
  }
  if (part == 0 && row < p.tokens) {
    const float lse = m + logf(s);
    p.lse[row] = lse;
    const int64_t t = target_of(p.targets, p.targets64, p.ignore, p.vocab, row);
    const int64_t given = p.targets64 ? ((const int64_t*)p.targets)[row] : (int64_t)((const int32_t*)p.targets)[row];
    if (t < 0 && given != p.ignore) atomicOr(p.status, kStatusToken);
    __hip_atomic_store(p.losses + row, t >= 0 ? lse - p.target_logit[row] : 0.0f, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (!p.total) return;
  // The losses are stored past this XCD's L2 and have arrived before the count
  // goes up (a fence would write back all of the L2, which holds nothing else
  // that the last workgroup reads).
  __builtin_amdgcn_s_waitcnt((0 & 15) | (7 << 4) | (15 << 8));
  __syncthreads();
  if (threadIdx.x == 0) last = __hip_atomic_fetch_add(p.done, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  double sum = 0.0, n = 0.0;
  for (int64_t i = threadIdx.x; i < p.tokens; i += 1024) {
    sum += (double)__hip_atomic_load(p.losses + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    n += target_of(p.targets, p.targets64, p.ignore, p.vocab, i) >= 0 ? 1.0 : 0.0;
  }
  sum = wave_sum_d(sum);
  n = wave_sum_d(n);
  __shared__ double sums[2][16];
  if ((threadIdx.x & 63) == 0) sums[0][threadIdx.x >> 6] = sum, sums[1][threadIdx.x >> 6] = n;
  __syncthreads();
  if (threadIdx.x) return;
  sum = n = 0.0;
  for (int k = 0; k < 16; ++k) sum += sums[0][k], n += sums[1][k];
  p.total[0] = (float)(p.mean ? (n > 0.0 ? sum / n : 0.0) : sum);
  p.total[1] = (float)n;
}

// C (+)= the sum of the splits' C in order, binary32 or rounded to bf16: V
// neighbouring values a thread (four where rows allow it: 8192 x 4096 sums to
// bf16 99 us with one, 37 with four).
template <int V>
__global__ __launch_bounds__(256) void split_join_kernel(const float* part, int splits, int64_t split_ld, int64_t rows,
                                                         int64_t cols, void* C, int bf16, int64_t ldc, int add) {
  typedef float vec_t __attribute__((ext_vector_type(V)));
  const int64_t per = cols / V, n = rows * per;
  for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < n; id += (int64_t)gridDim.x * 256) {
    const int64_t row = n <= UINT32_MAX ? (int64_t)((uint32_t)id / (uint32_t)per) : id / per, col = (id - row * per) * V;
    vec_t s = 0.0f;
    for (int k = 0; k < splits; k += 8) {
      vec_t v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = k + u < splits ? *(const vec_t*)(part + (k + u) * split_ld + id * V) : 0.0f;
#pragma unroll
      for (int u = 0; u < 8; ++u) s += v[u];
    }
    const int64_t at = row * ldc + col;
    if constexpr (V == 1) {
      if (add) s += load1(C, bf16, at);
      store1(C, bf16, at, s[0]);
    } else if (bf16) {
      *(uint2*)((uint16_t*)C + at) = make_uint2(pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3]));
    } else {
      if (add) s += *(const vec_t*)((const float*)C + at);
      *(vec_t*)((float*)C + at) = s;
    }
  }
}

__global__ __launch_bounds__(256) void zero_rows_kernel(void* p, int bf16, int64_t rows, int64_t cols, int64_t ld) {
  for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < rows * cols; id += (int64_t)gridDim.x * 256) {
    const int64_t row = id / cols;
    store1(p, bf16, row * ld + id - row * cols, 0.0f);
  }
}

}  // namespace metis
