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
// whose epilogue forms P (rounded to bf16, or to a pair of bf16 planes where a
// gradient is binary32), then the two products of the gradients.  So the
// backward pass spends 8 operations where keeping all logits would spend 6,
// and its memory does not grow with the vocabulary.
//
// A token whose target is ignore_index, or not a word (which raises the status
// flag), has loss 0 and gradients 0, whatever its x holds.
#pragma once

#include "bf16_gemm.hpp"

namespace metis {

// bf16 planes of rows: dst[plane][row][pitch] with zeros behind cols, in the
// rows behind `rows` up to out_rows, and in the rows of tokens without a part
// in the loss (targets not null); the high plane is x rounded to bf16, the low
// one the rest rounded.  Eight values a thread.
struct PlanesParams {
  const void* src;
  int64_t rows, cols, ld;
  int bf16, vec;
  uint16_t* dst;
  int64_t out_rows, pitch, plane;  // pitch and plane in values; plane 0: high plane alone
  const void* targets;
  int targets64;
  int64_t vocab, ignore;
};

__device__ __forceinline__ void store_planes(uint16_t* dst, int64_t at, int64_t plane, const float* v) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    l[i] = pack_bf16(v[2 * i] - unpack_bf16(h[i], 0), v[2 * i + 1] - unpack_bf16(h[i], 1));
  }
  *(uint4*)(dst + at) = make_uint4(h[0], h[1], h[2], h[3]);
  if (plane) *(uint4*)(dst + plane + at) = make_uint4(l[0], l[1], l[2], l[3]);
}

__global__ __launch_bounds__(256) void planes_kernel(PlanesParams p) {
  const int64_t per = p.pitch >> 3, total = p.out_rows * per;
  for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < total; id += (int64_t)gridDim.x * 256) {
    const int64_t row = id / per, c = (id - row * per) * 8;
    float v[8] = {};
    if (row < p.rows && (!p.targets || target_of(p.targets, p.targets64, p.ignore, p.vocab, row) >= 0)) {
      if (p.vec && c + 8 <= p.cols) {
        load8(p.src, p.bf16, row * p.ld + c, v);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = c + e < p.cols ? load1(p.src, p.bf16, row * p.ld + c + e) : 0.0f;
      }
    }
    store_planes(p.dst, row * p.pitch + c, p.plane, v);
  }
}

// loss and log-sum-exp of each token from its statistics: four waves of a
// workgroup share 64 tokens, each wave a quarter of the blocks in order.
struct LossJoinParams {
  const float2* stat;  // [blocks][tokens]
  int64_t blocks, tokens;
  const float* target_logit;
  const void* targets;
  int targets64;
  int64_t vocab, ignore;
  float *losses, *lse;  // losses may be null
  int* status;
};

__global__ __launch_bounds__(256) void loss_join_kernel(LossJoinParams p) {
  __shared__ float2 red[4][64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 64 + lane;
  float m = -__builtin_inff(), s = 0.0f;
  auto join = [&](float m2, float s2) {
    const float top = fmaxf(m, m2), at = top == -__builtin_inff() ? 0.0f : top;
    // (max leaves out a NaN; it comes back through the sum)
    s = s * __builtin_amdgcn_exp2f((m - at) * kLog2E) + s2 * __builtin_amdgcn_exp2f((m2 - at) * kLog2E);
    m = top;
  };
  if (row < p.tokens) {
    const int64_t per = (p.blocks + 3) / 4, end = min(p.blocks, (wave + 1) * per);
    int64_t b = wave * per;
    for (; b + 8 <= end; b += 8) {
      float2 v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = p.stat[(b + k) * p.tokens + row];
#pragma unroll
      for (int k = 0; k < 8; ++k) join(v[k].x, v[k].y);
    }
    for (; b < end; ++b) {
      const float2 v = p.stat[b * p.tokens + row];
      join(v.x, v.y);
    }
  }
  red[wave][lane] = make_float2(m, s);
  __syncthreads();
  if (wave || row >= p.tokens) return;
  m = red[0][lane].x, s = red[0][lane].y;
  for (int k = 1; k < 4; ++k) join(red[k][lane].x, red[k][lane].y);
  const float lse = m + logf(s);
  p.lse[row] = lse;
  const int64_t t = p.targets64 ? ((const int64_t*)p.targets)[row] : (int64_t)((const int32_t*)p.targets)[row];
  const bool in = t >= 0 && t < p.vocab;
  if (t != p.ignore && !in) atomicOr(p.status, kStatusToken);
  if (p.losses) p.losses[row] = t != p.ignore && in ? lse - p.target_logit[row] : 0.0f;
}

// total[0]: the sum of the losses, or their mean over the tokens that have one
// (0 where none has); total[1]: the number of those tokens.  Summed in
// binary64 in a fixed order.
__global__ __launch_bounds__(1024) void loss_total_kernel(const float* losses, const void* targets, int targets64, int64_t vocab,
                                                          int64_t ignore, int64_t tokens, int mean, float* total) {
  __shared__ double red[2][16];
  double s = 0.0, n = 0.0;
  for (int64_t i = threadIdx.x; i < tokens; i += 1024) {
    s += (double)losses[i];
    n += target_of(targets, targets64, ignore, vocab, i) >= 0 ? 1.0 : 0.0;
  }
  s = wave_sum_d(s);
  n = wave_sum_d(n);
  if ((threadIdx.x & 63) == 0) red[0][threadIdx.x >> 6] = s, red[1][threadIdx.x >> 6] = n;
  __syncthreads();
  if (threadIdx.x) return;
  s = n = 0.0;
  for (int k = 0; k < 16; ++k) s += red[0][k], n += red[1][k];
  total[0] = (float)(mean ? (n > 0.0 ? s / n : 0.0) : s);
  total[1] = (float)n;
}

// C (+)= the sum of the splits' C in order, binary32 or rounded to bf16
__global__ __launch_bounds__(256) void split_join_kernel(const float* part, int splits, int64_t split_ld, int64_t rows,
                                                         int64_t cols, void* C, int bf16, int64_t ldc, int add) {
  const int64_t n = rows * cols;
  for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < n; id += (int64_t)gridDim.x * 256) {
    const int64_t row = id / cols, col = id - row * cols;
    float s = 0.0f;
    for (int k = 0; k < splits; k += 8) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = k + u < splits ? part[(k + u) * split_ld + id] : 0.0f;
#pragma unroll
      for (int u = 0; u < 8; ++u) s += v[u];
    }
    if (add) s += load1(C, bf16, row * ldc + col);
    store1(C, bf16, row * ldc + col, s);
  }
}

__global__ __launch_bounds__(256) void zero_rows_kernel(void* p, int bf16, int64_t rows, int64_t cols, int64_t ld) {
  for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < rows * cols; id += (int64_t)gridDim.x * 256) {
    const int64_t row = id / cols;
    store1(p, bf16, row * ld + id - row * cols, 0.0f);
  }
}

}  // namespace metis
