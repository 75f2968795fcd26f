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
