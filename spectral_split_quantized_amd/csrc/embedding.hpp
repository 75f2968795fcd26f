// embedding.hpp -- rows of a table by token number, scaled, and the gradient
// of the table from the tokens in sorted order.  Both are bound by memory: the
// rows read and written, and all of dW.
//
// (16384 tokens of a table of 128256 x 4096 bf16: forward 52 us, 5.2 TB/s;
// backward 267 us, of which sorting 20, the sums and zeros 229 at 5.2 TB/s, the
// joins 18.  Rows that 16 bytes do not divide go a value at a time: x 4097 99 us
// and 521; binary32, 8192 of 50257 x 769, 13 and 76, x 768 10 and 47.)
//
//   y_i = scale W[id_i],   dW_v = scale (sum over i with id_i = v of dy_i),
// the sum in binary32 over ascending i within pieces of kEmbedRun sorted
// tokens and over the pieces in order: no atomics touch a value, equal calls
// give equal bits.  All of dW is written, zeros where no token points.
//
// A token outside [0, vocab) raises the status flag, gives a row of zeros and
// has no part in dW; neither has the padding token.
//
// Sorting: least significant digit first, kEmbedBits bits a pass.  A pass is
// a histogram for each tile of tokens and a stable scatter; a scatter's
// workgroup forms its own offsets from all histograms (at most kEmbedTiles).
// Within a tile of 1024 tokens the rank of a token among those of the same
// digit is the number of earlier ones in its wave (lanes compared by ballots,
// a bit at a time) plus the counts of the earlier waves.
#pragma once

#include "rows.hpp"

namespace metis {

constexpr int kEmbedBits = 9, kEmbedDigits = 1 << kEmbedBits;
constexpr int kEmbedTile = 1024, kEmbedTiles = 256;
// Sorted tokens whose rows one workgroup adds (a whole call, in us, with 8, 16
// and 32: 8192 tokens of 50257 x 768 binary32 54, 53, 57; 16384 of 5000 x 512
// bf16 38.5, 33.6, 38.9; 16384 of 128256 x 4096 bf16 274, 269, 271).
constexpr int kEmbedRun = 16;

struct EmbedFwdParams {
  const void* w;
  int64_t vocab, cols, ldw, tokens, ldy;
  const void* ids;
  int ids64, w_bf16, y_bf16, vec;
  float scale;
  void* y;
  int* status;
};

__device__ __forceinline__ int64_t load_id(const void* ids, int ids64, int64_t i) {
  return ids64 ? ((const int64_t*)ids)[i] : (int64_t)((const int32_t*)ids)[i];
}

// T threads a row, a power of two of at most 256
__global__ __launch_bounds__(256) void embed_fwd_kernel(EmbedFwdParams p, int T) {
  const int t = threadIdx.x & (T - 1), per = 256 / T;
  for (int64_t i = (int64_t)blockIdx.x * per + threadIdx.x / T; i < p.tokens; i += (int64_t)gridDim.x * per) {
    const int64_t id = load_id(p.ids, p.ids64, i);
    const bool in = id >= 0 && id < p.vocab;
    if (!in && t == 0) atomicOr(p.status, kStatusToken);
    const int64_t from = in ? id * p.ldw : 0, to = i * p.ldy;
    if (p.vec) {
      for (int64_t c = t * 8; c < p.cols; c += T * 8) {
        float v[8] = {};
        if (c + 8 <= p.cols) {
          if (in) load8(p.w, p.w_bf16, from + c, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] *= p.scale;
          store8(p.y, p.y_bf16, to + c, v);
        } else {
          for (int64_t k = c; k < p.cols; ++k)
            store1(p.y, p.y_bf16, to + k, in ? load1(p.w, p.w_bf16, from + k) * p.scale : 0.0f);
        }
      }
    } else {
      for (int64_t c = t; c < p.cols; c += T)
        store1(p.y, p.y_bf16, to + c, in ? load1(p.w, p.w_bf16, from + c) * p.scale : 0.0f);
    }
  }
}

struct EmbedSortParams {
  const void* ids;       // first pass: keys from the tokens
  int ids64;
  int64_t tokens, vocab, padding;
  const uint32_t* key;   // later passes
  const uint32_t* pos;
  uint32_t* key_to;
  uint32_t* pos_to;
  uint32_t* hist;        // [tiles][kEmbedDigits]
  int tiles;
  int64_t tile;          // tokens of a tile, a multiple of kEmbedTile
  int shift, first;
  int* status;
};

// a token's key: its number, or vocab (behind all) where it has no part
__device__ __forceinline__ uint32_t embed_key(const EmbedSortParams& p, int64_t i) {
  if (!p.first) return p.key[i];
  const int64_t id = load_id(p.ids, p.ids64, i);
  if (id < 0 || id >= p.vocab) {
    atomicOr(p.status, kStatusToken);
    return (uint32_t)p.vocab;
  }
  return id == p.padding ? (uint32_t)p.vocab : (uint32_t)id;
}

__global__ __launch_bounds__(kEmbedTile) void embed_hist_kernel(EmbedSortParams p) {
  __shared__ uint32_t h[kEmbedDigits];
  for (int d = threadIdx.x; d < kEmbedDigits; d += kEmbedTile) h[d] = 0;
  __syncthreads();
  const int64_t end = min((blockIdx.x + 1) * p.tile, p.tokens);
  for (int64_t i = blockIdx.x * p.tile + threadIdx.x; i < end; i += kEmbedTile)
    atomicAdd(&h[embed_key(p, i) >> p.shift & (kEmbedDigits - 1)], 1u);
  __syncthreads();
  for (int d = threadIdx.x; d < kEmbedDigits; d += kEmbedTile) p.hist[(int64_t)blockIdx.x * kEmbedDigits + d] = h[d];
}

// The lanes of the wave that have a token of this lane's digit: a bit of the
// digit at a time.
__device__ __forceinline__ uint64_t same_digit(uint32_t digit, bool have) {
  uint64_t same = __ballot(have);
#pragma unroll
  for (int b = 0; b < kEmbedBits; ++b) {
    const uint64_t set = __ballot(digit >> b & 1);
    same &= digit >> b & 1 ? set : ~set;
  }
  return same;
}

// Inclusive sums over the lanes of a wave.
__device__ __forceinline__ uint32_t sums_up(uint32_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t u = __shfl_up(v, o, 64);
    if (lane >= o) v += u;
  }
  return v;
}

// One tile of tokens: all passes in one workgroup, between them in LDS.
// (200 tokens of 30000 words: 5.2 us, and 17 of the host for a call; as two
// passes of histogram and scatter 11.4, and 26.)
__global__ __launch_bounds__(kEmbedTile) void embed_sort_kernel(EmbedSortParams p) {
  constexpr int W = kEmbedTile / 64;
  __shared__ uint32_t base[kEmbedDigits], sums[kEmbedDigits / 64], keys[kEmbedTile], from[kEmbedTile];
  __shared__ uint16_t count[W][kEmbedDigits];  // at most 1024 each
  const int i = threadIdx.x, wave = i >> 6, lane = i & 63;
  const bool have = i < p.tokens;
  uint32_t key = have ? embed_key(p, i) : 0, pos = i;
  for (int shift = 0;;) {
    for (int d = i; d < W * kEmbedDigits / 2; d += kEmbedTile) ((uint32_t*)count)[d] = 0;
    __syncthreads();
    const uint32_t digit = key >> shift & (kEmbedDigits - 1);
    const uint64_t same = same_digit(digit, have);
    const uint32_t rank = __popcll(same & ((1ull << lane) - 1));
    if (have && rank == 0) count[wave][digit] = (uint16_t)__popcll(same);
    __syncthreads();
    uint32_t up = 0, all = 0;
    if (i < kEmbedDigits) {  // counts of earlier waves, and all of smaller digits
#pragma unroll
      for (int k = 0; k < W; ++k) {
        const uint32_t c = count[k][i];
        count[k][i] = (uint16_t)all;
        all += c;
      }
      up = sums_up(all, lane);
      if (lane == 63) sums[wave] = up;
    }
    __syncthreads();
    if (i < kEmbedDigits) {
      uint32_t before = up - all;
      for (int k = 0; k < wave; ++k) before += sums[k];
      base[i] = before;
    }
    __syncthreads();
    const uint32_t to = base[digit] + rank + count[wave][digit];
    shift += kEmbedBits;
    if (!(p.vocab >> shift)) {  // keys go up to vocab
      if (have) p.key_to[to] = key, p.pos_to[to] = pos;
      return;
    }
    if (have) keys[to] = key, from[to] = pos;
    __syncthreads();
    if (have) key = keys[i], pos = from[i];
  }
}

__global__ __launch_bounds__(kEmbedTile) void embed_scatter_kernel(EmbedSortParams p) {
  constexpr int W = kEmbedTile / 64;
  __shared__ uint32_t base[kEmbedDigits], sums[kEmbedDigits / 64];
  __shared__ uint16_t count[W][kEmbedDigits];  // at most 64 each
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t begin = blockIdx.x * p.tile, end = min(begin + p.tile, p.tokens);
  uint32_t key = 0, from = 0;
  auto fetch = [&](int64_t i) {
    key = embed_key(p, i);
    from = p.first ? (uint32_t)i : p.pos[i];
  };
  if (begin + threadIdx.x < end) fetch(begin + threadIdx.x);
  // the digit's tokens of earlier tiles, and all of smaller digits
  uint32_t before = 0, all = 0;
  if (threadIdx.x < kEmbedDigits) {
    for (int k0 = 0; k0 < p.tiles; k0 += 16) {  // 16 loads in flight
      uint32_t c[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) c[k] = k0 + k < p.tiles ? p.hist[(int64_t)(k0 + k) * kEmbedDigits + threadIdx.x] : 0;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        before += k0 + k < (int)blockIdx.x ? c[k] : 0;
        all += c[k];
      }
    }
    const uint32_t up = sums_up(all, lane);
    if (lane == 63) sums[wave] = up;
    before += up - all;
  }
  __syncthreads();
  if (threadIdx.x < kEmbedDigits) {
    for (int k = 0; k < wave; ++k) before += sums[k];
    base[threadIdx.x] = before;
  }
  for (int64_t i0 = begin; i0 < end; i0 += kEmbedTile) {
    for (int d = threadIdx.x; d < W * kEmbedDigits / 2; d += kEmbedTile) ((uint32_t*)count)[d] = 0;
    __syncthreads();
    const int64_t i = i0 + threadIdx.x;
    const bool have = i < end;
    if (i0 > begin && have) fetch(i);
    const uint32_t digit = have ? key >> p.shift & (kEmbedDigits - 1) : 0;
    const uint64_t same = same_digit(digit, have);
    const uint32_t rank = __popcll(same & ((1ull << lane) - 1));
    if (have && rank == 0) count[wave][digit] = (uint16_t)__popcll(same);
    __syncthreads();
    uint32_t to = 0;
    if (have) {
      to = base[digit] + rank;
#pragma unroll
      for (int k = 0; k < W; ++k) to += k < wave ? count[k][digit] : 0;
      p.key_to[to] = key;
      p.pos_to[to] = from;
    }
    __syncthreads();
    if (threadIdx.x < kEmbedDigits) {
      uint32_t c = 0;
#pragma unroll
      for (int k = 0; k < W; ++k) c += count[k][threadIdx.x];
      base[threadIdx.x] += c;
    }
    __syncthreads();
  }
}

struct EmbedSumParams {
  const uint32_t *key, *pos;  // sorted
  int64_t tokens, vocab, cols, lddy, lddw;
  const void* dy;
  int dy_bf16, dw_bf16;
  float scale;
  void* dw;
  float* part;       // [runs][2][cols]: sums of a run's first and last token that a neighbour shares
  int64_t runs, zero_groups;
};

// Workgroups below `runs`: the rows of kEmbedRun sorted tokens, a row's
// columns over the threads.  A token whose tokens all lie here is written, the
// others leave partial sums.  The rest: rows of dW without a token, 64 a wave,
// each lane looking for one in the sorted tokens.  Zeros are
// written 16 bytes a lane, whole lines at a time (8192 tokens of 50257 x 768
// binary32: 28 us, with 32 bytes a lane 35; past the caches 35).
template <int VEC>
__global__ __launch_bounds__(256) void embed_sum_kernel(EmbedSumParams p) {
  if (blockIdx.x >= p.runs) {
    const int lane = threadIdx.x & 63;
    for (int64_t g = (int64_t)(blockIdx.x - p.runs) * 4 + (threadIdx.x >> 6); g * 64 < p.vocab; g += p.zero_groups * 4) {
      const int64_t v = g * 64 + lane;
      int64_t lo = 0, hi = p.tokens;  // first sorted token of at least v
      while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (p.key[mid] < v) lo = mid + 1;
        else hi = mid;
      }
      uint64_t todo = __ballot(v < p.vocab && (lo == p.tokens || p.key[lo] != v));
      while (todo) {
        const int64_t row = (g * 64 + __builtin_ctzll(todo)) * p.lddw;
        todo &= todo - 1;
        // 16 bytes a lane
        const int per = VEC == 1 ? 1 : p.dw_bf16 ? 8 : 4;
        for (int64_t c = lane * per; c < p.cols; c += 64 * per) {
          if (VEC == 8 && c + per <= p.cols) {
            *(uint4*)((char*)p.dw + (row + c) * (p.dw_bf16 ? 2 : 4)) = make_uint4(0, 0, 0, 0);
          } else {
            for (int e = 0; e < per; ++e)
              if (c + e < p.cols) store1(p.dw, p.dw_bf16, row + c + e, 0.0f);
          }
        }
      }
    }
    return;
  }
  __shared__ uint32_t key[kEmbedRun + 2], pos[kEmbedRun];
  const int64_t i0 = (int64_t)blockIdx.x * kEmbedRun;
  const int n = (int)min((int64_t)kEmbedRun, p.tokens - i0);
  const uint32_t none = 0xFFFFFFFFu;  // no token's key: vocab < 2^31
  if (threadIdx.x < kEmbedRun + 2) {  // with the neighbours before and behind
    const int64_t i = i0 - 1 + threadIdx.x;
    key[threadIdx.x] = i >= 0 && i < p.tokens ? p.key[i] : none;
    if (threadIdx.x < n) pos[threadIdx.x] = p.pos[i0 + threadIdx.x];
  }
  __syncthreads();
  for (int64_t c = threadIdx.x * VEC; c < p.cols; c += 256 * VEC) {
    const int m = (int)min((int64_t)VEC, p.cols - c);
    float s[VEC] = {};
    for (int k0 = 0; k0 < n; k0 += 8) {
      float v[8][VEC];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k0 + k >= n || key[k0 + k + 1] >= p.vocab) continue;
        const int64_t at = (int64_t)pos[k0 + k] * p.lddy + c;
        if (VEC == 8 && m == 8) {
          load8(p.dy, p.dy_bf16, at, v[k]);
        } else {
          for (int e = 0; e < VEC; ++e) v[k][e] = e < m ? load1(p.dy, p.dy_bf16, at + e) : 0.0f;
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int j = k0 + k;
        if (j >= n) continue;
        const uint32_t here = key[j + 1];
        if (here >= p.vocab) continue;
#pragma unroll
        for (int e = 0; e < VEC; ++e) s[e] += v[k][e];
        if (j + 1 < n && key[j + 2] == here) continue;
        // the token's last row here
        const bool shared_before = key[0] == here, shared_behind = j + 1 == n && key[j + 2] == here;
        if (shared_before || shared_behind) {
          float* const to = p.part + ((int64_t)blockIdx.x * 2 + (shared_before ? 0 : 1)) * p.cols + c;
          for (int e = 0; e < VEC; ++e)
            if (e < m) to[e] = s[e];
        } else {
          const int64_t row = here * p.lddw + c;
#pragma unroll
          for (int e = 0; e < VEC; ++e) s[e] *= p.scale;
          if (VEC == 8 && m == 8) {
            store8(p.dw, p.dw_bf16, row, s);
          } else {
            for (int e = 0; e < VEC; ++e)
              if (e < m) store1(p.dw, p.dw_bf16, row + e, s[e]);
          }
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) s[e] = 0.0f;
      }
    }
  }
}

// Tokens whose rows lie in more than one run: the workgroup of the run where
// one begins adds its partial sums in order.  V columns a thread (4 where rows
// of partial sums are 16-byte aligned); a token's runs are counted 64 at a time
// by the lanes of a wave, and 16 partial sums are in flight.  (16384 tokens of
// 4096 columns: 23 us with one column a thread, whose many workgroups mostly
// look at their run and end; a workgroup that looks at 16 runs, 34.)
template <int V>
__global__ __launch_bounds__(256) void embed_join_kernel(EmbedSumParams p) {
  const int64_t run = blockIdx.x, next = (run + 1) * kEmbedRun;
  if (next >= p.tokens) return;
  const uint32_t here = p.key[next - 1], behind = p.key[next], before = run ? p.key[run * kEmbedRun - 1] : ~0u;
  if (here >= p.vocab || behind != here || before == here) return;  // none begins here
  int64_t end = run + 1;  // the first run that does not begin with the token
  for (uint64_t same = ~0ull; same == ~0ull;) {
    const int64_t r = end + (threadIdx.x & 63);
    same = __ballot(r < p.runs && p.key[r * kEmbedRun] == here);
    end += same == ~0ull ? 64 : __builtin_ctzll(~same);
  }
  typedef float vec_t __attribute__((ext_vector_type(V)));
  for (int64_t c = (blockIdx.y * 256 + threadIdx.x) * V; c < p.cols; c += (int64_t)gridDim.y * 256 * V) {
    vec_t s = *(const vec_t*)(p.part + (run * 2 + 1) * p.cols + c);
    for (int64_t r = run + 1; r < end; r += 16) {
      vec_t v[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] = r + k < end ? *(const vec_t*)(p.part + (r + k) * 2 * p.cols + c) : vec_t{};
#pragma unroll
      for (int k = 0; k < 16; ++k) s += v[k];
    }
#pragma unroll
    for (int e = 0; e < V; ++e) store1(p.dw, p.dw_bf16, here * p.lddw + c + e, s[e] * p.scale);
  }
}

}  // namespace metis
