// model.hip -- host side of the operators around the linear layers (layer
// norm, dropout, embedding, loss over a vocabulary), declared in
// include/metis.h.
#include <math.h>

#include <algorithm>

#include "bf16_gemm.hpp"
#include "dropout.hpp"
#include "embedding.hpp"
#include "gemm_launch.hpp"
#include "host.hpp"
#include "loss.hpp"
#include "norm.hpp"

using namespace metis;

namespace {

int64_t value_size(int32_t dt) { return dt == METIS_BF16 ? 2 : 4; }

bool aligned(const void* p, int64_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

// rows of which any eight consecutive values from a multiple of eight can be
// taken at once
bool vec_rows(const void* p, int32_t dt, int64_t ld, int64_t rows) {
  return aligned(p, 16) && (rows <= 1 || ld * value_size(dt) % 16 == 0);
}

// a grid for `items` over workgroups of `per`; kernels stride over the rest
unsigned grid_for(int64_t items, int64_t per, int64_t most = 1 << 20) {
  return (unsigned)std::min<int64_t>(std::max<int64_t>(ceil_div<int64_t>(items, per), 1), most);
}

metis_status rows_check(const char* what, const void* p, int32_t dt, int64_t rows, int64_t cols, int64_t ld) {
  if (!dtype_ok(dt)) return fail(METIS_E_INVALID, "%s: dtype %d", what, dt);
  if (rows < 0 || cols < 1 || cols > INT32_MAX || (rows > 1 && ld < cols))
    return fail(METIS_E_INVALID, "%s: %lld rows of %lld, leading dimension %lld", what, (long long)rows, (long long)cols,
                (long long)ld);
  if (rows && !p) return fail(METIS_E_INVALID, "%s: null pointer", what);
  if (!aligned(p, value_size(dt))) return fail(METIS_E_INVALID, "%s: misaligned pointer", what);
  return METIS_OK;
}

metis_status ws_check(const char* what, const void* ws, size_t bytes, size_t need) {
  if (need && (!ws || bytes < need)) return fail(METIS_E_WORKSPACE, "%s: workspace %zu < %zu", what, bytes, need);
  if (need && !aligned(ws, 256)) return fail(METIS_E_INVALID, "%s: workspace not 256-byte aligned", what);
  return METIS_OK;
}

#define TRY(expr)                     \
  do {                                \
    const metis_status s__ = (expr);  \
    if (s__ != METIS_OK) return s__;  \
  } while (0)

// ------------------------------------------------------------- layer norm --

// Workgroups of a forward pass, which stride over the rows (us with 640, 1280
// and 4096: 16384 x 4096 bf16 48, 45, 42; 8192 x 768 binary32 11.6, 11.3, 12.5;
// 4096 x 8192 bf16 25.5, 25.4, 29.2; 16384 x 1500 binary32 37, 38, 46).
constexpr int64_t kNormFwdGroups = 1280;

// Threads of a row (us forward and backward with a wave up to 2048 columns and
// up to 1024: 16384 x 2048 bf16 25 + 41, 35 + 57; 16384 x 1500 binary32 38 +
// 68, 41 + 87).
int64_t norm_threads(int64_t cols) { return cols <= 2048 ? 64 : cols <= 8192 ? 256 : 512; }

// Workgroups of a backward pass, two on a CU (one of 512 threads), each with a
// partial sum of dw and db (us with half as many, these and twice as many:
// 4096 x 8192 bf16 52, 45, 59; 16384 x 2048 bf16 49, 41, 47; with these and half
// as many more, where registers leave room for three on a CU: 16384 x 4096
// bf16 80, 85; 8192 x 768 binary32 20.5, 20.9).  Of longer rows one for each
// kNormSumRows rows.
int64_t norm_groups(int64_t rows, int64_t cols) {
  if (cols > kNormCols) return std::min<int64_t>(ceil_div<int64_t>(rows, kNormSumRows), INT32_MAX);
  const int64_t T = norm_threads(cols), per = std::max<int64_t>(1, 256 / T);
  const int64_t most = T == 512 ? 256 : 512;
  return std::min<int64_t>(ceil_div<int64_t>(rows, per), most);
}

template <int VEC, int T, int NV>
void launch_norm(const NormParams& p, bool bwd, unsigned grid, hipStream_t st) {
  const dim3 block(norm_block(T));
  if (bwd) hipLaunchKernelGGL((norm_bwd_kernel<VEC, T, NV>), dim3(grid), block, 0, st, p);
  else hipLaunchKernelGGL((norm_fwd_kernel<VEC, T, NV>), dim3(grid), block, 0, st, p);
}

template <int VEC>
void launch_norm_rows(const NormParams& p, bool bwd, hipStream_t st) {
  constexpr int K = 8 / VEC;
  const int64_t T = norm_threads(p.cols), per = std::max<int64_t>(1, 256 / T);
  const unsigned grid = bwd ? (unsigned)norm_groups(p.rows, p.cols) : grid_for(p.rows, per, T == 512 ? 512 : kNormFwdGroups);
  if (T == 64) {
    if (p.cols <= 512) launch_norm<VEC, 64, 1 * K>(p, bwd, grid, st);
    else if (p.cols <= 1024) launch_norm<VEC, 64, 2 * K>(p, bwd, grid, st);
    else launch_norm<VEC, 64, 4 * K>(p, bwd, grid, st);
  } else if (T == 256) {
    if (p.cols <= 4096) launch_norm<VEC, 256, 2 * K>(p, bwd, grid, st);
    else launch_norm<VEC, 256, 4 * K>(p, bwd, grid, st);
  } else {
    launch_norm<VEC, 512, 4 * K>(p, bwd, grid, st);
  }
}

// -------------------------------------------------------------- embedding --

// Workgroups for the rows of zeros, at most, and the tokens whose runs fit one
// launch beside them.
constexpr int64_t kEmbedZeroGroups = 8192, kEmbedBwdTokens = (1 << 28) - (1 << 18);
static_assert(kEmbedBwdTokens / kEmbedRun + kEmbedZeroGroups <= UINT32_MAX / 256, "one launch");

struct EmbedWs {
  uint32_t *key[2], *pos[2], *hist;
  float* part;
};

EmbedWs carve_embed(Carver& cv, int64_t tokens, int64_t cols) {
  EmbedWs w;
  for (int i = 0; i < 2; ++i) {
    w.key[i] = cv.take<uint32_t>(tokens);
    w.pos[i] = cv.take<uint32_t>(tokens);
  }
  w.hist = cv.take<uint32_t>((size_t)kEmbedTiles * kEmbedDigits);
  w.part = cv.take<float>((size_t)ceil_div<int64_t>(tokens, kEmbedRun) * 2 * cols);
  return w;
}

metis_status ids_check(const char* what, const void* ids, int32_t bits, int64_t tokens, int64_t vocab) {
  if (bits != 32 && bits != 64) return fail(METIS_E_INVALID, "%s: %d bits a token", what, bits);
  if (tokens < 0 || vocab < 1) return fail(METIS_E_INVALID, "%s: %lld tokens, vocabulary %lld", what, (long long)tokens,
                                           (long long)vocab);
  if (tokens > INT32_MAX || vocab > INT32_MAX)
    return fail(METIS_E_UNSUPPORTED, "%s: %lld tokens, vocabulary %lld", what, (long long)tokens, (long long)vocab);
  if (tokens && (!ids || !aligned(ids, bits / 8))) return fail(METIS_E_INVALID, "%s: token pointer", what);
  return METIS_OK;
}

// ------------------------------------------------------------------- loss --

constexpr int64_t kLossMax = 1 << 22;

// the parts of a product's operand: planes of rows
struct Planes {
  const uint8_t* at = nullptr;
  int64_t pitch = 0;  // bytes
  int64_t plane = 0;  // bytes between planes
  int count = 1;
  const int* shift = nullptr;  // binary16 planes: their s
};

// whether rows can be an operand as they lie in memory
bool operand_as_is(const void* p, int32_t dt, int64_t ld, int64_t rows, int64_t cols) {
  return dt == METIS_BF16 && cols % 64 == 0 && vec_rows(p, dt, ld, rows) && (rows <= 1 || ld % 64 == 0) && ld < 1 << 23;
}

int64_t pad64(int64_t n) { return round_up64(n, 64); }

// Words of one piece: at most about 2^28 probabilities, but 4096 words at least
// (P takes 512 MB, or 8 KB a token; twice that for two planes); at most 2^29
// values of the weight, but 256 words at least (its copy takes 1 GB, or 512
// bytes a column; twice that for two planes); at most 2^22 words (the product
// counts the bytes of 256 rows of P in 32 bits).  None of it grows with the
// vocabulary.  Where they allow it, it is a number whose dw = P^T x fills whole
// rounds of the chip's 256 CUs with tiles of 256 x 256 (50257 words, 768
// features, 8192 tokens: dw in three pieces of 21760 and the rest, not in two
// of 25152, which take two rounds of tiles each).  Backward pass in us with at
// most 2^27, 2^28 and 2^29 probabilities: 8192 x 50257 x 768 2193, 2136, 2174;
// 8192 x 128256 x 4096 20470, 20183, 20632; 2048 x 50257 x 1024 binary32 1850,
// 1738, 1905; with at most 2^27, 2^28 and 2^29 values of the weight: 256 x
// 128256 x 4096 1860, 1717, 1605; 64 tokens of it 1384, 1388, 1329, binary32
// 3337, 3204, 3046.
int64_t loss_piece(int64_t tokens, int64_t cols) {
  const int64_t by_p = std::max<int64_t>(((int64_t)1 << 28) / std::max<int64_t>(tokens, 1), 4096);
  const int64_t by_w = std::max<int64_t>(((int64_t)1 << 29) / pad64(cols), 256);
  const int64_t most = std::min<int64_t>({by_p, by_w, 1 << 22});
  const int64_t round = std::max<int64_t>(256 / ceil_div<int64_t>(cols, 256), 1) * 256;
  return round <= most ? most / round * round : most / 256 * 256;
}

struct LossPlan {
  bool x_as_is, w_as_is;  // forward, both bf16
  bool pair;              // an operand is binary32: P has two planes, forward is of binary16 planes too
  int xp, wp;                   // planes of x and w
  int64_t N, V, D, Dp, Np, piece;
};

LossPlan loss_plan(const metis_loss& l) {
  LossPlan p;
  p.N = l.tokens, p.V = l.vocab, p.D = l.cols;
  p.Dp = pad64(p.D), p.Np = pad64(p.N);
  p.xp = l.x_dtype == METIS_F32 ? 2 : 1;
  p.wp = l.w_dtype == METIS_F32 ? 2 : 1;
  p.pair = p.xp == 2 || p.wp == 2;
  p.x_as_is = !p.pair && operand_as_is(l.x, l.x_dtype, l.ldx, p.N, p.D);
  p.w_as_is = !p.pair && operand_as_is(l.w, l.w_dtype, l.ldw, p.V, p.D);
  p.piece = loss_piece(p.N, p.D);
  return p;
}

struct LossWs {
  uint16_t *x, *w;             // planes of x, of a piece of w (where not as they are)
  uint16_t* weighed;           // backward: planes of x by the tokens' gradients
  uint32_t* top;               // [3][kTopBlocks] largest values of x, w, the gradients of the losses
  int* shift;                  // [3] their s, and a zero
  float2* stat;                // forward
  float *target, *losses;
  uint32_t* done;              // counter of the join
  uint16_t* p;                 // backward: P of a piece
  float *dx, *part;            // a bf16 dx summed over the pieces, parts of K
};

// parts of K of dx = P w over so many words
int dx_splits(const LossPlan& p, int64_t words) {
  const int runs = p.xp == 1 ? 1 : 1 + (p.wp == 2) + p.pair;  // as product() counts them
  return words ? bf_gemm_splits(p.N, p.D, runs * (int)(pad64(words) / 64)) : 1;
}

LossWs carve_loss(Carver& cv, const metis_loss& l, const LossPlan& p, bool backward) {
  LossWs w{};
  if (backward || !p.x_as_is) w.x = cv.take<uint16_t>((size_t)p.xp * p.Np * p.Dp);
  if (backward || !p.w_as_is) w.w = cv.take<uint16_t>((size_t)p.wp * std::min(p.piece, p.V) * p.Dp);
  if (backward || p.pair) {
    w.top = cv.take<uint32_t>(3 * kTopBlocks);
    w.shift = cv.take<int>(4);
  }
  if (!backward) {
    w.stat = cv.take<float2>((size_t)ceil_div<int64_t>(p.V, 64) * p.N);
    w.target = cv.take<float>(p.N);
    w.losses = cv.take<float>(p.N);
    w.done = cv.take<uint32_t>(1);
    return w;
  }
  w.weighed = cv.take<uint16_t>((size_t)p.xp * p.Np * p.Dp);
  const int64_t words = pad64(std::min(p.piece, p.V));
  w.p = cv.take<uint16_t>((size_t)(p.pair ? 2 : 1) * p.Np * words);
  if (l.x_dtype == METIS_BF16) w.dx = cv.take<float>((size_t)p.N * p.D);  // (a binary32 one is summed in place)
  int s = dx_splits(p, words);
  if (p.V > p.piece) s = std::max(s, dx_splits(p, pad64(p.V % p.piece)));
  if (s > 1) w.part = cv.take<float>((size_t)s * p.N * p.D);
  return w;
}

metis_status loss_check(const metis_loss* l, const char* what) {
  if (!l) return fail(METIS_E_INVALID, "%s: null argument", what);
  TRY(ids_check(what, l->targets, l->target_bits, l->tokens, l->vocab));
  TRY(rows_check(what, l->x, l->x_dtype, l->tokens, l->cols, l->ldx));
  TRY(rows_check(what, l->w, l->w_dtype, l->vocab, l->cols, l->ldw));
  if (l->tokens > kLossMax || l->cols > kLossMax)
    return fail(METIS_E_UNSUPPORTED, "%s: %lld tokens of %lld", what, (long long)l->tokens, (long long)l->cols);
  return METIS_OK;
}

// Planes of x (job 0) and w (job 1) and the s of the gradient of the losses, or
// planes of x weighed by their gradients (job 2), as planes_kernel and top_kernel
// make them.
struct PlaneJobs {
  PlanesParams p{};
  const LossWs& ws;
  bool any = false, scaled = false;

  PlaneJobs(const metis_loss& l, const LossWs& w) : ws(w) {
    p.targets = l.targets, p.targets64 = l.target_bits == 64, p.vocab = l.vocab, p.ignore = l.ignore_index;
  }
  static int blocks_for(int64_t blocks_of_8, int most) {
    return (int)std::min<int64_t>(std::max<int64_t>(ceil_div<int64_t>(blocks_of_8, 1024), 1), most);
  }
  // `half`: binary16 planes, `masked`: rows up to a multiple of 64 and zeros in
  // those of tokens that the loss leaves out
  Planes rows(int at, const void* src, int32_t dt, int64_t ld, int64_t rows, int64_t cols, int planes, uint16_t* dst, bool half,
              bool masked) {
    PlanesJob& j = p.job[at];
    const int64_t pitch = pad64(cols), out_rows = masked ? pad64(rows) : rows;
    j = PlanesJob{};
    j.src = src, j.rows = rows, j.cols = cols, j.ld = ld;
    j.bf16 = dt == METIS_BF16, j.masked = masked;
    j.dst = dst, j.out_rows = out_rows, j.pitch = pitch, j.plane = planes > 1 ? out_rows * pitch : 0;
    j.blocks = blocks_for(out_rows * (pitch / 8), 4096);
    if (half) top_of(at, src, rows * ceil_div<int64_t>(cols, 8));
    any = true;
    return {(const uint8_t*)dst, pitch * 2, out_rows * pitch * 2, planes, j.shift};
  }
  Planes weighed(const metis_loss& l, const LossPlan& plan, const float* grad, const float* count, uint16_t* dst) {
    const Planes x = rows(2, l.x, l.x_dtype, l.ldx, plan.N, plan.D, plan.xp, dst, true, true);
    p.job[2].weigh = grad, p.job[2].count = count;
    return x;
  }
  const int* gradient(const float* grad, const float* count) {
    PlanesJob& j = p.job[2];
    j = PlanesJob{};
    j.rows = 1, j.cols = j.ld = 1, j.count = count;
    j.blocks = 1;
    top_of(2, grad, j.rows);
    return j.shift;
  }
  metis_status run(hipStream_t st) {
    if (!any) return METIS_OK;
    const bool weigh = p.job[2].weigh != nullptr;
    if (scaled) {
      const dim3 grid(p.job[0].top_blocks + p.job[1].top_blocks + p.job[2].top_blocks);
      if (weigh) hipLaunchKernelGGL(top_kernel<true>, grid, dim3(256), 0, st, p);
      else hipLaunchKernelGGL(top_kernel<false>, grid, dim3(256), 0, st, p);
      LAUNCH_CHECK();
    }
    const dim3 grid(p.job[0].blocks + p.job[1].blocks + p.job[2].blocks);
    if (weigh) hipLaunchKernelGGL(planes_kernel<true>, grid, dim3(256), 0, st, p);
    else hipLaunchKernelGGL(planes_kernel<false>, grid, dim3(256), 0, st, p);
    LAUNCH_CHECK();
    return METIS_OK;
  }

 private:
  void top_of(int at, const void* values, int64_t blocks_of_8) {
    PlanesJob& j = p.job[at];
    if (!j.masked && j.ld == j.cols) j.flat = 1;
    j.values = values, j.top = ws.top + at * kTopBlocks, j.top_blocks = blocks_for(blocks_of_8, kTopBlocks), j.shift = ws.shift + at;
    scaled = true;
  }
};

// rows that are an operand as they lie in memory
Planes as_is(const void* src, int64_t ld, int64_t rows, int64_t cols) {
  return {(const uint8_t*)src, rows > 1 ? ld * 2 : cols * 2, 0, 1, nullptr};
}

// the operands and the products of their planes; `all`: with the low planes
BfGemmParams product(const Planes& a, int64_t M, const Planes& b, int64_t N, int64_t K, bool all) {
  BfGemmParams g{};
  g.M = M, g.N = N;
  g.a = a.at, g.b = b.at;
  g.pitch_a = a.pitch, g.pitch_b = b.pitch;
  g.run_stages = (int)(pad64(K) / 64);
  g.shift_a = a.shift, g.shift_b = b.shift;
  g.splits = 1;
  g.runs = 1;
  if (all && b.count > 1) g.at_b[g.runs++] = b.plane;
  if (all && a.count > 1) g.at_a[g.runs++] = a.plane;
  return g;
}

metis_status run_product(const BfGemmParams& g, BfOut out, hipStream_t st) {
  const hipError_t e = launch_bf_gemm(g, out, st);
  return e == hipSuccess ? METIS_OK : fail(METIS_E_HIP, "product launch: %s", hipGetErrorString(e));
}

// C (+)= the sum of the splits (add: to a binary32 C)
metis_status join_splits(const float* part, int splits, int64_t rows, int64_t cols, void* C, bool bf16, int64_t ldc, bool add,
                         hipStream_t st) {
  const bool four = cols % 4 == 0 && vec_rows(C, bf16 ? METIS_BF16 : METIS_F32, ldc, rows);
  const int64_t n = rows * cols;
  if (four)
    hipLaunchKernelGGL(split_join_kernel<4>, dim3(grid_for(n / 4, 256)), dim3(256), 0, st, part, splits, n, rows, cols, C, (int)bf16,
                       ldc, (int)add);
  else
    hipLaunchKernelGGL(split_join_kernel<1>, dim3(grid_for(n, 256)), dim3(256), 0, st, part, splits, n, rows, cols, C, (int)bf16, ldc,
                       (int)add);
  LAUNCH_CHECK();
  return METIS_OK;
}

void set_targets(BfGemmParams& g, const metis_loss& l, int64_t v0) {
  g.v0 = v0;
  g.targets = l.targets;
  g.targets64 = l.target_bits == 64;
  g.vocab = l.vocab;
  g.ignore = l.ignore_index;
}

const void* rows_from(const void* p, int32_t dt, int64_t ld, int64_t row) { return (const char*)p + row * ld * value_size(dt); }

}  // namespace

extern "C" {

// ------------------------------------------------------------- layer norm --

metis_status metis_layernorm_fwd(const void* X, int32_t x_dtype, int64_t rows, int64_t cols, int64_t ldx, const void* weight,
                                 const void* bias, int32_t w_dtype, double eps, void* Y, int32_t y_dtype, int64_t ldy,
                                 float* mean, float* rstd, void* stream) {
  TRY(rows_check("layernorm: X", X, x_dtype, rows, cols, ldx));
  TRY(rows_check("layernorm: Y", Y, y_dtype, rows, cols, ldy));
  if (!dtype_ok(w_dtype) || !aligned(weight, value_size(w_dtype)) || !aligned(bias, value_size(w_dtype)))
    return fail(METIS_E_INVALID, "layernorm: weight or bias");
  if (!(eps >= 0) || !isfinite(eps)) return fail(METIS_E_INVALID, "layernorm: eps %g", eps);
  if (!mean != !rstd || !aligned(mean, 4) || !aligned(rstd, 4)) return fail(METIS_E_INVALID, "layernorm: mean and rstd");
  if (rows == 0) return METIS_OK;
  hipStream_t st = (hipStream_t)stream;
  NormParams p{};
  p.rows = rows, p.cols = (int)cols;
  p.x = X, p.w = weight, p.b = bias;
  p.ldx = ldx, p.ldy = ldy;
  p.x_bf16 = x_dtype == METIS_BF16, p.w_bf16 = w_dtype == METIS_BF16, p.y_bf16 = y_dtype == METIS_BF16;
  p.eps = (float)eps, p.inv = (float)(1.0 / (double)cols);
  p.y = Y, p.mean = mean, p.rstd = rstd;
  if (cols > kNormCols) {
    hipLaunchKernelGGL(norm_fwd_long_kernel, dim3(grid_for(rows, 1, 512)), dim3(kNormThreads), 0, st, p);
  } else if (vec_rows(X, x_dtype, ldx, rows) && vec_rows(Y, y_dtype, ldy, rows) && aligned(weight, 16) && aligned(bias, 16)) {
    launch_norm_rows<8>(p, false, st);
  } else {
    launch_norm_rows<1>(p, false, st);
  }
  LAUNCH_CHECK();
  return METIS_OK;
}

size_t metis_layernorm_bwd_workspace(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0) return 256;
  return std::max<size_t>(256, (size_t)norm_groups(rows, cols) * 2 * cols * sizeof(float));
}

metis_status metis_layernorm_bwd(const void* dY, int32_t y_dtype, int64_t lddy, const void* X, int32_t x_dtype, int64_t rows,
                                 int64_t cols, int64_t ldx, const void* weight, int32_t w_dtype, const float* mean,
                                 const float* rstd, void* dX, int64_t lddx, void* dweight, void* dbias, void* ws, size_t ws_bytes,
                                 void* stream) {
  TRY(rows_check("layernorm_bwd: dY", dY, y_dtype, rows, cols, lddy));
  TRY(rows_check("layernorm_bwd: X", X, x_dtype, rows, cols, ldx));
  if (dX) TRY(rows_check("layernorm_bwd: dX", dX, x_dtype, rows, cols, lddx));
  if (!dtype_ok(w_dtype) || !aligned(weight, value_size(w_dtype)) || !aligned(dweight, value_size(w_dtype)) ||
      !aligned(dbias, value_size(w_dtype)))
    return fail(METIS_E_INVALID, "layernorm_bwd: weight, dweight or dbias");
  if (rows && (!mean || !rstd || !aligned(mean, 4) || !aligned(rstd, 4))) return fail(METIS_E_INVALID, "layernorm_bwd: mean and rstd");
  const bool sums = dweight || dbias;
  if (sums) TRY(ws_check("layernorm_bwd", ws, ws_bytes, metis_layernorm_bwd_workspace(rows, cols)));
  if (!dX && !sums) return METIS_OK;
  hipStream_t st = (hipStream_t)stream;
  NormParams p{};
  p.rows = rows, p.cols = (int)cols;
  p.x = X, p.w = weight;
  p.ldx = ldx, p.lddy = lddy, p.lddx = lddx;
  p.x_bf16 = x_dtype == METIS_BF16, p.w_bf16 = w_dtype == METIS_BF16, p.y_bf16 = y_dtype == METIS_BF16;
  p.inv = (float)(1.0 / (double)cols);
  p.mean = (float*)mean, p.rstd = (float*)rstd;
  p.dy = dY, p.dx = dX;
  p.part = sums ? (float*)ws : nullptr;
  if (rows > 0) {
    if (cols > kNormCols) {
      if (sums) {  // first: dX may be dY
        const dim3 grid((unsigned)ceil_div<int64_t>(cols, 256), (unsigned)std::min<int64_t>(norm_groups(rows, cols), 4096));
        hipLaunchKernelGGL(norm_dw_long_kernel, grid, dim3(256), 0, st, p);
        LAUNCH_CHECK();
      }
      if (dX) hipLaunchKernelGGL(norm_dx_long_kernel, dim3(grid_for(rows, 1, 512)), dim3(kNormThreads), 0, st, p);
    } else if (vec_rows(X, x_dtype, ldx, rows) && vec_rows(dY, y_dtype, lddy, rows) &&
               (!dX || vec_rows(dX, x_dtype, lddx, rows)) && aligned(weight, 16) && (!sums || cols % 4 == 0)) {
      launch_norm_rows<8>(p, true, st);
    } else {
      launch_norm_rows<1>(p, true, st);
    }
    LAUNCH_CHECK();
  }
  if (sums) {  // (no rows: zeros)
    // (a launch takes fewer than 2^32 work items a dimension)
    hipLaunchKernelGGL(norm_sum_kernel, dim3(grid_for(cols, 64), 2), dim3(1024), 0, st, (const float*)ws,
                       rows > 0 ? norm_groups(rows, cols) : 0, cols, dweight, dbias, (int)(w_dtype == METIS_BF16));
    LAUNCH_CHECK();
  }
  return METIS_OK;
}

// ---------------------------------------------------------------- dropout --

metis_status metis_dropout(const void* X, int32_t dtype, int64_t rows, int64_t cols, int64_t ldx, const void* residual,
                           int64_t ldr, double p, uint64_t seed, uint32_t tag, int64_t step, const int64_t* step_count, void* Y,
                           int64_t ldy, void* stream) {
  TRY(rows_check("dropout: X", X, dtype, rows, cols, ldx));
  TRY(rows_check("dropout: Y", Y, dtype, rows, cols, ldy));
  if (residual) TRY(rows_check("dropout: residual", residual, dtype, rows, cols, ldr));
  if (!(p >= 0 && p <= 1)) return fail(METIS_E_INVALID, "dropout: p %g", p);
  if (step < 0) return fail(METIS_E_INVALID, "dropout: step %lld", (long long)step);
  if (!aligned(step_count, 8)) return fail(METIS_E_INVALID, "dropout: step count pointer");
  if (rows > INT64_MAX / cols) return fail(METIS_E_UNSUPPORTED, "dropout: %lld x %lld", (long long)rows, (long long)cols);
  if (rows == 0) return METIS_OK;
  const uint32_t t = (uint32_t)rint(65536.0 * p);
  DropoutParams d{X, residual, Y, rows, cols, ldx, ldr, ldy, dtype == METIS_BF16, t,
                  t < 65536 ? (float)(65536.0 / (65536 - t)) : 0.0f, seed, tag_with_role(tag, kRoleDropout), (uint32_t)step,
                  step_count};
  const bool flat = (rows == 1 || (ldx == cols && ldy == cols && (!residual || ldr == cols))) && aligned(X, 16) && aligned(Y, 16) &&
                    aligned(residual, 16);
  hipStream_t st = (hipStream_t)stream;
  const dim3 grid(grid_for(ceil_div<int64_t>(rows * cols, 8), 256));
  if (flat) {
    d.cols = rows * cols;
    hipLaunchKernelGGL((dropout_kernel<true>), grid, dim3(256), 0, st, d);
  } else {
    hipLaunchKernelGGL((dropout_kernel<false>), grid, dim3(256), 0, st, d);
  }
  LAUNCH_CHECK();
  return METIS_OK;
}

// -------------------------------------------------------------- embedding --

metis_status metis_embedding_fwd(const void* W, int32_t w_dtype, int64_t vocab, int64_t cols, int64_t ldw, const void* ids,
                                 int32_t id_bits, int64_t tokens, double scale, void* Y, int32_t y_dtype, int64_t ldy,
                                 void* stream) {
  TRY(ids_check("embedding", ids, id_bits, tokens, vocab));
  TRY(rows_check("embedding: W", W, w_dtype, vocab, cols, ldw));
  TRY(rows_check("embedding: Y", Y, y_dtype, tokens, cols, ldy));
  if (tokens == 0) return METIS_OK;
  TRY(ensure_device_tables());
  EmbedFwdParams p{W, vocab, cols, ldw, tokens, ldy, ids, id_bits == 64, w_dtype == METIS_BF16, y_dtype == METIS_BF16,
                   vec_rows(W, w_dtype, ldw, vocab) && vec_rows(Y, y_dtype, ldy, tokens), (float)scale, Y, device_status()};
  int T = 1;
  while (T < 256 && T * (p.vec ? 8 : 1) < cols) T *= 2;
  hipLaunchKernelGGL(embed_fwd_kernel, dim3(grid_for(tokens, 256 / T)), dim3(256), 0, (hipStream_t)stream, p, T);
  LAUNCH_CHECK();
  return METIS_OK;
}

size_t metis_embedding_bwd_workspace(int64_t tokens, int64_t cols) {
  if (tokens <= 0 || cols <= 0) return 256;
  Carver cv(nullptr, 0);
  carve_embed(cv, tokens, cols);
  return cv.used();
}

metis_status metis_embedding_bwd(const void* dY, int32_t y_dtype, int64_t tokens, int64_t cols, int64_t lddy, const void* ids,
                                 int32_t id_bits, int64_t vocab, int64_t padding, double scale, void* dW, int32_t w_dtype,
                                 int64_t lddw, void* ws, size_t ws_bytes, void* stream) {
  TRY(ids_check("embedding_bwd", ids, id_bits, tokens, vocab));
  TRY(rows_check("embedding_bwd: dY", dY, y_dtype, tokens, cols, lddy));
  TRY(rows_check("embedding_bwd: dW", dW, w_dtype, vocab, cols, lddw));
  if (tokens >= kEmbedBwdTokens) return fail(METIS_E_UNSUPPORTED, "embedding_bwd: %lld tokens", (long long)tokens);
  if (padding >= vocab) return fail(METIS_E_INVALID, "embedding_bwd: padding token %lld of %lld", (long long)padding, (long long)vocab);
  TRY(ws_check("embedding_bwd", ws, ws_bytes, metis_embedding_bwd_workspace(tokens, cols)));
  TRY(ensure_device_tables());
  hipStream_t st = (hipStream_t)stream;
  Carver cv(ws, ws_bytes);
  const EmbedWs w = carve_embed(cv, std::max<int64_t>(tokens, 1), cols);
  EmbedSumParams s{};
  if (tokens > 0) {
    EmbedSortParams p{};
    p.ids = ids, p.ids64 = id_bits == 64;
    p.tokens = tokens, p.vocab = vocab, p.padding = padding;
    p.hist = w.hist;
    p.tile = kEmbedTile * ceil_div<int64_t>(tokens, (int64_t)kEmbedTile * kEmbedTiles);
    p.tiles = (int)ceil_div<int64_t>(tokens, p.tile);
    p.status = device_status();
    int at = 0;  // where the sorted tokens lie
    if (tokens <= kEmbedTile) {
      p.first = 1;
      p.key_to = w.key[0], p.pos_to = w.pos[0];
      hipLaunchKernelGGL(embed_sort_kernel, dim3(1), dim3(kEmbedTile), 0, st, p);
      LAUNCH_CHECK();
    } else {
      at = 1;
      for (p.shift = 0; p.shift == 0 || vocab >> p.shift; p.shift += kEmbedBits) {  // keys go up to vocab
        p.first = p.shift == 0;
        p.key = w.key[at], p.pos = w.pos[at];
        at ^= 1;
        p.key_to = w.key[at], p.pos_to = w.pos[at];
        hipLaunchKernelGGL(embed_hist_kernel, dim3((unsigned)p.tiles), dim3(kEmbedTile), 0, st, p);
        hipLaunchKernelGGL(embed_scatter_kernel, dim3((unsigned)p.tiles), dim3(kEmbedTile), 0, st, p);
        LAUNCH_CHECK();
      }
    }
    s.key = w.key[at], s.pos = w.pos[at];
  }
  s.tokens = tokens, s.vocab = vocab, s.cols = cols, s.lddy = lddy, s.lddw = lddw;
  s.dy = dY, s.dw = dW;
  s.dy_bf16 = y_dtype == METIS_BF16, s.dw_bf16 = w_dtype == METIS_BF16;
  s.scale = (float)scale;
  s.part = w.part;
  s.runs = ceil_div<int64_t>(tokens, kEmbedRun);
  s.zero_groups = grid_for(ceil_div<int64_t>(vocab, 64), 4, kEmbedZeroGroups);
  const dim3 grid((unsigned)(s.runs + s.zero_groups));
  if (vec_rows(dY, y_dtype, lddy, tokens) && vec_rows(dW, w_dtype, lddw, vocab))
    hipLaunchKernelGGL((embed_sum_kernel<8>), grid, dim3(256), 0, st, s);
  else
    hipLaunchKernelGGL((embed_sum_kernel<1>), grid, dim3(256), 0, st, s);
  LAUNCH_CHECK();
  if (s.runs > 1) {
    const int V = cols % 4 == 0 ? 4 : 1;
    const dim3 join((unsigned)s.runs, (unsigned)std::min<int64_t>(ceil_div<int64_t>(cols, 256 * V), 64));
    if (V == 4) hipLaunchKernelGGL((embed_join_kernel<4>), join, dim3(256), 0, st, s);
    else hipLaunchKernelGGL((embed_join_kernel<1>), join, dim3(256), 0, st, s);
    LAUNCH_CHECK();
  }
  return METIS_OK;
}

// ------------------------------------------------------------------- loss --

size_t metis_cross_entropy_workspace(const metis_loss* l, int32_t backward) {
  if (!l || l->tokens <= 0 || l->vocab <= 0 || l->cols <= 0) return 256;
  Carver cv(nullptr, 0);
  carve_loss(cv, *l, loss_plan(*l), backward != 0);
  return cv.used();
}

metis_status metis_cross_entropy_fwd(const metis_loss* l, float* losses, float* lse, int32_t mean, float* total, void* ws,
                                     size_t ws_bytes, void* stream) {
  TRY(loss_check(l, "cross_entropy"));
  if ((l->tokens && !lse) || !aligned(lse, 4) || !aligned(losses, 4) || !aligned(total, 4))
    return fail(METIS_E_INVALID, "cross_entropy: output pointer");
  if (mean != 0 && mean != 1) return fail(METIS_E_INVALID, "cross_entropy: mean %d", mean);
  hipStream_t st = (hipStream_t)stream;
  const int t64 = l->target_bits == 64;
  if (l->tokens > 0) {
    TRY(ws_check("cross_entropy", ws, ws_bytes, metis_cross_entropy_workspace(l, 0)));
    TRY(ensure_device_tables());
    const LossPlan p = loss_plan(*l);
    Carver cv(ws, ws_bytes);
    const LossWs w = carve_loss(cv, *l, p, false);
    Planes x, v;
    // a weight that needs no copies goes through in one piece
    // (as long as its tiles can be counted in 32 bits)
    const int64_t piece = p.w_as_is && ceil_div<int64_t>(p.N, 64) * ceil_div<int64_t>(p.V, 128) < 1 << 30 ? p.V : p.piece;
    for (int64_t v0 = 0; v0 < p.V; v0 += piece) {
      const int64_t n = std::min(piece, p.V - v0);
      PlaneJobs jobs(*l, w);
      if (v0 == 0)
        x = p.x_as_is ? as_is(l->x, l->ldx, p.N, p.D) : jobs.rows(0, l->x, l->x_dtype, l->ldx, p.N, p.D, p.xp, w.x, p.pair, p.pair);
      const void* wv = rows_from(l->w, l->w_dtype, l->ldw, v0);
      v = p.w_as_is ? as_is(wv, l->ldw, n, p.D) : jobs.rows(1, wv, l->w_dtype, l->ldw, n, p.D, p.wp, w.w, p.pair, false);
      TRY(jobs.run(st));
      BfGemmParams g = product(x, p.N, v, n, p.D, true);
      set_targets(g, *l, v0);
      g.stat = w.stat, g.target_logit = w.target;
      g.done = w.done;
      TRY(run_product(g, kBfStats, st));
    }
    LossJoinParams j{w.stat, ceil_div<int64_t>(p.V, 64), p.N, w.target, l->targets, t64, l->vocab, l->ignore_index,
                     losses ? losses : w.losses, lse, mean, total, w.done, device_status()};
    hipLaunchKernelGGL(loss_join_kernel, dim3((unsigned)ceil_div<int64_t>(p.N, 16)), dim3(1024), 0, st, j);
    LAUNCH_CHECK();
  } else if (total) {
    hipLaunchKernelGGL(zero_rows_kernel, dim3(1), dim3(256), 0, st, (void*)total, 0, (int64_t)1, (int64_t)2, (int64_t)2);
    LAUNCH_CHECK();
  }
  return METIS_OK;
}

metis_status metis_cross_entropy_bwd(const metis_loss* l, const float* lse, const float* grad, int32_t grad_each,
                                     const float* count, void* dX, int64_t lddx, void* dW, int64_t lddw, void* ws, size_t ws_bytes,
                                     void* stream) {
  TRY(loss_check(l, "cross_entropy_bwd"));
  if (dX) TRY(rows_check("cross_entropy_bwd: dX", dX, l->x_dtype, l->tokens, l->cols, lddx));
  if (dW) TRY(rows_check("cross_entropy_bwd: dW", dW, l->w_dtype, l->vocab, l->cols, lddw));
  if (l->tokens && (!lse || !grad || !aligned(lse, 4) || !aligned(grad, 4) || !aligned(count, 4)))
    return fail(METIS_E_INVALID, "cross_entropy_bwd: lse, grad or count");
  if (grad_each != 0 && grad_each != 1) return fail(METIS_E_INVALID, "cross_entropy_bwd: grad_each %d", grad_each);
  if (!dX && !dW) return METIS_OK;
  hipStream_t st = (hipStream_t)stream;
  const LossPlan p = loss_plan(*l);
  if (p.N == 0) {
    if (dW) {
      hipLaunchKernelGGL(zero_rows_kernel, dim3(grid_for(p.V * p.D, 256)), dim3(256), 0, st, dW, (int)(l->w_dtype == METIS_BF16),
                         p.V, p.D, lddw);
      LAUNCH_CHECK();
    }
    return METIS_OK;
  }
  TRY(ws_check("cross_entropy_bwd", ws, ws_bytes, metis_cross_entropy_workspace(l, 1)));
  TRY(ensure_device_tables());
  Carver cv(ws, ws_bytes);
  const LossWs w = carve_loss(cv, *l, p, true);
  Planes x, x_dw;
  const int* shift_p = w.shift + 3;  // (each token's own: by its gradient, in all 0)
  const bool dx_f32 = l->x_dtype == METIS_F32;
  const bool one = p.piece >= p.V;
  for (int64_t v0 = 0; v0 < p.V; v0 += p.piece) {
    const int64_t n = std::min(p.piece, p.V - v0), np = pad64(n);
    const void* wv = rows_from(l->w, l->w_dtype, l->ldw, v0);
    PlaneJobs jobs(*l, w);
    if (v0 == 0) {
      x = jobs.rows(0, l->x, l->x_dtype, l->ldx, p.N, p.D, p.xp, w.x, true, true);
      x_dw = x;
      if (!grad_each) shift_p = jobs.gradient(grad, count);
      else if (dW) x_dw = jobs.weighed(*l, p, grad, count, w.weighed);
      jobs.p.zero = w.shift + 3;
    }
    const Planes v = jobs.rows(1, wv, l->w_dtype, l->ldw, n, p.D, p.wp, w.w, true, false);
    TRY(jobs.run(st));
    BfGemmParams g = product(x, p.N, v, n, p.D, true);
    set_targets(g, *l, v0);
    g.lse = lse, g.grad = grad, g.count = count, g.grad_each = grad_each;
    g.prob = w.p, g.ldp = np, g.lo_plane = p.pair ? p.Np * np : 0;
    g.shift_p = shift_p;
    TRY(run_product(g, kBfProb, st));
    const Planes pr{(const uint8_t*)w.p, np * 2, p.Np * np * 2, p.pair ? 2 : 1, shift_p};
    if (dX) {
      g = product(pr, p.N, v, p.D, n, dx_f32);
      g.rows_b = n;
      g.grad = grad, g.count = count, g.grad_each = grad_each;
      const int splits = dx_splits(p, n);
      // one piece: straight to dX; else summed in binary32, in dX itself where it is binary32
      void* const sum = dx_f32 ? dX : (void*)w.dx;
      const int64_t ld = dx_f32 ? lddx : p.D;
      const bool direct = one && !dx_f32;
      if (splits > 1) {
        g.splits = splits;
        g.C = w.part, g.ldc = p.D, g.split_ld = p.N * p.D;
        TRY(run_product(g, kBfF32, st));
        TRY(join_splits(w.part, splits, p.N, p.D, direct ? dX : sum, direct, direct ? lddx : ld, v0 > 0, st));
      } else {
        g.C = direct ? dX : sum, g.ldc = direct ? lddx : ld;
        g.add = v0 > 0;
        TRY(run_product(g, direct ? kBfBF16 : kBfF32, st));
      }
    }
    if (dW) {
      g = product(pr, n, x_dw, p.D, p.N, p.wp == 2);
      g.rows_a = g.rows_b = p.Np;
      g.C = (char*)dW + v0 * lddw * value_size(l->w_dtype), g.ldc = lddw;
      TRY(run_product(g, p.wp == 2 ? kBfF32 : kBfBF16, st));
    }
  }
  if (dX && !dx_f32 && !one) {
    TRY(join_splits(w.dx, 1, p.N, p.D, dX, true, lddx, false, st));
  }
  return METIS_OK;
}

}  // extern "C"
