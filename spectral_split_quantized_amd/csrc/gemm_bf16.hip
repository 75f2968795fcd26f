// gemm_bf16.hip -- translation unit of the bf16 product (bf16_gemm.hpp), in
// its own unit for the scheduling strategy that its loop wants.
#include "bf16_gemm.hpp"
#include "gemm_launch.hpp"

namespace metis {

namespace {

template <int WM, int WN, int TM, int NS, int ER>
void launch_tiles(const BfGemmParams& g, BfOut out, hipStream_t st) {
  const int64_t units = ceil_div<int64_t>(g.M, WM * TM * 32) * ceil_div<int64_t>(g.N, WN * 64) * g.splits;
  // workgroups that fit the chip at once: one of 8 waves a CU, or two of 4
  const dim3 grid((unsigned)std::min<int64_t>(256 * (8 / (WM * WN)), ceil_div<int64_t>(units, 8) * 8));
  const dim3 block(WM * WN * 64);
#define LAUNCH(...) hipLaunchKernelGGL((bf_gemm_kernel<WM, WN, TM, NS, ER, __VA_ARGS__>), grid, block, 0, st, g)
  // the logits' product has K along both rows, dx = P W has W transposed, dw =
  // P^T x both
  if (out == kBfStats) LAUNCH(kBfStats, false, false);
  else if (out == kBfProb) LAUNCH(kBfProb, false, false);
  else if (out == kBfBF16 && g.rows_a) LAUNCH(kBfBF16, true, true);
  else if (out == kBfBF16) LAUNCH(kBfBF16, false, true);
  else if (g.rows_a) LAUNCH(kBfF32, true, true);
  else LAUNCH(kBfF32, false, true);
#undef LAUNCH
}

int tile_of(int64_t M, int64_t N) {
  auto tiles = [&](int m, int n) { return ceil_div<int64_t>(M, m) * ceil_div<int64_t>(N, n); };
  if (tiles(256, 256) >= 256) return 256;
  return tiles(128, 128) >= 256 ? 128 : 64;
}

}  // namespace

int bf_gemm_most_splits(int64_t M, int64_t N) {
  const int64_t t = ceil_div<int64_t>(M, 64) * ceil_div<int64_t>(N, 128);
  return tile_of(M, N) != 64 || t >= 128 ? 1 : (int)std::min<int64_t>(256 / t, 32);
}

int bf_gemm_splits(int64_t M, int64_t N, int stages) {
  const int s = std::min(bf_gemm_most_splits(M, N), stages / 16);
  if (s < 2) return 1;
  return ceil_div(stages, ceil_div(stages, s));  // none is empty
}

hipError_t launch_bf_gemm(const BfGemmParams& in, BfOut out, hipStream_t st) {
  BfGemmParams g = in;
  const int stages = g.runs * g.run_stages;
  g.split_stages = (int)ceil_div<int64_t>(stages, g.splits);
  const int tile = g.splits > 1 ? 64 : tile_of(g.M, g.N);
  if (tile == 256) launch_tiles<2, 4, 4, 2, 32>(g, out, st);
  else if (tile == 128) launch_tiles<2, 2, 2, 2, 32>(g, out, st);
  else launch_tiles<2, 2, 1, 3, 16>(g, out, st);
  return hipGetLastError();
}

}  // namespace metis
