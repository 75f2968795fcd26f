// gemm_bf16.hip -- translation unit of the product of 16-bit operands
// (bf16_gemm.hpp): its instances and the choice among them, apart from the host
// side that calls them.
#include "bf16_gemm.hpp"
#include "gemm_launch.hpp"

namespace metis {

namespace {

template <int WM, int WN, int TM, int NS, int ER>
void launch_tiles(const BfGemmParams& g, BfOut out, hipStream_t st) {
  const int64_t units = ceil_div<int64_t>(g.M, WM * TM * 16) * ceil_div<int64_t>(g.N, WN * 64) * g.splits;
  // workgroups that fit the chip at once: one of 8 waves a CU, or two of 4
  const dim3 grid((unsigned)std::min<int64_t>(256 * (8 / (WM * WN)), ceil_div<int64_t>(units, 8) * 8));
  const dim3 block(WM * WN * 64);
#define LAUNCH(...) hipLaunchKernelGGL((bf_gemm_kernel<WM, WN, TM, NS, ER, __VA_ARGS__>), grid, block, 0, st, g)
  // the logits' product has K along both rows, dx = P W has W transposed, dw =
  // P^T x both; all but the statistics of bf16 rows are of binary16 planes
  if (out == kBfStats && !g.shift_a) LAUNCH(kBfStats, false, false, false);
  else if (out == kBfStats) LAUNCH(kBfStats, false, false, true);
  else if (out == kBfProb) LAUNCH(kBfProb, false, false, true);
  else if (out == kBfBF16 && g.rows_a) LAUNCH(kBfBF16, true, true, true);
  else if (out == kBfBF16) LAUNCH(kBfBF16, false, true, true);
  else if (g.rows_a) LAUNCH(kBfF32, true, true, true);
  else LAUNCH(kBfF32, false, true, true);
#undef LAUNCH
}

// Tiles: rows, columns, and what a stage takes, in us, with one workgroup on a
// CU and with two (measured on products that fill the chip once or many
// times).
struct Tile {
  int m, n;
  double one, two;
};
constexpr Tile kTiles[3] = {{256, 256, 1.55, 0}, {128, 128, 0.63, 0.98}, {64, 128, 0.31, 0.77}};

// us that M x N x 64 stages take in `splits` parts of K: whole rounds of
// workgroups and the rest of one, what a workgroup starts and ends with, and
// the sums that the parts write and their join reads.  (What a tile of 256 x 256
// starts and ends with is about 5 us with statistics and 11 with probabilities,
// which the choice does not know of: 8192 x 50257 x 768 584 us in 25 rounds of 12
// stages, 8192 x 21760 x 768 326 in 11.)
double time_of(const Tile& t, int64_t M, int64_t N, int stages, int splits) {
  const int64_t units = ceil_div<int64_t>(M, t.m) * ceil_div<int64_t>(N, t.n) * splits, slots = t.two ? 512 : 256;
  const int64_t rounds = units / slots, rest = units % slots;
  const double full = t.two ? t.two : t.one, part = rest == 0 ? 0 : rest <= 256 ? t.one : t.two;
  const double us = (double)(rounds + (rest > 0)) * 2 + ceil_div(stages, splits) * (rounds * full + part);
  return splits == 1 ? us : us + 4 + splits * (double)M * N * 8 / 4.5e6;
}

// the fastest tile and splits by that estimate (us measured, without the join):
//   8192 x 768 x 21760: 256 x 256 whole 502, in 2 279, in 8 322; 128 x 128
//     whole 359, in 4 338; 64 x 128 383
//   1024 x 1024 x 480 stages: 256 x 256 in 8 79, in 16 66; 128 x 128 in 8 85; 64 x
//     128 whole 148, in 2 83
//   100 x 512 x 5760: 64 x 128 whole 32, in 12 7; 128 x 128 in 12 9
//   37 x 50304 x 768: 64 x 128 16, 128 x 128 16, 256 x 256 21
//   12608 x 768 x 8192: 256 x 256 161, 128 x 128 189, 64 x 128 189
struct Plan {
  int tile, splits;
};

Plan plan_of(int64_t M, int64_t N, int stages, int most_splits) {
  Plan best{0, 1};
  double us = 1e30;
  for (int t = 0; t < 3; ++t)
    for (int s = 1; s <= most_splits && s <= stages; s += s < 4 ? 1 : s < 8 ? 2 : 4) {
      const int splits = ceil_div(stages, ceil_div(stages, s));  // none is empty
      const double here = time_of(kTiles[t], M, N, stages, splits);
      if (here < us) us = here, best = {t, splits};
    }
  return best;
}

}  // namespace

int bf_gemm_splits(int64_t M, int64_t N, int stages) { return plan_of(M, N, stages, kBfMostSplits).splits; }

hipError_t launch_bf_gemm(const BfGemmParams& in, BfOut out, hipStream_t st) {
  BfGemmParams g = in;
  const int stages = g.runs * g.run_stages;
  const int tile = plan_of(g.M, g.N, stages, g.splits > 1 ? kBfMostSplits : 1).tile;
  g.split_stages = ceil_div(stages, g.splits);
  if (tile == 0) launch_tiles<2, 4, 8, 2, 32>(g, out, st);
  else if (tile == 1) launch_tiles<2, 2, 4, 2, 32>(g, out, st);
  else launch_tiles<2, 2, 2, 3, 16>(g, out, st);
  return hipGetLastError();
}

}  // namespace metis
