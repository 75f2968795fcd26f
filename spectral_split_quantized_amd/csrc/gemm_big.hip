// gemm_big.hip -- translation unit of the register-dequant GEMM (built with
// an instruction-level-parallelism scheduling strategy; see build.py).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "gemm_launch.hpp"
#include "gemm_reg.hpp"
#include "mxfp4_gemm.hpp"
#include "int8_gemm.hpp"

namespace metis {

hipError_t launch_gemm_big(const GemmParams& gp, int splits, hipStream_t st) {
  using Cfg = RegCfg<2, 2, 4, 4>;
  const int64_t tiles = ceil_div<int64_t>(gp.M, Cfg::BM) * ceil_div<int64_t>(gp.N, Cfg::BN);
  if (tiles <= 0) return hipSuccess;
  // LDS is static (one array per pipeline stage)
  hipLaunchKernelGGL((gemm_fp4_reg_kernel<2, 2, 4, 4>), dim3((unsigned)tiles, (unsigned)splits), dim3(Cfg::NT),
                     0, st, gp);
  return hipGetLastError();
}

hipError_t launch_mx_gemm(const MxGemmParams& g, hipStream_t st) {
  const int64_t tiles = ceil_div<int64_t>(g.M, 256) * ceil_div<int64_t>(g.N, 256);
  if (tiles <= 0) return hipSuccess;
  hipLaunchKernelGGL((mx_gemm_kernel<2, 2, 4, 4>), dim3((unsigned)tiles), dim3(256), 0, st, g);
  return hipGetLastError();
}

namespace {

template <int WM, int WN, int TM, int NS, int ER>
void launch_i8_tiles(const I8GemmParams& g, hipStream_t st) {
  const int64_t units = ceil_div<int64_t>(g.M, WM * TM * 32) * ceil_div<int64_t>(g.N, WN * 64) * g.splits;
  // workgroups that fit the chip at once: one of 8 waves a CU, or two of 4
  const dim3 grid((unsigned)std::min<int64_t>(256 * (8 / (WM * WN)), ceil_div<int64_t>(units, 8) * 8));
  const dim3 block(WM * WN * 64);
  if constexpr (TM == 1) {  // the larger tiles take the products that fill the chip without a cut
    if (g.splits > 1) {
      I8GemmParams q = g;
      q.C = g.part;
      q.ldc = g.N;
      hipLaunchKernelGGL((i8_gemm_kernel<WM, WN, TM, NS, ER, kOutPart>), grid, block, 0, st, q);
      const dim3 join((unsigned)ceil_div<int64_t>(g.M * ((g.N + 3) >> 2), 64));
      if (g.bf16) hipLaunchKernelGGL((i8_join_kernel<true>), join, dim3(64), 0, st, g);
      else hipLaunchKernelGGL((i8_join_kernel<false>), join, dim3(64), 0, st, g);
      return;
    }
  }
  if (g.bf16) {
    hipLaunchKernelGGL((i8_gemm_kernel<WM, WN, TM, NS, ER, kOutBF16>), grid, block, 0, st, g);
  } else {
    hipLaunchKernelGGL((i8_gemm_kernel<WM, WN, TM, NS, ER, kOutF32>), grid, block, 0, st, g);
  }
}

}  // namespace

size_t i8_gemm_workspace(int64_t M, int64_t N, int64_t pitch) {
  if (M <= 0 || N <= 0 || pitch <= 0) return 0;
  const I8Plan pl = i8_plan(M, N, pitch);
  return pl.splits > 1 ? (size_t)pl.splits * M * N * sizeof(int32_t) : 0;
}

hipError_t launch_i8_gemm(const I8GemmParams& in, hipStream_t st) {
  I8GemmParams g = in;
  const I8Plan pl = i8_plan(g.M, g.N, g.pitch);
  g.splits = pl.splits;
  g.run = pl.run;
  if (pl.tile == 256) launch_i8_tiles<2, 4, 4, 2, 32>(g, st);
  else if (pl.tile == 128) launch_i8_tiles<2, 2, 2, 2, 32>(g, st);
  else if (pl.tile == 64 && pl.slots == 3) launch_i8_tiles<2, 2, 1, 3, 16>(g, st);
  else if (pl.tile == 64) launch_i8_tiles<2, 2, 1, 2, 32>(g, st);
  else {
    // one batch of loads for the whole row where four waves can hold it
    // (16 x 4096 bytes: 13.1 us at 14336 rows of B against 14.6 with eight
    // waves of four loads; at 14336 bytes 14.8 against 13.5)
    const int64_t steps = g.pitch >> 6, lines = max_groups(512) * 16;
    for (int64_t n0 = 0; n0 < in.N; n0 += lines) {
      g.N = std::min(lines, in.N - n0);
      g.b = in.b + n0 * in.pitch;
      g.sb = in.sb + n0;
      g.C = (char*)in.C + n0 * (in.bf16 ? 2 : 4);
      const dim3 grid((unsigned)ceil_div<int64_t>(g.N, 16));
      if (steps > 32 && steps <= 64) hipLaunchKernelGGL((i8_gemm_skinny_kernel<4, 16>), grid, dim3(256), 0, st, g);
      else hipLaunchKernelGGL((i8_gemm_skinny_kernel<8, 4>), grid, dim3(512), 0, st, g);
    }
  }
  return hipGetLastError();
}

}  // namespace metis
