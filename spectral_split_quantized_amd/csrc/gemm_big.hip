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

hipError_t launch_i8_gemm(const I8GemmParams& g, hipStream_t st) {
  if (g.M <= 64) {
    const dim3 grid((unsigned)ceil_div<int64_t>(g.N, 16), 1);
    if (g.M <= 16) hipLaunchKernelGGL((i8_gemm_skinny_kernel<8, 1, 4>), grid, dim3(512), 0, st, g);
    else if (g.M <= 32) hipLaunchKernelGGL((i8_gemm_skinny_kernel<8, 2, 4>), grid, dim3(512), 0, st, g);
    else hipLaunchKernelGGL((i8_gemm_skinny_kernel<8, 4, 2>), grid, dim3(512), 0, st, g);
    return hipGetLastError();
  }
  const int64_t big = ceil_div<int64_t>(g.M, 256) * ceil_div<int64_t>(g.N, 256);
  if (big >= 256) {
    if (g.bf16) hipLaunchKernelGGL((i8_gemm_kernel<2, 4, 4, true>), dim3(256), dim3(512), 0, st, g);
    else hipLaunchKernelGGL((i8_gemm_kernel<2, 4, 4, false>), dim3(256), dim3(512), 0, st, g);
  } else {
    const int64_t tiles = ceil_div<int64_t>(g.M, 128) * ceil_div<int64_t>(g.N, 128);
    const dim3 grid((unsigned)std::min<int64_t>(512, ceil_div<int64_t>(tiles, 8) * 8));
    if (g.bf16) hipLaunchKernelGGL((i8_gemm_kernel<2, 2, 2, true>), grid, dim3(256), 0, st, g);
    else hipLaunchKernelGGL((i8_gemm_kernel<2, 2, 2, false>), grid, dim3(256), 0, st, g);
  }
  return hipGetLastError();
}

}  // namespace metis
