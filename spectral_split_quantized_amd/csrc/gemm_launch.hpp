// gemm_launch.hpp -- host entry of the register-dequant GEMM translation unit.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace metis {

// Workgroups that one launch takes: a dispatch has fewer than 2^32 work items.
inline int64_t max_groups(int64_t threads) { return (int64_t)UINT32_MAX / threads; }

struct GemmParams;

// C = alpha A B^T (+ K-extension) with 256 x 256 tiles; requires K % 256 == 0
// and 16-byte aligned code, scale and extension rows.
// splits > 1 writes raw partial sums per split (see gemm_fp4_kernel).
hipError_t launch_gemm_big(const GemmParams& gp, int splits, hipStream_t st);

struct MxGemmParams;

// C = A B^T of two MXFP4 operands with 256 x 256 tiles; requires K % 1024 == 0
// and 16-byte aligned code and scale rows.
hipError_t launch_mx_gemm(const MxGemmParams& g, hipStream_t st);

struct I8GemmParams;

// C = diag(s_a) A B^T diag(s_b) of two int8 operands; code rows 16-byte
// aligned with a pitch that is a multiple of 128.  part: i8_gemm_workspace
// bytes (0: may be null), 16-byte aligned; splits and run are set here.
size_t i8_gemm_workspace(int64_t M, int64_t N, int64_t pitch);
hipError_t launch_i8_gemm(const I8GemmParams& g, hipStream_t st);

}  // namespace metis
