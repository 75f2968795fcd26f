// rows.hpp -- access to rows of binary32 or bf16 values, and sums over waves
// and workgroups, shared by the kernels around the linear layers.
#pragma once

#include <type_traits>

#include "common.hpp"

namespace metis {

constexpr int kStatusToken = 8;  // bit of the device's status word: a token number outside the vocabulary

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// two values rounded to bf16 (nearest even), a in the low half
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2_t v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ float unpack_bf16(uint32_t w, int i) {
  return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
}

__device__ __forceinline__ float load1(const void* p, int bf16, int64_t at) {
  return bf16 ? __uint_as_float((uint32_t)((const uint16_t*)p)[at] << 16) : ((const float*)p)[at];
}

__device__ __forceinline__ void store1(void* p, int bf16, int64_t at, float v) {
  if (bf16) ((uint16_t*)p)[at] = (uint16_t)pack_bf16(v, v);
  else ((float*)p)[at] = v;
}

// eight consecutive values at an address that 16 divides
__device__ __forceinline__ void load8(const void* p, int bf16, int64_t at, float* v) {
  if (bf16) {
    const uint4 q = *(const uint4*)((const uint16_t*)p + at);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = unpack_bf16(w[i >> 1], i);
  } else {
    const float4 a = *(const float4*)((const float*)p + at), b = *((const float4*)((const float*)p + at) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}

__device__ __forceinline__ void store8(void* p, int bf16, int64_t at, const float* v) {
  if (bf16) {
    *(uint4*)((uint16_t*)p + at) =
        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  } else {
    float4* const q = (float4*)((float*)p + at);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// Sum over the wave, the same bits in every lane: a butterfly, whose partners
// add the same two values.  Sixteen lanes by DPP, then the lanes of a half
// exchanged, then the halves.
__device__ __forceinline__ float wave_sum(float v) {
  auto dpp = [](float x, auto ctrl) {
    return __int_as_float(
        __builtin_amdgcn_update_dpp(0, __float_as_int(x), decltype(ctrl)::value, 0xF, 0xF, false));
  };
  v += dpp(v, std::integral_constant<int, 0xB1>{});   // quad_perm 1,0,3,2
  v += dpp(v, std::integral_constant<int, 0x4E>{});   // quad_perm 2,3,0,1
  v += dpp(v, std::integral_constant<int, 0x141>{});  // row_half_mirror
  v += dpp(v, std::integral_constant<int, 0x140>{});  // row_mirror
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Sum over T threads that share a row (T a multiple of 64; T = 64: the wave).
// `red` holds T / 64 values; the caller keeps a barrier between two uses of
// the same array (alternating arrays do, since each use has one).
template <int T>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = wave_sum(v);
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < T / 64; ++w) v += red[w];
  }
  return v;
}

}  // namespace metis
