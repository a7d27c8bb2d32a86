// The 128-point Walsh-Hadamard transform of one head vector held by 4 lanes
// (32 values each) or by a whole warp (4 values each), unnormalised, float32.
//
// Both run the butterfly stages in the order of the rotate+quantise kernel for
// g = 128 (index bits 6, 0, 1, 2, 4, 5, 3), so that the sums round alike and the
// codes of a vector do not depend on which kernel made them.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fwht_dev.cuh"

namespace convrot {

namespace fwht {

constexpr float kInvSqrt128 = 0.0883883461356163f;  // nearest float to 1/sqrt(128)

// Two 16-bit values (bf16, or IEEE fp16) widened to float32, and rounded back.
template <bool F16>
__device__ __forceinline__ float2 widen_pair(uint32_t w) {
  if (F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

template <bool F16>
__device__ __forceinline__ uint32_t narrow_pair(float a, float b) {
  if (F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// One stage between lanes: the lower lane keeps a + b, the upper a - b.
template <int N>
__device__ __forceinline__ void lane_stage(float (&v)[N], int mask, bool upper) {
  const float own = upper ? -1.0f : 1.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = fmaf(own, v[i], __shfl_xor_sync(0xFFFFFFFFu, v[i], mask));
}

// One stage between the values a thread holds, on index bit H of the register.
template <int N, int H>
__device__ __forceinline__ void reg_stage(float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if ((i & H) == 0) {
      const float a = v[i], b = v[i + H];
      v[i] = a + b;
      v[i + H] = a - b;
    }
  }
}

// One stage between lanes on packed pairs.
template <int N>
__device__ __forceinline__ void lane_stage2(float2 (&v)[N], int mask, bool upper) {
  const float own = upper ? -1.0f : 1.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float2 q = make_float2(__shfl_xor_sync(0xFFFFFFFFu, v[i].x, mask), __shfl_xor_sync(0xFFFFFFFFu, v[i].y, mask));
    v[i] = __ffma2_rn(make_float2(own, own), v[i], q);
  }
}

// One stage between the packed pairs a thread holds, on index bit H.
template <int N, int H>
__device__ __forceinline__ void reg_stage2(float2 (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if ((i & H) == 0) {
      const float2 a = v[i], b = v[i + H];
      v[i] = bfly_sum(a, b);
      v[i + H] = bfly_diff(a, b);
    }
  }
}

// Lane l (0..3) of a vector holds channels 32 j + 8 l + e (.x) and 64 more (.y) in
// v[8 j + e], j in {0, 1}. The stage on index bit 6, between .x and .y, has been
// done where the pairs were made; this does the other six.
__device__ __forceinline__ void fwht128_quad(float2 (&v)[16], int l) {
  reg_stage2<16, 1>(v);
  reg_stage2<16, 2>(v);
  reg_stage2<16, 4>(v);
  lane_stage2(v, 2, (l & 2) != 0);
  reg_stage2<16, 8>(v);
  lane_stage2(v, 1, (l & 1) != 0);
}

// Lane l (0..31) holds channels 4 l .. 4 l + 3.
__device__ __forceinline__ void fwht128_warp(float (&v)[4], int l) {
  lane_stage(v, 16, (l & 16) != 0);
  reg_stage<4, 1>(v);
  reg_stage<4, 2>(v);
  lane_stage(v, 1, (l & 1) != 0);
  lane_stage(v, 4, (l & 4) != 0);
  lane_stage(v, 8, (l & 8) != 0);
  lane_stage(v, 2, (l & 2) != 0);
}

}  // namespace fwht

}  // namespace convrot
