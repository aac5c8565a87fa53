// Rows of bf16 or fp32 in 16-byte pieces, and sums over a wave.
#pragma once

#include "moe_internal.h"

namespace moe {

template <typename T> constexpr int kVec = 16 / (int)sizeof(T);   // elements in 16 bytes

__device__ __forceinline__ void unpack(const u32x4_t v, float *f, const bf16_t *) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_bits_to_f32(v[i] & 0xffffu);
    f[2 * i + 1] = bf16_bits_to_f32(v[i] >> 16);
  }
}
__device__ __forceinline__ void unpack(const u32x4_t v, float *f, const float *) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
}
__device__ __forceinline__ u32x4_t pack(const float *f, const bf16_t *) {
  u32x4_t v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  return v;
}
__device__ __forceinline__ u32x4_t pack(const float *f, const float *) {
  u32x4_t v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(f[i]);
  return v;
}

// Sum over the 64 lanes, the same in all of them, in a fixed order.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
  return v;
}

}  // namespace moe
