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

// A row as a buffer: what lies past its end, or a row that is not there (0
// bytes), reads as zero and takes no stores.  Without branches the compiler
// knows how many accesses are on their way and waits for the ones it needs;
// behind a store in a branch it waits for all, the stores' ends among them.
// Non-temporal, as every row here is read or written once: four streams read
// and two written at 6.2 TB/s against 5.5 without (16384 rows of 5760 bytes).
constexpr int kNt = 2;   // the cache-policy operand's bit
struct Row {
  __amdgpu_buffer_rsrc_t rs;
  __device__ Row(const void *p, int64_t at, bool there, uint32_t bytes)
      : rs(__builtin_amdgcn_make_buffer_rsrc((void *)((const char *)p + (there ? at : 0)), 0,
                                             (int)(there ? bytes : 0u), 0x00020000)) {}
  __device__ __forceinline__ u32x4_t load(uint32_t off) const {
    return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, (int)off, 0, kNt));
  }
  // for a row that others read too
  __device__ __forceinline__ u32x4_t keep(uint32_t off) const {
    return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, (int)off, 0, 0));
  }
  __device__ __forceinline__ void store(uint32_t off, u32x4_t v) const {
    __builtin_amdgcn_raw_buffer_store_b128(v, rs, (int)off, 0, kNt);
  }
};

// Sum over the 64 lanes, the same in all of them, in a fixed order: within rows
// of 16 lanes, then lanes 15, 31 and 47 into the rows behind them.  Six vector
// instructions; through LDS (shuffles) the same six steps wait ~100 cycles each.
template <int CTRL, int ROWS>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xf, true));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = add_dpp<0x111, 0xf>(v);   // row_shr 1, 2, 4, 8
  v = add_dpp<0x112, 0xf>(v);
  v = add_dpp<0x114, 0xf>(v);
  v = add_dpp<0x118, 0xf>(v);
  v = add_dpp<0x142, 0xa>(v);   // row_bcast 15 into rows 1 and 3
  v = add_dpp<0x143, 0xc>(v);   // row_bcast 31 into rows 2 and 3
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

}  // namespace moe
