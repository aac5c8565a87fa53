// Expert rows back to their tokens with the combine weights applied here (the
// rows are "weighted by the top-k probabilities" where they return: "Halo's
// 2.8x over TRL is not a kernel, and its own benchmark proves it", section
// "Where the gap actually is"), and the gradient, written as gathers with no
// atomic adds.
//   y[t] = store(sum_j w[t,j] y_perm[row(t,j)])
//   dy_perm[row(t,j)] = store(w[t,j] dy[t]),  d_row_scale[row(t,j)] = <dy[t], y_perm[row(t,j)]>
// Both move each row once and compute 2 to 3 operations an element: HBM bounds them.
#include "rows.h"

namespace moe {
namespace {

// One wave for kPieces x 64 16-byte pieces of a token's row, four expert rows in
// flight, so that several waves share a token whose rows come from far apart.
constexpr int kPieces = 2;
template <typename T>
__global__ __launch_bounds__(256) void k_combine_weighted(const T *__restrict__ y_perm,
                                                          const int32_t *__restrict__ slot_to_row,
                                                          const float *__restrict__ w, int64_t ntok,
                                                          int64_t nrow, int d, int k,
                                                          T *__restrict__ y) {
  constexpr int N = kVec<T>;
  const int nvec = d / N, parts = (nvec + 64 * kPieces - 1) / (64 * kPieces);
  const int64_t wid = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int64_t t = wid / parts;
  if (t >= ntok) return;
  const int lane = threadIdx.x & 63;
  const uint32_t c0 = (uint32_t)((int)(wid - t * parts) * 64 * kPieces + lane) * 16u;
  const uint32_t bytes = (uint32_t)d * sizeof(T);
  int myr = lane < k ? slot_to_row[t * k + lane] : -1;   // k <= 32
  if (myr >= nrow) myr = -1;
  const float myw = myr < 0 ? 0.0f : w[t * k + lane];
  float acc[kPieces][N];
#pragma unroll
  for (int h = 0; h < kPieces; ++h)
#pragma unroll
    for (int i = 0; i < N; ++i) acc[h][i] = 0.0f;
  for (int j = 0; j < k; j += 4) {   // a row that is not there adds 0 * 0
    u32x4_t v[4][kPieces];
#pragma unroll
    for (int u = 0; u < 4; ++u) {   // lanes from k on hold -1 (j + u <= 34)
      const int r = __builtin_amdgcn_readlane(myr, j + u);
      const Row row(y_perm, (int64_t)r * bytes, r >= 0, bytes);
#pragma unroll
      for (int h = 0; h < kPieces; ++h) v[u][h] = row.load(c0 + 1024u * h);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float wj = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(myw), j + u));
#pragma unroll
      for (int h = 0; h < kPieces; ++h) {
        float f[N];
        unpack(v[u][h], f, (const T *)nullptr);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[h][i] = fmaf(wj, f[i], acc[h][i]);
      }
    }
  }
  const Row to(y, t * bytes, true, bytes);
#pragma unroll
  for (int h = 0; h < kPieces; ++h) to.store(c0 + 1024u * h, pack(acc[h], (const T *)nullptr));
}

// One wave for each slot; the waves of a token's slots lie next to each other,
// so that its row of dy comes from HBM once (read past the caches it would
// take 171 us where it takes 162).  16384 tokens with 4 rows of 2880 (850 MB):
// 150 to 170 us as cards differ; with the rows in slot order 142, so it is the
// order of the rows that HBM is slower with.  A wave for each token, which
// keeps dy in registers, takes 169.
constexpr int kSteps = 6;   // 16-byte pieces of a row that a lane has in flight (3: 164 us)
template <typename T>
__global__ __launch_bounds__(256) void k_combine_weighted_bwd(
    const T *__restrict__ dy, const T *__restrict__ y_perm, const int32_t *__restrict__ slot_to_row,
    const float *__restrict__ w, int64_t nslot, int64_t nrow, int d, int k, T *__restrict__ dy_perm,
    float *__restrict__ d_row_scale) {
  constexpr int N = kVec<T>;
  const int64_t slot = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  if (slot >= nslot) return;
  const int r = slot_to_row[slot];
  if (r < 0 || r >= nrow) return;
  const float wj = w[slot];
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)((uint32_t)slot / (uint32_t)k);   // slots are below 2^31
  const uint32_t bytes = (uint32_t)d * sizeof(T);
  const Row g(dy, t * bytes, true, bytes), yr(y_perm, (int64_t)r * bytes, d_row_scale, bytes);
  const Row to(dy_perm, (int64_t)r * bytes, dy_perm, bytes);
  float dot = 0.0f;
  for (uint32_t c = lane * 16u; c < bytes; c += 1024u * kSteps) {
    u32x4_t a[kSteps], b[kSteps];
#pragma unroll
    for (int h = 0; h < kSteps; ++h) {
      a[h] = g.keep(c + 1024u * h);
      b[h] = yr.load(c + 1024u * h);
    }
#pragma unroll
    for (int h = 0; h < kSteps; ++h) {
      float f[N], q[N];
      unpack(a[h], f, (const T *)nullptr);
      unpack(b[h], q, (const T *)nullptr);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        dot = fmaf(f[i], q[i], dot);
        f[i] *= wj;
      }
      to.store(c + 1024u * h, pack(f, (const T *)nullptr));
    }
  }
  if (!d_row_scale) return;
  dot = wave_sum(dot);
  if (lane == 0) d_row_scale[r] = dot;
}

int check(const char *fn, int64_t T, int64_t R, int d, int k, int dtype) {
  MOE_REQUIRE(T >= 0 && R >= 0, MOE_ERR_INVALID_ARG, "%s: T or R < 0", fn);
  MOE_REQUIRE(d > 0 && d % 8 == 0, MOE_ERR_UNSUPPORTED, "%s: d=%d not a positive multiple of 8", fn, d);
  MOE_REQUIRE(k >= 1 && k <= kMaxTopK, MOE_ERR_UNSUPPORTED, "%s: k=%d", fn, k);
  MOE_REQUIRE(T < ((int64_t)1 << 31) / k, MOE_ERR_UNSUPPORTED, "%s: T*k >= 2^31", fn);
  MOE_REQUIRE(dtype == MOE_BF16 || dtype == MOE_F32, MOE_ERR_UNSUPPORTED, "%s: dtype %d", fn, dtype);
  // places in a row, and up to 6 KB past its end, are 32 bits of bytes in the kernels
  MOE_REQUIRE((int64_t)d * (dtype == MOE_BF16 ? 2 : 4) < ((int64_t)1 << 31), MOE_ERR_UNSUPPORTED,
              "%s: rows of 2^31 bytes and more (d=%d)", fn, d);
  return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" {

int moe_combine_weighted(const void *y_perm, int64_t R, const int32_t *slot_to_row,
                         const float *weights, int dtype, int64_t T, int d, int k, void *y, void *stream) {
  using namespace moe;
  const char *fn = "moe_combine_weighted";
  clear_error();
  const int rc = check(fn, T, R, d, k, dtype);
  if (rc != MOE_OK) return rc;
  if (T == 0) return MOE_OK;
  MOE_REQUIRE(y_perm && slot_to_row && weights && y, MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
  MOE_REQUIRE(aligned16(y_perm) && aligned16(y), MOE_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", fn);
  const int64_t nvec = (int64_t)d * (dtype == MOE_BF16 ? 2 : 4) / 16;
  const int64_t blocks = (T * ((nvec + 64 * kPieces - 1) / (64 * kPieces)) + 3) / 4;
  MOE_REQUIRE(blocks < ((int64_t)1 << 24), MOE_ERR_UNSUPPORTED, "%s: too many tokens (T=%lld d=%d)",
              fn, (long long)T, d);   // a launch has below 2^32 threads
  hipStream_t s = (hipStream_t)stream;
  MOE_LAUNCH("combine_weighted", s, {
    if (dtype == MOE_BF16)
      k_combine_weighted<bf16_t><<<(unsigned)blocks, 256, 0, s>>>(
          (const bf16_t *)y_perm, slot_to_row, weights, T, R, d, k, (bf16_t *)y);
    else
      k_combine_weighted<float><<<(unsigned)blocks, 256, 0, s>>>(
          (const float *)y_perm, slot_to_row, weights, T, R, d, k, (float *)y);
  });
  return check_launch(fn);
}

int moe_combine_weighted_bwd(const void *dy, const void *y_perm, int64_t R,
                             const int32_t *slot_to_row, const float *weights, int dtype, int64_t T, int d, int k,
                             void *dy_perm, float *d_row_scale, void *stream) {
  using namespace moe;
  const char *fn = "moe_combine_weighted_bwd";
  clear_error();
  const int rc = check(fn, T, R, d, k, dtype);
  if (rc != MOE_OK) return rc;
  if (T == 0) return MOE_OK;
  MOE_REQUIRE(dy && slot_to_row && weights && (dy_perm || d_row_scale) && (y_perm || !d_row_scale),
              MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
  MOE_REQUIRE(aligned16(dy) && aligned16(y_perm) && aligned16(dy_perm), MOE_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", fn);
  const int64_t slots = T * k, blocks = (slots + 3) / 4;
  MOE_REQUIRE(blocks < ((int64_t)1 << 24), MOE_ERR_UNSUPPORTED, "%s: too many rows (T=%lld k=%d)",
              fn, (long long)T, k);   // a launch has below 2^32 threads
  hipStream_t s = (hipStream_t)stream;
  MOE_LAUNCH("combine_weighted_bwd", s, {
    if (dtype == MOE_BF16)
      k_combine_weighted_bwd<bf16_t><<<(unsigned)blocks, 256, 0, s>>>(
          (const bf16_t *)dy, (const bf16_t *)y_perm, slot_to_row, weights, slots, R, d, k,
          (bf16_t *)dy_perm, d_row_scale);
    else
      k_combine_weighted_bwd<float><<<(unsigned)blocks, 256, 0, s>>>(
          (const float *)dy, (const float *)y_perm, slot_to_row, weights, slots, R, d, k,
          (float *)dy_perm, d_row_scale);
  });
  return check_launch(fn);
}

}  // extern "C"
