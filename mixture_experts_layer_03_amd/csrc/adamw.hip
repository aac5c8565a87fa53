// An AdamW step over many tensors in one launch for each 40 of them.
//
//   m = b1 m + (1-b1) g,  v = b2 v + (1-b2) g g,
//   p = p (1 - lr wd) - lr/(1-b1^t) m / (sqrt(v)/sqrt(1-b2^t) + eps)
//
// States in 32 bits, or in 8 with a power of two for each 128 elements: m in
// e4m3, v in e5m2 (its values are squares, so it gets the wider exponent).
// Both are rounded up or down at random in proportion to where the value lies
// between its neighbours: v moves by 1-b2 = 1e-3 of itself in a step, far
// below half an 8-bit step, and rounding to nearest would never move it.  bf16
// parameters without a 32-bit copy are rounded the same way, for the same
// reason.  The random bits are a hash of (seed, step, tensor, element).
//
// Per element 28 bytes move with fp32 parameters, 30 with bf16 ones and a
// copy, 12 with bf16 ones and 8-bit states: HBM bounds the step, with the
// hash and roundings (~100 instructions an element) close behind at 12.
#include <algorithm>
#include <cmath>
#include <functional>
#include <vector>

#include "rows.h"

namespace moe {
namespace {

constexpr int kPerLaunch = 40;   // tensors whose pointers fit the kernel's arguments (below 4 KB)

struct AdamTensor {
  void *p;
  const void *g;
  float *master;
  void *m, *v;
  uint8_t *m_scale, *v_scale;
  int64_t n;
  double decay;                  // the host's 1 - lr wd, or wd where lr is on the device
  uint32_t index;                // place in the caller's list, for the random bits
};

struct AdamArgs {
  AdamTensor t[kPerLaunch];
  uint32_t first[kPerLaunch];    // each tensor's first block
  int count;
  float b1, a1, b2, a2, eps;     // a = 1 - b, rounded from 64 bits
  float step_size, inv_sqrt_bc2; // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  float ln_b1, ln_b2;
  uint32_t seed_lo, seed_hi, step;
  const float *grad_scale, *lr;
  const int64_t *step_dev;
};

__device__ __forceinline__ uint32_t mix(uint32_t a) {
  a ^= a >> 16;
  a *= 0x971cbef1u;
  a ^= a >> 15;
  a *= 0x6a695495u;
  a ^= a >> 16;
  return a;
}

// The largest of 16 neighbouring lanes' values, in all of them.
__device__ __forceinline__ float max16(float v) {
#define MOE_ROR(n) \
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x120 + n, 0xf, 0xf, true)))
  MOE_ROR(8);
  MOE_ROR(4);
  MOE_ROR(2);
  MOE_ROR(1);
#undef MOE_ROR
  return v;
}

__device__ __forceinline__ bool finite(float v) { return (__float_as_uint(v) & 0x7f800000u) != 0x7f800000u; }

// The smallest s >= -126 with amax <= 1.75 * 2^top * 2^s; 0 for an empty block.
template <int TOP>
__device__ __forceinline__ int block_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int s = (int)(b >> 23) - 127 - TOP + ((b & 0x7fffffu) > 0x600000u);
  return b == 0 ? 0 : max(s, -126);
}

// |x| times the block's inverse scale, at most 1.75 * 2^(its largest exponent),
// to 8 bits: MANT mantissa bits, exponent bias BIAS, 16 random bits below the
// last.  The scaling is exact but for values that are far below the smallest
// code.  No carry leaves the format: the largest value has no bits below its last.
template <int MANT, int BIAS>
__device__ __forceinline__ uint32_t to8(float a, uint32_t r16) {
  constexpr int cut = 23 - MANT;
  constexpr float least = 1.0f / (float)(1 << (BIAS - 1));            // smallest normal
  const uint32_t r = r16 << (cut - 16);
  const uint32_t normal = ((__float_as_uint(a) + r) >> cut) - (uint32_t)((127 - BIAS) << MANT);
  const uint32_t low = ((uint32_t)(fminf(a, least) * __uint_as_float((uint32_t)(127 + BIAS - 1 + MANT + cut) << 23)) + r) >> cut;
  return a >= least ? normal : low;
}

template <typename T, int V>
__device__ __forceinline__ void load_row(const void *base, int64_t i, int64_t n, float (&f)[V]) {
  if (i + V <= n) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int q = 0; q < V / 4; ++q) {
        const u32x4_t v = *reinterpret_cast<const u32x4_t *>((const float *)base + i + 4 * q);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[4 * q + e] = __uint_as_float(v[e]);
      }
    } else {
      uint32_t w[V / 2];
      __builtin_memcpy(w, __builtin_assume_aligned((const bf16_t *)base + i, 2 * V), 2 * V);
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        f[2 * e] = bf16_bits_to_f32(w[e] & 0xffffu);
        f[2 * e + 1] = bf16_bits_to_f32(w[e] >> 16);
      }
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < V; ++e) f[e] = i + e < n ? Store<T>::load((const T *)base + i + e) : 0.0f;
}

template <typename T, int V>
__device__ __forceinline__ void store_row(void *base, int64_t i, int64_t n, const float (&f)[V]) {
  uint32_t w[V * sizeof(T) / 4];
#pragma unroll
  for (int e = 0; e < V; e += (sizeof(T) == 4 ? 1 : 2)) {
    if constexpr (sizeof(T) == 4) w[e] = __float_as_uint(f[e]);
    else w[e / 2] = pack_bf16x2(f[e], f[e + 1]);
  }
  T *p = (T *)base + i;
  if (i + V <= n) {
    __builtin_memcpy(__builtin_assume_aligned(p, sizeof(T) * V < 16 ? sizeof(T) * V : 16), w, sizeof(T) * V);
    return;
  }
#pragma unroll
  for (int e = 0; e < V; ++e) {
    if (i + e >= n) continue;
    if constexpr (sizeof(T) == 4) p[e] = f[e];
    else p[e] = (bf16_t)(w[e / 2] >> (16 * (e & 1)));
  }
}

__device__ __forceinline__ u32x2_t load8(const void *base, int64_t i, int64_t n) {
  const uint8_t *p = (const uint8_t *)base + i;
  if (i + 8 <= n) return *reinterpret_cast<const u32x2_t *>(p);
  u32x2_t w = {0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (i + e < n) w[e / 4] |= (uint32_t)p[e] << (8 * (e & 3));
  return w;
}
__device__ __forceinline__ void store8(void *base, int64_t i, int64_t n, u32x2_t w) {
  uint8_t *p = (uint8_t *)base + i;
  if (i + 8 <= n) {
    *reinterpret_cast<u32x2_t *>(p) = w;
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (i + e < n) p[e] = (uint8_t)(w[e / 4] >> (8 * (e & 3)));
}

// P, G: types of parameter and gradient.  A thread takes V neighbouring
// elements, a block 256 V of them; 16 lanes share the scale of 128 (i >> 7).
template <typename P, typename G, bool MASTER, bool EIGHT>
__global__ __launch_bounds__(256) void k_adamw(const AdamArgs a) {
#pragma clang fp contract(off)
  constexpr int V = EIGHT ? 8 : 4;
  constexpr bool RANDOM_P = sizeof(P) == 2 && !MASTER;
  int lo = 0, hi = a.count - 1;
  while (lo < hi) {   // the tensor of this block
    const int mid = (lo + hi + 1) >> 1;
    if (a.first[mid] <= blockIdx.x) lo = mid;
    else hi = mid - 1;
  }
  const AdamTensor &t = a.t[lo];
  const int64_t n = t.n;
  const int64_t i = ((int64_t)(blockIdx.x - a.first[lo]) * 256 + threadIdx.x) * V;

  float g[V], p[V], m[V], v[V];
  load_row<G>(t.g, i, n, g);
  if constexpr (MASTER) load_row<float>(t.master, i, n, p);
  else load_row<P>(t.p, i, n, p);
  if constexpr (EIGHT) {
    const u32x2_t mq = load8(t.m, i, n), vq = load8(t.v, i, n);
    const int64_t b = i >> 7;
    const float ms = i < n ? __uint_as_float((uint32_t)t.m_scale[b] << 23) : 0.0f;
    const float vs = i < n ? __uint_as_float((uint32_t)t.v_scale[b] << 23) : 0.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const bool up = q & 1;
      const f32x2_t mf = up ? __builtin_amdgcn_cvt_pk_f32_fp8((int)mq[q / 2], true)
                            : __builtin_amdgcn_cvt_pk_f32_fp8((int)mq[q / 2], false);
      const f32x2_t vf = up ? __builtin_amdgcn_cvt_pk_f32_bf8((int)vq[q / 2], true)
                            : __builtin_amdgcn_cvt_pk_f32_bf8((int)vq[q / 2], false);
      m[2 * q] = mf[0] * ms;
      m[2 * q + 1] = mf[1] * ms;
      v[2 * q] = vf[0] * vs;
      v[2 * q + 1] = vf[1] * vs;
    }
  } else {
    load_row<float>(t.m, i, n, m);
    load_row<float>(t.v, i, n, v);
  }

  const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
  float decay = (float)t.decay, step_size = a.step_size, rbc2 = a.inv_sqrt_bc2;
  uint32_t step = a.step;
  if (a.lr) {   // a captured step: the learning rate and the step count are the device's
    const int64_t s = *a.step_dev;
    step = (uint32_t)s;
    const float lr = *a.lr;
    decay = (float)(1.0 - (double)lr * t.decay);
    step_size = lr / -expm1f((float)s * a.ln_b1);
    rbc2 = 1.0f / sqrtf(-expm1f((float)s * a.ln_b2));
  }
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float ge = g[e] * gs;
    m[e] = m[e] * a.b1 + ge * a.a1;
    v[e] = v[e] * a.b2 + ge * a.a2 * ge;
    // 1-ulp root and reciprocal: off by 2^-22 of the update, below the
    // rounding of p wherever the update is below p/4
    const float den = __builtin_amdgcn_sqrtf(v[e]) * rbc2 + a.eps;
    p[e] = p[e] * decay - step_size * (m[e] * __builtin_amdgcn_rcpf(den));
  }

  uint32_t r[V];
  if constexpr (RANDOM_P || EIGHT) {
    const uint32_t key =
        mix(mix(mix(mix(a.seed_lo) ^ a.seed_hi) ^ step) ^ t.index) ^ (uint32_t)(i >> 32);
#pragma unroll
    for (int e = 0; e < V; ++e) r[e] = mix(key ^ ((uint32_t)i + e));
  }
  if constexpr (EIGHT) {
    float m_max = 0.0f, v_max = 0.0f;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      m_max = finite(m[e]) ? fmaxf(m_max, fabsf(m[e])) : m_max;
      v_max = finite(v[e]) ? fmaxf(v_max, fabsf(v[e])) : v_max;
    }
    const int ms = block_exponent<8>(max16(m_max)), vs = block_exponent<15>(max16(v_max));
    const float mi = __uint_as_float((uint32_t)(127 - ms) << 23), vi = __uint_as_float((uint32_t)(127 - vs) << 23);
    u32x2_t mq = {0u, 0u}, vq = {0u, 0u};
#pragma unroll
    for (int e = 0; e < V; ++e) {
      uint32_t cm = to8<3, 7>(fabsf(m[e]) * mi, r[e] >> 16) | ((__float_as_uint(m[e]) >> 24) & 0x80u);
      uint32_t cv = to8<2, 15>(fabsf(v[e]) * vi, (r[e] * 0x30e9132du) >> 16);
      // a second moment that is not zero never becomes it: its root divides
      if (v[e] > 0.0f) cv = max(cv, 1u);
      if (!finite(m[e])) cm = 0x7fu;
      if (!finite(v[e])) cv = 0x7fu;
      mq[e / 4] |= cm << (8 * (e & 3));
      vq[e / 4] |= cv << (8 * (e & 3));
    }
    store8(t.m, i, n, mq);
    store8(t.v, i, n, vq);
    if ((threadIdx.x & 15) == 0 && i < n) {
      t.m_scale[i >> 7] = (uint8_t)(ms + 127);
      t.v_scale[i >> 7] = (uint8_t)(vs + 127);
    }
  } else {
    store_row<float>(t.m, i, n, m);
    store_row<float>(t.v, i, n, v);
  }
  if constexpr (MASTER) store_row<float>(t.master, i, n, p);
  if constexpr (RANDOM_P) {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (finite(p[e])) p[e] = __uint_as_float((__float_as_uint(p[e]) + (r[e] & 0xffffu)) & 0xffff0000u);
  }
  store_row<P>(t.p, i, n, p);
}

constexpr int64_t kMaxBlocks = ((int64_t)1 << 24) - 1;   // a launch has below 2^32 threads

// Whether no two tensors with elements have the same pointer; without a copy
// of the list where the pointers ascend, as tensors allocated in order do.
template <typename F>
bool distinct(const moe_adamw_tensor *t, int n, F of) {
  const void *last = nullptr;
  bool ascending = true;
  for (int i = 0; i < n && ascending; ++i) {
    if (t[i].numel == 0) continue;
    ascending = std::less<const void *>()(last, of(t[i]));
    last = of(t[i]);
  }
  if (ascending) return true;
  std::vector<const void *> all;
  for (int i = 0; i < n; ++i)
    if (t[i].numel) all.push_back(of(t[i]));
  std::sort(all.begin(), all.end(), std::less<const void *>());
  return std::adjacent_find(all.begin(), all.end()) == all.end();
}

template <typename P, typename G, bool MASTER>
void launch(const AdamArgs &a, unsigned blocks, bool eight, hipStream_t s) {
  if (eight) k_adamw<P, G, MASTER, true><<<blocks, 256, 0, s>>>(a);
  else k_adamw<P, G, MASTER, false><<<blocks, 256, 0, s>>>(a);
}

}  // namespace
}  // namespace moe

extern "C" int moe_adamw_step(const moe_adamw_tensor *tensors, int n, int param_dtype,
                              int grad_dtype, int state_bits, double lr, double beta1, double beta2,
                              double eps, int64_t step, uint64_t seed, const float *grad_scale,
                              const float *lr_dev, const int64_t *step_dev, void *stream) {
  using namespace moe;
  const char *fn = "moe_adamw_step";
  clear_error();
  MOE_REQUIRE(n >= 0 && (n == 0 || tensors), MOE_ERR_INVALID_ARG, "%s: bad tensor list", fn);
  MOE_REQUIRE((param_dtype == MOE_BF16 || param_dtype == MOE_F32) &&
                  (grad_dtype == MOE_F32 || (grad_dtype == MOE_BF16 && param_dtype == MOE_BF16)),
              MOE_ERR_UNSUPPORTED, "%s: parameters of dtype %d with gradients of dtype %d", fn,
              param_dtype, grad_dtype);
  MOE_REQUIRE(state_bits == 32 || state_bits == 8, MOE_ERR_UNSUPPORTED, "%s: states of %d bits", fn,
              state_bits);
  MOE_REQUIRE(beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0 && eps >= 1e-30 && eps < 1e30,
              MOE_ERR_INVALID_ARG, "%s: beta1=%g beta2=%g eps=%g", fn, beta1, beta2, eps);
  MOE_REQUIRE(!lr_dev == !step_dev, MOE_ERR_INVALID_ARG, "%s: lr_dev and step_dev go together", fn);
  MOE_REQUIRE(lr_dev || (step >= 1 && step < ((int64_t)1 << 32) && std::isfinite(lr)),
              MOE_ERR_INVALID_ARG, "%s: step=%lld lr=%g", fn, (long long)step, lr);
  const bool eight = state_bits == 8, master = n > 0 && tensors[0].master;
  const int64_t per_block = 256 * (eight ? 8 : 4);
  for (int i = 0; i < n; ++i) {
    const moe_adamw_tensor &t = tensors[i];
    MOE_REQUIRE(t.numel >= 0 && t.numel <= per_block * kMaxBlocks, MOE_ERR_UNSUPPORTED,
                "%s: tensor %d has %lld elements", fn, i, (long long)t.numel);
    MOE_REQUIRE((t.master != nullptr) == master && !(master && param_dtype == MOE_F32),
                MOE_ERR_INVALID_ARG, "%s: tensor %d: all bf16 parameters have a 32-bit copy, or none",
                fn, i);
    MOE_REQUIRE(std::isfinite(t.weight_decay), MOE_ERR_INVALID_ARG, "%s: tensor %d: weight_decay %g", fn,
                i, t.weight_decay);
    if (t.numel == 0) continue;
    MOE_REQUIRE(t.param && t.grad && t.m && t.v && (!eight || (t.m_scale && t.v_scale)),
                MOE_ERR_INVALID_ARG, "%s: tensor %d: null pointer", fn, i);
    MOE_REQUIRE(aligned16(t.param) && aligned16(t.grad) && aligned16(t.master) && aligned16(t.m) &&
                    aligned16(t.v),
                MOE_ERR_INVALID_ARG, "%s: tensor %d: pointers must be 16-byte aligned", fn, i);
  }
  bool once = true;   // two updates of one tensor would race
  try {
    once = distinct(tensors, n, [](const moe_adamw_tensor &t) { return (const void *)t.param; }) &&
           distinct(tensors, n, [](const moe_adamw_tensor &t) { return (const void *)t.m; }) &&
           distinct(tensors, n, [](const moe_adamw_tensor &t) { return (const void *)t.v; }) &&
           (!master || distinct(tensors, n, [](const moe_adamw_tensor &t) { return (const void *)t.master; }));
  } catch (...) {
    MOE_REQUIRE(false, MOE_ERR_INVALID_ARG, "%s: no memory for a list of %d tensors", fn, n);
  }
  MOE_REQUIRE(once, MOE_ERR_INVALID_ARG, "%s: a parameter or state is listed twice", fn);

  AdamArgs a;
  a.b1 = (float)beta1, a.a1 = (float)(1.0 - beta1), a.b2 = (float)beta2, a.a2 = (float)(1.0 - beta2);
  a.eps = (float)eps;
  a.ln_b1 = (float)std::log(beta1), a.ln_b2 = (float)std::log(beta2);   // -inf for 0
  a.step_size = lr_dev ? 0.0f : (float)(lr / (1.0 - std::pow(beta1, (double)step)));
  a.inv_sqrt_bc2 = lr_dev ? 0.0f : (float)(1.0 / std::sqrt(1.0 - std::pow(beta2, (double)step)));
  a.seed_lo = (uint32_t)seed, a.seed_hi = (uint32_t)(seed >> 32), a.step = (uint32_t)step;
  a.grad_scale = grad_scale, a.lr = lr_dev, a.step_dev = step_dev;
  hipStream_t s = (hipStream_t)stream;
  for (int i = 0; i < n;) {
    int64_t blocks = 0;
    a.count = 0;
    for (; i < n && a.count < kPerLaunch; ++i) {
      const moe_adamw_tensor &t = tensors[i];
      if (t.numel == 0) continue;
      const int64_t mine = (t.numel + per_block - 1) / per_block;
      if (blocks + mine > kMaxBlocks) break;
      a.t[a.count] = {t.param,   t.grad,    t.master, t.m, t.v,
                      t.m_scale, t.v_scale, t.numel,  lr_dev ? t.weight_decay : 1.0 - lr * t.weight_decay,
                      (uint32_t)i};
      a.first[a.count++] = (uint32_t)blocks;
      blocks += mine;
    }
    if (!a.count) break;
    MOE_LAUNCH("adamw", s, {
      const unsigned b = (unsigned)blocks;
      if (param_dtype == MOE_F32) launch<float, float, false>(a, b, eight, s);
      else if (master && grad_dtype == MOE_F32) launch<bf16_t, float, true>(a, b, eight, s);
      else if (master) launch<bf16_t, bf16_t, true>(a, b, eight, s);
      else if (grad_dtype == MOE_F32) launch<bf16_t, float, false>(a, b, eight, s);
      else launch<bf16_t, bf16_t, false>(a, b, eight, s);
    });
    const int e = check_launch(fn);
    if (e != MOE_OK) return e;
  }
  return MOE_OK;
}
