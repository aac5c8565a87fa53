// An AdamW step over many tensors in a launch for each 55 to 83 of them.
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
// copy, 12 with bf16 ones and 8-bit states, each once and in order: HBM bounds
// the step.  Measured: 796M bf16 weights with copies 3.78 ms (6.3 TB/s), 604M
// with 8-bit states 1.16 ms (6.3 TB/s; ~48 instructions an element, five of
// them at quarter rate).
#include <algorithm>
#include <cmath>
#include <functional>
#include <type_traits>
#include <vector>

#include "rows.h"

namespace moe {
namespace {

// Up to kMost tensors of a launch: their pointers fit the kernel's 4 KB of
// arguments (62 with 8-bit states and no master copies).  A launch costs 5 to
// 10 us beside its share of the work: its first blocks' way to the code and
// its last blocks.
constexpr int kArgBytes = 4096, kScalarBytes = 96;
enum { kP, kG, kM, kV, kMore };   // kMore: master, or the scales of m and v behind it

template <int PTRS>
struct AdamArgs {
  static constexpr int kMost = (kArgBytes - kScalarBytes) / (8 * PTRS + 16);
  void *ptr[PTRS][kMost];
  int64_t n[kMost];
  float decay[kMost];            // 1 - lr wd, or wd where lr is on the device
  uint32_t first[kMost];         // each tensor's first block
  const float *grad_scale, *lr;
  const int64_t *step_dev;
  int count;
  uint32_t base;                 // place of the first in the caller's list
  float b1, a1, b2, a2, eps;     // a = 1 - b, rounded from 64 bits
  float step_size, inv_sqrt_bc2; // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  float ln_b1, ln_b2;
  uint32_t seed_lo, seed_hi, step;
};

// Shifts and odd factors chosen here: a flipped bit of the argument flips each
// bit of the result with a probability of 0.487 to 0.513 (2^18 arguments).
__device__ __forceinline__ uint32_t mix(uint32_t a) {
  a ^= a >> 16;
  a *= 0x971cbef1u;
  a ^= a >> 15;
  a *= 0x6a695495u;
  a ^= a >> 16;
  return a;
}

// The largest of 16 neighbouring lanes' values, in all of them.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
#define MOE_ROR(n) v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x120 + n, 0xf, 0xf, true))
  MOE_ROR(8);
  MOE_ROR(4);
  MOE_ROR(2);
  MOE_ROR(1);
#undef MOE_ROR
  return v;
}

constexpr uint32_t kInf = 0x7f800000u;
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The smallest s >= -126 with amax <= 1.75 * 2^top * 2^s; 0 for an empty block.
template <int TOP>
__device__ __forceinline__ int block_exponent(uint32_t amax) {
  const int s = (int)(amax >> 23) - 127 - TOP + ((amax & 0x7fffffu) > 0x600000u);
  return amax == 0 ? 0 : max(s, -126);
}

// TAIL: the elements may end here; elsewhere whole vectors, without a branch.
template <bool TAIL, typename T, int V>
__device__ __forceinline__ void load_row(const void *base, int64_t i, int64_t n, float (&f)[V]) {
  if (!TAIL || i + V <= n) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int q = 0; q < V / 4; ++q) {
        const u32x4_t v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t *>((const float *)base + i + 4 * q));
#pragma unroll
        for (int e = 0; e < 4; ++e) f[4 * q + e] = __uint_as_float(v[e]);
      }
    } else {
      typedef uint32_t words __attribute__((ext_vector_type(V / 2)));
      const words w = __builtin_nontemporal_load(reinterpret_cast<const words *>((const bf16_t *)base + i));
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

// V elements as words (two bf16 in one)
template <bool TAIL, typename T, int V>
__device__ __forceinline__ void store_words(void *base, int64_t i, int64_t n,
                                            const uint32_t (&w)[V * sizeof(T) / 4]) {
  constexpr int kWords = V * (int)sizeof(T) / 4, kEach = kWords < 4 ? kWords : 4;
  typedef uint32_t words __attribute__((ext_vector_type(kEach)));
  T *p = (T *)base + i;
  if (!TAIL || i + V <= n) {
#pragma unroll
    for (int q = 0; q < kWords; q += kEach) {
      words x;
#pragma unroll
      for (int e = 0; e < kEach; ++e) x[e] = w[q + e];
      __builtin_nontemporal_store(x, reinterpret_cast<words *>(p) + q / kEach);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < V; ++e) {
    if (i + e >= n) continue;
    if constexpr (sizeof(T) == 4) p[e] = __uint_as_float(w[e]);
    else p[e] = (bf16_t)(w[e / 2] >> (16 * (e & 1)));
  }
}
template <bool TAIL, typename T, int V>
__device__ __forceinline__ void store_row(void *base, int64_t i, int64_t n, const float (&f)[V]) {
  uint32_t w[V * sizeof(T) / 4];
#pragma unroll
  for (int e = 0; e < V; e += (sizeof(T) == 4 ? 1 : 2)) {
    if constexpr (sizeof(T) == 4) w[e] = __float_as_uint(f[e]);
    else w[e / 2] = pack_bf16x2(f[e], f[e + 1]);
  }
  store_words<TAIL, T, V>(base, i, n, w);
}

template <bool TAIL>
__device__ __forceinline__ u32x2_t load8(const void *base, int64_t i, int64_t n) {
  const uint8_t *p = (const uint8_t *)base + i;
  if (!TAIL || i + 8 <= n) return __builtin_nontemporal_load(reinterpret_cast<const u32x2_t *>(p));
  u32x2_t w = {0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (i + e < n) w[e / 4] |= (uint32_t)p[e] << (8 * (e & 3));
  return w;
}
template <bool TAIL>
__device__ __forceinline__ void store8(void *base, int64_t i, int64_t n, u32x2_t w) {
  uint8_t *p = (uint8_t *)base + i;
  if (!TAIL || i + 8 <= n) {
    __builtin_nontemporal_store(w, reinterpret_cast<u32x2_t *>(p));
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (i + e < n) p[e] = (uint8_t)(w[e / 4] >> (8 * (e & 3)));
}

// P, G: types of parameter and gradient.  A thread takes V neighbouring
// elements, a block 256 V of them; 16 lanes share the scale of 128 (i >> 7).
template <typename P, typename G, bool MASTER, bool EIGHT, bool TAIL>
__device__ __forceinline__ void adamw_block(const AdamArgs<4 + (MASTER ? 1 : 0) + (EIGHT ? 2 : 0)> &a,
                                            int lo, int64_t i, int64_t n) {
#pragma clang fp contract(off)
  constexpr int V = EIGHT ? 8 : 4;
  constexpr bool RANDOM_P = sizeof(P) == 2 && !MASTER;
  void *const t_p = a.ptr[kP][lo], *const t_m = a.ptr[kM][lo], *const t_v = a.ptr[kV][lo];
  float *const t_master = MASTER ? (float *)a.ptr[MASTER ? kMore : 0][lo] : nullptr;
  uint8_t *const m_scale = EIGHT ? (uint8_t *)a.ptr[EIGHT ? kMore + MASTER : 0][lo] : nullptr;
  uint8_t *const v_scale = EIGHT ? (uint8_t *)a.ptr[EIGHT ? kMore + MASTER + 1 : 0][lo] : nullptr;

  float g[V], p[V], m[V], v[V];
  load_row<TAIL, G>(a.ptr[kG][lo], i, n, g);
  if constexpr (MASTER) load_row<TAIL, float>(t_master, i, n, p);
  else load_row<TAIL, P>(t_p, i, n, p);
  if constexpr (EIGHT) {
    const u32x2_t mq = load8<TAIL>(t_m, i, n), vq = load8<TAIL>(t_v, i, n);
    const int64_t b = i >> 7;
    const float ms = !TAIL || i < n ? __uint_as_float((uint32_t)m_scale[b] << 23) : 0.0f;
    const float vs = !TAIL || i < n ? __uint_as_float((uint32_t)v_scale[b] << 23) : 0.0f;
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
    load_row<TAIL, float>(t_m, i, n, m);
    load_row<TAIL, float>(t_v, i, n, v);
  }

  const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
  float decay = a.decay[lo], step_size = a.step_size, rbc2 = a.inv_sqrt_bc2;
  uint32_t step = a.step;
  if (a.lr) {   // a captured step: the learning rate and the step count are the device's
    const int64_t s = *a.step_dev;
    step = (uint32_t)s;
    const float lr = *a.lr;
    decay = (float)(1.0 - (double)lr * (double)decay);
    step_size = lr / -expm1f((float)s * a.ln_b1);
    rbc2 = 1.0f / sqrtf(-expm1f((float)s * a.ln_b2));
  }
  // The root instruction takes what is below 2^-126 for zero, and eps may be
  // far below the root of that: there it is the root of v 2^64.
  auto lifted_root = [&](int e) {
    const bool low = v[e] < 0x1p-126f;
    return __builtin_amdgcn_sqrtf(low ? v[e] * 0x1p64f : v[e]) * (low ? 0x1p-32f : 1.0f);
  };
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float ge = g[e] * gs;
    m[e] = m[e] * a.b1 + ge * a.a1;
    v[e] = v[e] * a.b2 + ge * a.a2 * ge;
    // 1-ulp root and reciprocal: off by 2^-22 of the update, below the
    // rounding of p wherever the update is below p/4.  (In this loop: from a
    // function of its own the loads come out in another order, and 796M
    // elements take 3.85 ms for 3.78.)
    const float den = fmaf(EIGHT ? __builtin_amdgcn_sqrtf(v[e]) : lifted_root(e), rbc2, a.eps);
    p[e] = fmaf(-step_size, m[e] * __builtin_amdgcn_rcpf(den), p[e] * decay);
  }
  if constexpr (EIGHT) {
    // Here the choice for each element would cost every step (604M weights
    // 1165 -> 1224 us); where a v is that low and not zero, p is read again.
    uint32_t least = ~0u;
#pragma unroll
    for (int e = 0; e < V; ++e) least = min(least, __float_as_uint(v[e]) - 1u);
    if (__any(least < 0x7fffffu)) {
      if constexpr (MASTER) load_row<TAIL, float>(t_master, i, n, p);
      else load_row<TAIL, P>(t_p, i, n, p);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float den = fmaf(lifted_root(e), rbc2, a.eps);
        p[e] = fmaf(-step_size, m[e] * __builtin_amdgcn_rcpf(den), p[e] * decay);
      }
    }
  }

  // The conversions below round a magnitude up where the bits that it loses
  // and the top bits of the random operand carry (measured: as bit arithmetic
  // on the fp32 pattern does, denormal results included; infinities and NaN stay).
  uint32_t r[V];
  if constexpr (RANDOM_P || EIGHT) {
    const uint32_t key =
        mix(mix(mix(mix(a.seed_lo) ^ a.seed_hi) ^ step) ^ (a.base + lo)) ^ (uint32_t)(i >> 32) ^ (uint32_t)i;
#pragma unroll
    for (int e = 0; e < V; ++e) r[e] = mix(key ^ e);   // i is a multiple of V
  }
  if constexpr (EIGHT) {
    uint32_t m_max = 0, v_max = 0;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      m_max = max(m_max, magnitude(m[e]));
      v_max = max(v_max, magnitude(v[e]));
    }
    m_max = max16(m_max), v_max = max16(v_max);
    const bool bad = __any(max(m_max, v_max) >= kInf);   // somewhere in the wave
    if (bad) {   // only what is finite scales a block
      m_max = v_max = 0;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        uint32_t mm = magnitude(m[e]), vm = magnitude(v[e]);
        asm volatile("" : "+v"(mm), "+v"(vm));   // keeps the branch: no selects for every block
        m_max = max(m_max, mm < kInf ? mm : 0u);
        v_max = max(v_max, vm < kInf ? vm : 0u);
      }
      m_max = max16(m_max), v_max = max16(v_max);
    }
    const int ms = block_exponent<8>(m_max), vs = block_exponent<15>(v_max);
    const float mi = __uint_as_float((uint32_t)(127 - ms) << 23), vi = __uint_as_float((uint32_t)(127 - vs) << 23);
    uint32_t mq[2] = {0u, 0u}, vq[2] = {0u, 0u};
    auto code = [&](int e, auto sel) {
      const float am = m[e] * mi;
      // a second moment that is not zero never becomes it, since its root
      // divides: at least the smallest code, 2^-16
      const float av = v[e] > 0.0f ? fmaxf(v[e] * vi, 0x1p-16f) : v[e] * vi;
      mq[e / 4] = (uint32_t)__builtin_amdgcn_cvt_sr_fp8_f32(am, r[e] & 0xffff0000u, (int)mq[e / 4], decltype(sel)::value);
      vq[e / 4] = (uint32_t)__builtin_amdgcn_cvt_sr_bf8_f32(av, (r[e] * 0x30e9132du) & 0xffff0000u, (int)vq[e / 4],
                                                            decltype(sel)::value);
    };
#pragma unroll
    for (int e = 0; e < V; e += 4) {
      code(e, std::integral_constant<int, 0>());
      code(e + 1, std::integral_constant<int, 1>());
      code(e + 2, std::integral_constant<int, 2>());
      code(e + 3, std::integral_constant<int, 3>());
    }
    if (bad) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const uint32_t at = 0xffu << (8 * (e & 3)), nan = 0x7fu << (8 * (e & 3));
        uint32_t mm = magnitude(m[e]), vm = magnitude(v[e]);
        asm volatile("" : "+v"(mm), "+v"(vm));
        if (mm >= kInf) mq[e / 4] = (mq[e / 4] & ~at) | nan;
        if (vm >= kInf) vq[e / 4] = (vq[e / 4] & ~at) | nan;
      }
    }
    store8<TAIL>(t_m, i, n, u32x2_t{mq[0], mq[1]});
    store8<TAIL>(t_v, i, n, u32x2_t{vq[0], vq[1]});
    if ((threadIdx.x & 15) == 0 && (!TAIL || i < n)) {
      m_scale[i >> 7] = (uint8_t)(ms + 127);
      v_scale[i >> 7] = (uint8_t)(vs + 127);
    }
  } else {
    store_row<TAIL, float>(t_m, i, n, m);
    store_row<TAIL, float>(t_v, i, n, v);
  }
  if constexpr (MASTER) store_row<TAIL, float>(t_master, i, n, p);
  if constexpr (RANDOM_P) {
    uint32_t w[V / 2];
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      bf16x2v_t q = {(__bf16)0.0f, (__bf16)0.0f};
      q = __builtin_amdgcn_cvt_sr_bf16_f32(q, p[e], r[e] << 16, false);
      q = __builtin_amdgcn_cvt_sr_bf16_f32(q, p[e + 1], r[e + 1] << 16, true);
      w[e / 2] = __builtin_bit_cast(uint32_t, q);
    }
    store_words<TAIL, P, V>(t_p, i, n, w);
  } else {
    store_row<TAIL, P>(t_p, i, n, p);
  }
}

// Five waves a SIMD with 32-bit states: more of them have more lines under way
// than HBM serves in order (30 bytes an element: 6.3 TB/s with 5, 6.1 with 8 or
// 4); 8-bit states need the sixth for their arithmetic.
template <typename P, typename G, bool MASTER, bool EIGHT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(EIGHT ? 6 : 5, EIGHT ? 6 : 5))) void k_adamw(
    const AdamArgs<4 + (MASTER ? 1 : 0) + (EIGHT ? 2 : 0)> a) {
  constexpr int V = EIGHT ? 8 : 4;
  int lo = 0, hi = a.count - 1;
  while (lo < hi) {   // the tensor of this block: the last that begins here or before, so none without elements
    const int mid = (lo + hi + 1) >> 1;
    if (a.first[mid] <= blockIdx.x) lo = mid;
    else hi = mid - 1;
  }
  const int64_t n = a.n[lo], at = (int64_t)(blockIdx.x - a.first[lo]) * 256 * V;
  const int64_t i = at + threadIdx.x * V;
  // Whole blocks without the code for ends between their accesses: 8-bit
  // states' instructions are then half as many to fetch when a launch begins
  // (120 tensors of 47M elements 106 -> 95 us).  With 32-bit states the
  // branches between the accesses spread them out, and long tensors take 3.80
  // ms with them, 3.98 without (796M elements).
  if (EIGHT && at + 256 * V <= n) adamw_block<P, G, MASTER, EIGHT, false>(a, lo, i, n);
  else adamw_block<P, G, MASTER, EIGHT, true>(a, lo, i, n);
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

struct AdamCall {
  const moe_adamw_tensor *tensors;
  int n;
  double lr, beta1, beta2, eps;
  int64_t step;
  uint64_t seed;
  const float *grad_scale, *lr_dev;
  const int64_t *step_dev;
};

template <typename P, typename G, bool MASTER, bool EIGHT>
int run(const char *fn, const AdamCall &c, hipStream_t s) {
  AdamArgs<4 + (MASTER ? 1 : 0) + (EIGHT ? 2 : 0)> a;
  static_assert(sizeof(a) <= kArgBytes, "a kernel's arguments");
  const int64_t per_block = 256 * (EIGHT ? 8 : 4);
  a.b1 = (float)c.beta1, a.a1 = (float)(1.0 - c.beta1);
  a.b2 = (float)c.beta2, a.a2 = (float)(1.0 - c.beta2);
  a.eps = (float)c.eps;
  a.ln_b1 = (float)std::log(c.beta1), a.ln_b2 = (float)std::log(c.beta2);   // -inf for 0
  a.step_size = c.lr_dev ? 0.0f : (float)(c.lr / (1.0 - std::pow(c.beta1, (double)c.step)));
  a.inv_sqrt_bc2 = c.lr_dev ? 0.0f : (float)(1.0 / std::sqrt(1.0 - std::pow(c.beta2, (double)c.step)));
  a.seed_lo = (uint32_t)c.seed, a.seed_hi = (uint32_t)(c.seed >> 32), a.step = (uint32_t)c.step;
  a.grad_scale = c.grad_scale, a.lr = c.lr_dev, a.step_dev = c.step_dev;
  for (int i = 0; i < c.n;) {
    int64_t blocks = 0;
    a.count = 0;
    a.base = (uint32_t)i;
    for (; i < c.n && a.count < a.kMost; ++i) {
      const moe_adamw_tensor &t = c.tensors[i];
      const int64_t mine = (t.numel + per_block - 1) / per_block;
      if (blocks + mine > kMaxBlocks) break;
      const int k = a.count++;
      a.ptr[kP][k] = t.param, a.ptr[kG][k] = const_cast<void *>(t.grad);
      a.ptr[kM][k] = t.m, a.ptr[kV][k] = t.v;
      if constexpr (MASTER) a.ptr[kMore][k] = t.master;
      if constexpr (EIGHT) a.ptr[kMore + MASTER][k] = t.m_scale, a.ptr[kMore + MASTER + 1][k] = t.v_scale;
      a.n[k] = t.numel;
      a.decay[k] = (float)(c.lr_dev ? t.weight_decay : 1.0 - c.lr * t.weight_decay);
      a.first[k] = (uint32_t)blocks;
      blocks += mine;
    }
    if (!blocks) continue;   // tensors without elements
    MOE_LAUNCH("adamw", s, k_adamw<P, G, MASTER, EIGHT><<<(unsigned)blocks, 256, 0, s>>>(a));
    const int e = check_launch(fn);
    if (e != MOE_OK) return e;
  }
  return MOE_OK;
}

template <typename P, typename G, bool MASTER>
int run(const char *fn, const AdamCall &c, bool eight, hipStream_t s) {
  return eight ? run<P, G, MASTER, true>(fn, c, s) : run<P, G, MASTER, false>(fn, c, s);
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
  const bool eight = state_bits == 8;
  bool master = false, first = true;   // of the first tensor with elements
  const int64_t per_block = 256 * (eight ? 8 : 4);
  for (int i = 0; i < n; ++i) {
    const moe_adamw_tensor &t = tensors[i];
    MOE_REQUIRE(t.numel >= 0 && t.numel <= per_block * kMaxBlocks, MOE_ERR_UNSUPPORTED,
                "%s: tensor %d has %lld elements", fn, i, (long long)t.numel);
    MOE_REQUIRE(std::isfinite(t.weight_decay), MOE_ERR_INVALID_ARG, "%s: tensor %d: weight_decay %g", fn,
                i, t.weight_decay);
    if (t.numel == 0) continue;
    if (first) master = t.master, first = false;
    MOE_REQUIRE((t.master != nullptr) == master && !(master && param_dtype == MOE_F32),
                MOE_ERR_INVALID_ARG, "%s: tensor %d: all bf16 parameters have a 32-bit copy, or none",
                fn, i);
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

  const AdamCall c = {tensors, n, lr, beta1, beta2, eps, step, seed, grad_scale, lr_dev, step_dev};
  hipStream_t s = (hipStream_t)stream;
  if (param_dtype == MOE_F32) return run<float, float, false>(fn, c, eight, s);
  if (master && grad_dtype == MOE_F32) return run<bf16_t, float, true>(fn, c, eight, s);
  if (master) return run<bf16_t, bf16_t, true>(fn, c, eight, s);
  if (grad_dtype == MOE_F32) return run<bf16_t, float, false>(fn, c, eight, s);
  return run<bf16_t, bf16_t, false>(fn, c, eight, s);
}
