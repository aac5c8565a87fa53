// Routing by scores over all experts (softmax or sigmoid), with a selection
// bias, expert groups, top-k and optionally renormalised weights, and the
// adjoint of its weights.
#include "moe_internal.h"

namespace moe {
namespace {

// Value descending, equal values by lower id, NaN below every number.
template <typename F>
__device__ __forceinline__ bool ranks_before(F va, int ia, F vb, int ib) {
  const bool na = va != va, nb = vb != vb;
  if (na || nb) return nb && (!na || ia < ib);
  return va > vb || (va == vb && ia < ib);
}

__device__ __forceinline__ double score64(double x, bool sigmoid, double shift, double inv_sum) {
  return sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - shift) * inv_sum;
}

constexpr float kLowest = -INFINITY;
constexpr int64_t kFewTokens = 2048;   // up to here a token takes twice the lanes: latency counts

// A float as an integer of the same order (and back): integer maxima need no
// care for NaNs.  -0 has to be +0 before.
__device__ __forceinline__ int to_key(float v) {
  const int i = __float_as_int(v);
  return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float from_key(int k) {
  return __int_as_float(k ^ ((k >> 31) & 0x7fffffff));
}
constexpr int kLowestKey = (int)0x807fffff;   // of -inf

// Exchange with lane ^ 1, ^ 2, the other quad of 8, the other 8 of 16: after
// the steps below M, every lane of an M-lane block holds the same value, so a
// mirror serves as the exchange with lane ^ M.
template <int M>
__device__ __forceinline__ int dpp(int v) {
  constexpr int ctrl = M == 1 ? 0xB1 : M == 2 ? 0x4E : M == 4 ? 0x141 : 0x140;
  return __builtin_amdgcn_update_dpp(0, v, ctrl, 0xf, 0xf, false);
}
// (a, b) of the two blocks of 16 (32) lanes that a pair of blocks holds
template <int M>
__device__ __forceinline__ void blocks(int v, int &a, int &b) {
  if constexpr (M == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    a = (int)r[0];
    b = (int)r[1];
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    a = (int)r[0];
    b = (int)r[1];
  }
}
// One step of a reduction over blocks of 2 M lanes.
template <int M, typename T, typename Op>
__device__ __forceinline__ T step(T v, Op op) {
  int a = __builtin_bit_cast(int, v), b;
  if constexpr (M <= 8) b = dpp<M>(a);
  else blocks<M>(a, a, b);
  return op(__builtin_bit_cast(T, a), __builtin_bit_cast(T, b));
}
template <int G, typename T, typename Op>
__device__ __forceinline__ T reduce(T v, Op op) {
  if constexpr (G > 1) v = step<1>(v, op);
  if constexpr (G > 2) v = step<2>(v, op);
  if constexpr (G > 4) v = step<4>(v, op);
  if constexpr (G > 8) v = step<8>(v, op);
  if constexpr (G > 16) v = step<16>(v, op);
  if constexpr (G > 32) v = step<32>(v, op);
  return v;
}
struct Max {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
  __device__ __forceinline__ int operator()(int a, int b) const { return max(a, b); }
};
struct Min {
  __device__ __forceinline__ int operator()(int a, int b) const { return min(a, b); }
};
struct Add {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
// (largest, second largest) keys over blocks of n lanes, n a power of two
template <int M>
__device__ __forceinline__ void top2_step(int &a, int &b) {
  int oa, ob;
  if constexpr (M <= 8) {
    oa = dpp<M>(a);
    ob = dpp<M>(b);
  } else {
    blocks<M>(a, a, oa);
    blocks<M>(b, b, ob);
  }
  b = max(min(a, oa), max(b, ob));
  a = max(a, oa);
}
__device__ __forceinline__ void top2(int &a, int &b, int n) {
  if (n > 1) top2_step<1>(a, b);
  if (n > 2) top2_step<2>(a, b);
  if (n > 4) top2_step<4>(a, b);
  if (n > 8) top2_step<8>(a, b);
  if (n > 16) top2_step<16>(a, b);
  if (n > 32) top2_step<32>(a, b);
}

struct RouteArgs {
  const float *logits, *bias;
  int64_t T;
  int E, k;
  bool sigmoid, renorm, pairs;   // pairs: a group's value is the sum of its two best
  int groups, keep, size;        // groups that compete (1: no restriction), kept, experts each
  int span, span_log;            // lanes per group, a power of two
  float scale;
  int32_t *idx;
  float *w;
};

// The lane's V values of a group's, `none` where it has no expert.
typedef float f32x4u_t __attribute__((ext_vector_type(4), aligned(4)));
template <int V>
__device__ __forceinline__ void load(const RouteArgs &g, const float *p, bool in, int li, float none,
                                     float (&c)[V]) {
  if (V % 4 == 0 && g.size % 4 == 0) {   // four or none of four
#pragma unroll
    for (int v = 0; v < V; v += 4) {
      f32x4u_t r = {none, none, none, none};
      if (in && li * V + v < g.size) r = *reinterpret_cast<const f32x4u_t *>(p + li * V + v);
#pragma unroll
      for (int i = 0; i < 4; ++i) c[(v + i) % V] = r[i];
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = in && li * V + v < g.size ? p[li * V + v] : none;
  }
}

// The lane's choices in fp64 (0 where it has no expert), and as a mask where
// it has one; ranked: what the groups compare.
template <int G, int V>
__device__ __forceinline__ unsigned choices64(const RouteArgs &g, const float *x, int s, float shift,
                                              double (&c)[V], double &first, double &second) {
  const int li = s % g.span, gi = s / g.span, base = gi * g.size;
  double inv = 0.0;
  if (!g.sigmoid) {
    double sum = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int o = li * V + v;
      if (gi < g.groups && o < g.size) sum += exp((double)x[base + o] - (double)shift);
    }
    for (int m = 1; m < G; m <<= 1) sum += __shfl_xor(sum, m, 64);
    inv = sum == 0.0 ? 0.0 : 1.0 / sum;
  }
  unsigned open = 0;
  first = second = kLowest;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int o = li * V + v;
    c[v] = 0.0;
    if (gi >= g.groups || o >= g.size) continue;
    const double xe = x[base + o];
    const double sc = score64(xe, g.sigmoid, shift, inv);
    c[v] = g.bias ? sc + (double)g.bias[base + o] : xe;
    open |= 1u << v;
    const double r = !g.bias && g.pairs ? sc : c[v];   // a NaN is passed over
    if (r > first) {
      second = first;
      first = r;
    } else if (r > second) {
      second = r;
    }
  }
  return open;
}
// Whether the lane's group stays, by its values in fp64.
template <int G>
__device__ __forceinline__ bool kept64(const RouteArgs &g, int s, double a, double b) {
  for (int m = 1; m < g.span; m <<= 1) {
    const double oa = __shfl_xor(a, m, 64), ob = __shfl_xor(b, m, 64);
    b = fmax(fmin(a, oa), fmax(b, ob));
    a = fmax(a, oa);
  }
  double val = g.pairs ? a + b : a;
  if (val != val) val = kLowest;
  int rank = 0;
  for (int i = 0; i < g.groups; ++i) {
    const double o = __shfl(val, i * g.span, G);
    rank += ranks_before(o, i, val, s / g.span) ? 1 : 0;
  }
  return rank < g.keep;
}

// The whole selection in fp64: lane s of a token's G lanes returns the expert
// at place s.
template <int G, int V>
__device__ __forceinline__ int select64(const RouteArgs &g, const float *x, int s, float shift) {
  const int li = s % g.span, gi = s / g.span, base = gi * g.size;
  double c[V], a, b;
  unsigned open = choices64<G, V>(g, x, s, shift, c, a, b);
  if (g.keep < g.groups && !kept64<G>(g, s, a, b)) open = 0;
  int mine = 0;
  for (int j = 0; j < g.k; ++j) {
    double bv = 0.0;
    int bi = 0x7fffffff;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = base + li * V + v;
      if (((open >> v) & 1) && (bi == 0x7fffffff || ranks_before(c[v], e, bv, bi))) {
        bv = c[v];
        bi = e;
      }
    }
    const int own = bi;
    for (int m = 1; m < G; m <<= 1) {
      const double ov = __shfl_xor(bv, m, 64);
      const int oi = __shfl_xor(bi, m, 64);
      if (oi != 0x7fffffff && (bi == 0x7fffffff || ranks_before(ov, oi, bv, bi))) {
        bv = ov;
        bi = oi;
      }
    }
    if (own == bi && bi != 0x7fffffff) open &= ~(1u << (bi - base - li * V));
    if (s == j) mine = bi;
  }
  return mine;
}

// G lanes per token, V experts per lane: lane s holds experts size * (s / span)
// + V (s % span) + v, so that a group's experts lie in span adjacent lanes and
// are read 16 bytes at a time.
//
// Quick form, in fp32: the group values, then k rounds of a maximum over the
// lane's V values and the G lanes (one instruction per step), the winner
// taken out where it is found.  Logits are ordered exactly as they are.
// Choices with a bias and sums of scores carry the errors of fp32, so a
// decision between two of them counts only if they differ by more than those
// errors can explain: for sigmoid scores 2^-21 + 2^-23 |c| each (exponential,
// sum, reciprocal: 6 units of 2^-24; the bias's sum 2^-24 |c|), for softmax
// scores 2^-24 (2 + 40 s_max) + 2^-23 |c| (the argument's error is in
// proportion to it, |d| exp(-|d|) < 0.4; sum and reciprocal 32 units of the
// score); a sum of two choices has the errors of both.  Where the last group
// that stays and the first that goes are nearer than that, the wave takes the
// groups' values in fp64; where neighbours in the order are, the first k + 1
// are ranked again in fp64; where that cannot settle it (the k + 2nd is close
// too, a NaN, scores of -inf), the wave selects in fp64 from the start.
//
// The vector units bound it, not memory: 32768 tokens x 256 experts in 8
// groups, sigmoid, bias, top-8 take 22 us (31 at V = 4, 24 at V = 16; the
// logits' 34 MB alone 7), about 750 instructions per two tokens, of which a
// round is 37.
template <int G, int V>
__global__ __launch_bounds__(256) void k_route_scored(RouteArgs g) {
  __shared__ int2 s_place[256 / G][G];   // the selected experts and their keys, and the next
  const int s = threadIdx.x % G;
  const int64_t t = ((int64_t)blockIdx.x * 256 + threadIdx.x) / G;
  const bool live = t < g.T;
  const int gi = s >> g.span_log, li = s - (gi << g.span_log), base = gi * g.size;
  const float *x = g.logits + (live ? t : 0) * g.E;
  float c[V];
  load<V>(g, x + base, gi < g.groups, li, kLowest, c);
  bool unsure = false;
  float shift = 0.0f, sum = 0.0f, top = 1.0f;
  const bool scored = g.bias || (g.pairs && g.keep < g.groups);   // scores are compared
  if (!g.sigmoid && (scored || !g.renorm)) {
    float m = c[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = fmaxf(m, c[v]);
    m = reduce<G>(m, Max());
    shift = m == kLowest ? 0.0f : m;
#pragma unroll
    for (int v = 0; v < V; ++v) sum += __expf(c[v] - shift);
    sum = reduce<G>(sum, Add());
    top = sum == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(sum);   // the largest score
  }
  auto sigmoid = [](float v) { return __builtin_amdgcn_rcpf(1.0f + __expf(-v)); };
  // what two compared values may be off together
  const float tol = g.sigmoid ? 0x1p-20f : 0x1p-23f * (2.0f + 40.0f * top);
  auto slack = [&](float v) { return tol + 0x1p-22f * fabsf(v); };
  float r[V];
  if (g.bias) {   // (no expert: 0 - infinity)
    load<V>(g, g.bias + base, gi < g.groups, li, kLowest, r);
    if (g.sigmoid) {
#pragma unroll
      for (int v = 0; v < V; ++v) r[v] += sigmoid(c[v]);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) r[v] += __expf(c[v] - shift) * top;
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) r[v] = c[v];
  }
  int key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    unsure |= r[v] != r[v];
    key[v] = to_key(r[v] + 0.0f);
  }
  if (g.keep < g.groups) {
    int a = kLowestKey, b = kLowestKey;
    auto take = [&](int k) {
      b = max(b, min(a, k));
      a = max(a, k);
    };
    if (g.pairs && !g.bias) {   // the scores' sum; a score of no expert would be 0
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float sc = g.sigmoid ? sigmoid(c[v]) : __expf(c[v] - shift) * top;
        unsure |= sc != sc;   // a logit of +inf: no logit is a NaN, but all scores are
        take(gi < g.groups && li * V + v < g.size ? to_key(sc) : kLowestKey);
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) take(key[v]);
    }
    top2(a, b, g.span);
    const float val = g.pairs ? from_key(a) + from_key(b) : from_key(a);
    // How near two groups' values are that fp32 cannot tell apart.  The errors of
    // a sum are those of its addends: where they differ in sign (a bias may be
    // of any size) they are larger than the sum by far, and any group's count.
    float near = 2.0f * slack(val);
    if (g.pairs && g.bias && __any(gi < g.groups && b < 0)) {
      const float own = slack(from_key(a)) + slack(from_key(b));
      near = reduce<G>(gi < g.groups ? own : 0.0f, Max());
    }
    int rank = 0;
    bool close = false;   // a group behind this one, nearer than the errors
    for (int i = 0; i < g.groups; ++i) {
      const float o = __shfl(val, i * g.span, G);
      const bool before = o > val || (o == val && i < gi);
      rank += before ? 1 : 0;
      close |= scored && !before && i != gi && !(val - o > near);   // (sums of one infinity too)
    }
    bool kept = rank < g.keep;
    if (__any(live && gi < g.groups && rank == g.keep - 1 && close)) {
      double c64[V], a64, b64;
      choices64<G, V>(g, x, s, shift, c64, a64, b64);
      kept = kept64<G>(g, s, a64, b64);
    }
    if (!kept) {
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = kLowestKey;
    }
  }
  int2 *const place = s_place[threadIdx.x / G];
  auto best_key = [&](int &lane_best) {
    lane_best = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) lane_best = max(lane_best, key[v]);
    return reduce<G>(lane_best, Max());
  };
  const int rounds = g.bias ? g.k + 1 : g.k;   // with a bias, the first that is not selected too
  for (int j = 0; j < rounds; ++j) {
    int m;
    const int best = best_key(m);
    bool has = m == best;
    if (__popcll(__ballot(has)) != 64 / G) {   // equal values in several lanes: the lowest id
      int at = 0;
#pragma unroll
      for (int v = V - 1; v >= 0; --v) at = key[v] == best ? v : at;
      const int e = base + li * V + at;
      const int low = reduce<G>(has ? e : 0x7fffffff, Min());
      has = has && e == low;
    }
    // the lane that has it takes out the first of its values that is it
    int at = 0;
    bool rest = has;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const bool hit = rest && key[v] == best;
      at = hit ? v : at;
      key[v] = hit ? kLowestKey : key[v];
      rest = rest && !hit;
    }
    if (has) place[j] = int2{base + li * V + at, best};
  }
  // (a token's lanes are lanes of one wave, whose LDS operations keep their order)
  asm volatile("" ::: "memory");
  int mine = -1, got = kLowestKey;
  if (s < rounds) {
    mine = place[s].x;
    got = place[s].y;
    if (got == kLowestKey) mine = -1;
  }
  unsure |= s < g.k && mine < 0;
  bool close = false;   // to the one behind
  if (g.bias && s < g.k) close = from_key(got) - from_key(place[s + 1].y) <= slack(from_key(got));
  if (__any(close && live)) {
    // Neighbours in the order are too close: lane s takes the choice of the
    // s-th in fp64, and they are ranked again.  Enough unless the next one is
    // close to them too.
    int m;
    const float next = from_key(best_key(m)), last = from_key(place[g.k].y);
    unsure |= last - next <= slack(last);
    double inv = 0.0;
    if (!g.sigmoid) {
      double z = 0.0;
#pragma unroll
      for (int v = 0; v < V; ++v) z += exp((double)c[v] - (double)shift);
      for (int i = 1; i < G; i <<= 1) z += __shfl_xor(z, i, 64);
      inv = z == 0.0 ? 0.0 : 1.0 / z;
    }
    double mv = kLowest;
    if (mine >= 0) mv = score64(x[mine], g.sigmoid, shift, inv) + (double)g.bias[mine];
    int rank = 0;
    for (int j = 0; j < rounds; ++j) {
      const double ov = __shfl(mv, j, G);
      const int oi = __shfl(mine, j, G);
      rank += oi >= 0 && ranks_before(ov, oi, mv, mine) ? 1 : 0;
    }
    if (mine >= 0) place[rank].x = mine;
    asm volatile("" ::: "memory");
    if (s < g.k && mine >= 0) mine = place[s].x;
  }
  if (__any(unsure && live)) mine = select64<G, V>(g, x, s, shift);

  // ---- weights of the k selected
  const bool sel = s < g.k;
  const float v = sel && live ? x[mine] : kLowest;
  float w;
  if (g.renorm) {
    // s_j / sum s: the common factor of the selected scores is taken out
    // first, so that no score is too small to be a number
    const float low = g.sigmoid ? fminf(v, 0.0f) : v;
    const float m = reduce<G>(low, Max());
    float r = 0.0f;
    if (sel && m != kLowest) r = g.sigmoid ? expf(low - m) / (1.0f + expf(-fabsf(v))) : expf(v - m);
    if (sel && v != v) r = v;
    const float total = reduce<G>(r, Add());
    w = total == 0.0f ? 0.0f : r / total;
  } else if (g.sigmoid) {
    w = 1.0f / (1.0f + expf(-v));
  } else {
    w = sum == 0.0f ? 0.0f : expf(v - shift) / sum;
  }
  if (sel && live) {
    g.idx[t * g.k + s] = mine;
    g.w[t * g.k + s] = w * g.scale;
  }
}

// ------------------------------------------------------------------ adjoint
//
// G lanes per token; lane s < k holds selection s.  d_logits is a row that is
// dense only for softmax scores without renormalisation: it is formed in LDS
// (zeros or -s_e m), the k selected terms are added, and it leaves with U-wide
// stores (U = 4 where rows are 16-byte aligned); NV units per lane.
template <int G, int U, int NV>
__global__ __launch_bounds__(256) void k_route_scored_bwd(
    const float *__restrict__ logits, const int32_t *__restrict__ topk_idx,
    const float *__restrict__ topk_w, const float *__restrict__ d_row_scale,
    const int32_t *__restrict__ slot_to_row, int64_t T, int E, int k, bool sigmoid, bool renorm,
    float scale, float *__restrict__ d_topk_w, float *__restrict__ d_logits) {
  typedef float unit_t __attribute__((ext_vector_type(U)));
  __shared__ unit_t s_row[256 / G][G * NV];
  const int s = threadIdx.x % G;
  const int64_t t = ((int64_t)blockIdx.x * 256 + threadIdx.x) / G;
  const bool live = t < T;
  const float *x = logits + (live ? t : 0) * E;
  const bool sel = live && s < k;
  const bool dense = !sigmoid && !renorm;
  int idx = -1;
  float w = 0.0f, g = 0.0f;
  if (sel) {
    const int64_t slot = t * k + s;
    idx = topk_idx[slot];
    w = topk_w[slot];
    const int64_t row = slot_to_row ? slot_to_row[slot] : slot;
    g = row >= 0 ? d_row_scale[row] : 0.0f;
    if (d_topk_w) d_topk_w[slot] = g;
  }
  const bool in = sel && idx >= 0 && idx < E;
  float rest = 1.0f;
  if (sigmoid && in) rest = 1.0f / (1.0f + expf(x[idx]));   // 1 - s
  const float mean = reduce<G>(w * g, Add()) / scale;
  const float d = w * rest * (renorm ? g - mean : g);
  unit_t u[NV];
  const int n = E / U;   // units of a row
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int i = 0; i < U; ++i) u[v][i] = 0.0f;
  if (dense) {
    float m = kLowest;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int at = s + G * v;
      if (at < n) u[v] = *reinterpret_cast<const unit_t *>(x + at * U);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (at >= n) u[v][i] = kLowest;
        m = fmaxf(m, u[v][i]);
      }
    }
    m = reduce<G>(m, Max());
    const float shift = m == kLowest ? 0.0f : m;
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < U; ++i) {
        u[v][i] = expf(u[v][i] - shift);
        sum += u[v][i];
      }
    sum = reduce<G>(sum, Add());
    const float f = sum == 0.0f ? 0.0f : -scale * mean / sum;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < U; ++i) u[v][i] *= f;
  }
  unit_t *row = s_row[threadIdx.x / G];
#pragma unroll
  for (int v = 0; v < NV; ++v) row[s + G * v] = u[v];
  // (a token's lanes are lanes of one wave, whose LDS operations keep their order)
  asm volatile("" ::: "memory");
  if (in) {   // a token's selections are distinct
    float *const p = reinterpret_cast<float *>(row) + idx;
    *p = *p + d;
  }
  asm volatile("" ::: "memory");
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int at = s + G * v;
    if (live && at < n) *reinterpret_cast<unit_t *>(d_logits + t * E + at * U) = row[at];
  }
}

int check_scored(const char *fn, int64_t T, int E, int k, int score, float scale) {
  MOE_REQUIRE(T >= 0, MOE_ERR_INVALID_ARG, "%s: T < 0", fn);
  MOE_REQUIRE(E >= 1 && E <= kMaxExperts, MOE_ERR_UNSUPPORTED, "%s: E=%d outside [1,%d]", fn, E,
              kMaxExperts);
  MOE_REQUIRE(k >= 1 && k <= E && k <= kMaxTopK, MOE_ERR_UNSUPPORTED, "%s: k=%d E=%d", fn, k, E);
  // (a launch has at most 2^32 threads, a token up to 64)
  MOE_REQUIRE(T < ((int64_t)1 << 26), MOE_ERR_UNSUPPORTED, "%s: T >= 2^26", fn);
  MOE_REQUIRE(score == MOE_SCORE_SOFTMAX || score == MOE_SCORE_SIGMOID, MOE_ERR_UNSUPPORTED,
              "%s: score %d", fn, score);
  MOE_REQUIRE(scale > 0.0f && scale <= 3.402823466e38f, MOE_ERR_INVALID_ARG,
              "%s: scale must be positive and finite", fn);
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_route_scored(const float *logits, const float *sel_bias, int64_t T, int E, int k,
                                int score, int n_group, int topk_group, int group_top, int renorm,
                                float scale, int32_t *topk_idx, float *topk_w, void *stream) {
  const char *fn = "moe_route_scored";
  clear_error();
  int rc = check_scored(fn, T, E, k, score, scale);
  if (rc) return rc;
  MOE_REQUIRE(n_group >= 1 && n_group <= 32 && E % n_group == 0, MOE_ERR_UNSUPPORTED,
              "%s: n_group=%d (1 to 32, a divisor of E=%d)", fn, n_group, E);
  MOE_REQUIRE(topk_group >= 1 && topk_group <= n_group, MOE_ERR_UNSUPPORTED,
              "%s: topk_group=%d of %d", fn, topk_group, n_group);
  MOE_REQUIRE(group_top == 1 || (group_top == 2 && E / n_group >= 2), MOE_ERR_UNSUPPORTED,
              "%s: group_top=%d with groups of %d", fn, group_top, E / n_group);
  MOE_REQUIRE(k <= topk_group * (E / n_group), MOE_ERR_UNSUPPORTED,
              "%s: k=%d exceeds the %d experts of %d groups", fn, k, topk_group * (E / n_group),
              topk_group);
  if (T == 0) return MOE_OK;
  MOE_REQUIRE(logits && topk_idx && topk_w, MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
  MOE_REQUIRE(aligned16(logits), MOE_ERR_INVALID_ARG, "%s: logits must be 16-byte aligned", fn);
  hipStream_t s = (hipStream_t)stream;
  RouteArgs g{};
  g.logits = logits;
  g.bias = sel_bias;
  g.T = T;
  g.E = E;
  g.k = k;
  g.sigmoid = score == MOE_SCORE_SIGMOID;
  g.renorm = renorm != 0;
  g.pairs = group_top == 2;
  g.groups = topk_group < n_group ? n_group : 1;
  g.keep = g.groups > 1 ? topk_group : 1;
  g.size = E / g.groups;
  g.scale = scale;
  g.idx = topk_idx;
  g.w = topk_w;
  // Lanes per token: enough for the k places and the groups, then as many as
  // bring the experts per lane to the wanted number.
  const int want = T <= kFewTokens ? 4 : 8;
  int span2 = 1;   // groups, rounded up to a power of two
  while (span2 < g.groups) span2 <<= 1;
  int G = 8, V = 1;
  while (G < k + (sel_bias ? 1 : 0) || G < span2) G <<= 1;
  while (G < 64 && (g.size + G / span2 - 1) / (G / span2) > want) G <<= 1;
  g.span = G / span2;
  while (1 << g.span_log < g.span) ++g.span_log;
  while (V * g.span < g.size) V <<= 1;
  const unsigned blocks = (unsigned)((T * G + 255) / 256);
#define ROUTE_CASE(GV, VV)                                                                        \
  case GV * 64 + VV:                                                                               \
    MOE_LAUNCH("route_scored", s, (k_route_scored<GV, VV><<<blocks, 256, 0, s>>>(g)));             \
    break
#define ROUTE_CASES(GV) \
  ROUTE_CASE(GV, 1); ROUTE_CASE(GV, 2); ROUTE_CASE(GV, 4); ROUTE_CASE(GV, 8)
  switch (G * 64 + V) {
    ROUTE_CASES(8);
    ROUTE_CASES(16);
    ROUTE_CASES(32);
    ROUTE_CASES(64);
    ROUTE_CASE(64, 16);
    ROUTE_CASE(64, 32);
    default:
      MOE_REQUIRE(false, MOE_ERR_UNSUPPORTED, "%s: E=%d n_group=%d", fn, E, n_group);
  }
#undef ROUTE_CASES
#undef ROUTE_CASE
  return check_launch(fn);
}

extern "C" int moe_route_scored_bwd(const float *logits, const int32_t *topk_idx,
                                    const float *topk_w, const float *d_row_scale,
                                    const int32_t *slot_to_row, int64_t T, int E, int k, int score,
                                    int renorm, float scale, float *d_topk_w, float *d_logits,
                                    void *stream) {
  const char *fn = "moe_route_scored_bwd";
  clear_error();
  int rc = check_scored(fn, T, E, k, score, scale);
  if (rc) return rc;
  if (T == 0) return MOE_OK;
  MOE_REQUIRE(logits && topk_idx && topk_w && d_row_scale && d_logits, MOE_ERR_INVALID_ARG,
              "%s: null pointer", fn);
  MOE_REQUIRE(aligned16(logits) && aligned16(d_logits), MOE_ERR_INVALID_ARG,
              "%s: logits and d_logits must be 16-byte aligned", fn);
  hipStream_t s = (hipStream_t)stream;
  // lanes per token: a unit of the row or a selection each, at most 64
  const int U = E % 4 == 0 ? 4 : 1, n = E / U;
  int G = 8, NV = 1;
  while (G < 64 && (G < k || G < n)) G <<= 1;
  while (NV * G < n) NV <<= 1;
  const unsigned blocks = (unsigned)((T * G + 255) / 256);
#define BWD_CASE(GV, UV, NVV)                                                                     \
  case GV * 1024 + UV * 64 + NVV:                                                                 \
    MOE_LAUNCH("route_scored_bwd", s,                                                             \
               (k_route_scored_bwd<GV, UV, NVV><<<blocks, 256, 0, s>>>(                             \
                   logits, topk_idx, topk_w, d_row_scale, slot_to_row, T, E, k,                    \
                   score == MOE_SCORE_SIGMOID, renorm != 0, scale, d_topk_w, d_logits)));          \
    break
  switch (G * 1024 + U * 64 + NV) {
    BWD_CASE(8, 1, 1); BWD_CASE(16, 1, 1); BWD_CASE(32, 1, 1); BWD_CASE(64, 1, 1);
    BWD_CASE(64, 1, 2); BWD_CASE(64, 1, 4); BWD_CASE(64, 1, 8); BWD_CASE(64, 1, 16);
    BWD_CASE(8, 4, 1); BWD_CASE(16, 4, 1); BWD_CASE(32, 4, 1); BWD_CASE(64, 4, 1);
    BWD_CASE(64, 4, 2); BWD_CASE(64, 4, 4);
    default:
      MOE_REQUIRE(false, MOE_ERR_UNSUPPORTED, "%s: E=%d", fn, E);
  }
#undef BWD_CASE
  return check_launch(fn);
}
