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

// One wave per token, decisions in fp64.
__global__ __launch_bounds__(64) void k_route_scored(const float *__restrict__ logits,
                                                     const float *__restrict__ sel_bias, int E,
                                                     int k, bool sigmoid, int n_group,
                                                     int topk_group, int group_top, bool renorm,
                                                     float scale, int32_t *__restrict__ topk_idx,
                                                     float *__restrict__ topk_w) {
  __shared__ double s_c[kMaxExperts];
  const int lane = threadIdx.x;
  const int64_t t = blockIdx.x;
  const float *x = logits + t * E;
  double shift = 0.0, inv_sum = 0.0;
  float fshift = 0.0f, fsum = 0.0f;
  if (!sigmoid) {
    float m = -INFINITY;
    for (int e = lane; e < E; e += 64) m = fmaxf(m, x[e]);
    for (int s = 1; s < 64; s <<= 1) m = fmaxf(m, __shfl_xor(m, s, 64));
    fshift = m == -INFINITY ? 0.0f : m;
    shift = fshift;
    double sum = 0.0;
    for (int e = lane; e < E; e += 64) sum += exp((double)x[e] - shift);
    for (int s = 1; s < 64; s <<= 1) sum += __shfl_xor(sum, s, 64);
    inv_sum = sum == 0.0 ? 0.0 : 1.0 / sum;
    fsum = (float)sum;
  }
  const int gs = E / n_group;
  uint64_t kept = ~0ull;
  if (topk_group < n_group) {
    for (int e = lane; e < E; e += 64) {
      const bool plain = !sel_bias && group_top == 1;
      double c = plain ? (double)x[e] : score64(x[e], sigmoid, shift, inv_sum);
      if (sel_bias) c += sel_bias[e];
      s_c[e] = c;
    }
    __syncthreads();
    double g = -INFINITY;
    if (lane < n_group) {
      double a = -INFINITY, b = -INFINITY;
      for (int i = 0; i < gs; ++i) {
        const double c = s_c[lane * gs + i];
        if (c > a) { b = a; a = c; }
        else if (c > b) b = c;
      }
      g = group_top == 2 ? a + b : a;
      if (g != g) g = -INFINITY;
    }
    int before = 0;
    for (int i = 0; i < n_group; ++i) {
      const double o = __shfl(g, i, 64);
      before += ranks_before(o, i, g, lane) ? 1 : 0;
    }
    kept = __ballot(lane < n_group && before < topk_group);
    __syncthreads();
  }
  constexpr int V = kMaxExperts / 64;
  double c[V];
  uint32_t open = 0;
  for (int v = 0; v < V; ++v) {
    const int e = lane + 64 * v;
    c[v] = 0.0;
    if (e < E && (kept >> (e / gs)) & 1) {
      open |= 1u << v;
      c[v] = sel_bias ? score64(x[e], sigmoid, shift, inv_sum) + (double)sel_bias[e] : (double)x[e];
    }
  }
  int my = 0;
  for (int j = 0; j < k; ++j) {
    double bv = 0.0;
    int bi = 0x7fffffff;
    for (int v = 0; v < V; ++v) {
      const int e = lane + 64 * v;
      if (((open >> v) & 1) && (bi == 0x7fffffff || ranks_before(c[v], e, bv, bi))) { bv = c[v]; bi = e; }
    }
    for (int s = 1; s < 64; s <<= 1) {
      const double ov = __shfl_xor(bv, s, 64);
      const int oi = __shfl_xor(bi, s, 64);
      if (oi != 0x7fffffff && (bi == 0x7fffffff || ranks_before(ov, oi, bv, bi))) { bv = ov; bi = oi; }
    }
    if ((bi & 63) == lane) open &= ~(1u << (bi >> 6));
    if (lane == j) my = bi;
  }
  const bool sel = lane < k;
  const float v = sel ? x[my] : -INFINITY;
  float w;
  if (renorm) {
    // s_j / sum s: the common factor of the selected scores is taken out
    // first, so that no score is too small to be a number
    const float low = sigmoid ? fminf(v, 0.0f) : v;
    float m = low;
    for (int s = 1; s < 64; s <<= 1) m = fmaxf(m, __shfl_xor(m, s, 64));
    float r = 0.0f;
    if (sel && m != -INFINITY) r = sigmoid ? expf(low - m) / (1.0f + expf(-fabsf(v))) : expf(v - m);
    if (sel && v != v) r = v;
    float sum = r;
    for (int s = 1; s < 64; s <<= 1) sum += __shfl_xor(sum, s, 64);
    w = sum == 0.0f ? 0.0f : r / sum;
  } else if (sigmoid) {
    w = 1.0f / (1.0f + expf(-v));
  } else {
    w = fsum == 0.0f ? 0.0f : expf(v - fshift) / fsum;
  }
  if (sel) {
    topk_idx[t * k + lane] = my;
    topk_w[t * k + lane] = w * scale;
  }
}

// One wave per token.
__global__ __launch_bounds__(64) void k_route_scored_bwd(
    const float *__restrict__ logits, const int32_t *__restrict__ topk_idx,
    const float *__restrict__ topk_w, const float *__restrict__ d_row_scale,
    const int32_t *__restrict__ slot_to_row, int E, int k, bool sigmoid, bool renorm, float scale,
    float *__restrict__ d_topk_w, float *__restrict__ d_logits) {
  const int lane = threadIdx.x;
  const int64_t t = blockIdx.x;
  const float *x = logits + t * E;
  const bool sel = lane < k;
  int idx = -1;
  float w = 0.0f, g = 0.0f;
  if (sel) {
    const int64_t slot = t * k + lane;
    idx = topk_idx[slot];
    w = topk_w[slot];
    const int64_t row = slot_to_row ? slot_to_row[slot] : slot;
    g = row >= 0 ? d_row_scale[row] : 0.0f;
    if (d_topk_w) d_topk_w[slot] = g;
  }
  float mean = w * g;
  for (int s = 1; s < 64; s <<= 1) mean += __shfl_xor(mean, s, 64);
  mean /= scale;
  float d = w * (renorm ? g - mean : g);
  const bool dense = !sigmoid && !renorm;
  if (sigmoid && sel && idx >= 0 && idx < E) d *= 1.0f / (1.0f + expf(x[idx]));
  float shift = 0.0f, inv = 0.0f;
  if (dense) {
    float m = -INFINITY;
    for (int e = lane; e < E; e += 64) m = fmaxf(m, x[e]);
    for (int s = 1; s < 64; s <<= 1) m = fmaxf(m, __shfl_xor(m, s, 64));
    shift = m == -INFINITY ? 0.0f : m;
    float sum = 0.0f;
    for (int e = lane; e < E; e += 64) sum += expf(x[e] - shift);
    for (int s = 1; s < 64; s <<= 1) sum += __shfl_xor(sum, s, 64);
    inv = sum == 0.0f ? 0.0f : scale / sum;
  }
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    float out = dense && e < E ? -expf(x[e] - shift) * inv * mean : 0.0f;
    for (int j = 0; j < k; ++j) {
      const int ij = __shfl(idx, j, 64);
      const float dj = __shfl(d, j, 64);
      if (ij == e) out += dj;
    }
    if (e < E) d_logits[t * E + e] = out;
  }
}

int check_scored(const char *fn, int64_t T, int E, int k, int score, float scale) {
  MOE_REQUIRE(T >= 0, MOE_ERR_INVALID_ARG, "%s: T < 0", fn);
  MOE_REQUIRE(E >= 1 && E <= kMaxExperts, MOE_ERR_UNSUPPORTED, "%s: E=%d outside [1,%d]", fn, E,
              kMaxExperts);
  MOE_REQUIRE(k >= 1 && k <= E && k <= kMaxTopK, MOE_ERR_UNSUPPORTED, "%s: k=%d E=%d", fn, k, E);
  MOE_REQUIRE(T * k < ((int64_t)1 << 31), MOE_ERR_UNSUPPORTED, "%s: T*k >= 2^31", fn);
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
  MOE_LAUNCH("route_scored", s,
             k_route_scored<<<(unsigned)T, 64, 0, s>>>(logits, sel_bias, E, k,
                                                       score == MOE_SCORE_SIGMOID, n_group,
                                                       topk_group, group_top, renorm != 0, scale,
                                                       topk_idx, topk_w));
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
  MOE_LAUNCH("route_scored_bwd", s,
             k_route_scored_bwd<<<(unsigned)T, 64, 0, s>>>(
                 logits, topk_idx, topk_w, d_row_scale, slot_to_row, E, k,
                 score == MOE_SCORE_SIGMOID, renorm != 0, scale, d_topk_w, d_logits));
  return check_launch(fn);
}
