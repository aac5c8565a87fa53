// The residual stream around the block: the norm of the block's output, its
// gate, the scaled residual and the norm before the next block, forward and
// backward; the forward also straight from the expert rows (weighted combine).
//
// With z = the stored block output (dense, or the combine of its k rows,
// rounded to its type as the combine alone stores it), r(v) = (mean(v^2) +
// eps)^-1/2 over a row:
//   p   = z r(z) w_post          (z without w_post)
//   out = store(s x + gate p)
//   n   = store(out r(out) w_pre), of the stored out: the backward has no other
// A pass moves x, z, out and n once (or k rows in z's place) and does ~10
// operations an element: HBM bounds it, launch latency for few rows.
#include "rows.h"

namespace moe {
namespace {

constexpr int kGateNone = 0, kGateChannel = 1, kGateToken = 2, kGateElement = 3;
constexpr int kMaxNormD = 16384;

// Sums of N values over a row's lanes: a wave, or a block of `waves` waves
// through LDS (`part`: 16 x N floats of its own for each call between two
// uses of the same array, so that one barrier is enough).
template <bool WIDE, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*part)[N], int waves) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (WIDE) {
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) part[threadIdx.x >> 6][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.0f;
    for (int w = 0; w < waves; ++w) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += part[w][i];
    }
  }
}

struct FwdArgs {
  const void *x, *y, *gate, *w_post, *w_pre;
  const int32_t *slot_to_row;   // y holds expert rows
  const float *weights;         // [T,k] or NULL
  void *y_out, *out, *n;
  float *rstd_post, *rstd_pre;
  int64_t T;
  int d, k, gate_kind;
  float scale, eps;
};

// One row for each wave (four in a block), or with WIDE one for a block of
// up to 16 waves.  A lane holds NV pieces of 16 bytes of the row.
template <typename T, int NV, bool WIDE, bool GATHER>
__global__ __launch_bounds__(WIDE ? 1024 : 256) void k_residual_norm(const FwdArgs a) {
  constexpr int N = kVec<T>;
  __shared__ float part[2][16][1];
  const int nvec = a.d / N;
  const int waves = WIDE ? (int)blockDim.x >> 6 : 1;
  const int li = WIDE ? (int)threadIdx.x : (int)threadIdx.x & 63;
  const int stride = WIDE ? (int)blockDim.x : 64;
  const int64_t t = WIDE ? (int64_t)blockIdx.x
                         : (int64_t)blockIdx.x * 4 +
                               __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  if (t >= a.T) return;   // whole waves (WIDE: never)
  const u32x4_t zero = {0u, 0u, 0u, 0u};
  const T *tag = nullptr;
  bool ok[NV];
#pragma unroll
  for (int h = 0; h < NV; ++h) ok[h] = li + h * stride < nvec;

  u32x4_t xv[NV], gv[NV];
  const u32x4_t *xr = (const u32x4_t *)((const T *)a.x + t * a.d);
#pragma unroll
  for (int h = 0; h < NV; ++h) xv[h] = a.x && ok[h] ? xr[li + h * stride] : zero;
  const bool rows = a.gate_kind == kGateElement;
  const u32x4_t *gr = (const u32x4_t *)((const T *)a.gate + (rows ? t * a.d : 0));
#pragma unroll
  for (int h = 0; h < NV; ++h)
    gv[h] = (rows || a.gate_kind == kGateChannel) && ok[h] ? gr[li + h * stride] : zero;

  float p[NV][N];   // the block's output, then out
  if constexpr (GATHER) {
    const int lane = threadIdx.x & 63;
    const int myr = lane < a.k ? a.slot_to_row[t * a.k + lane] : -1;   // k <= 32
    const float myw = lane < a.k && a.weights ? a.weights[t * a.k + lane] : 1.0f;
#pragma unroll
    for (int h = 0; h < NV; ++h)
#pragma unroll
      for (int i = 0; i < N; ++i) p[h][i] = 0.0f;
    for (int j = 0; j < a.k; j += 4) {   // four rows in flight
      u32x4_t v[4][NV];
      int r[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        r[u] = j + u < a.k ? __builtin_amdgcn_readlane(myr, j + u) : -1;
        const u32x4_t *row = (const u32x4_t *)((const T *)a.y + (int64_t)max(r[u], 0) * a.d);
#pragma unroll
        for (int h = 0; h < NV; ++h) v[u][h] = r[u] >= 0 && ok[h] ? row[li + h * stride] : zero;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (r[u] < 0) continue;
        const float w = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(myw), j + u));
#pragma unroll
        for (int h = 0; h < NV; ++h) {
          float f[N];
          unpack(v[u][h], f, tag);
#pragma unroll
          for (int i = 0; i < N; ++i) p[h][i] = fmaf(w, f[i], p[h][i]);
        }
      }
    }
    u32x4_t *yo = (u32x4_t *)((T *)a.y_out + t * a.d);
#pragma unroll
    for (int h = 0; h < NV; ++h) {   // the stored row, as the combine alone leaves it
      const u32x4_t v = pack(p[h], tag);
      if (a.y_out && ok[h]) yo[li + h * stride] = v;
      unpack(v, p[h], tag);
    }
  } else {
    const u32x4_t *yr = (const u32x4_t *)((const T *)a.y + t * a.d);
#pragma unroll
    for (int h = 0; h < NV; ++h) unpack(a.y && ok[h] ? yr[li + h * stride] : zero, p[h], tag);
  }

  if (a.w_post) {
    float s[1] = {0.0f};
#pragma unroll
    for (int h = 0; h < NV; ++h)
#pragma unroll
      for (int i = 0; i < N; ++i) s[0] = fmaf(p[h][i], p[h][i], s[0]);
    row_sum<WIDE, 1>(s, part[0], waves);
    const float r = 1.0f / sqrtf(s[0] / (float)a.d + a.eps);
    if (a.rstd_post && li == 0) a.rstd_post[t] = r;
    const u32x4_t *wr = (const u32x4_t *)a.w_post;
#pragma unroll
    for (int h = 0; h < NV; ++h) {
      float w[N];
      unpack(ok[h] ? wr[li + h * stride] : zero, w, tag);
#pragma unroll
      for (int i = 0; i < N; ++i) p[h][i] = p[h][i] * r * w[i];
    }
  }
  const float gt = a.gate_kind == kGateToken ? ((const float *)a.gate)[t] : 1.0f;
  u32x4_t *orow = (u32x4_t *)((T *)a.out + t * a.d);
  float s[1] = {0.0f};
#pragma unroll
  for (int h = 0; h < NV; ++h) {
    float x[N], g[N];
    unpack(xv[h], x, tag);
    unpack(gv[h], g, tag);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float gi = rows || a.gate_kind == kGateChannel ? g[i] : gt;
      p[h][i] = a.y ? fmaf(a.scale, x[i], gi * p[h][i]) : x[i];
    }
    const u32x4_t v = pack(p[h], tag);
    if (a.out && ok[h]) orow[li + h * stride] = v;
    unpack(v, p[h], tag);
#pragma unroll
    for (int i = 0; i < N; ++i) s[0] = fmaf(p[h][i], p[h][i], s[0]);
  }
  if (!a.w_pre) return;
  row_sum<WIDE, 1>(s, part[1], waves);
  const float r = 1.0f / sqrtf(s[0] / (float)a.d + a.eps);
  if (a.rstd_pre && li == 0) a.rstd_pre[t] = r;
  const u32x4_t *wr = (const u32x4_t *)a.w_pre;
  u32x4_t *nrow = (u32x4_t *)((T *)a.n + t * a.d);
#pragma unroll
  for (int h = 0; h < NV; ++h) {
    float w[N], f[N];
    unpack(ok[h] ? wr[li + h * stride] : zero, w, tag);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = p[h][i] * r * w[i];
    if (ok[h]) nrow[li + h * stride] = pack(f, tag);
  }
}

struct BwdArgs {
  const void *d_out, *d_n, *out, *y, *gate, *w_post, *w_pre;
  const float *rstd_post, *rstd_pre;
  void *d_x, *d_y, *d_gate;
  float *partial;               // [blocks][columns][d]: sums over a block's rows
  int64_t T;
  int d, gate_kind, columns;
  int c_pre, c_post, c_gate;    // which of the partial's columns, -1: not formed
  float scale;
};

// With o = the stored out, q = d_n w_pre, rn and rp the forward's 1/rms:
//   D   = d_out + rn q - o rn^3/d sum(q o)
//   d_x = store(s D),  P = gate D
//   d_y = store(rp (P w_post - y rp^2/d sum(P w_post y)))
//   d_w_pre = sum_t d_n o rn,  d_w_post = sum_t P y rp,  d_gate: D p summed over
//   what the gate is shared by.
// D is linear in sum(q o), so with A = y w_post (gate) the three sums of a row
// (q o;  A (d_out + rn q);  A o) come from one pass over it and one reduction.
// A block of W waves takes rows b, b + G, ...; its lanes keep their columns'
// weight gradients in registers over all of them.
template <typename T, int NV>
__global__ __launch_bounds__(1024) void k_residual_norm_bwd(const BwdArgs a) {
  constexpr int N = kVec<T>;
  __shared__ float part[2][16][3];
  const int nvec = a.d / N, li = threadIdx.x, stride = blockDim.x, waves = blockDim.x >> 6;
  const u32x4_t zero = {0u, 0u, 0u, 0u};
  const T *tag = nullptr;
  bool ok[NV];
#pragma unroll
  for (int h = 0; h < NV; ++h) ok[h] = li + h * stride < nvec;
  float gw_pre[NV][N], gw_post[NV][N], gw_gate[NV][N];
  u32x4_t wpre[NV], wpost[NV], gch[NV];
#pragma unroll
  for (int h = 0; h < NV; ++h) {
#pragma unroll
    for (int i = 0; i < N; ++i) gw_pre[h][i] = gw_post[h][i] = gw_gate[h][i] = 0.0f;
    wpre[h] = a.w_pre && ok[h] ? ((const u32x4_t *)a.w_pre)[li + h * stride] : zero;
    wpost[h] = a.w_post && ok[h] ? ((const u32x4_t *)a.w_post)[li + h * stride] : zero;
    gch[h] = a.gate_kind == kGateChannel && ok[h] ? ((const u32x4_t *)a.gate)[li + h * stride] : zero;
  }
  const float inv_d = 1.0f / (float)a.d;
  int flip = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, flip ^= 1) {
    const int64_t row = t * a.d;
    u32x4_t dov[NV], dnv[NV], ov[NV], yv[NV], gv[NV];
#pragma unroll
    for (int h = 0; h < NV; ++h) {
      const int c = li + h * stride;
      dov[h] = a.d_out && ok[h] ? ((const u32x4_t *)((const T *)a.d_out + row))[c] : zero;
      dnv[h] = a.d_n && ok[h] ? ((const u32x4_t *)((const T *)a.d_n + row))[c] : zero;
      ov[h] = a.d_n && ok[h] ? ((const u32x4_t *)((const T *)a.out + row))[c] : zero;
      yv[h] = a.y && ok[h] ? ((const u32x4_t *)((const T *)a.y + row))[c] : zero;
      gv[h] = a.gate_kind == kGateElement && ok[h] ? ((const u32x4_t *)((const T *)a.gate + row))[c] : gch[h];
    }
    const float rn = a.rstd_pre ? a.rstd_pre[t] : 0.0f;
    const float rp = a.rstd_post ? a.rstd_post[t] : 1.0f;
    const float gt = a.gate_kind == kGateToken ? ((const float *)a.gate)[t] : 1.0f;
    const bool vec_gate = a.gate_kind == kGateChannel || a.gate_kind == kGateElement;
    // s: sum(q o), sum(A (d_out + rn q)), sum(A o)
    float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int h = 0; h < NV; ++h) {
      float o[N], dn[N], dd[N], y[N], g[N], w1[N], w2[N];
      unpack(ov[h], o, tag);
      unpack(dnv[h], dn, tag);
      unpack(dov[h], dd, tag);
      unpack(yv[h], y, tag);
      unpack(gv[h], g, tag);
      unpack(wpre[h], w1, tag);
      unpack(wpost[h], w2, tag);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float q = dn[i] * w1[i];
        const float base = fmaf(rn, q, dd[i]);
        float A = a.w_post ? y[i] * w2[i] : y[i];
        if (vec_gate) A *= g[i];
        s[0] = fmaf(q, o[i], s[0]);
        s[1] = fmaf(A, base, s[1]);
        s[2] = fmaf(A, o[i], s[2]);
      }
    }
    row_sum<true, 3>(s, part[flip], waves);
    const float c1 = rn * rn * rn * inv_d * s[0];         // D = d_out + rn q - c1 o
    const float dot = fmaf(-c1, s[2], s[1]);              // sum(A D), without a token's gate
    const float c2 = a.w_post ? rp * rp * inv_d * gt * dot : 0.0f;
    if (a.gate_kind == kGateToken && a.d_gate && li == 0) ((float *)a.d_gate)[t] = rp * dot;
#pragma unroll
    for (int h = 0; h < NV; ++h) {
      float o[N], dn[N], dd[N], y[N], g[N], w1[N], w2[N], dx[N], dy[N], dg[N];
      unpack(ov[h], o, tag);
      unpack(dnv[h], dn, tag);
      unpack(dov[h], dd, tag);
      unpack(yv[h], y, tag);
      unpack(gv[h], g, tag);
      unpack(wpre[h], w1, tag);
      unpack(wpost[h], w2, tag);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float D = fmaf(-c1, o[i], fmaf(rn, dn[i] * w1[i], dd[i]));
        const float P = D * (vec_gate ? g[i] : gt);
        const float yn = y[i] * rp;
        const float w = a.w_post ? w2[i] : 1.0f;
        dx[i] = a.scale * D;
        dy[i] = rp * fmaf(-c2, y[i], P * w);
        dg[i] = D * yn * w;
        gw_pre[h][i] = fmaf(dn[i] * rn, o[i], gw_pre[h][i]);
        gw_post[h][i] = fmaf(P, yn, gw_post[h][i]);
        gw_gate[h][i] += dg[i];
      }
      if (ok[h]) {
        const int c = li + h * stride;
        if (a.d_x) ((u32x4_t *)((T *)a.d_x + row))[c] = pack(dx, tag);
        if (a.d_y) ((u32x4_t *)((T *)a.d_y + row))[c] = pack(dy, tag);
        if (a.gate_kind == kGateElement && a.d_gate)
          ((u32x4_t *)((T *)a.d_gate + row))[c] = pack(dg, tag);
      }
    }
  }
  float *o = a.partial + (int64_t)blockIdx.x * a.columns * a.d;
#pragma unroll
  for (int h = 0; h < NV; ++h) {
    if (!ok[h]) continue;
    const int c = (li + h * stride) * N;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (a.c_pre >= 0) o[(int64_t)a.c_pre * a.d + c + i] = gw_pre[h][i];
      if (a.c_post >= 0) o[(int64_t)a.c_post * a.d + c + i] = gw_post[h][i];
      if (a.c_gate >= 0) o[(int64_t)a.c_gate * a.d + c + i] = gw_gate[h][i];
    }
  }
}

// The partial sums of `blocks` blocks in a fixed order: a block of 16 waves
// takes 64 columns, wave w blocks w, w + 16, ...
__global__ __launch_bounds__(1024) void k_norm_weights(const float *__restrict__ partial, int blocks,
                                                       int columns, int d, float *d0, float *d1,
                                                       float *d2) {
  __shared__ float part[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (c < d) {
    const float *p = partial + (int64_t)blockIdx.y * d + c;
#pragma unroll 4
    for (int b = wave; b < blocks; b += 16) s += p[(int64_t)b * columns * d];
  }
  part[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < d) {
    for (int w = 1; w < 16; ++w) s += part[w][lane];
    (blockIdx.y == 0 ? d0 : blockIdx.y == 1 ? d1 : d2)[c] = s;
  }
}

// How a row is spread: NV pieces of 16 bytes for each of 64 W lanes.
struct Spread {
  int nv, waves;
};
Spread spread_wide(int nvec) {
  const int nv = nvec <= 8 * 64 ? 1 : nvec <= 16 * 64 ? 2 : 4;
  return {nv, (nvec + 64 * nv - 1) / (64 * nv)};
}

int bwd_blocks(int64_t T) { return (int)(T < 768 ? T : 768); }

template <typename T, bool GATHER>
void launch_fwd(const FwdArgs &a, hipStream_t s) {
  const int nvec = a.d / kVec<T>;
  // a wave for each row once they fill the card and a row fits its registers
  if (nvec <= 64 * 8 && a.T >= 2048) {
    const unsigned grid = (unsigned)((a.T + 3) / 4);
    const int nv = (nvec + 63) / 64;
    if (nv <= 1) k_residual_norm<T, 1, false, GATHER><<<grid, 256, 0, s>>>(a);
    else if (nv <= 2) k_residual_norm<T, 2, false, GATHER><<<grid, 256, 0, s>>>(a);
    else if (nv <= 4) k_residual_norm<T, 4, false, GATHER><<<grid, 256, 0, s>>>(a);
    else if (nv <= 6) k_residual_norm<T, 6, false, GATHER><<<grid, 256, 0, s>>>(a);
    else k_residual_norm<T, 8, false, GATHER><<<grid, 256, 0, s>>>(a);
    return;
  }
  const Spread sp = spread_wide(nvec);
  const unsigned grid = (unsigned)a.T, block = 64u * sp.waves;
  if (sp.nv == 1) k_residual_norm<T, 1, true, GATHER><<<grid, block, 0, s>>>(a);
  else if (sp.nv == 2) k_residual_norm<T, 2, true, GATHER><<<grid, block, 0, s>>>(a);
  else k_residual_norm<T, 4, true, GATHER><<<grid, block, 0, s>>>(a);
}

template <typename T>
void launch_bwd(const BwdArgs &a, unsigned grid, hipStream_t s) {
  const Spread sp = spread_wide(a.d / kVec<T>);
  const unsigned block = 64u * sp.waves;
  if (sp.nv == 1) k_residual_norm_bwd<T, 1><<<grid, block, 0, s>>>(a);
  else if (sp.nv == 2) k_residual_norm_bwd<T, 2><<<grid, block, 0, s>>>(a);
  else k_residual_norm_bwd<T, 4><<<grid, block, 0, s>>>(a);
}

// what both directions ask of their sizes, types and gate
int check_common(const char *fn, int64_t T, int d, int dtype, const void *gate, int gate_kind,
                 float eps_or_one) {
  MOE_REQUIRE(T >= 0 && d > 0, MOE_ERR_INVALID_ARG, "%s: bad sizes (T=%lld d=%d)", fn, (long long)T, d);
  MOE_REQUIRE(d % 8 == 0 && d <= kMaxNormD, MOE_ERR_UNSUPPORTED,
              "%s: d must be a multiple of 8 and at most %d (d=%d)", fn, kMaxNormD, d);
  MOE_REQUIRE(dtype == MOE_BF16 || dtype == MOE_F32, MOE_ERR_UNSUPPORTED, "%s: dtype %d", fn, dtype);
  const int nvec = d * (dtype == MOE_BF16 ? 2 : 4) / 16;   // a launch has below 2^32 threads
  MOE_REQUIRE(T < ((int64_t)1 << 26) && T * 64 * spread_wide(nvec).waves < ((int64_t)1 << 32),
              MOE_ERR_UNSUPPORTED, "%s: too many tokens (T=%lld d=%d)", fn, (long long)T, d);
  MOE_REQUIRE(gate_kind >= kGateNone && gate_kind <= kGateElement, MOE_ERR_INVALID_ARG,
              "%s: gate_kind %d", fn, gate_kind);
  MOE_REQUIRE((gate != nullptr) == (gate_kind != kGateNone) || T == 0, MOE_ERR_INVALID_ARG,
              "%s: gate and gate_kind %d do not go together", fn, gate_kind);
  MOE_REQUIRE(eps_or_one > 0.0f, MOE_ERR_INVALID_ARG, "%s: eps must be positive", fn);
  return MOE_OK;
}

int run_fwd(const char *fn, const FwdArgs &a, bool gather, int dtype, void *stream) {
  const int rc = check_common(fn, a.T, a.d, dtype, a.gate, a.gate_kind, a.eps);
  if (rc != MOE_OK) return rc;
  if (gather) {
    MOE_REQUIRE(a.k >= 1 && a.k <= kMaxTopK && a.T * a.k < ((int64_t)1 << 31), MOE_ERR_INVALID_ARG,
                "%s: bad sizes (T=%lld k=%d)", fn, (long long)a.T, a.k);
  }
  if (a.T == 0) return MOE_OK;   // tensors without elements have no address
  MOE_REQUIRE(!a.n == !a.w_pre, MOE_ERR_INVALID_ARG, "%s: n and w_pre go together", fn);
  MOE_REQUIRE((a.w_post || !a.rstd_post) && (a.w_pre || !a.rstd_pre), MOE_ERR_INVALID_ARG,
              "%s: rstd of a norm without its weight", fn);
  if (gather || a.y) {
    MOE_REQUIRE(a.out && a.y && (!gather || a.slot_to_row), MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
  } else {
    MOE_REQUIRE(a.x && a.n, MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
    MOE_REQUIRE(!a.out && !a.w_post && !a.gate && a.scale == 1.0f, MOE_ERR_INVALID_ARG,
                "%s: without y there is only the norm of x (no out, w_post, gate or scale)", fn);
  }
  MOE_REQUIRE(aligned16(a.x) && aligned16(a.y) && aligned16(a.gate) && aligned16(a.w_post) &&
                  aligned16(a.w_pre) && aligned16(a.y_out) && aligned16(a.out) && aligned16(a.n),
              MOE_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", fn);
  hipStream_t s = (hipStream_t)stream;
  MOE_LAUNCH(gather ? "combine_residual_norm" : "residual_norm", s, {
    if (dtype == MOE_BF16) {
      if (gather) launch_fwd<bf16_t, true>(a, s);
      else launch_fwd<bf16_t, false>(a, s);
    } else {
      if (gather) launch_fwd<float, true>(a, s);
      else launch_fwd<float, false>(a, s);
    }
  });
  return check_launch(fn);
}

}  // namespace
}  // namespace moe

extern "C" {

int moe_residual_norm(const void *x, const void *y, const void *gate, int gate_kind,
                      const void *w_post, const void *w_pre, float res_scale, float eps, int dtype,
                      int64_t T, int d, void *out, void *n, float *rstd_post, float *rstd_pre,
                      void *stream) {
  moe::clear_error();
  const moe::FwdArgs a = {x,   y,         gate,     w_post, w_pre, nullptr, nullptr,   nullptr,   out,
                          n,   rstd_post, rstd_pre, T,      d,     1,       gate_kind, res_scale, eps};
  return moe::run_fwd("moe_residual_norm", a, false, dtype, stream);
}

int moe_combine_residual_norm(const void *y_perm, const int32_t *slot_to_row, const float *weights,
                              int k, const void *x, const void *gate, int gate_kind,
                              const void *w_post, const void *w_pre, float res_scale, float eps,
                              int dtype, int64_t T, int d, void *y, void *out, void *n,
                              float *rstd_post, float *rstd_pre, void *stream) {
  moe::clear_error();
  const moe::FwdArgs a = {x,         y_perm,   gate, w_post, w_pre, slot_to_row, weights, y, out, n,
                          rstd_post, rstd_pre, T,    d,      k,     gate_kind,   res_scale, eps};
  return moe::run_fwd("moe_combine_residual_norm", a, true, dtype, stream);
}

size_t moe_residual_norm_bwd_workspace_size(int64_t T, int d) {
  if (T < 0 || d <= 0) return 0;
  return moe::align_up((size_t)(T < 768 ? T : 768) * 3 * (size_t)d * 4, 256);
}

int moe_residual_norm_bwd(const void *d_out, const void *d_n, const void *out, const void *y,
                          const void *gate, int gate_kind, const void *w_post, const void *w_pre,
                          const float *rstd_post, const float *rstd_pre, float res_scale, int dtype,
                          int64_t T, int d, void *d_x, void *d_y, float *d_w_post, float *d_w_pre,
                          void *d_gate, void *ws, size_t ws_bytes, void *stream) {
  using namespace moe;
  const char *fn = "moe_residual_norm_bwd";
  clear_error();
  const int rc = check_common(fn, T, d, dtype, gate, gate_kind, 1.0f);
  if (rc != MOE_OK) return rc;
  MOE_REQUIRE(!d_w_post || w_post, MOE_ERR_INVALID_ARG, "%s: d_w_post without w_post", fn);
  MOE_REQUIRE(!d_w_pre || w_pre, MOE_ERR_INVALID_ARG, "%s: d_w_pre without w_pre", fn);
  MOE_REQUIRE(!d_gate || gate_kind != kGateNone, MOE_ERR_INVALID_ARG, "%s: d_gate without gate", fn);
  const int columns = (d_w_pre != nullptr) + (d_w_post != nullptr) +
                      (d_gate && gate_kind == kGateChannel);
  if (T > 0) {
    MOE_REQUIRE(d_out || d_n, MOE_ERR_INVALID_ARG, "%s: d_out and d_n are both null", fn);
    MOE_REQUIRE(!d_n == !w_pre, MOE_ERR_INVALID_ARG, "%s: d_n and w_pre go together", fn);
    MOE_REQUIRE(!w_pre || (rstd_pre && out), MOE_ERR_INVALID_ARG,
                "%s: w_pre needs out and rstd_pre", fn);
    MOE_REQUIRE(!w_post || (rstd_post && y), MOE_ERR_INVALID_ARG,
                "%s: w_post needs y and rstd_post", fn);
    MOE_REQUIRE(!d_gate || y, MOE_ERR_INVALID_ARG, "%s: d_gate needs y", fn);
    MOE_REQUIRE(d_x || d_y || columns || d_gate, MOE_ERR_INVALID_ARG, "%s: nothing to compute", fn);
    MOE_REQUIRE(!columns || (ws && ws_bytes >= moe_residual_norm_bwd_workspace_size(T, d)),
                MOE_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", fn, ws ? ws_bytes : 0,
                moe_residual_norm_bwd_workspace_size(T, d));
  }
  MOE_REQUIRE(aligned16(d_out) && aligned16(d_n) && aligned16(out) && aligned16(y) && aligned16(gate) &&
                  aligned16(w_post) && aligned16(w_pre) && aligned16(d_x) && aligned16(d_y) && aligned16(d_w_post) &&
                  aligned16(d_w_pre) && aligned16(d_gate) && aligned16(ws),
              MOE_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", fn);
  hipStream_t s = (hipStream_t)stream;
  BwdArgs a = {};
  a.d_out = d_out, a.d_n = d_n, a.out = out, a.y = y, a.gate = gate, a.w_post = w_post, a.w_pre = w_pre;
  a.rstd_post = w_post ? rstd_post : nullptr, a.rstd_pre = w_pre ? rstd_pre : nullptr;
  a.d_x = d_x, a.d_y = d_y, a.d_gate = d_gate, a.partial = (float *)ws;
  a.T = T, a.d = d, a.gate_kind = gate_kind, a.columns = columns, a.scale = res_scale;
  float *dst[3] = {nullptr, nullptr, nullptr};
  int c = 0;
  a.c_pre = a.c_post = a.c_gate = -1;
  if (d_w_pre) dst[a.c_pre = c++] = d_w_pre;
  if (d_w_post) dst[a.c_post = c++] = d_w_post;
  if (d_gate && gate_kind == kGateChannel) dst[a.c_gate = c++] = (float *)d_gate;
  const int blocks = bwd_blocks(T);
  if (T > 0) {
    MOE_LAUNCH("residual_norm_bwd", s, {
      if (dtype == MOE_BF16) launch_bwd<bf16_t>(a, (unsigned)blocks, s);
      else launch_bwd<float>(a, (unsigned)blocks, s);
    });
    const int e = check_launch(fn);
    if (e != MOE_OK) return e;
  }
  if (columns) {   // T = 0: zeros
    MOE_LAUNCH("norm_weights", s,
               k_norm_weights<<<dim3((unsigned)((d + 63) / 64), (unsigned)columns), 1024, 0, s>>>(
                   (const float *)ws, blocks, columns, d, dst[0], dst[1], dst[2]));
    return check_launch(fn);
  }
  return MOE_OK;
}

}  // extern "C"
