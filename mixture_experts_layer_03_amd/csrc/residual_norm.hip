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
// Measured, bf16: 32768 rows of 2880 (755 MB) 130 us, 5.8 TB/s; 8 expert rows
// of 2048 for each of 32768 tokens (1.48 GB) 254 us, 5.8 TB/s; 16 rows 4 us.
#include <algorithm>

#include "rows.h"

namespace moe {
namespace {

constexpr int kGateNone = 0, kGateChannel = 1, kGateToken = 2, kGateElement = 3;
constexpr int kMaxNormD = 16384;

// Sums of N values over a row's lanes: a wave, or with WIDE a block of up to
// 16 waves through `part`, whose entries of waves that are not there are zero.
// One barrier: two uses of the same array need another sum in between.
constexpr int kMaxWaves = 16;
template <bool WIDE, int N, int WAVES = kMaxWaves>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*part)[kMaxWaves]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (WIDE) {
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) part[i][threadIdx.x >> 6] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = 0.0f;
#pragma unroll
      for (int w = 0; w < WAVES; w += 4) {
        const f32x4_t q = *reinterpret_cast<const f32x4_t *>(&part[i][w]);
        v[i] += (q[0] + q[1]) + (q[2] + q[3]);
      }
    }
  }
}
// part = 0, before the first sum
template <int COUNT>
__device__ __forceinline__ void clear(float *part) {
  for (int i = threadIdx.x; i < COUNT; i += blockDim.x) part[i] = 0.0f;
  __syncthreads();
}

struct FwdArgs {
  const void *x, *y, *gate, *w_post, *w_pre;
  const int32_t *slot_to_row;   // y holds expert rows
  const float *weights;         // [T,k] or NULL
  void *y_out, *out, *n;
  float *rstd_post, *rstd_pre;
  int64_t T, R;                 // R: rows of y where it holds expert rows
  int d, k, gate_kind;
  float scale, eps;
};

// One row for each wave (four in a block), or with WIDE one for a block of
// up to 16 waves.  A lane holds NV pieces of 16 bytes of the row, from one read
// to the last write.  A wave has no barriers (32768 rows of 2880: 130 us, a
// block for each 140); a block spreads a row where waves would not fill the
// card or a row does not fit their registers.
template <typename T, int NV, bool WIDE, bool GATHER>
__global__ __launch_bounds__(WIDE ? 1024 : 256) void k_residual_norm(const FwdArgs a) {
  constexpr int N = kVec<T>;
  __shared__ __attribute__((aligned(16))) float part[2][1][kMaxWaves];
  if constexpr (WIDE) clear<2 * kMaxWaves>(&part[0][0][0]);
  const int li = WIDE ? (int)threadIdx.x : (int)threadIdx.x & 63;
  const int stride = WIDE ? (int)blockDim.x : 64;
  const int64_t t = WIDE ? (int64_t)blockIdx.x
                         : (int64_t)blockIdx.x * 4 +
                               __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  if (t >= a.T) return;   // whole waves (WIDE: never)
  const T *tag = nullptr;
  const uint32_t bytes = (uint32_t)a.d * sizeof(T);
  const int64_t at = t * bytes;
  uint32_t c[NV];
#pragma unroll
  for (int h = 0; h < NV; ++h) c[h] = (uint32_t)(li + h * stride) * 16u;

  float p[NV][N];   // the block's output, then out
  u32x4_t yv[NV], xv[NV], gv[NV];
  const bool rows = a.gate_kind == kGateElement, vec_gate = rows || a.gate_kind == kGateChannel;
  auto load_x = [&]() {
    const Row x(a.x, at, a.x, bytes), g(a.gate, rows ? at : 0, vec_gate, bytes);
#pragma unroll
    for (int h = 0; h < NV; ++h) xv[h] = x.load(c[h]);
#pragma unroll
    for (int h = 0; h < NV; ++h) gv[h] = g.keep(c[h]);   // a channel's is every row's
  };
  if constexpr (GATHER) {
    const int lane = threadIdx.x & 63;
    int myr = lane < a.k ? a.slot_to_row[t * a.k + lane] : -1;   // k <= 32
    if (myr >= a.R) myr = -1;
    const float myw = myr < 0 ? 0.0f : a.weights ? a.weights[t * a.k + lane] : 1.0f;
#pragma unroll
    for (int h = 0; h < NV; ++h)
#pragma unroll
      for (int i = 0; i < N; ++i) p[h][i] = 0.0f;
    for (int j = 0; j < a.k; j += 4) {   // four rows in flight; one that is not there adds 0 * 0
      u32x4_t v[4][NV];
#pragma unroll
      for (int u = 0; u < 4; ++u) {   // lanes from k on hold -1 (j + u <= 34)
        const int r = __builtin_amdgcn_readlane(myr, j + u);
        const Row row(a.y, (int64_t)r * bytes, r >= 0, bytes);
#pragma unroll
        for (int h = 0; h < NV; ++h) v[u][h] = row.load(c[h]);
      }
      if (j + 4 >= a.k) load_x();
#pragma unroll
      for (int u = 0; u < 4; ++u) {
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
    const Row to_y(a.y_out, at, a.y_out, bytes);
#pragma unroll
    for (int h = 0; h < NV; ++h) {   // the stored row, as the combine alone leaves it
      yv[h] = pack(p[h], tag);
      to_y.store(c[h], yv[h]);
    }
  } else {
    const Row y(a.y, at, a.y, bytes);
#pragma unroll
    for (int h = 0; h < NV; ++h) yv[h] = y.load(c[h]);
    load_x();
  }
#pragma unroll
  for (int h = 0; h < NV; ++h) unpack(yv[h], p[h], tag);

  if (a.w_post) {
    float s[1] = {0.0f};
#pragma unroll
    for (int h = 0; h < NV; ++h)
#pragma unroll
      for (int i = 0; i < N; ++i) s[0] = fmaf(p[h][i], p[h][i], s[0]);
    row_sum<WIDE, 1>(s, part[0]);
    const float r = 1.0f / sqrtf(s[0] / (float)a.d + a.eps);
    if (a.rstd_post && li == 0) a.rstd_post[t] = r;
    const Row wr(a.w_post, 0, true, bytes);
#pragma unroll
    for (int h = 0; h < NV; ++h) {
      float w[N];
      unpack(wr.keep(c[h]), w, tag);
#pragma unroll
      for (int i = 0; i < N; ++i) p[h][i] = p[h][i] * r * w[i];
    }
  }
  const float gt = a.gate_kind == kGateToken ? ((const float *)a.gate)[t] : 1.0f;
  const Row to_out(a.out, at, a.out, bytes);
  float s[1] = {0.0f};
#pragma unroll
  for (int h = 0; h < NV; ++h) {
    float x[N], g[N];
    unpack(xv[h], x, tag);
    unpack(gv[h], g, tag);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float gi = vec_gate ? g[i] : gt;
      p[h][i] = a.y ? fmaf(a.scale, x[i], gi * p[h][i]) : x[i];
    }
    const u32x4_t v = pack(p[h], tag);
    to_out.store(c[h], v);
    unpack(v, p[h], tag);
#pragma unroll
    for (int i = 0; i < N; ++i) s[0] = fmaf(p[h][i], p[h][i], s[0]);
  }
  if (!a.w_pre) return;
  row_sum<WIDE, 1>(s, part[1]);
  const float r = 1.0f / sqrtf(s[0] / (float)a.d + a.eps);
  if (a.rstd_pre && li == 0) a.rstd_pre[t] = r;
  const Row wr(a.w_pre, 0, true, bytes), to_n(a.n, at, true, bytes);
#pragma unroll
  for (int h = 0; h < NV; ++h) {
    float w[N], f[N];
    unpack(wr.keep(c[h]), w, tag);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = p[h][i] * r * w[i];
    to_n.store(c[h], pack(f, tag));
  }
}

struct BwdArgs {
  const void *d_out, *d_n, *out, *y, *gate, *w_post, *w_pre;
  const float *rstd_post, *rstd_pre;
  void *d_x, *d_y, *d_gate;
  float *partial;               // [blocks][columns][d]: sums over a block's rows
  int64_t T;
  int d, gate_kind, columns;
  int c_pre, c_post;            // the columns of d_n out rn and of P y rp (a channel's gate:
                                // D y rp), -1: not formed
  float scale;
};

// With o = the stored out, q = d_n w_pre, rn and rp the forward's 1/rms:
//   D   = d_out + rn q - c1 o,  c1 = rn^3/d sum(q o)
//   d_x = store(s D),  P = gate D
//   d_y = store(rp (P w_post - y rp^2/d sum(P w_post y)))
//   d_w_pre = sum_t d_n o rn,  d_w_post = sum_t P y rp,  d_gate: D p summed over
//   what the gate is shared by.
// D is linear in sum(q o), so with A = y w_post (gate) the three sums of a row
// (q o;  A (d_out + rn q);  A o) come from one pass over it and one reduction.
// A channel's d_w_post and d_gate are its sum of D y rp times the other's factor.
// A block of W waves takes rows b, b + G, ...; its lanes keep their columns'
// sums in registers over all of them and load two rows ahead of the one they work
// on.  One block a CU: more rows under way at once come slower from HBM (16384 rows
// of 5760 bytes with its weights' pass: 104 us with one block of 6 waves two rows
// ahead, 117 one row ahead, 111 with two blocks, one or two ahead; a wave for each
// row, with no barriers, 139).
template <int NV>
struct BwdRow {
  u32x4_t dd[NV], dn[NV], o[NV], y[NV], g[NV];
  float rn, rp, gt;
};

template <typename T, int NV, int GATE>
__global__ __launch_bounds__(512) void k_residual_norm_bwd(const BwdArgs a) {
  constexpr int N = kVec<T>;
  // with more than one piece a lane its registers hold one row, in its stored
  // type, and the weights too, and no row is under way meanwhile (8192 rows of
  // 5120 in bf16: 122 us, their bytes at 6.3 TB/s 80)
  constexpr bool kAhead = NV == 1;
  constexpr bool kChannel = GATE == kGateChannel, kToken = GATE == kGateToken, kElement = GATE == kGateElement;
  __shared__ __attribute__((aligned(16))) float part[3][3][kMaxWaves];
  clear<3 * 3 * kMaxWaves>(&part[0][0][0]);
  const int nvec = a.d / N, li = threadIdx.x, stride = blockDim.x;
  const u32x4_t zero = {0u, 0u, 0u, 0u};
  const T *tag = nullptr;
  bool ok[NV];
#pragma unroll
  for (int h = 0; h < NV; ++h) ok[h] = li + h * stride < nvec;
  float g_pre[NV][N], g_post[NV][N];
  u32x4_t wv_pre[NV], wv_post[NV], gv[NV];
#pragma unroll
  for (int h = 0; h < NV; ++h) {
    const int c = li + h * stride;
    wv_pre[h] = a.w_pre && ok[h] ? ((const u32x4_t *)a.w_pre)[c] : zero;
    wv_post[h] = a.w_post && ok[h] ? ((const u32x4_t *)a.w_post)[c] : zero;
    gv[h] = kChannel && ok[h] ? ((const u32x4_t *)a.gate)[c] : zero;
#pragma unroll
    for (int i = 0; i < N; ++i) g_pre[h][i] = g_post[h][i] = 0.0f;
  }
  // the weight of the second norm; that of the first, with a channel's gate
  auto unpack_weights = [&](int h, float (&w1)[N], float (&w2)[N]) {
    float g[N];
    unpack(wv_pre[h], w1, tag);
    unpack(wv_post[h], w2, tag);
    unpack(gv[h], g, tag);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (!a.w_post) w2[i] = 1.0f;
      if (kChannel) w2[i] *= g[i];
    }
  };
  float w1_held[N], w2_held[N];
  if (kAhead) unpack_weights(0, w1_held, w2_held);
  auto weights = [&](int h, float (&w1)[N], float (&w2)[N]) {
    if (!kAhead) return unpack_weights(h, w1, w2);
#pragma unroll
    for (int i = 0; i < N; ++i) w1[i] = w1_held[i], w2[i] = w2_held[i];
  };
  const uint32_t bytes = (uint32_t)a.d * sizeof(T);
  auto load = [&](int64_t t, BwdRow<NV> &r) {   // t past the end: zeros
    const bool in = t < a.T;
    const int64_t at = in ? t : 0, row = at * bytes;
    const Row dd(a.d_out, row, in && a.d_out, bytes), dn(a.d_n, row, in && a.d_n, bytes);
    const Row o(a.out, row, in && a.d_n, bytes), y(a.y, row, in && a.y, bytes);
    const Row g(a.gate, row, in && kElement, bytes);
#pragma unroll
    for (int h = 0; h < NV; ++h) {
      const uint32_t c = (uint32_t)(li + h * stride) * 16u;
      r.dd[h] = dd.load(c);
      r.dn[h] = dn.load(c);
      r.o[h] = o.load(c);
      r.y[h] = y.load(c);
      if (kElement) r.g[h] = g.load(c);
    }
    r.rn = a.rstd_pre ? a.rstd_pre[at] : 0.0f;
    r.rp = a.rstd_post ? a.rstd_post[at] : 1.0f;
    r.gt = kToken ? ((const float *)a.gate)[at] : 1.0f;
    __builtin_amdgcn_sched_barrier(0);
  };
  const float inv_d = 1.0f / (float)a.d;
  auto work = [&](int64_t t, BwdRow<NV> &r, float (*lds)[kMaxWaves]) {
    const float rn = r.rn, rp = r.rp;
    // s: sum(q o), sum(A (d_out + rn q)), sum(A o)
    float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int h = 0; h < NV; ++h) {
      float dd[N], dn[N], o[N], y[N], g[N], w1[N], w2[N];
      unpack(r.o[h], o, tag);
      unpack(r.dn[h], dn, tag);
      unpack(r.dd[h], dd, tag);
      unpack(r.y[h], y, tag);
      weights(h, w1, w2);
      if (kElement) unpack(r.g[h], g, tag);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float q = dn[i] * w1[i];
        float A = y[i] * w2[i];
        if (kElement) A *= g[i];
        s[0] = fmaf(q, o[i], s[0]);
        s[1] = fmaf(A, fmaf(rn, q, dd[i]), s[1]);
        s[2] = fmaf(A, o[i], s[2]);
      }
      if (!kAhead) {   // unpacked again below, rather than held
        asm volatile("" : "+v"(r.o[h]), "+v"(r.dn[h]), "+v"(r.dd[h]), "+v"(r.y[h]));
        asm volatile("" : "+v"(wv_pre[h]), "+v"(wv_post[h]), "+v"(gv[h]));
      }
    }
    row_sum<true, 3, 8>(s, lds);
    const float c1 = rn * inv_d * s[0] * rn * rn;   // in this order a row of zeros gives 0
    // sum(A D), without a token's gate; where there is no second norm, an infinite y times its zeros is left out
    const float dot = a.w_pre ? fmaf(-c1, s[2], s[1]) : s[1];
    const float c2 = a.w_post ? rp * inv_d * r.gt * dot * rp * rp : 0.0f;
    if (kToken && a.d_gate && li == 0) ((float *)a.d_gate)[t] = rp * dot;
    const float rpg = rp * r.gt;
    const int64_t row = t * bytes;
    const Row to_x(a.d_x, row, a.d_x, bytes), to_y(a.d_y, row, a.d_y, bytes);
    const Row to_g(a.d_gate, row, kElement && a.d_gate, bytes);
#pragma unroll
    for (int h = 0; h < NV; ++h) {
      float dd[N], dn[N], o[N], y[N], g[N], w1[N], w2[N], dx[N], dy[N], dg[N];
      unpack(r.o[h], o, tag);
      unpack(r.dn[h], dn, tag);
      unpack(r.dd[h], dd, tag);
      unpack(r.y[h], y, tag);
      weights(h, w1, w2);
      if (kElement) unpack(r.g[h], g, tag);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float D = fmaf(-c1, o[i], fmaf(rn, dn[i] * w1[i], dd[i]));
        const float yn = y[i] * rpg;
        const float P = kElement ? D * g[i] : D;
        dx[i] = a.scale * D;
        dy[i] = fmaf(P * w2[i], rpg, a.w_post ? -c2 * y[i] : 0.0f);   // no y in it without its norm
        if (kElement) dg[i] = D * yn * w2[i];
        g_pre[h][i] = fmaf(dn[i], rn * o[i], g_pre[h][i]);
        g_post[h][i] = fmaf(P, yn, g_post[h][i]);
      }
      const uint32_t c = (uint32_t)(li + h * stride) * 16u;
      to_x.store(c, pack(dx, tag));
      to_y.store(c, pack(dy, tag));
      if (kElement) to_g.store(c, pack(dg, tag));
    }
  };
  int64_t t = blockIdx.x;   // below T
  if constexpr (kAhead) {
    const int64_t G = gridDim.x;
    BwdRow<NV> r0, r1, r2;
    load(t, r0);
    load(t + G, r1);
    for (;;) {
      load(t + 2 * G, r2);
      work(t, r0, part[0]);
      if ((t += G) >= a.T) break;
      load(t + 2 * G, r0);
      work(t, r1, part[1]);
      if ((t += G) >= a.T) break;
      load(t + 2 * G, r1);
      work(t, r2, part[2]);
      if ((t += G) >= a.T) break;
    }
  } else {
    BwdRow<NV> r0;
    for (int flip = 0; t < a.T; t += gridDim.x, flip ^= 1) {
      load(t, r0);
      work(t, r0, part[flip]);
    }
  }
  float *out = a.partial + (int64_t)blockIdx.x * a.columns * a.d;
#pragma unroll
  for (int h = 0; h < NV; ++h) {
    if (!ok[h]) continue;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t at = (int64_t)(li + h * stride) * N + i;
      if (a.c_pre >= 0) out[(int64_t)a.c_pre * a.d + at] = g_pre[h][i];
      if (a.c_post >= 0) out[(int64_t)a.c_post * a.d + at] = g_post[h][i];
    }
  }
}

// The same for rows of more than 1024 pieces: each is read twice, the second
// time from the L2 where the rows of an XCD's 32 blocks fit it (4 MB at 16384
// in bf16), and the sums over the tokens are kept in LDS (128 KB), where a lane
// has its columns to itself.  4096 rows of 10240 in bf16: 130 us, their bytes
// at 6.3 TB/s 80.
template <typename T, int GATE>
__global__ __launch_bounds__(1024) void k_residual_norm_bwd_long(const BwdArgs a) {
  constexpr int N = kVec<T>;
  constexpr bool kChannel = GATE == kGateChannel, kToken = GATE == kGateToken, kElement = GATE == kGateElement;
  __shared__ float acc[2][kMaxNormD];
  __shared__ __attribute__((aligned(16))) float part[2][3][kMaxWaves];
  const int nvec = a.d / N;
  const T *tag = nullptr;
  const float inv_d = 1.0f / (float)a.d;
  for (int c = threadIdx.x * N; c < a.d; c += 1024 * N) {
#pragma unroll
    for (int i = 0; i < N; ++i) acc[0][c + i] = acc[1][c + i] = 0.0f;
  }
  struct Piece {
    float dd[N], dn[N], o[N], y[N], g[N], w1[N], w2[N];
  };
  auto get = [&](const void *p, int64_t at, int c, float (&f)[N]) {
    const u32x4_t zero = {0u, 0u, 0u, 0u};
    unpack(p ? ((const u32x4_t *)((const T *)p + at))[c] : zero, f, tag);
  };
  auto load = [&](int64_t t, int c, Piece &p) {
    const int64_t row = t * a.d;
    get(a.d_out, row, c, p.dd);
    get(a.d_n, row, c, p.dn);
    get(a.d_n ? a.out : nullptr, row, c, p.o);
    get(a.y, row, c, p.y);
    get(a.w_pre, 0, c, p.w1);
    get(a.w_post, 0, c, p.w2);
    if (kElement) get(a.gate, row, c, p.g);
    if (kChannel) get(a.gate, 0, c, p.g);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (!a.w_post) p.w2[i] = 1.0f;
      if (kChannel) p.w2[i] *= p.g[i];
    }
  };
  int flip = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, flip ^= 1) {
    const float rn = a.rstd_pre ? a.rstd_pre[t] : 0.0f, rp = a.rstd_post ? a.rstd_post[t] : 1.0f;
    const float gt = kToken ? ((const float *)a.gate)[t] : 1.0f;
    float s[3] = {0.0f, 0.0f, 0.0f};
    for (int c = threadIdx.x; c < nvec; c += 1024) {
      Piece p;
      load(t, c, p);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float q = p.dn[i] * p.w1[i];
        float A = p.y[i] * p.w2[i];
        if (kElement) A *= p.g[i];
        s[0] = fmaf(q, p.o[i], s[0]);
        s[1] = fmaf(A, fmaf(rn, q, p.dd[i]), s[1]);
        s[2] = fmaf(A, p.o[i], s[2]);
      }
    }
    row_sum<true, 3>(s, part[flip]);
    const float c1 = rn * inv_d * s[0] * rn * rn, dot = a.w_pre ? fmaf(-c1, s[2], s[1]) : s[1];
    const float c2 = a.w_post ? rp * inv_d * gt * dot * rp * rp : 0.0f, rpg = rp * gt;
    if (kToken && a.d_gate && threadIdx.x == 0) ((float *)a.d_gate)[t] = rp * dot;
    const int64_t row = t * a.d;
    for (int c = threadIdx.x; c < nvec; c += 1024) {
      Piece p;
      load(t, c, p);
      float dx[N], dy[N], dg[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float D = fmaf(-c1, p.o[i], fmaf(rn, p.dn[i] * p.w1[i], p.dd[i]));
        const float yn = p.y[i] * rpg, P = kElement ? D * p.g[i] : D;
        dx[i] = a.scale * D;
        dy[i] = fmaf(P * p.w2[i], rpg, a.w_post ? -c2 * p.y[i] : 0.0f);
        if (kElement) dg[i] = D * yn * p.w2[i];
        acc[0][c * N + i] = fmaf(p.dn[i], rn * p.o[i], acc[0][c * N + i]);
        acc[1][c * N + i] = fmaf(P, yn, acc[1][c * N + i]);
      }
      if (a.d_x) ((u32x4_t *)((T *)a.d_x + row))[c] = pack(dx, tag);
      if (a.d_y) ((u32x4_t *)((T *)a.d_y + row))[c] = pack(dy, tag);
      if (kElement && a.d_gate) ((u32x4_t *)((T *)a.d_gate + row))[c] = pack(dg, tag);
    }
  }
  __syncthreads();
  float *out = a.partial + (int64_t)blockIdx.x * a.columns * a.d;
  for (int at = threadIdx.x; at < a.d; at += 1024) {
    if (a.c_pre >= 0) out[(int64_t)a.c_pre * a.d + at] = acc[0][at];
    if (a.c_post >= 0) out[(int64_t)a.c_post * a.d + at] = acc[1][at];
  }
}

// The partial sums of `blocks` blocks in a fixed order: a block of 16 waves
// takes 64 columns, wave w blocks w, w + 16, ...  A channel's d_w_post and
// d_gate are the one sum times the other's factor; without rows (blocks 0) the
// sums are zero whatever the factors hold.
template <typename T>
__global__ __launch_bounds__(1024) void k_norm_weights(const BwdArgs a, int blocks, float *d_pre,
                                                       float *d_post, float *d_gate) {
  __shared__ float part[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (c < a.d) {
    const float *p = a.partial + (int64_t)blockIdx.y * a.d + c;
#pragma unroll 8
    for (int b = wave; b < blocks; b += 16) s += p[(int64_t)b * a.columns * a.d];
  }
  part[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < a.d) {
    for (int w = 1; w < 16; ++w) s += part[w][lane];
    if ((int)blockIdx.y == a.c_pre) {
      d_pre[c] = s;
    } else {
      // asked for alone, d_w_post still has the gate in it
      if (d_post) d_post[c] = a.gate_kind == kGateChannel && blocks ? s * Store<T>::load((const T *)a.gate + c) : s;
      if (d_gate) d_gate[c] = a.w_post && blocks ? s * Store<T>::load((const T *)a.w_post + c) : s;
    }
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

// How the backward's rows are worked: pieces of a lane, waves of a block (0:
// the long rows' kernel), blocks: up to six waves a CU (with twelve
// 2048 columns run at 5.3 TB/s instead of 5.9); for few tokens a block for each row, and between them at least 8 rows each, since every block
// leaves its sums over the tokens to be added up.
struct BwdPlan {
  int nv, waves, blocks;
};
BwdPlan bwd_plan(int64_t T, int d, int dtype) {
  const int nvec = d * (dtype == MOE_BF16 ? 2 : 4) / 16;
  BwdPlan p;
  p.nv = nvec <= 512 ? 1 : 2;
  p.waves = nvec > 1024 ? 0 : (nvec + 64 * p.nv - 1) / (64 * p.nv);
  int64_t b = p.waves == 0 ? 256 : 256 * (p.waves < 6 ? 6 / p.waves : 1);
  if (b > T / 8) b = T / 8 > 256 ? T / 8 : 256;
  p.blocks = (int)(b < T ? b : T);
  return p;
}

template <typename T, bool GATHER>
void launch_fwd(const FwdArgs &a, hipStream_t s) {
  const int nvec = a.d / kVec<T>;
  // A wave for each row once they fill the card and a row fits its registers
  // (us a block : a wave, dense rows of 2880: 1024 rows 5.8 : 7.6, 2048 12.1 :
  // 9.5, 32768 140 : 130; eight expert rows of 2048 for each of 32768 tokens
  // 261 : 254, of 4096 33.1 : 35.5), and where a lane holds one piece of it
  // (rows of 512: 16 of them 2.9 : 2.7, 16384 14.2 : 13.8).  The two add a row's
  // squares in different orders, so the combined call goes by the same rule as
  // the two calls that it stands for, and its sums are theirs (gathered rows of 4
  // to 8 KB were not measured).
  if (nvec <= 64 || (nvec <= 64 * 8 && a.T >= 2048)) {
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

template <typename T, int GATE>
void launch_bwd(const BwdArgs &a, const BwdPlan &p, hipStream_t s) {
  if (p.waves == 0) k_residual_norm_bwd_long<T, GATE><<<p.blocks, 1024, 0, s>>>(a);
  else if (p.nv == 1) k_residual_norm_bwd<T, 1, GATE><<<p.blocks, 64 * p.waves, 0, s>>>(a);
  else k_residual_norm_bwd<T, 2, GATE><<<p.blocks, 64 * p.waves, 0, s>>>(a);
}
template <typename T>
void launch_bwd(const BwdArgs &a, const BwdPlan &p, hipStream_t s) {
  if (a.gate_kind == kGateChannel) launch_bwd<T, kGateChannel>(a, p, s);
  else if (a.gate_kind == kGateToken) launch_bwd<T, kGateToken>(a, p, s);
  else if (a.gate_kind == kGateElement) launch_bwd<T, kGateElement>(a, p, s);
  else launch_bwd<T, kGateNone>(a, p, s);
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
  // a gate of [T,1] or [T,d] without elements has no address; a channel's always has its d
  MOE_REQUIRE((gate != nullptr) == (gate_kind != kGateNone) || (T == 0 && gate_kind != kGateChannel),
              MOE_ERR_INVALID_ARG,
              "%s: gate and gate_kind %d do not go together", fn, gate_kind);
  MOE_REQUIRE(eps_or_one > 0.0f, MOE_ERR_INVALID_ARG, "%s: eps must be positive", fn);
  return MOE_OK;
}

int run_fwd(const char *fn, const FwdArgs &a, bool gather, int dtype, void *stream) {
  const int rc = check_common(fn, a.T, a.d, dtype, a.gate, a.gate_kind, a.eps);
  if (rc != MOE_OK) return rc;
  // four rows to a block of 256 threads
  MOE_REQUIRE((a.T + 3) / 4 < ((int64_t)1 << 24), MOE_ERR_UNSUPPORTED, "%s: too many tokens (T=%lld)", fn, (long long)a.T);
  if (gather) {
    MOE_REQUIRE(a.R >= 0 && a.k >= 1 && a.k <= kMaxTopK && a.T * a.k < ((int64_t)1 << 31),
                MOE_ERR_INVALID_ARG, "%s: bad sizes (T=%lld k=%d R=%lld)", fn, (long long)a.T, a.k,
                (long long)a.R);
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
  moe::FwdArgs a = {};
  a.x = x, a.y = y, a.gate = gate, a.gate_kind = gate_kind, a.w_post = w_post, a.w_pre = w_pre;
  a.scale = res_scale, a.eps = eps, a.T = T, a.d = d;
  a.out = out, a.n = n, a.rstd_post = rstd_post, a.rstd_pre = rstd_pre;
  return moe::run_fwd("moe_residual_norm", a, false, dtype, stream);
}

int moe_combine_residual_norm(const void *y_perm, int64_t R, const int32_t *slot_to_row,
                              const float *weights, int k, const void *x, const void *gate,
                              int gate_kind, const void *w_post, const void *w_pre, float res_scale,
                              float eps, int dtype, int64_t T, int d, void *y, void *out, void *n,
                              float *rstd_post, float *rstd_pre, void *stream) {
  moe::clear_error();
  moe::FwdArgs a = {};
  a.x = x, a.y = y_perm, a.gate = gate, a.gate_kind = gate_kind, a.w_post = w_post, a.w_pre = w_pre;
  a.slot_to_row = slot_to_row, a.weights = weights, a.k = k, a.R = R, a.y_out = y;
  a.scale = res_scale, a.eps = eps, a.T = T, a.d = d;
  a.out = out, a.n = n, a.rstd_post = rstd_post, a.rstd_pre = rstd_pre;
  return moe::run_fwd("moe_combine_residual_norm", a, true, dtype, stream);
}

size_t moe_residual_norm_bwd_workspace_size(int64_t T, int d) {
  if (T < 0 || d <= 0) return 0;
  const int b = moe::bwd_plan(T, d, MOE_BF16).blocks, f = moe::bwd_plan(T, d, MOE_F32).blocks;
  return moe::align_up((size_t)std::max(b, f) * 2 * (size_t)d * 4, 256);
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
  float *d_channel = gate_kind == kGateChannel ? (float *)d_gate : nullptr;
  const int columns = (d_w_pre != nullptr) + (d_w_post || d_channel);
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
  a.d_out = d_out, a.d_n = d_n, a.out = out, a.y = w_post || d_gate ? y : nullptr, a.gate = gate, a.w_post = w_post, a.w_pre = w_pre;
  a.rstd_post = w_post ? rstd_post : nullptr, a.rstd_pre = w_pre ? rstd_pre : nullptr;
  a.d_x = d_x, a.d_y = d_y, a.d_gate = d_gate, a.partial = (float *)ws;
  a.T = T, a.d = d, a.gate_kind = gate_kind, a.columns = columns, a.scale = res_scale;
  a.c_pre = d_w_pre ? 0 : -1;
  a.c_post = columns > (d_w_pre != nullptr) ? columns - 1 : -1;
  const BwdPlan p = bwd_plan(T, d, dtype);
  if (T > 0) {
    MOE_LAUNCH("residual_norm_bwd", s, {
      if (dtype == MOE_BF16) launch_bwd<bf16_t>(a, p, s);
      else launch_bwd<float>(a, p, s);
    });
    const int e = check_launch(fn);
    if (e != MOE_OK) return e;
  }
  if (columns) {   // T = 0: zeros
    const dim3 grid((unsigned)((d + 63) / 64), (unsigned)columns);
    const int blocks = T > 0 ? p.blocks : 0;
    MOE_LAUNCH("norm_weights", s, {
      if (dtype == MOE_BF16) k_norm_weights<bf16_t><<<grid, 1024, 0, s>>>(a, blocks, d_w_pre, d_w_post, d_channel);
      else k_norm_weights<float><<<grid, 1024, 0, s>>>(a, blocks, d_w_pre, d_w_post, d_channel);
    });
    return check_launch(fn);
  }
  return MOE_OK;
}

}  // extern "C"
