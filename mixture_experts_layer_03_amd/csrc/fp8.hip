// Block-scaled 8-bit expert products: quantisation of rows and weights, the
// grouped product C[r] = w_r A[r] B[e]^T, and the grouped SwiGLU FFN on it.
//
// Format: e4m3 values (sign, 4 exponent bits, 3 mantissa bits, largest 448)
// with one power-of-two scale 2^s per block of 128 along K (rows) or of
// 128 x 128 (weights); s is the smallest integer >= -127 that keeps the
// block's largest finite magnitude within 448 * 2^s, so x * 2^-s is exact in
// fp32 and the conversion is the one rounding.  The byte s + 127 is what
// v_mfma_scale_f32_16x16x128_f8f6f4 takes as an operand: the scales of a
// 128-wide K block enter the product inside the matrix instruction, and the
// fp32 accumulator runs over all of K with no work between the blocks (an
// arbitrary fp32 scale would need a multiply-add of every accumulator per
// block).
//
// Accumulation: the instruction adds the products of each 8 consecutive k
// first, cut at 2^-13 of the largest one's power of two (measured), then the
// groups' sums and the accumulator in fp32.  The cut is taken for its rate
// (twice that of bf16): the values have 4 significant bits, and the error it
// leaves, about 1e-4 of a result, is a tenth of the bf16 store's.
#include "moe_internal.h"

namespace moe {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

constexpr int kBlk = 128;                                   // elements of a scale block
constexpr float kMaxE4m3 = 448.0f;

__host__ __device__ inline int scale_blocks(int K) { return (K + kBlk - 1) / kBlk; }
// bytes of one row of scales: a multiple of four, so that a dword holds the
// scales of four K blocks
__host__ __device__ inline int scale_cols(int K) { return (scale_blocks(K) + 3) / 4 * 4; }

// ------------------------------------------------------------------ scalars

__device__ __forceinline__ float finite_abs(float v) {
  const float a = fabsf(v);
  return a <= 3.402823466e38f ? a : 0.0f;   // NaN and infinities count as 0
}

// The scale byte of a block whose largest finite magnitude is amax:
// floor(log2(amax)) - 8, one more where the mantissa exceeds 448 = 1.75 * 2^8;
// at least 0 (2^-127).  A block of zeros gets 2^0.
__device__ __forceinline__ uint32_t scale_byte(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int s = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return amax == 0.0f ? 127u : (uint32_t)max(s, 0);
}
// 2^-s for the scale byte s + 127 (byte <= 247: the result is a normal number)
__device__ __forceinline__ float inv_scale(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}
// x * 2^-s with infinities turned to NaN (the format has no infinity)
__device__ __forceinline__ float scaled(float x, float inv) {
  return fabsf(x) <= 3.402823466e38f ? x * inv : __uint_as_float(0x7fc00000u);
}
// four values to four e4m3 bytes, nearest even
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}

// Eight consecutive elements as fp32.
__device__ __forceinline__ void load8(const bf16_t *p, float (&v)[8]) {
  const u32x4_t r = *reinterpret_cast<const u32x4_t *>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_bits_to_f32(r[i] & 0xffffu);
    v[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// ------------------------------------------------------------------ rows
//
// One wave per row: 16 lanes x 8 elements hold a block, so a step of the
// wave covers four blocks with 16-byte loads and 8-byte stores.
template <typename T>
__global__ __launch_bounds__(256) void k_quant_rows(const T *__restrict__ x, int64_t R, int K,
                                                    uint8_t *__restrict__ q,
                                                    uint8_t *__restrict__ scale) {
  const int lane = threadIdx.x & 63;
  const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (r >= R) return;
  const int nb = scale_blocks(K), cols = scale_cols(K);
  const T *row = x + r * K;
  for (int b0 = 0; b0 < cols; b0 += 4) {
    const int blk = b0 + (lane >> 4), c = blk * kBlk + (lane & 15) * 8;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    if (c < K) load8(row + c, v);
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, finite_abs(v[i]));
#pragma unroll
    for (int s = 1; s < 16; s <<= 1) m = fmaxf(m, __shfl_xor(m, s, 64));
    const uint32_t byte = blk < nb ? scale_byte(m) : 127u;
    const float inv = inv_scale(byte);
    if (c < K) {
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = scaled(v[i], inv);
      *reinterpret_cast<u32x2_t *>(q + r * K + c) =
          u32x2_t{pack_e4m3x4(w[0], w[1], w[2], w[3]), pack_e4m3x4(w[4], w[5], w[6], w[7])};
    }
    if ((lane & 15) == 0) scale[r * cols + blk] = (uint8_t)byte;
  }
}

// ------------------------------------------------------------------ weights
//
// One block of threads per 128 x 128 weight block: thread t holds columns
// 8 (t % 16).. of rows t / 16 + 16 i.  The transposed copy goes through LDS,
// and its scale is the same byte: a square block keeps its scale when it is
// transposed.
template <typename T, bool TR>
__global__ __launch_bounds__(256) void k_quant_weights(const T *__restrict__ w, int N, int K,
                                                       uint8_t *__restrict__ q,
                                                       uint8_t *__restrict__ scale,
                                                       uint8_t *__restrict__ qt,
                                                       uint8_t *__restrict__ scale_t) {
  __shared__ float s_max[4];
  __shared__ __attribute__((aligned(16))) uint8_t s_t[TR ? 128 * 144 : 16];
  const int tid = threadIdx.x, cg = tid & 15, rg = tid >> 4;
  const int kb = blockIdx.x, mb = blockIdx.y;
  const int64_t e = blockIdx.z;
  const int c = kb * kBlk + cg * 8;
  const T *we = w + e * N * K;
  float v[8][8];
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = mb * kBlk + rg + 16 * i;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    if (n < N && c < K) load8(we + (int64_t)n * K + c, v[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, finite_abs(v[i][j]));
  }
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) m = fmaxf(m, __shfl_xor(m, s, 64));
  if ((tid & 63) == 0) s_max[tid >> 6] = m;
  __syncthreads();
  m = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
  const uint32_t byte = scale_byte(m);
  const float inv = inv_scale(byte);
  const int mbs = scale_blocks(N), nbs = scale_blocks(K);
  const int cols = scale_cols(K), cols_t = scale_cols(N);
  // the scale's own byte, and the padding after the last block of a row
  if (tid == 0) scale[(e * mbs + mb) * cols + kb] = (uint8_t)byte;
  if (kb == nbs - 1 && tid > 0 && tid < cols - kb) scale[(e * mbs + mb) * cols + kb + tid] = 127;
  if (TR) {
    if (tid == 64) scale_t[(e * nbs + kb) * cols_t + mb] = (uint8_t)byte;
    if (mb == mbs - 1 && tid > 64 && tid - 64 < cols_t - mb)
      scale_t[(e * nbs + kb) * cols_t + mb + tid - 64] = 127;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = mb * kBlk + rg + 16 * i;
    float u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = scaled(v[i][j], inv);
    const uint32_t lo = pack_e4m3x4(u[0], u[1], u[2], u[3]);
    const uint32_t hi = pack_e4m3x4(u[4], u[5], u[6], u[7]);
    if (n < N && c < K) *reinterpret_cast<u32x2_t *>(q + (e * N + n) * K + c) = u32x2_t{lo, hi};
    if (TR) {
      const int rl = rg + 16 * i;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s_t[(cg * 8 + j) * 144 + rl] = (uint8_t)(lo >> (8 * j));
        s_t[(cg * 8 + 4 + j) * 144 + rl] = (uint8_t)(hi >> (8 * j));
      }
    }
  }
  if (TR) {
    __syncthreads();
    // rows of the transposed block: 8 lanes x 16 bytes each
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int kr = (tid >> 3) + 32 * i, n = mb * kBlk + (tid & 7) * 16;
      if (kb * kBlk + kr < K && n < N)
        *reinterpret_cast<u32x4_t *>(qt + (e * K + kb * kBlk + kr) * N + n) =
            *reinterpret_cast<const u32x4_t *>(s_t + kr * 144 + (tid & 7) * 16);
    }
  }
}

// ------------------------------------------------------------------ product
//
// A block of threads forms one tile D[p][q] = sum_k P[p][k] Q[q][k]: p runs
// over BP output columns (weight rows; in the gate/up product BP/2 gate rows
// and the BP/2 up rows of the same features), q over BQ rows of one expert.
// K runs in stages of 128 bytes, one scale block: both operands of a stage
// go to LDS with direct loads of 16 bytes per lane, NS stages deep.
//
// LDS: operand row r of a stage is 8 chunks of 16 bytes, chunk c at place
// c ^ ((r >> 1) & 7), so that the fragment reads (16 rows, one chunk each)
// spread over the banks.
//
// MFMA 16x16x128: lane l holds 32 bytes of row l % 16 of each operand; which
// of the 128 k they are does not matter as long as both operands agree and
// share one scale per row: chunks g and g + 4 of the stage, g = l / 16.  The
// result holds D[4 g + v][l % 16].
struct Fp8Args {
  const uint8_t *a, *a_scale;     // rows [.., K], scales [.., scale_cols(K)]
  const int32_t *row_to_slot;     // gathered rows: row r is slot / k; or null
  uint64_t kmagic;                // floor(2^32 / k) + 1
  int64_t slots;                  // rows of the sorted order (R)
  int64_t a_rows;                 // rows of a
  const int32_t *offsets;         // [E + 1]
  int E, N, K;                    // N: output columns (gate/up: f)
  const uint8_t *b, *b_scale;     // [E, N, K] (gate/up: [E, 2 f, K]), [E, blocks, scale_cols(K)]
  const float *row_scale;         // [R] or null
  bf16_t *c;                      // [R, N]
  uint8_t *h, *h_scale;           // gate/up: [R, f], [R, scale_cols(f)]
  int PT;                         // tiles along the output columns
};

#define LDS_AS __attribute__((address_space(3)))

// Raw buffer resource over [base, base + bytes): loads at or past the byte
// count return zeros.
__device__ __forceinline__ u32x4_t make_rsrc(const void *base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  return u32x4_t{(uint32_t)a, (uint32_t)(a >> 32) & 0xffffu, bytes, 0x00020000u};
}
constexpr uint32_t kOOB = 0x80000000u;   // at or past every resource's byte count

// 16 bytes per lane from global memory to LDS (lane l at lds + 16 l).  In
// assembly, so that the compiler puts no waits of its own around it; the
// kernel waits (wait_vm) before the barrier that publishes the stage.
__device__ __forceinline__ void dma16(u32x4_t rs, uint32_t lds, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(voff), "s"(rs)
               : "memory", "m0");
}
// s_waitcnt vmcnt(N) lgkmcnt(0)
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | ((N >> 4) << 14));
}

// Rows of expert e inside [0, R], whatever the offsets hold.
__device__ __forceinline__ void segment(const Fp8Args &g, int e, int &seg0, int &rows) {
  const int64_t a = min(max((int64_t)g.offsets[e], (int64_t)0), g.slots);
  const int64_t b = min(max((int64_t)g.offsets[e + 1], a), g.slots);
  seg0 = (int)a;
  rows = (int)(b - a);
}

// The tile of this block of threads: the wave scans the experts' tile counts
// (64 per step).  Tiles are numbered expert, then output columns, then rows
// (fastest), and the numbers are split into 8 contiguous chunks, one per XCD
// (blocks go round the XCDs), so that the tiles in flight on an XCD share
// their weight slab in its L2.  Returns false if there is none.
template <int BQ>
__device__ __forceinline__ bool find_tile(const Fp8Args &g, int lane, int &e, int &pt, int &q0,
                                          int &seg0, int &rows) {
  int total = 0;
  for (int e0 = 0; e0 < g.E; e0 += 64) {
    int s = 0, n = 0;
    if (e0 + lane < g.E) segment(g, e0 + lane, s, n);
    n = (n + BQ - 1) / BQ;
    for (int m = 1; m < 64; m <<= 1) n += __shfl_xor(n, m, 64);
    total += n;
  }
  // tiles fit 32 bits: the host bounds the grid
  const int all = __builtin_amdgcn_readfirstlane(total) * g.PT;
  const int chunk = (all + 7) >> 3;
  const int slot = (int)(blockIdx.x >> 3);
  const int id = (int)(blockIdx.x & 7) * chunk + slot;
  if (slot >= chunk || id >= all) return false;
  int base = 0;
  for (int e0 = 0; e0 < g.E; e0 += 64) {
    int s = 0, n = 0;
    if (e0 + lane < g.E) segment(g, e0 + lane, s, n);
    const int t = (n + BQ - 1) / BQ * g.PT;
    int end = t;   // inclusive scan
    for (int m = 1; m < 64; m <<= 1) {
      const int o = __shfl_up(end, m, 64);
      if (lane >= m) end += o;
    }
    const uint64_t hit = __ballot(base + end > id);
    if (hit) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      const int tl = __builtin_amdgcn_readlane(t, l);
      const int at = id - base - (__builtin_amdgcn_readlane(end, l) - tl);
      rows = __builtin_amdgcn_readlane(n, l);
      seg0 = __builtin_amdgcn_readlane(s, l);
      e = e0 + l;
      const int qt = (rows + BQ - 1) / BQ;
      pt = at / qt;
      q0 = (at % qt) * BQ;
      return true;
    }
    base += __builtin_amdgcn_readlane(end, 63);
  }
  return false;
}

// h = silu(g) u in fp32
__device__ __forceinline__ float swiglu(float g, float u) { return g / (1.0f + __expf(-g)) * u; }

constexpr int kScaleChunk = 64;   // K blocks whose scales are in LDS at a time

template <bool GU, int BP, int BQ, int WP, int WQ, int NS>
__global__ __launch_bounds__(WP *WQ * 64) void k_grouped_fp8(Fp8Args g) {
  constexpr int NW = WP * WQ;
  constexpr int FP = BP / WP / 16, FQ = BQ / WQ / 16;   // a wave's fragments
  constexpr int TQ = BQ * 8, TP = BP * 8;               // 16-byte chunks of a stage
  constexpr int NIP = TP / 64 / NW;                     // loads per wave and stage
  constexpr int NIQ = (TQ / 64 + NW - 1) / NW;
  constexpr int LOADS = NIP + NIQ;
  static_assert(NIP * 64 * NW == TP, "the P tile splits evenly over the waves");
  static_assert(!GU || (BP == 256 && FP % 2 == 0), "a gate/up tile holds one block of 128 h");
  static_assert(FP >= 1 && FQ >= 1 && NS >= 2 && (NS - 2) * LOADS < 64, "shape");
  constexpr int STAGE = (TP + TQ) * 16;                 // bytes
  constexpr int PITCH = (GU ? FP * 8 : FP * 32) + 16;   // epilogue: bytes of a row of 16 FP columns
  static_assert(NW * 16 * PITCH <= NS * STAGE, "the epilogue's slots reuse the stages");
  // P scale rows of a tile: gate/up, one block of gate rows and the two
  // blocks that the up rows can touch; else BP / 128 (at least one)
  constexpr int PB = GU ? 3 : (BP + 127) / 128;
  __shared__ u32x4_t smem[NS * (TP + TQ)];
  __shared__ u32x4_t s_dummy[64];
  __shared__ uint32_t s_qs[kScaleChunk / 4][BQ];
  __shared__ uint32_t s_ps[kScaleChunk / 4][4];
  __shared__ float s_amax[GU ? WP : 1][GU ? BQ : 1];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wp = wave % WP, wq = wave / WP;
  int e, pt, q0, seg0, rows;
  if (!find_tile<BQ>(g, lane, e, pt, q0, seg0, rows)) return;
  const int K = g.K, N = g.N, cols = scale_cols(K), nk = scale_blocks(K);
  const int p0 = pt * (GU ? BP / 2 : BP);
  const int64_t nmat = GU ? 2 * (int64_t)N : N;         // rows of an expert's weights

  // ---- row offsets of this wave's loads
  uint32_t voffP[NIP], voffQ[NIQ];
  const u32x4_t zero_rs = make_rsrc(g.offsets, 0);
  // P: rows 0 .. BP-1 of the tile; gate/up: the second half from row N + p0
  const bool second = GU && wave * NIP * 8 >= BP / 2;
  const int prow_shift = second ? BP / 2 : 0;
  const int pvalid = min(N - p0, GU ? BP / 2 : BP);
  const uint8_t *pbase = g.b + (e * nmat + p0 + (second ? N : 0)) * K;
#pragma unroll
  for (int i = 0; i < NIP; ++i) {
    const int row = 8 * (wave * NIP + i) + (lane >> 3);
    const int ch = (lane & 7) ^ ((row >> 1) & 7);
    voffP[i] = (uint32_t)(row - prow_shift) * (uint32_t)K + (uint32_t)ch * 16u;
  }
  const int qvalid = min(rows - q0, BQ);
  const bool gathered = g.row_to_slot != nullptr;
  const uint8_t *qbase = gathered ? g.a : g.a + ((int64_t)seg0 + q0) * K;
  const uint32_t qbytes = gathered ? (uint32_t)(g.a_rows * K) : (uint32_t)qvalid * (uint32_t)K;
  // row of a that holds row q of the tile; -1 past the segment
  auto source_row = [&](int q) -> int {
    if (q >= qvalid) return -1;
    if (!gathered) return q;
    const uint32_t slot = (uint32_t)g.row_to_slot[(int64_t)seg0 + q0 + q];
    return slot < (uint64_t)g.slots ? (int)(((uint64_t)slot * g.kmagic) >> 32) : -1;
  };
#pragma unroll
  for (int i = 0; i < NIQ; ++i) {
    const int row = 8 * (wave * NIQ + i) + (lane >> 3);
    const int ch = (lane & 7) ^ ((row >> 1) & 7);
    const int src = row < BQ ? source_row(row) : -1;
    voffQ[i] = src >= 0 ? (uint32_t)src * (uint32_t)K + (uint32_t)ch * 16u : kOOB;
  }

  // Loads of K stage n into its place of the ring; past the last stage they
  // read nothing into the spare slot (the count of loads per stage stays).
  const uint32_t lds0 = (uint32_t)(uintptr_t)((const LDS_AS void *)smem);
  const uint32_t dummy = (uint32_t)(uintptr_t)((const LDS_AS void *)s_dummy);
  auto issue = [&](int n) {
    const bool live = n < nk;
    const uint32_t k0 = (uint32_t)n * 128u;
    const u32x4_t rp = live ? make_rsrc(pbase + k0, (uint32_t)pvalid * (uint32_t)K - k0) : zero_rs;
    const u32x4_t rq = live ? make_rsrc(qbase + k0, qbytes - k0) : zero_rs;
    const uint32_t st = lds0 + (uint32_t)(n % NS) * STAGE;
    const bool tail = k0 + 128u > (uint32_t)K;
#pragma unroll
    for (int i = 0; i < NIP; ++i) {
      const int row = 8 * (wave * NIP + i) + (lane >> 3);
      const uint32_t ch = (uint32_t)((lane & 7) ^ ((row >> 1) & 7));
      const uint32_t off = tail && k0 + ch * 16u >= (uint32_t)K ? kOOB : voffP[i];
      dma16(rp, live ? st + (uint32_t)(wave * NIP + i) * 1024u : dummy, off);
    }
#pragma unroll
    for (int i = 0; i < NIQ; ++i) {
      const int row = 8 * (wave * NIQ + i) + (lane >> 3);
      const uint32_t ch = (uint32_t)((lane & 7) ^ ((row >> 1) & 7));
      const uint32_t off = tail && k0 + ch * 16u >= (uint32_t)K ? kOOB : voffQ[i];
      const bool in = live && (wave * NIQ + i) * 8 < BQ;
      dma16(in ? rq : zero_rs, in ? st + TP * 16u + (uint32_t)(wave * NIQ + i) * 1024u : dummy, off);
    }
  };
#pragma unroll
  for (int n = 0; n < NS - 1; ++n) issue(n);

  // ---- scales of kScaleChunk K blocks from block kc, as dwords of four
  const int mbs = scale_blocks((int)nmat);
  auto load_scales = [&](int kc) {
    const int nd = min(kScaleChunk, cols - kc) >> 2;
    for (int i = tid; i < nd * BQ; i += NW * 64) {
      const int q = i % BQ, w = i / BQ;
      const int src = source_row(q);
      const int64_t r = gathered ? src : (int64_t)seg0 + q0 + src;
      s_qs[w][q] = src >= 0 ? *reinterpret_cast<const uint32_t *>(g.a_scale + r * cols + kc + 4 * w)
                            : 0x7f7f7f7fu;
    }
    for (int i = tid; i < nd * PB; i += NW * 64) {
      const int b = i % PB, w = i / PB;
      const int first = GU && b > 0 ? (N + p0) / kBlk + b - 1 : p0 / kBlk + b;
      s_ps[w][b] = first < mbs ? *reinterpret_cast<const uint32_t *>(
                                     g.b_scale + ((int64_t)e * mbs + first) * cols + kc + 4 * w)
                               : 0x7f7f7f7fu;
    }
  };
  load_scales(0);

  // ---- fragments
  int prow[FP];   // first row of fragment i in the tile
#pragma unroll
  for (int i = 0; i < FP; ++i)
    prow[i] = GU ? (i < FP / 2 ? 0 : BP / 2) + wp * (BP / 2 / WP) + 16 * (i % (FP / 2))
                 : wp * (BP / WP) + 16 * i;
  const int qrow0 = wq * (BQ / WQ);
  // which of the PB scale rows fragment i takes (a fragment of 16 rows never
  // straddles two blocks: N is a multiple of 16)
  int pblk[FP];
#pragma unroll
  for (int i = 0; i < FP; ++i) {
    if (!GU) pblk[i] = prow[i] / kBlk;
    else if (i < FP / 2) pblk[i] = 0;
    else pblk[i] = 1 + (N + p0 + prow[i] - BP / 2) / kBlk - (N + p0) / kBlk;
  }
  f32x4_t acc[FP][FQ];
#pragma unroll
  for (int i = 0; i < FP; ++i)
#pragma unroll
    for (int j = 0; j < FQ; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int lrow = lane & 15, lg = lane >> 4;
  const uint32_t lane_off = (uint32_t)lrow * 128u + (uint32_t)((lg ^ ((lrow >> 1) & 7)) * 16);
  const LDS_AS char *lds = (const LDS_AS char *)smem;
  auto frag = [&](uint32_t at) -> i32x8_t {
    const u32x4_t lo = *reinterpret_cast<const LDS_AS u32x4_t *>(lds + at);
    const u32x4_t hi = *reinterpret_cast<const LDS_AS u32x4_t *>(lds + (at ^ 64u));
    return i32x8_t{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
                   (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  };
  const int nlive = min(FQ, max(0, (qvalid - qrow0 + 15) >> 4));   // Q fragments with rows

  uint32_t sp[FP], sq[FQ];
#pragma unroll
  for (int i = 0; i < FP; ++i) sp[i] = 0;
#pragma unroll
  for (int j = 0; j < FQ; ++j) sq[j] = 0;
  for (int n = 0; n < nk; ++n) {
    if (n > 0 && n % kScaleChunk == 0) {
      __syncthreads();
      load_scales(n);
    }
    wait_vm<(NS - 2) * LOADS>();
    __syncthreads();   // stage n (and the scales) are in LDS; stage n - 1 is read
    asm volatile("" ::: "memory");
    issue(n + NS - 1);
    const int kc = n % kScaleChunk;
    if ((kc & 3) == 0) {
#pragma unroll
      for (int i = 0; i < FP; ++i) sp[i] = s_ps[kc >> 2][pblk[i]];
#pragma unroll
      for (int j = 0; j < FQ; ++j) sq[j] = s_qs[kc >> 2][qrow0 + 16 * j + lrow];
    }
    const uint32_t st = (uint32_t)(n % NS) * STAGE;
    i32x8_t pf[FP];
#pragma unroll
    for (int i = 0; i < FP; ++i) pf[i] = frag(st + (uint32_t)prow[i] * 128u + lane_off);
#pragma unroll
    for (int j = 0; j < FQ; ++j) {
      if (j < nlive) {
        const i32x8_t qf = frag(st + TP * 16u + (uint32_t)(qrow0 + 16 * j) * 128u + lane_off);
#pragma unroll
        for (int i = 0; i < FP; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              pf[i], qf, acc[i][j], 0, 0, 0, (int)sp[i], 0, (int)sq[j]);
      }
    }
#pragma unroll
    for (int i = 0; i < FP; ++i) sp[i] >>= 8;
#pragma unroll
    for (int j = 0; j < FQ; ++j) sq[j] >>= 8;
  }

  // ---- epilogue: 16 rows x the wave's columns at a time through the wave's
  // own LDS slot, so that the stores are 16 bytes per lane
  wait_vm<0>();
  __syncthreads();   // every wave is done with the stages, whose space the slots take
  LDS_AS char *slot = (LDS_AS char *)smem + wave * 16 * PITCH;
  if constexpr (GU) {
    constexpr int FH = FP / 2;
    // h in the gate accumulators, and the largest magnitude of each row
#pragma unroll
    for (int j = 0; j < FQ; ++j) {
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < FH; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float h = swiglu(acc[i][j][v], acc[i + FH][j][v]);
          acc[i][j][v] = h;
          m = fmaxf(m, finite_abs(h));
        }
      m = fmaxf(m, __shfl_xor(m, 16, 64));
      m = fmaxf(m, __shfl_xor(m, 32, 64));
      if (lane < 16) s_amax[wp][qrow0 + 16 * j + lane] = m;
    }
    __syncthreads();
    const int hcols = scale_cols(N);
#pragma unroll
    for (int j = 0; j < FQ; ++j) {
      if (j >= nlive) continue;
      const int q = qrow0 + 16 * j + lrow;
      float m = 0.0f;
#pragma unroll
      for (int w = 0; w < WP; ++w) m = fmaxf(m, s_amax[w][q]);
      const uint32_t byte = scale_byte(m);
      const float inv = inv_scale(byte);
      const int64_t r = (int64_t)seg0 + q0 + q;
      if (wp == 0 && lg == 0 && q < qvalid) {
        g.h_scale[r * hcols + pt] = (uint8_t)byte;
        if (pt == g.PT - 1)
          for (int b = pt + 1; b < hcols; ++b) g.h_scale[r * hcols + b] = 127;
      }
#pragma unroll
      for (int i = 0; i < FH; ++i)
        *reinterpret_cast<LDS_AS uint32_t *>(slot + lrow * PITCH + 16 * i + 4 * lg) =
            pack_e4m3x4(scaled(acc[i][j][0], inv), scaled(acc[i][j][1], inv),
                        scaled(acc[i][j][2], inv), scaled(acc[i][j][3], inv));
      constexpr int CPR = FH, RPI = 64 / CPR;   // 16-byte chunks per row, rows per step
#pragma unroll
      for (int rr = 0; rr < 16; rr += RPI) {
        const int row = rr + lane / CPR, ch = lane % CPR;
        if (row >= 16) continue;
        const u32x4_t val = *reinterpret_cast<const LDS_AS u32x4_t *>(slot + row * PITCH + 16 * ch);
        const int qq = qrow0 + 16 * j + row, n = p0 + wp * (BP / 2 / WP) + 16 * ch;
        if (qq < qvalid && n < N)
          *reinterpret_cast<u32x4_t *>(g.h + ((int64_t)seg0 + q0 + qq) * N + n) = val;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < FQ; ++j) {
      if (j >= nlive) continue;
      const int q = qrow0 + 16 * j + lrow;
      const float w = g.row_scale && q < qvalid ? g.row_scale[(int64_t)seg0 + q0 + q] : 1.0f;
#pragma unroll
      for (int i = 0; i < FP; ++i)
        *reinterpret_cast<LDS_AS u32x2_t *>(slot + lrow * PITCH + 32 * i + 8 * lg) =
            u32x2_t{pack_bf16x2(w * acc[i][j][0], w * acc[i][j][1]),
                    pack_bf16x2(w * acc[i][j][2], w * acc[i][j][3])};
      constexpr int CPR = 2 * FP, RPI = 64 / CPR;
#pragma unroll
      for (int rr = 0; rr < 16; rr += RPI) {
        const int row = rr + lane / CPR, ch = lane % CPR;
        if (row >= 16) continue;
        const u32x4_t val = *reinterpret_cast<const LDS_AS u32x4_t *>(slot + row * PITCH + 16 * ch);
        const int qq = qrow0 + 16 * j + row, n = p0 + wp * (BP / WP) + 8 * ch;
        if (qq < qvalid && n < N)
          *reinterpret_cast<u32x4_t *>(g.c + ((int64_t)seg0 + q0 + qq) * N + n) = val;
      }
    }
  }
}

// Blocks for a product over R rows: every expert ends with a partial tile at
// most, and no more experts have rows than there are rows.
int64_t grid_blocks(int64_t R, int E, int BQ, int PT) {
  const int64_t q = R / BQ + (E < R ? (int64_t)E : R);
  return (q * PT + 7) / 8 * 8;
}

template <bool GU, int BP, int BQ, int WP, int WQ, int NS>
int launch_product(const Fp8Args &args, const char *name, const char *fn, hipStream_t s) {
  Fp8Args g = args;
  const int per = GU ? BP / 2 : BP;
  g.PT = (g.N + per - 1) / per;
  const int64_t blocks = grid_blocks(g.slots, g.E, BQ, g.PT);
  MOE_REQUIRE(blocks < ((int64_t)1 << 31), MOE_ERR_UNSUPPORTED, "%s: too many tiles", fn);
  MOE_LAUNCH(name, s,
             (k_grouped_fp8<GU, BP, BQ, WP, WQ, NS><<<(unsigned)blocks, WP * WQ * 64, 0, s>>>(g)));
  return check_launch(fn);
}

template <bool GU>
int product(const Fp8Args &g, const char *name, const char *fn, hipStream_t s) {
  return launch_product<GU, 256, 128, 4, 2, 2>(g, name, fn, s);
}

constexpr int kMaxDim = 1 << 16;

// Checks shared by the product and the FFN.
int check_rows(const char *fn, int64_t R, const int32_t *row_to_slot, int k, int E, int K) {
  MOE_REQUIRE(R >= 0, MOE_ERR_INVALID_ARG, "%s: R < 0", fn);
  MOE_REQUIRE(R < ((int64_t)1 << 31), MOE_ERR_UNSUPPORTED, "%s: R >= 2^31", fn);
  MOE_REQUIRE(E >= 1 && E <= kMaxExperts, MOE_ERR_UNSUPPORTED, "%s: E=%d outside [1,%d]", fn, E,
              kMaxExperts);
  MOE_REQUIRE(K >= 16 && K % 16 == 0 && K <= kMaxDim, MOE_ERR_UNSUPPORTED,
              "%s: inner size %d is not a multiple of 16 in [16,%d]", fn, K, kMaxDim);
  if (row_to_slot) {
    MOE_REQUIRE(k >= 1 && k <= kMaxTopK, MOE_ERR_UNSUPPORTED, "%s: k=%d", fn, k);
    MOE_REQUIRE(R % k == 0, MOE_ERR_INVALID_ARG, "%s: R is not a multiple of k", fn);
    MOE_REQUIRE(R / k * K < ((int64_t)1 << 31), MOE_ERR_UNSUPPORTED,
                "%s: gathered rows of 2^31 bytes or more", fn);
    MOE_REQUIRE(R * k < ((int64_t)1 << 32), MOE_ERR_UNSUPPORTED, "%s: R*k >= 2^32", fn);
  }
  return MOE_OK;
}

int check_cols(const char *fn, int N) {
  MOE_REQUIRE(N >= 16 && N % 16 == 0 && N <= kMaxDim, MOE_ERR_UNSUPPORTED,
              "%s: size %d is not a multiple of 16 in [16,%d]", fn, N, kMaxDim);
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

// ====================================================================== C ABI

extern "C" int moe_fp8_scale_cols(int K) { return K > 0 ? scale_cols(K) : 0; }

extern "C" int moe_quant_rows_fp8(const void *x, int dtype, int64_t R, int K, uint8_t *q,
                                  uint8_t *scale, void *stream) {
  const char *fn = "moe_quant_rows_fp8";
  clear_error();
  MOE_REQUIRE(dtype == MOE_BF16 || dtype == MOE_F32, MOE_ERR_UNSUPPORTED, "%s: dtype %d", fn, dtype);
  int rc = check_rows(fn, R, nullptr, 1, 1, K);
  if (rc) return rc;
  if (R == 0) return MOE_OK;
  MOE_REQUIRE(x && q && scale, MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
  MOE_REQUIRE(aligned16(x) && aligned16(q) && aligned16(scale), MOE_ERR_INVALID_ARG,
              "%s: pointers must be 16-byte aligned", fn);
  hipStream_t s = (hipStream_t)stream;
  const unsigned blocks = (unsigned)((R + 3) / 4);
  if (dtype == MOE_BF16)
    MOE_LAUNCH("quant_rows_fp8", s,
               k_quant_rows<bf16_t><<<blocks, 256, 0, s>>>((const bf16_t *)x, R, K, q, scale));
  else
    MOE_LAUNCH("quant_rows_fp8", s,
               k_quant_rows<float><<<blocks, 256, 0, s>>>((const float *)x, R, K, q, scale));
  return check_launch(fn);
}

extern "C" int moe_quant_weights_fp8(const void *w, int dtype, int E, int N, int K, uint8_t *q,
                                     uint8_t *scale, uint8_t *qt, uint8_t *scale_t, void *stream) {
  const char *fn = "moe_quant_weights_fp8";
  clear_error();
  MOE_REQUIRE(dtype == MOE_BF16 || dtype == MOE_F32, MOE_ERR_UNSUPPORTED, "%s: dtype %d", fn, dtype);
  int rc = check_rows(fn, 0, nullptr, 1, E, K);
  if (rc) return rc;
  rc = check_cols(fn, N);
  if (rc) return rc;
  MOE_REQUIRE(w && q && scale, MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
  MOE_REQUIRE(!qt == !scale_t, MOE_ERR_INVALID_ARG, "%s: qt and scale_t go together", fn);
  MOE_REQUIRE(aligned16(w) && aligned16(q) && aligned16(scale) && aligned16(qt) && aligned16(scale_t),
              MOE_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", fn);
  hipStream_t s = (hipStream_t)stream;
  const dim3 grid((unsigned)scale_blocks(K), (unsigned)scale_blocks(N), (unsigned)E);
#define QUANT_CASE(TT, TRV)                                                                   \
  MOE_LAUNCH("quant_weights_fp8", s,                                                          \
             (k_quant_weights<TT, TRV><<<grid, 256, 0, s>>>((const TT *)w, N, K, q, scale, qt, \
                                                            scale_t)))
  if (dtype == MOE_BF16) {
    if (qt) QUANT_CASE(bf16_t, true);
    else QUANT_CASE(bf16_t, false);
  } else {
    if (qt) QUANT_CASE(float, true);
    else QUANT_CASE(float, false);
  }
#undef QUANT_CASE
  return check_launch(fn);
}

extern "C" int moe_grouped_gemm_fp8(const uint8_t *a, const uint8_t *a_scale,
                                    const int32_t *row_to_slot, int k, const int32_t *offsets,
                                    int E, int64_t R, int N, int K, const uint8_t *b,
                                    const uint8_t *b_scale, const float *row_scale, void *c,
                                    void *stream) {
  const char *fn = "moe_grouped_gemm_fp8";
  clear_error();
  int rc = check_rows(fn, R, row_to_slot, k, E, K);
  if (rc) return rc;
  rc = check_cols(fn, N);
  if (rc) return rc;
  if (R == 0) return MOE_OK;
  MOE_REQUIRE(a && a_scale && offsets && b && b_scale && c, MOE_ERR_INVALID_ARG, "%s: null pointer",
              fn);
  MOE_REQUIRE(aligned16(a) && aligned16(a_scale) && aligned16(b) && aligned16(b_scale) &&
                  aligned16(c),
              MOE_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", fn);
  Fp8Args g{};
  g.a = a;
  g.a_scale = a_scale;
  g.row_to_slot = row_to_slot;
  g.kmagic = row_to_slot ? ((uint64_t)1 << 32) / (uint64_t)k + 1 : 0;
  g.slots = R;
  g.a_rows = row_to_slot ? R / k : R;
  g.offsets = offsets;
  g.E = E;
  g.N = N;
  g.K = K;
  g.b = b;
  g.b_scale = b_scale;
  g.row_scale = row_scale;
  g.c = (bf16_t *)c;
  return product<false>(g, "gg_fp8", fn, (hipStream_t)stream);
}

extern "C" int moe_grouped_ffn_fwd_fp8(const uint8_t *x, const uint8_t *x_scale,
                                       const int32_t *row_to_slot, int k, const int32_t *offsets,
                                       int E, int64_t R, int d, int f, const uint8_t *w_gu,
                                       const uint8_t *w_gu_scale, const uint8_t *w_down,
                                       const uint8_t *w_down_scale, const float *row_scale,
                                       uint8_t *h, uint8_t *h_scale, void *y_perm, void *stream) {
  const char *fn = "moe_grouped_ffn_fwd_fp8";
  clear_error();
  int rc = check_rows(fn, R, row_to_slot, k, E, d);
  if (rc) return rc;
  rc = check_cols(fn, f);
  if (rc) return rc;
  if (R == 0) return MOE_OK;
  MOE_REQUIRE(x && x_scale && offsets && w_gu && w_gu_scale && w_down && w_down_scale && h &&
                  h_scale && y_perm,
              MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
  MOE_REQUIRE(aligned16(x) && aligned16(x_scale) && aligned16(w_gu) && aligned16(w_gu_scale) &&
                  aligned16(w_down) && aligned16(w_down_scale) && aligned16(h) &&
                  aligned16(h_scale) && aligned16(y_perm),
              MOE_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", fn);
  hipStream_t s = (hipStream_t)stream;
  Fp8Args g{};
  g.a = x;
  g.a_scale = x_scale;
  g.row_to_slot = row_to_slot;
  g.kmagic = row_to_slot ? ((uint64_t)1 << 32) / (uint64_t)k + 1 : 0;
  g.slots = R;
  g.a_rows = row_to_slot ? R / k : R;
  g.offsets = offsets;
  g.E = E;
  g.N = f;
  g.K = d;
  g.b = w_gu;
  g.b_scale = w_gu_scale;
  g.h = h;
  g.h_scale = h_scale;
  rc = product<true>(g, "gg_fp8_gate_up", fn, s);
  if (rc) return rc;
  Fp8Args w{};
  w.a = h;
  w.a_scale = h_scale;
  w.slots = R;
  w.a_rows = R;
  w.offsets = offsets;
  w.E = E;
  w.N = d;
  w.K = f;
  w.b = w_down;
  w.b_scale = w_down_scale;
  w.row_scale = row_scale;
  w.c = (bf16_t *)y_perm;
  return product<false>(w, "gg_fp8_down", fn, s);
}
