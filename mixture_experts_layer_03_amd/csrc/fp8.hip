// Block-scaled 8-bit expert products: quantisation of rows and weights, the
// grouped product C[r] = w_r A[r] B[e]^T, and the grouped SwiGLU FFN on it.
//
// Format: e4m3 values (sign, 4 exponent bits, 3 mantissa bits, largest 448)
// with one power-of-two scale 2^s per block of 128 along K (rows) or of
// 128 x 128 (weights); s is the smallest integer >= -127 that keeps the
// block's largest finite magnitude within 448 * 2^s, so x * 2^-s is exact in
// fp32 and the conversion is the one rounding.  The byte s + 127 is what
// v_mfma_scale_f32_*_f8f6f4 takes as an operand: the scales of a
// 128-wide K block enter the product inside the matrix instruction, and the
// fp32 accumulator runs over all of K with no work between the blocks (an
// arbitrary fp32 scale would need a multiply-add of every accumulator per
// block).
//
// Accumulation: the instruction adds the products of each 8 consecutive k
// first, cut at 2^-13 of the largest one's power of two (measured), then the
// groups' sums and the accumulator in fp32.  The cut is taken for its rate
// (twice that of bf16): the values have 4 significant bits, and the error it
// leaves, about 1e-4 of a result, is a tenth of the bf16 store's.  The gate/up
// product of few rows does without it: h is rounded to 8 bits at once, and
// where the cut moves a value over a border h changes by a step of 6 to 12%.
// In many values that adds a little to the rounding's own error (0.0020
// against 0.0017 of y); one token's few values can meet one such step too many
// (0.0038), so there the bytes become bf16, whose products are exact.
#include <type_traits>

#include "moe_internal.h"

namespace moe {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

constexpr int kBlk = 128;                                   // elements of a scale block

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
// 16 lanes x 8 elements hold a block, so a step of a wave covers four blocks
// with 16-byte loads and 8-byte stores.  A wave takes a whole row (26928 rows
// of 2880 bf16: 43 us, 5.4 TB/s read and written; 54 us with a wave per step);
// where that makes few waves, one step of it each (1 row: 2.0 against 4.1 us,
// 2048 rows: 5.3 against 6.9, 4096: 8.4 and 8.6, 8192: 14.2 and 13.6).
template <typename T>
__global__ __launch_bounds__(256) void k_quant_rows(const T *__restrict__ x, int64_t R, int K,
                                                    uint8_t *__restrict__ q,
                                                    uint8_t *__restrict__ scale, int steps) {
  const int lane = threadIdx.x & 63;
  const int nb = scale_blocks(K), cols = scale_cols(K);
  const int first = (int)blockIdx.y * steps * 4, end = min(first + steps * 4, cols);
  for (int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); r < R; r += (int64_t)gridDim.x * 4) {
    const T *row = x + r * K;
    for (int b0 = first; b0 < end; b0 += 4) {
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
}

// ------------------------------------------------------------------ weights
//
// One block of threads per 128 x 128 weight block: thread t holds columns
// 8 (t % 16).. of rows 4 (t / 16) .. + 3 and 64 further.  The transposed copy
// goes through LDS, four rows of a column to a dword, chunk c of 16 bytes of
// the transposed row r at place c ^ (r / 8 % 8); its scale is the same byte: a
// square block keeps its scale when it is transposed.  32 x 5760 x 2880 bf16
// into both layouts: 393 us (5.4 TB/s read and written; 411 with stores that
// stay in L2, 521 with those and byte writes to LDS).
template <typename T, bool TR>
__global__ __launch_bounds__(256) void k_quant_weights(const T *__restrict__ w, int N, int K,
                                                       uint8_t *__restrict__ q,
                                                       uint8_t *__restrict__ scale,
                                                       uint8_t *__restrict__ qt,
                                                       uint8_t *__restrict__ scale_t) {
  __shared__ float s_max[4];
  __shared__ __attribute__((aligned(16))) uint8_t s_t[TR ? 128 * 128 : 16];
  const int tid = threadIdx.x, cg = tid & 15, rg = tid >> 4;
  const int kb = blockIdx.x, mb = blockIdx.y;
  const int64_t e = blockIdx.z;
  const int c = kb * kBlk + cg * 8;
  const T *we = w + e * N * K;
  float v[8][8];
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = mb * kBlk + 4 * rg + i % 4 + 16 * (i & 4);
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
  uint32_t lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = mb * kBlk + 4 * rg + i % 4 + 16 * (i & 4);
    float u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = scaled(v[i][j], inv);
    lo[i] = pack_e4m3x4(u[0], u[1], u[2], u[3]);
    hi[i] = pack_e4m3x4(u[4], u[5], u[6], u[7]);
    if (n < N && c < K)
      __builtin_nontemporal_store(u32x2_t{lo[i], hi[i]}, reinterpret_cast<u32x2_t *>(q + (e * N + n) * K + c));
  }
  if (TR) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {      // rows 4 rg .. of the upper and the lower half
      const int chunk = (4 * h + (rg >> 2)) ^ (cg & 7);
      uint8_t *const to = s_t + cg * 8 * 128 + chunk * 16 + (rg & 3) * 4;
#pragma unroll
      for (int d = 0; d < 2; ++d) {    // columns 8 cg + 4 d ..
        const uint32_t *const w4 = (d ? hi : lo) + 4 * h;
        const uint32_t a = __builtin_amdgcn_perm(w4[1], w4[0], 0x05010400u);   // columns 0, 1 of rows 0, 1
        const uint32_t b = __builtin_amdgcn_perm(w4[1], w4[0], 0x07030602u);   // columns 2, 3
        const uint32_t f = __builtin_amdgcn_perm(w4[3], w4[2], 0x05010400u);
        const uint32_t g = __builtin_amdgcn_perm(w4[3], w4[2], 0x07030602u);
        *reinterpret_cast<uint32_t *>(to + (4 * d + 0) * 128) = __builtin_amdgcn_perm(f, a, 0x05040100u);
        *reinterpret_cast<uint32_t *>(to + (4 * d + 1) * 128) = __builtin_amdgcn_perm(f, a, 0x07060302u);
        *reinterpret_cast<uint32_t *>(to + (4 * d + 2) * 128) = __builtin_amdgcn_perm(g, b, 0x05040100u);
        *reinterpret_cast<uint32_t *>(to + (4 * d + 3) * 128) = __builtin_amdgcn_perm(g, b, 0x07060302u);
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
        __builtin_nontemporal_store(
            *reinterpret_cast<const u32x4_t *>(s_t + kr * 128 + (((tid & 7) ^ (kr >> 3)) & 7) * 16),
            reinterpret_cast<u32x4_t *>(qt + (e * K + kb * kBlk + kr) * N + n));
    }
  }
}

// ------------------------------------------------------------------ product
//
// A block of threads forms one tile D[p][q] = sum_k P[p][k] Q[q][k]: p runs
// over BP output columns (weight rows; in the gate/up product BP/2 gate rows
// and the BP/2 up rows of the same features), q over BQ rows of one expert.
// K runs in stages of 128 bytes, one scale block: both operands of a stage
// go to a ring in LDS with direct loads of 16 bytes per lane.
//
// LDS: operand row r of a stage is 8 chunks of 16 bytes, chunk c at place
// c ^ ((r >> 1) & 7), so that the fragment reads (16 rows, one chunk each)
// spread over the banks.
//
// MFMA 16x16x128 (few rows): lane l holds 32 bytes of row l % 16 of each
// operand; which of the 128 k they are does not matter as long as both
// operands agree and share one scale per row: chunks g and g + 4 of the stage,
// g = l / 16.  The result holds D[4 g + v][l % 16].
// MFMA 32x32x64 (many rows): row l % 32, chunks g and g + 2 of the stage's
// first 64 k and 4 + g, 6 + g of its last, g = l / 32; the result holds
// D[8 (v / 4) + 4 g + v % 4][l % 32].
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

// Raw buffer resource over [base, base + bytes), uniform over the wave: loads
// at or past the byte count return zeros.
__device__ __forceinline__ u32x4_t make_rsrc(const void *base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  return u32x4_t{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
                 (uint32_t)__builtin_amdgcn_readfirstlane((int)(a >> 32)) & 0xffffu,
                 (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), 0x00020000u};
}
constexpr uint32_t kOOB = 0x80000000u;   // at or past every resource's byte count
// Bytes (fewer than 2^31) of a resource whose base has moved by `moved`.  Signed,
// for a scalar maximum: the saturating difference is a vector instruction, and
// a load stands five wait states behind one that writes its resource, which the
// compiler does not keep before inline assembly.
__device__ __forceinline__ uint32_t left_of(uint32_t bytes, uint32_t moved) {
  return (uint32_t)max((int)(bytes - moved), 0);
}

// 16 bytes per lane from global memory to LDS (lane l at lds + 16 l).  In
// assembly, so that the compiler puts no waits of its own around it; the
// kernel waits (wait_vm) before the barrier that publishes the stage.  (s_nop:
// a load to LDS stands a wait state behind the write of M0, which the compiler
// cannot see to in here.)
__device__ __forceinline__ void dma16(u32x4_t rs, uint32_t lds, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(voff), "s"(rs)
               : "memory", "m0");
}
// The same for what is read once: its lines do not stay in L2.
__device__ __forceinline__ void dma16_once(u32x4_t rs, uint32_t lds, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(voff), "s"(rs)
               : "memory", "m0");
}
// The same as dma16 with 4 bytes per lane (lane l at lds + 4 l).
__device__ __forceinline__ void dma4(u32x4_t rs, uint32_t lds, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(voff), "s"(rs)
               : "memory", "m0");
}
__device__ __forceinline__ uint32_t lds_addr(const void *p) {
  return (uint32_t)(uintptr_t)((const LDS_AS void *)p);
}
// s_waitcnt vmcnt(N) lgkmcnt(0)
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | ((N >> 4) << 14));
}

// h = silu(g) u in fp32, the quotient by the hardware reciprocal (1 ulp)
__device__ __forceinline__ float swiglu(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

// every LDS access of this wave is done
__device__ __forceinline__ void wait_lgkm() { __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (3 << 14)); }

constexpr int kScaleChunk = 64;   // K blocks whose scales are in LDS at a time

// A tile: expert, output columns from tile number pt, rows q0 .. q0 + qvalid - 1
// of the expert's segment, which starts at row seg0.
struct Tile {
  int e, pt, q0, seg0, qvalid;
};

// Tiles are numbered expert, then output columns, then rows (fastest), BQ rows
// each, and split into 8 contiguous chunks, one per XCD (blocks go round the
// XCDs): the tiles in flight on an XCD share their weight slab in its L2.
// KINDS = 2: an expert's last tile, if it has half the rows or fewer, is of
// the second kind, which has numbers and chunks of its own.
template <int BQ, int KINDS>
struct Tiles {
  int off[kMaxExperts + 1];            // the experts' first rows, in [0, R]
  int start[KINDS][kMaxExperts + 1];   // the experts' first tiles
  static __device__ __forceinline__ int row_tiles(int rows, int kind) {
    const int rest = rows % BQ;
    if (KINDS == 1) return rows / BQ + (rest != 0);
    return kind == 0 ? rows / BQ + (rest > BQ / 2) : rest > 0 && rest <= BQ / 2;
  }
  // by all threads of the block
  __device__ __forceinline__ void init(const Fp8Args &g) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int i = threadIdx.x; i <= g.E; i += blockDim.x)
      off[i] = (int)min(max((int64_t)g.offsets[i], (int64_t)0), g.slots);
    __syncthreads();
    if (wave < KINDS) {
      int base = 0;
      for (int e0 = 0; e0 < g.E; e0 += 64) {
        const int e = e0 + lane;
        // (offsets that go up and down could add up to more: sums stop at 2^30)
        uint32_t n = e < g.E ? (uint32_t)(row_tiles(max(off[e + 1] - off[e], 0), wave) * g.PT) : 0u;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
          const uint32_t o = (uint32_t)__shfl_up((int)n, m, 64);
          if (lane >= m) n = min(n + o, 1u << 30);
        }
        n = min(n + (uint32_t)base, 1u << 30);
        if (e < g.E) start[wave][e + 1] = (int)n;
        base = __builtin_amdgcn_readlane((int)n, 63);
      }
      if (lane == 0) start[wave][0] = 0;
    }
    __syncthreads();
  }
  __device__ __forceinline__ int total(const Fp8Args &g, int kind) const {
    return __builtin_amdgcn_readfirstlane(start[kind][g.E]);
  }
  __device__ __forceinline__ Tile decode(const Fp8Args &g, int kind, int at) const {
    const int lane = threadIdx.x & 63;
    for (int e0 = 0;; e0 += 64) {
      const uint64_t hit = __ballot(e0 + lane < g.E && start[kind][min(e0 + lane, g.E - 1) + 1] > at);
      if (hit) {
        Tile t;
        t.e = __builtin_amdgcn_readfirstlane(e0 + __ffsll((unsigned long long)hit) - 1);
        t.seg0 = __builtin_amdgcn_readfirstlane(off[t.e]);
        const int rows = __builtin_amdgcn_readfirstlane(off[t.e + 1]) - t.seg0;
        const int qt = row_tiles(rows, kind);
        const int in = at - __builtin_amdgcn_readfirstlane(start[kind][t.e]);
        t.pt = in / qt;
        t.q0 = kind ? rows / BQ * BQ : (in % qt) * BQ;
        t.qvalid = min(rows - t.q0, BQ);
        return t;
      }
    }
  }
};

// The direct loads of a tile's K stages.  Instruction i of a wave covers 8
// rows x 128 bytes; a lane's byte offset is fixed for the tile and the
// resource's base moves with the stage.  Chunks past K read nothing, and so
// does every chunk of a stage past the last one: such a stage leaves zeros.
//
// LATE, for K = 64 mod 128, where every second row begins in the middle of a
// 128-byte line: such a weight row is `late`.  Its stage n is bytes 128 n + 64
// .., a whole line, its first 64 bytes come as the second half of a stage -1
// (pre), and fragments are put together from the last stage's second half and
// this stage's first.  Stages that straddle lines ask for every such line
// twice: 92 blocks of threads reading 256 rows of 2880 bytes take 19.5 us, of
// 2944 bytes 14.8.  The gate/up product of few rows has it (d = f = 2880, 32
// experts: 28.9 -> 25.1 us at one token, 108 -> 104 at 64, 115 -> 109 at 256,
// before ONCE); in the product into d its start costs as much as it saves
// (13.8 -> 15.4, 59.5 -> 59.0).
//
// ONCE: the weight rows are read by one tile only and need not stay in L2 (d =
// f = 2880, 32 experts, gate/up + down, before bf16: 16 tokens 98 + 54 -> 89 +
// 54 us, 64 104 + 59 -> 94 + 58, 256 109 + 70 -> 101 + 71; where several tiles
// of rows share them, 5003 rows of 13 experts, 720 x 1136, it costs: 13 -> 18).
template <bool GU, int BP, int BQ, int NW, bool LATE, bool ONCE>
struct Loads {
  static constexpr int TP = BP * 8, TQ = BQ * 8;               // 16-byte chunks of a stage
  static constexpr int NIP = TP / 64 / NW;                     // instructions per wave and stage
  static constexpr int NIQ = TQ / 64 / NW;
  static constexpr int LOADS = NIP + NIQ;
  static constexpr uint32_t STAGE = (TP + TQ) * 16;            // bytes
  // every wave issues the same number of loads
  static_assert(NIP * 64 * NW == TP && NIQ * 64 * NW == TQ && (NIQ == 1 || NIQ % 2 == 0), "loads per wave");
  static_assert(NIP % 2 == 0, "the chunk a lane loads depends on its place's parity alone");
  uint32_t voffP[NIP], voffQ[NIQ];
  uint32_t leftP[2], leftQ[NIQ == 1 ? 1 : 2];   // K minus the lane's first byte, by parity of i
  const uint8_t *pbase, *qbase;
  uint32_t pbytes, qbytes;
  uint32_t ldsP, ldsQ;   // the wave's places in the ring's first stage
  int wave, lane;

  __device__ __forceinline__ void init(int wave_, int lane_, const void *smem) {
    wave = wave_;
    lane = lane_;
    ldsP = lds_addr(smem) + (uint32_t)wave * (NIP * 1024u);
    ldsQ = lds_addr(smem) + TP * 16u + (uint32_t)wave * (NIQ * 1024u);
  }
  // row and byte of the chunk that a lane loads with instruction q of an operand
  __device__ __forceinline__ int row(int q) const { return 8 * q + (lane >> 3); }
  __device__ __forceinline__ uint32_t chunk(int q) const {
    return (uint32_t)((lane & 7) ^ ((row(q) >> 1) & 7)) * 16u;
  }
  // whether a row that begins at p is late
  static __device__ __forceinline__ bool late(const Fp8Args &g, const uint8_t *p) {
    return LATE && g.K % 64 == 0 && ((uintptr_t)p & 64);
  }
  // src(r): the row of a (from qbase) that holds row r of the tile, or -1
  template <typename Src>
  __device__ __forceinline__ void tile(const Fp8Args &g, const Tile &t, Src src) {
    // P: rows p0 .. of the expert; gate/up: the second half of the tile from row N + p0
    const int K = g.K;
    const int p0 = t.pt * (GU ? BP / 2 : BP);
    const bool second = GU && wave * NIP * 8 >= BP / 2;
    const int shift = second ? BP / 2 : 0;
    const int64_t nmat = GU ? 2 * (int64_t)g.N : g.N;
    pbase = g.b + (t.e * nmat + p0 + (second ? g.N : 0)) * K;
    pbytes = (uint32_t)min(g.N - p0, GU ? BP / 2 : BP) * (uint32_t)K;
    const uint32_t ahead = late(g, pbase + (lane >> 3) * K) ? 64u : 0u;   // rows 8 apart are alike
#pragma unroll
    for (int i = 0; i < NIP; ++i)
      voffP[i] = (uint32_t)(row(NIP * wave + i) - shift) * (uint32_t)K + chunk(NIP * wave + i) + ahead;
#pragma unroll
    for (int i = 0; i < 2; ++i) leftP[i] = (uint32_t)max(K - (int)(chunk(NIP * wave + i) + ahead), 0);
    const bool gathered = g.row_to_slot != nullptr;
    qbase = gathered ? g.a : g.a + ((int64_t)t.seg0 + t.q0) * K;
    qbytes = gathered ? (uint32_t)(g.a_rows * K) : (uint32_t)t.qvalid * (uint32_t)K;
#pragma unroll
    for (int i = 0; i < NIQ; ++i) {
      const int q = NIQ * wave + i;
      const int r = src(row(q));
      voffQ[i] = r >= 0 ? (uint32_t)r * (uint32_t)K + chunk(q) : kOOB;
    }
#pragma unroll
    for (int i = 0; i < (NIQ == 1 ? 1 : 2); ++i) leftQ[i] = (uint32_t)max(K - (int)chunk(NIQ * wave + i), 0);
  }
  // one(i): instruction i of the stage at byte k0 of the rows, into the place
  // of the ring at `buf`
  __device__ __forceinline__ void one(int i, uint32_t k0, uint32_t buf) const {
    if (i < NIP) {
      const u32x4_t rs = make_rsrc(pbase + k0, left_of(pbytes, k0));
      const uint32_t to = ldsP + buf + (uint32_t)i * 1024u, voff = k0 < leftP[i & 1] ? voffP[i] : kOOB;
      if (ONCE) dma16_once(rs, to, voff);
      else dma16(rs, to, voff);
    } else {
      const int j = i - NIP;
      dma16(make_rsrc(qbase + k0, left_of(qbytes, k0)), ldsQ + buf + (uint32_t)j * 1024u,
            k0 < leftQ[NIQ == 1 ? 0 : j & 1] ? voffQ[j] : kOOB);
    }
  }
  // stage -1: the first 64 bytes of the late rows, as the stage's second half
  __device__ __forceinline__ void pre(const Fp8Args &g, uint32_t buf) const {
    const bool on = late(g, pbase + (lane >> 3) * g.K);
#pragma unroll
    for (int i = 0; i < NIP; ++i)
      dma16(make_rsrc(pbase, pbytes), ldsP + buf + (uint32_t)i * 1024u,
            on && chunk(NIP * wave + i) >= 64u ? voffP[i] - 128u : kOOB);
  }
  __device__ __forceinline__ void issue(uint32_t k0, uint32_t buf) const {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) one(i, k0, buf);
  }
};

// Scale row of row r of the tile: gate/up, 0 for the gate rows (one block)
// and 1, 2 for the two blocks that the up rows can touch; else one per 128.
template <bool GU, int BP>
__device__ __forceinline__ int p_block(const Fp8Args &g, int p0, int r) {
  if (!GU) return r / kBlk;
  return r < BP / 2 ? 0 : 1 + (g.N + p0 + r - BP / 2) / kBlk - (g.N + p0) / kBlk;
}

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

// Values 8 m .. of a fragment's 32 as bf16 (exact: 4 significant bits), unscaled.
__device__ __forceinline__ bf16x8_t as_bf16(const i32x8_t &f, int m) {
  typedef __bf16 pair_t __attribute__((ext_vector_type(2)));
  const pair_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)f[2 * m], 1.0f, false);
  const pair_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)f[2 * m], 1.0f, true);
  const pair_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)f[2 * m + 1], 1.0f, false);
  const pair_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)f[2 * m + 1], 1.0f, true);
  return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// 32 bytes of a fragment: chunks at `at` and at `at` with the bits `other` flipped.
__device__ __forceinline__ i32x8_t frag(const LDS_AS char *lds, uint32_t at, uint32_t other) {
  const u32x4_t lo = *reinterpret_cast<const LDS_AS u32x4_t *>(lds + at);
  const u32x4_t hi = *reinterpret_cast<const LDS_AS u32x4_t *>(lds + (at ^ other));
  return i32x8_t{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
                 (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// The same for the wide kernel's tiles of 256 x 256 and 8 waves, whose P rows
// come as two halves (gate/up: gate and up rows) of two instructions per wave
// each, and whose Q rows take four.
template <bool GU>
struct WideLoads {
  static constexpr uint32_t HALF = 128 * 128, ROWS = 256 * 128;   // bytes of a P half, of the Q rows
  static constexpr uint32_t STAGE = ROWS + 2 * HALF;              // Q rows, P half 0, P half 1
  uint32_t voffP[2], voffQ[4];
  uint32_t left[2];      // K minus the lane's chunk offset, by parity of the instruction
  const uint8_t *pbase[2], *qbase;
  uint32_t pbytes[2], qbytes;
  uint32_t ldsP, ldsQ;   // the wave's places in the ring's first stage
  int wave, lane;

  __device__ __forceinline__ void init(const Fp8Args &g, int wave_, int lane_, const void *smem) {
    wave = wave_;
    lane = lane_;
    ldsQ = lds_addr(smem) + (uint32_t)wave * 4096u;
    ldsP = lds_addr(smem) + ROWS + (uint32_t)wave * 2048u;
#pragma unroll
    for (int i = 0; i < 2; ++i) left[i] = (uint32_t)max(g.K - (int)chunk(i), 0);
  }
  // row (of the wave's) and byte of the chunk that a lane loads with instruction i
  __device__ __forceinline__ int row(int i) const { return 8 * i + (lane >> 3); }
  __device__ __forceinline__ uint32_t chunk(int i) const {
    return (uint32_t)((lane & 7) ^ ((row(i) >> 1) & 7)) * 16u;
  }
  // src(r): the row of a (from qbase) that holds row r of the tile, or -1
  template <typename Src>
  __device__ __forceinline__ void tile(const Fp8Args &g, const Tile &t, Src src) {
    const int K = g.K, p0 = t.pt * (GU ? 128 : 256);
    const uint8_t *const first = g.b + ((GU ? 2 : 1) * (int64_t)g.N * t.e + p0) * K;
    pbase[0] = first;
    pbase[1] = first + (int64_t)(GU ? g.N : 128) * K;
    pbytes[0] = (uint32_t)min(g.N - p0, 128) * (uint32_t)K;
    pbytes[1] = GU ? pbytes[0] : (uint32_t)min(max(g.N - p0 - 128, 0), 128) * (uint32_t)K;
#pragma unroll
    for (int i = 0; i < 2; ++i) voffP[i] = (uint32_t)(16 * wave + row(i)) * (uint32_t)K + chunk(i);
    const bool gathered = g.row_to_slot != nullptr;
    qbase = gathered ? g.a : g.a + ((int64_t)t.seg0 + t.q0) * K;
    qbytes = gathered ? (uint32_t)(g.a_rows * K) : (uint32_t)t.qvalid * (uint32_t)K;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = src(32 * wave + row(i));
      voffQ[i] = r >= 0 ? (uint32_t)r * (uint32_t)K + chunk(i) : kOOB;
    }
  }
  // Instruction i of P half h / of the Q rows, of the stage at byte k0 of the
  // rows, into the place of the ring at `buf`.
  __device__ __forceinline__ void p(int h, int i, uint32_t k0, uint32_t buf) const {
    dma16(make_rsrc(pbase[h] + k0, left_of(pbytes[h], k0)),
          ldsP + buf + (uint32_t)h * HALF + (uint32_t)i * 1024u, k0 < left[i] ? voffP[i] : kOOB);
  }
  __device__ __forceinline__ void q(int i, uint32_t k0, uint32_t buf) const {
    dma16(make_rsrc(qbase + k0, left_of(qbytes, k0)), ldsQ + buf + (uint32_t)i * 1024u,
          k0 < left[i & 1] ? voffQ[i] : kOOB);
  }
  // all offsets in registers here
  __device__ __forceinline__ void keep() {
    asm volatile("" : "+v"(voffP[0]), "+v"(voffP[1]), "+v"(voffQ[0]), "+v"(voffQ[1]), "+v"(voffQ[2]),
                 "+v"(voffQ[3]), "+v"(left[0]), "+v"(left[1]));
  }
  // Q rows and P half 0 (6 instructions), then P half 1 (2)
  __device__ __forceinline__ void front(int i, uint32_t k0, uint32_t buf) const {
    if (i < 4) q(i, k0, buf);
    else p(0, i - 4, k0, buf);
  }
  __device__ __forceinline__ void issue(uint32_t k0, uint32_t buf) const {
#pragma unroll
    for (int i = 0; i < 6; ++i) front(i, k0, buf);
#pragma unroll
    for (int i = 0; i < 2; ++i) p(1, i, k0, buf);
  }
};

// Many rows: tiles of 256 x 256, 8 waves of 128 x 64 (4 x 2 fragments of
// 32 x 32, MFMA 32x32x64).  Persistent: one block of threads per CU walks its
// tiles.
//
// A stage is worked on in two halves, its P rows 0 .. 127 and 128 .. 255 (gate
// and up), each against all Q rows: 8 MFMAs of a wave.  While the MFMAs of a
// half run, the next half's fragments come from LDS into the registers of
// those that are done with (the Q fragments every other half).  A barrier
// stands in the middle of each half: behind it the parts of the ring that the
// half's own fragments came from are free, and the next half's have landed.
// So a stage's Q rows and first P half are loaded three halves before they
// are read, and its second P half too, with two stages in the ring: loads may
// take one and a half stages.  After a tile's last stage the next tile's
// first stage and scales are loaded while the epilogue runs, which uses the
// ring's other place.
//
// 16384 rows x 32 experts, d = f = 2880: gate/up 545 GFLOP in 340 to 355 us
// (as cards differ), down 272 GFLOP in 185 to 190 us; 16384 x 2880 x 5760 over
// 8 experts of 2048 rows 223 to 237 us (2.4 PFLOP/s), over 32 of 512 rows 255
// to 262.  With the MFMAs taken out 251 us, with the loads taken out 270 us
// (gate/up): neither alone bounds, and half of the lines come from beyond the
// XCD's L2.  Where experts have a few rows more than a multiple of 256, their
// last tiles read all their weight rows again: experts of 479 to 558 rows take
// 330 us (350 with big and small tiles dealt out as one).  Tried: one barrier
// a stage with loads one stage ahead (379 and 204 us for the FFN's products),
// 4 waves of 128 x 128 with half the LDS reads and 512 registers (gate/up as
// fast, down 224 us: one wave per SIMD hides neither epilogue nor waits).
template <bool GU>
__global__ __launch_bounds__(512, 2) void k_grouped_fp8_wide(Fp8Args g) {
  constexpr int BP = 256, BQ = 256, WP = 2, NW = 8, FP = 4, FQ = 2, NSP = GU ? 3 : 2;
  using L = WideLoads<GU>;
  __shared__ u32x4_t smem[2 * L::STAGE / 16];
  __shared__ uint32_t s_qs[kScaleChunk / 4][BQ];   // scales of a chunk of K blocks, four to a dword
  __shared__ uint32_t s_ps[kScaleChunk / 4][4];
  __shared__ int s_slot[BQ];                        // gathered rows: the next tile's slots
  __shared__ float s_amax[GU ? WP : 1][GU ? BQ : 1];
  __shared__ Tiles<BQ, 2> tiles;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wp = wave % WP, wq = wave / WP;
  const int N = g.N, nk = scale_blocks(g.K), cols = scale_cols(g.K);
  const bool gathered = g.row_to_slot != nullptr;

  // The blocks of an XCD take its big tiles in turn, and its small ones in turn
  // from where the big ones ended, so that none gets one big tile more while
  // another has a small one left; a block works through both in the order of
  // the experts.
  tiles.init(g);
  const int per = (int)(gridDim.x >> 3);
  int at[2], last[2];   // the block's next tile of each kind, and the end of its XCD's
  {
    int first = (int)(blockIdx.x >> 3);
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      const int total = tiles.total(g, kind), chunk = (total + 7) >> 3, from = (int)(blockIdx.x & 7) * chunk;
      last[kind] = min(total, from + chunk);
      at[kind] = from + first;
      first -= max(last[kind] - from, 0) % per;
      if (first < 0) first += per;
    }
  }
  // the block's next tile; e = E after the last
  auto take = [&]() -> Tile {
    Tile t{g.E, 0, 0, 0, 0};
    bool small = false;
    if (at[0] < last[0]) t = tiles.decode(g, 0, at[0]);
    if (at[1] < last[1]) {
      const Tile u = tiles.decode(g, 1, at[1]);
      if (u.e < t.e || (u.e == t.e && u.pt < t.pt)) {
        t = u;
        small = true;
      }
    }
    at[0] += small ? 0 : per;
    at[1] += small ? per : 0;
    return t;
  };

  // ---- loads of a tile: its slots, its scales of a chunk of K blocks
  L ld;
  ld.init(g, wave, lane, smem);
  auto load_slots = [&](const Tile &t) {
    if (wave < BQ / 64)
      dma4(make_rsrc(g.row_to_slot + t.seg0 + t.q0, (uint32_t)t.qvalid * 4u),
           lds_addr(s_slot + wave * 64), (uint32_t)(wave * 64 + lane) * 4u);
  };
  uint32_t sc_off = 0;   // of row 64 (wave % 4) + lane in the scale rows
  auto set_tile = [&](const Tile &t) {
    int ln = lane;   // taken anew, as in the epilogue
    asm volatile("" : "+v"(ln));
    ld.lane = ln;
    auto src = [&](int r) -> int {   // row of a, -1 past the segment or for no token
      if (r >= t.qvalid) return -1;
      if (!gathered) return r;
      const uint32_t slot = (uint32_t)s_slot[r];
      return slot < (uint64_t)g.slots ? (int)(((uint64_t)slot * g.kmagic) >> 32) : -1;
    };
    ld.tile(g, t, src);
    const int r = src((wave & 3) * 64 + ln);
    sc_off = r >= 0 ? (uint32_t)r * (uint32_t)cols : kOOB;
  };
  auto load_scales = [&](const Tile &t, int kc) {
    const int nd = min(kScaleChunk, cols - kc) >> 2;
    const u32x4_t rs =
        gathered ? make_rsrc(g.a_scale, (uint32_t)(g.a_rows * cols))
                 : make_rsrc(g.a_scale + ((int64_t)t.seg0 + t.q0) * cols, (uint32_t)(t.qvalid * cols));
    for (int w = wave >> 2; w < nd; w += 2)
      dma4(rs, lds_addr(&s_qs[w][(wave & 3) * 64]), sc_off + (uint32_t)(kc + 4 * w));
    if (wave == 0) {   // lane 4 w + b: dword w of scale row b
      const int p0 = t.pt * (GU ? BP / 2 : BP);
      const int mbs = scale_blocks((GU ? 2 : 1) * N);
      const int b = lane & 3, w = lane >> 2;
      const int first = GU && b > 0 ? (N + p0) / kBlk + b - 1 : p0 / kBlk + b;
      const bool in = first < mbs && w < nd;
      dma4(make_rsrc(g.b_scale + (int64_t)t.e * mbs * cols, (uint32_t)(mbs * cols)),
           lds_addr(s_ps), in ? (uint32_t)(first * cols + kc + 4 * w) : kOOB);
    }
  };

  // ---- fragments
  const int lr = lane & 31, lg = lane >> 5;
  int prow[FP];   // first row in the tile: fragments 0, 1 in half 0, fragments 2, 3 in half 1
#pragma unroll
  for (int i = 0; i < FP; ++i) prow[i] = (i >> 1) * 128 + wp * 64 + 32 * (i & 1);
  // Q fragment j: rows 32 wq + 128 j, so that a tile's last rows are spread
  // over the SIMDs
  const int qrow0 = wq * 32;
  const LDS_AS char *lds = (const LDS_AS char *)smem;
  // lane's first chunk of the first 64 k: row lr, chunk lg; of the others:
  // chunk bit 2; the fragment's second chunk: bit 1
  const uint32_t at0 = (uint32_t)lr * 128u + (uint32_t)((lg ^ ((lr >> 1) & 7)) * 16);
  Tile t = take();
  if (t.e >= g.E) return;
  if (gathered) load_slots(t);
  wait_vm<0>();
  __syncthreads();
  set_tile(t);
  ld.issue(0, 0);
  load_scales(t, 0);
  wait_vm<0>();
  for (;;) {
    const Tile tn = take();
    const bool more = tn.e < g.E;
    f32x16_t acc[FP][FQ];
#pragma unroll
    for (int i = 0; i < FP; ++i)
#pragma unroll
      for (int j = 0; j < FQ; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
    const int p0 = t.pt * (GU ? BP / 2 : BP);
    // scale rows of the P fragments: gate/up, one for the gate rows and one for
    // each fragment of up rows; else one for each half of the tile
    int pblk[NSP];
#pragma unroll
    for (int i = 0; i < NSP; ++i) pblk[i] = GU && i > 0 ? p_block<GU, BP>(g, p0, prow[i + 1] + lr) : i;
    // every wave's loads of stage 0 and the scales have landed (it waited for
    // them), and every wave is done with the epilogue's slots
    wait_lgkm();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    // (what a spill brings back has to be here before the loop: a wait for it
    // among the stages would wait for all loads)
    ld.keep();
    uint32_t at_keep = at0;
    asm volatile("" : "+v"(at_keep));
    if (more && gathered) load_slots(tn);
    ld.issue(128, L::STAGE);

    i32x8_t pf[2][2], qf[FQ][2];   // [row fragment][first or last 64 k]
    auto read_p = [&](int h, int i, int s, uint32_t at) {
      pf[i][s] = frag(lds + L::ROWS + prow[2 * h + i] * 128, at ^ (s ? 64u : 0u), 32u);
    };
    auto read_q = [&](int j, int s, uint32_t at) {
      qf[j][s] = frag(lds + (qrow0 + 128 * j) * 128, at ^ (s ? 64u : 0u), 32u);
    };
    // scales: of the stage at hand in the lowest byte, of the next ones above it
    uint32_t sp[NSP], sq[FQ], sp4[NSP], sq4[FQ];
    auto scales = [&](int n) {
      const int w = ((unsigned)n % kScaleChunk) >> 2;
#pragma unroll
      for (int i = 0; i < NSP; ++i) sp4[i] = s_ps[w][pblk[i]];
#pragma unroll
      for (int j = 0; j < FQ; ++j) sq4[j] = s_qs[w][qrow0 + 128 * j + lr];
    };
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int j = 0; j < FQ; ++j) read_q(j, s, at0);
#pragma unroll
      for (int i = 0; i < 2; ++i) read_p(0, i, s, at0);
    }
    scales(0);
#pragma unroll
    for (int i = 0; i < NSP; ++i) sp[i] = sp4[i];
#pragma unroll
    for (int j = 0; j < FQ; ++j) sq[j] = sq4[j];
    // NL: the wave's Q fragments that hold rows
    auto run = [&](auto nl) {
      constexpr int NL = decltype(nl)::value;
      uint32_t at = at_keep, k0 = 256;   // stage n's place; byte of stage n + 2
      auto mfma = [&](int h, int i, int s) {
#pragma unroll
        for (int j = 0; j < NL; ++j)
          acc[2 * h + i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              pf[i][s], qf[j][s], acc[2 * h + i][j], 0, 0, 0, (int)sp[GU ? (h ? i + 1 : 0) : h], 0, (int)sq[j]);
      };
      // What the next half reads has landed everywhere (8 younger loads are on
      // their way), and what this half was read from is free.
      auto publish = [&]() {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        wait_vm<8>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
      };
      for (int n = 0;;) {
        const int end = min(nk, (n / kScaleChunk + 1) * kScaleChunk);
        // (no branch in the body: the compiler would move MFMAs over it)
        for (; n < end; ++n) {
          const uint32_t buf = n & 1 ? L::STAGE : 0u;
          // half 0; half 1's P fragments follow; Q rows and P half 0 of stage n + 2
          mfma(0, 0, 0);
          mfma(0, 1, 0);
          publish();
          read_p(1, 0, 0, at);
          read_p(1, 1, 0, at);
          ld.front(0, k0, buf);
          ld.front(1, k0, buf);
          __builtin_amdgcn_sched_barrier(0);
          mfma(0, 0, 1);
          ld.front(2, k0, buf);
          ld.front(3, k0, buf);
          __builtin_amdgcn_sched_barrier(0);
          read_p(1, 0, 1, at);
          mfma(0, 1, 1);
          ld.front(4, k0, buf);
          ld.front(5, k0, buf);
          __builtin_amdgcn_sched_barrier(0);
          read_p(1, 1, 1, at);
          // half 1; stage n + 1's half 0 and Q fragments follow; P half 1 of stage n + 2
          at ^= L::STAGE;
          mfma(1, 0, 0);
          mfma(1, 1, 0);
          publish();
          scales(n + 1);
          read_q(0, 0, at);
          read_q(1, 0, at);
          read_p(0, 0, 0, at);
          read_p(0, 1, 0, at);
          ld.p(1, 0, k0, buf);
          __builtin_amdgcn_sched_barrier(0);
          mfma(1, 0, 1);
          ld.p(1, 1, k0, buf);
          __builtin_amdgcn_sched_barrier(0);
          read_p(0, 0, 1, at);
          mfma(1, 1, 1);
          __builtin_amdgcn_sched_barrier(0);
          read_p(0, 1, 1, at);
          read_q(0, 1, at);
          read_q(1, 1, at);
          k0 += 128;
          const bool fresh = ((n + 1) & 3) == 0;
#pragma unroll
          for (int i = 0; i < NSP; ++i) sp[i] = fresh ? sp4[i] : sp[i] >> 8;
#pragma unroll
          for (int j = 0; j < FQ; ++j) sq[j] = fresh ? sq4[j] : sq[j] >> 8;
        }
        if (n >= nk) break;
        wait_lgkm();
        __builtin_amdgcn_s_barrier();
        load_scales(t, n);
        wait_vm<0>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        scales(n);
#pragma unroll
        for (int i = 0; i < NSP; ++i) sp[i] = sp4[i];
#pragma unroll
        for (int j = 0; j < FQ; ++j) sq[j] = sq4[j];
      }
    };
    const int nlive = (t.qvalid > qrow0) + (t.qvalid > qrow0 + 128);
    if (nlive == 2) run(std::integral_constant<int, 2>{});
    else if (nlive == 1) run(std::integral_constant<int, 1>{});
    else run(std::integral_constant<int, 0>{});

    // Epilogue.  The lane number is taken anew: addresses kept over the main
    // loop would not fit its registers.
    int ln = lane;
    asm volatile("" : "+v"(ln));
    const int er = ln & 31, eg = ln >> 5;
    const int64_t r0 = (int64_t)t.seg0 + t.q0;
    float w[FQ];   // row weights, asked for before the next tile's loads
    if (!GU) {
#pragma unroll
      for (int j = 0; j < FQ; ++j) {
        const int q = qrow0 + 128 * j + er;
        w[j] = g.row_scale && q < t.qvalid ? g.row_scale[r0 + q] : 1.0f;
      }
    }
    // every wave is done with the ring (the empty stages' zeros too) and the scales
    asm volatile("" ::: "memory");
    wait_vm<0>();
    __builtin_amdgcn_s_barrier();
    if (!GU) asm volatile("" : "+v"(w[0]), "+v"(w[1]) : : "memory");
    asm volatile("" ::: "memory");
    if (more) {
      set_tile(tn);
      ld.issue(0, 0);
      load_scales(tn, 0);
    }

    // Lane holds D[8 (v / 4) + 4 (lane / 32) + v % 4][lane % 32] of each fragment;
    // the results go through the wave's own slot in the ring's second place,
    // so that the stores are 16 bytes per lane.
    LDS_AS char *const slot = (LDS_AS char *)smem + L::STAGE + wave * (L::STAGE / NW);
    if constexpr (GU) {
      constexpr int PITCH = 64 + 16;
#pragma unroll
      for (int j = 0; j < FQ; ++j) {
        float m = 0.0f;
        if (j < nlive) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int v = 0; v < 16; ++v) {
              const float h = swiglu(acc[i][j][v], acc[i + 2][j][v]);
              acc[i][j][v] = h;
              m = fmaxf(m, fabsf(h));   // a NaN is passed over
            }
          // an infinity is passed over too, and turned to NaN: the rare case
          // costs a second pass over the values
          if (__any(m > 3.402823466e38f)) {
            m = 0.0f;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int v = 0; v < 16; ++v) {
                m = fmaxf(m, finite_abs(acc[i][j][v]));
                acc[i][j][v] = scaled(acc[i][j][v], 1.0f);
              }
          }
          m = fmaxf(m, __shfl_xor(m, 32, 64));
        }
        if (ln < 32) s_amax[wp][qrow0 + 128 * j + ln] = m;
      }
      wait_lgkm();
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      const int hcols = scale_cols(N);
#pragma unroll
      for (int j = 0; j < FQ; ++j) {
        if (j >= nlive) continue;
        const int q = qrow0 + 128 * j + er;
        const uint32_t byte = scale_byte(fmaxf(s_amax[0][q], s_amax[WP - 1][q]));
        const float inv = inv_scale(byte);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int v = 0; v < 16; v += 4)
            *reinterpret_cast<LDS_AS uint32_t *>(slot + er * PITCH + 32 * i + 2 * v + 4 * eg) =
                pack_e4m3x4(acc[i][j][v] * inv, acc[i][j][v + 1] * inv, acc[i][j][v + 2] * inv,
                            acc[i][j][v + 3] * inv);
        if (j == 0) wait_vm<0>();   // the next tile's loads; before the stores, which need not be waited for
        if (wp == 0 && eg == 0 && q < t.qvalid) {
          g.h_scale[(r0 + q) * hcols + t.pt] = (uint8_t)byte;
          if (t.pt == g.PT - 1)
            for (int b = t.pt + 1; b < hcols; ++b) g.h_scale[(r0 + q) * hcols + b] = 127;
        }
#pragma unroll
        for (int rr = 0; rr < 32; rr += 16) {   // 4 lanes x 16 bytes per row
          const int row = rr + (ln >> 2), ch = ln & 3;
          const u32x4_t val = *reinterpret_cast<const LDS_AS u32x4_t *>(slot + row * PITCH + 16 * ch);
          const int qq = qrow0 + 128 * j + row, n = p0 + wp * 64 + 16 * ch;
          if (qq < t.qvalid && n < N) *reinterpret_cast<u32x4_t *>(g.h + (r0 + qq) * N + n) = val;
        }
      }
    } else {
      // rows of 256 bytes, chunk c of 16 bytes at place c ^ (row & 15)
#pragma unroll
      for (int j = 0; j < FQ; ++j) {
        if (j >= nlive) continue;
#pragma unroll
        for (int i = 0; i < FP; ++i)
#pragma unroll
          for (int v = 0; v < 16; v += 4)
            *reinterpret_cast<LDS_AS u32x2_t *>(slot + er * 256 + ((4 * i + v / 4) ^ (er & 15)) * 16 + 8 * eg) =
                u32x2_t{pack_bf16x2(w[j] * acc[i][j][v], w[j] * acc[i][j][v + 1]),
                        pack_bf16x2(w[j] * acc[i][j][v + 2], w[j] * acc[i][j][v + 3])};
        if (j == 0) wait_vm<0>();   // the next tile's loads; before the stores, which need not be waited for
#pragma unroll
        for (int rr = 0; rr < 32; rr += 4) {   // 16 lanes x 16 bytes per row
          const int row = rr + (ln >> 4), ch = ln & 15;
          const u32x4_t val =
              *reinterpret_cast<const LDS_AS u32x4_t *>(slot + row * 256 + (ch ^ (row & 15)) * 16);
          const int qq = qrow0 + 128 * j + row, n = p0 + wp * 64 + (ch >> 3) * 128 + (ch & 7) * 8;
          // (written once, read by another kernel: kept out of the way of the weights in L2)
          if (qq < t.qvalid && n < N)
            __builtin_nontemporal_store(val, reinterpret_cast<u32x4_t *>(g.c + (r0 + qq) * N + n));
        }
      }
    }
    if (nlive == 0) wait_vm<0>();
    if (!more) break;
    t = tn;
  }
}

// Few rows per expert, where the weights' way from memory bounds (64 tokens, 4
// of 32 experts, d = f = 2880: 531 MB of gate/up weights in 96 us), and few
// tiles, where one tile's latency does: tiles of BP weight rows (gate/up: 128
// gate and 128 up, one block of h) and 64 rows, a block of threads each, over
// all of K with NS - 1 stages on their way.  NW waves side by side along the
// weight rows, 16 x 16 fragments (MFMA 16x16x128, one per stage and fragment
// pair; fragments past the expert's last row are left out).  The gate/up
// product of few rows converts its fragments to bf16 (the rounding of h, at the
// top); that costs 24.8 -> 28.3 us at one token, 92 -> 96 at 64.
//
// One CU draws about 50 GB/s from memory however much it has on its way, so
// few rows want many tiles: d = f = 2880, 32 experts, BP = 64 against 128, down
// product: 28 against 30 us at 4 tokens, 49 against 53 at 16, 57 against 58 at
// 64 (265 MB: 4.7 TB/s).  More rows want more work per byte loaded: 1024 rows,
// 8 experts, 608 x 608: 9.1 and 9.4 us; 4096 rows: 15.7 and 11.8 us.
template <bool GU, int BP, int NS, int NW, bool LATE, bool ONCE>
__global__ __launch_bounds__(NW * 64) void k_grouped_fp8_small(Fp8Args g) {
  constexpr int BQ = 64, FP = BP / NW / 16, FQ = BQ / 16;
  using L = Loads<GU, BP, BQ, NW, LATE, ONCE>;
  static_assert(!GU || BP == 256, "a gate/up tile holds one block of 128 h");
  constexpr bool EXACT = GU && ONCE;   // bf16 products, scales applied to their sums over a stage
  static_assert((NS - 2) * L::LOADS < 64, "vmcnt range");
  __shared__ u32x4_t smem[NS * (L::TP + L::TQ)];
  __shared__ uint32_t s_qs[kScaleChunk / 4][BQ];
  __shared__ uint32_t s_ps[kScaleChunk / 4][4];
  __shared__ float s_amax[GU ? NW : 1][GU ? BQ : 1];
  using Table = Tiles<BQ, 1>;
  static_assert(sizeof(Table) <= sizeof(smem), "the table shares the ring");
  Table &tiles = *reinterpret_cast<Table *>(smem);

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int N = g.N, nk = scale_blocks(g.K), cols = scale_cols(g.K);
  const bool gathered = g.row_to_slot != nullptr;

  tiles.init(g);
  const int total = tiles.total(g, 0), chunk = (total + 7) >> 3;
  const int id = (int)(blockIdx.x & 7) * chunk + (int)(blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= chunk || id >= total) return;
  const Tile t = tiles.decode(g, 0, id);
  __syncthreads();   // the table gives way to the ring
  const int p0 = t.pt * (GU ? BP / 2 : BP);
  const int lr = lane & 15, lg = lane >> 4;
  int prow[FP], pblk[FP];
#pragma unroll
  for (int i = 0; i < FP; ++i) {
    prow[i] = GU ? i * (BP / 2) + 16 * wave : 16 * (FP * wave + i);
    pblk[i] = p_block<GU, BP>(g, p0, prow[i]);   // 16 rows lie in one block: N is a multiple of 16
  }
  const LDS_AS char *lds = (const LDS_AS char *)smem;
  const uint32_t at0 = (uint32_t)lr * 128u + (uint32_t)((lg ^ ((lr >> 1) & 7)) * 16);
  L ld;
  ld.init(wave, lane, smem);

  auto src = [&](int r) -> int {   // row of a, -1 past the segment or for no token
    if (r >= t.qvalid) return -1;
    if (!gathered) return r;
    const uint32_t slot = (uint32_t)g.row_to_slot[(int64_t)t.seg0 + t.q0 + r];
    return slot < (uint64_t)g.slots ? (int)(((uint64_t)slot * g.kmagic) >> 32) : -1;
  };
  const int srow = src(lane);
  ld.tile(g, t, src);
  // Loads: whether the lane's weight rows (lr and multiples of 16) are late
  const bool late = L::late(g, ld.pbase + lr * g.K);
  auto load_scales = [&](int kc) {   // as in the wide kernel
    const int nd = min(kScaleChunk, cols - kc) >> 2;
    const u32x4_t rs =
        gathered ? make_rsrc(g.a_scale, (uint32_t)(g.a_rows * cols))
                 : make_rsrc(g.a_scale + ((int64_t)t.seg0 + t.q0) * cols, (uint32_t)(t.qvalid * cols));
    for (int w = wave; w < nd; w += NW)
      dma4(rs, lds_addr(&s_qs[w][0]), srow >= 0 ? (uint32_t)srow * (uint32_t)cols + (uint32_t)(kc + 4 * w) : kOOB);
    if (wave == 0) {
      const int mbs = scale_blocks((GU ? 2 : 1) * N);
      const int b = lane & 3, w = lane >> 2;
      const int first = GU && b > 0 ? (N + p0) / kBlk + b - 1 : p0 / kBlk + b;
      dma4(make_rsrc(g.b_scale + (int64_t)t.e * mbs * cols, (uint32_t)(mbs * cols)), lds_addr(s_ps),
           first < mbs && w < nd ? (uint32_t)(first * cols + kc + 4 * w) : kOOB);
    }
  };
  load_scales(0);
  if (LATE) ld.pre(g, (NS - 1) * L::STAGE);
#pragma unroll
  for (int n = 0; n < NS - 1; ++n) ld.issue(128u * n, n * L::STAGE);
  f32x4_t acc[FP][FQ];
#pragma unroll
  for (int i = 0; i < FP; ++i)
#pragma unroll
    for (int j = 0; j < FQ; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  uint32_t buf = 0, last = (NS - 1) * L::STAGE;   // places of stage n and of stage n + NS - 1
  const int nlive = (t.qvalid + 15) >> 4;
  auto half = [&](uint32_t at) { return *reinterpret_cast<const LDS_AS u32x4_t *>(lds + at); };
  u32x4_t old[FP];   // second half of the last stage: of late rows, the first 64 k of this one
  if constexpr (LATE) {
    asm volatile("" ::: "memory");
    wait_vm<(NS - 1) * L::LOADS>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = 0; i < FP; ++i) old[i] = half((prow[i] * 128 + last + at0) ^ 64u);
  }
  for (int n = 0; n < nk; ++n) {
    if (n > 0 && n % kScaleChunk == 0) {
      wait_lgkm();
      __builtin_amdgcn_s_barrier();
      load_scales(n);
      wait_vm<0>();
    }
    // stage n (and the scales, before it) has landed everywhere and stage n - 1 is read
    asm volatile("" ::: "memory");
    wait_vm<(NS - 2) * L::LOADS>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    ld.issue(128u * (n + NS - 1), last);
    const int w = (n % kScaleChunk) >> 2, sh = (n & 3) * 8;
    i32x8_t pf[FP];
    uint32_t sp[FP];
#pragma unroll
    for (int i = 0; i < FP; ++i) {
      const uint32_t at = prow[i] * 128 + buf + at0;
      const u32x4_t lo = half(at), hi = half(at ^ 64u);
      const u32x4_t a = LATE && late ? old[i] : lo, b = LATE && late ? lo : hi;
      old[i] = hi;
      pf[i] = i32x8_t{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
      sp[i] = s_ps[w][pblk[i]] >> sh;
    }
    bf16x8_t pb[EXACT ? FP : 1][4];
    if constexpr (EXACT)
#pragma unroll
      for (int i = 0; i < FP; ++i)
#pragma unroll
        for (int m = 0; m < 4; ++m) pb[i][m] = as_bf16(pf[i], m);
#pragma unroll
    for (int j = 0; j < FQ; ++j) {
      if (j < nlive) {
        const i32x8_t qf = frag(lds + L::TP * 16 + 16 * j * 128, buf + at0, 64u);
        const uint32_t sq = s_qs[w][16 * j + lr] >> sh;
        if constexpr (EXACT) {
          f32x4_t part[FP];
#pragma unroll
          for (int i = 0; i < FP; ++i) part[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const bf16x8_t qb = as_bf16(qf, m);
#pragma unroll
            for (int i = 0; i < FP; ++i)
              part[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pb[i][m], qb, part[i], 0, 0, 0);
          }
#pragma unroll
          for (int i = 0; i < FP; ++i)
#pragma unroll
            for (int v = 0; v < 4; ++v)
              acc[i][j][v] += ldexpf(part[i][v], (int)(sp[i] & 255u) + (int)(sq & 255u) - 254);
        } else {
#pragma unroll
          for (int i = 0; i < FP; ++i)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                pf[i], qf, acc[i][j], 0, 0, 0, (int)sp[i], 0, (int)sq);
        }
      }
    }
    buf = buf == (NS - 1) * L::STAGE ? 0u : buf + L::STAGE;
    last = last == (NS - 1) * L::STAGE ? 0u : last + L::STAGE;
  }
  asm volatile("" ::: "memory");
  wait_vm<0>();
  __builtin_amdgcn_s_barrier();   // every wave is done with the ring and the scales
  asm volatile("" ::: "memory");

  // Epilogue.  Lane holds D[4 lg + v][lr] of each fragment.
  const int64_t r0 = (int64_t)t.seg0 + t.q0;
  if constexpr (GU) {
#pragma unroll
    for (int j = 0; j < FQ; ++j) {
      float m = 0.0f;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        acc[0][j][v] = swiglu(acc[0][j][v], acc[1][j][v]);
        m = fmaxf(m, finite_abs(acc[0][j][v]));
      }
      m = fmaxf(m, __shfl_xor(m, 16, 64));
      m = fmaxf(m, __shfl_xor(m, 32, 64));
      if (lane < 16) s_amax[wave][16 * j + lane] = m;
    }
    wait_lgkm();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    const int hcols = scale_cols(N);
#pragma unroll
    for (int j = 0; j < FQ; ++j) {
      const int q = 16 * j + lr;
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < NW; ++i) m = fmaxf(m, s_amax[i][q]);
      const uint32_t byte = scale_byte(m);
      const float inv = inv_scale(byte);
      if (q < t.qvalid) {
        const int n = p0 + prow[0] + 4 * lg;
        if (n < N)
          *reinterpret_cast<uint32_t *>(g.h + (r0 + q) * N + n) =
              pack_e4m3x4(scaled(acc[0][j][0], inv), scaled(acc[0][j][1], inv),
                          scaled(acc[0][j][2], inv), scaled(acc[0][j][3], inv));
        if (wave == 0 && lg == 0) {
          g.h_scale[(r0 + q) * hcols + t.pt] = (uint8_t)byte;
          if (t.pt == g.PT - 1)
            for (int b = t.pt + 1; b < hcols; ++b) g.h_scale[(r0 + q) * hcols + b] = 127;
        }
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < FQ; ++j) {
      const int q = 16 * j + lr;
      if (q >= t.qvalid) continue;
      const float w = g.row_scale ? g.row_scale[r0 + q] : 1.0f;
#pragma unroll
      for (int i = 0; i < FP; ++i) {
        const int n = p0 + prow[i] + 4 * lg;
        if (n < N)
          *reinterpret_cast<u32x2_t *>(g.c + (r0 + q) * N + n) =
              u32x2_t{pack_bf16x2(w * acc[i][j][0], w * acc[i][j][1]),
                      pack_bf16x2(w * acc[i][j][2], w * acc[i][j][3])};
      }
    }
  }
}

// Rows per expert (on average, of those that can have rows) up to which the
// weights bound.  d = f = 2880, 32 experts, gate/up + down, small tiles (BP =
// 64) against the wide kernel: 95 + 56 us against 107 + 66 at 8 rows, 102 + 60
// against 108 + 67 at 16, 112 + 64 against 110 + 68 at 24, 116 + 67 against
// 110 + 69 at 32, 120 + 72 against 112 + 69 at 40.
template <bool GU>
constexpr int64_t kFewRows = GU ? 20 : 32;
constexpr int kCUs = 256;   // persistent kernels: one block of threads per CU, a multiple of 8

template <bool GU, int BP, int NS, int NW, bool LATE, bool ONCE>
int launch_small(Fp8Args g, int64_t active, const char *name, const char *fn, hipStream_t s) {
  constexpr int per = GU ? BP / 2 : BP;
  g.PT = (g.N + per - 1) / per;
  // an expert ends with a partial tile at most
  const int64_t tiles = (g.slots / 64 + active) * g.PT;
  MOE_REQUIRE(tiles < ((int64_t)1 << 30), MOE_ERR_UNSUPPORTED, "%s: too many tiles", fn);
  const unsigned blocks = (unsigned)((tiles + 7) / 8 * 8);
  MOE_LAUNCH(name, s, (k_grouped_fp8_small<GU, BP, NS, NW, LATE, ONCE><<<blocks, NW * 64, 0, s>>>(g)));
  return check_launch(fn);
}

template <bool GU>
int product(const Fp8Args &args, const char *name, const char *fn, hipStream_t s) {
  Fp8Args g = args;
  const int64_t active = g.E < g.slots ? (int64_t)g.E : g.slots;   // experts with rows, at most
  if (g.slots <= kFewRows<GU> * active) {
    if constexpr (GU)
      if (g.K % 128 == 64) return launch_small<GU, 256, 3, 8, true, true>(g, active, name, fn, s);
    return launch_small<GU, GU ? 256 : 64, GU ? 3 : 4, GU ? 8 : 4, false, true>(g, active, name, fn, s);
  }
  // Many rows, but so few small tiles (counting half a tile of 64 rows lost per
  // expert) that all run at once: gate/up one, else two blocks of threads to a
  // CU.  Event times against the wide kernel's: 608 x 608, 8 experts, 2048 rows
  // (180 tiles) 12.8 against 17.7 us gate/up, (180) 9.5 against 15.8; 4096 rows
  // (340) 21.5 against 18.8 and (340) 11.8 against 16.4; 8192 rows (660) 18.4
  // against 17.9; 1024 rows, 4 experts, 2880 x 2880 (414) 51 against 42 and 27
  // against 37; 2048 rows (782) 44 against 39.
  const int64_t small = (g.slots / 64 + active / 2) * ((g.N + 127) / 128);
  if (small <= (GU ? kCUs : 2 * kCUs))
    return launch_small<GU, GU ? 256 : 128, 3, 8, false, false>(g, active, name, fn, s);
  const int per = GU ? 128 : 256;
  g.PT = (g.N + per - 1) / per;
  const int64_t tiles = (g.slots / 256 + active) * g.PT;
  MOE_REQUIRE(tiles < ((int64_t)1 << 30), MOE_ERR_UNSUPPORTED, "%s: too many tiles", fn);
  const unsigned blocks = (unsigned)min((tiles + 7) / 8 * 8, (int64_t)kCUs);
  MOE_LAUNCH(name, s, (k_grouped_fp8_wide<GU><<<blocks, 512, 0, s>>>(g)));
  return check_launch(fn);
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
  const int steps = R < kCUs * 16 ? 1 : scale_cols(K) / 4;
  const dim3 blocks((unsigned)min((R + 3) / 4, (int64_t)1 << 22), (unsigned)(scale_cols(K) / 4 / steps));
  if (dtype == MOE_BF16)
    MOE_LAUNCH("quant_rows_fp8", s,
               k_quant_rows<bf16_t><<<blocks, 256, 0, s>>>((const bf16_t *)x, R, K, q, scale,
                                                      steps));
  else
    MOE_LAUNCH("quant_rows_fp8", s,
               k_quant_rows<float><<<blocks, 256, 0, s>>>((const float *)x, R, K, q, scale,
                                                     steps));
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
