// b2, b3. Products of 4-bit matrices on the sm_100a tensor cores (hinm.h): one matrix by
// another, by expert over ragged columns, and by expert over a ragged depth.
//
//   Y[m][n] = act(gA gB sum_k A[m][k] B[n][k] + bias[m])
//
// where A[m][k] = code * block scale.  tcgen05.mma multiplies e2m1 codes with their block
// scales, 64 of the depth an instruction, and accumulates in fp32 in tensor memory.  Both
// operands are stored row by row with the depth contiguous, as the instruction takes them
// (K-major), and the scales in the 512-byte chunks that tcgen05.cp spreads over the lanes.
//
// The product is symmetric in its operands, so the kernel speaks of P, whose rows are the
// accumulator's 128 lanes, and Q, whose rows are its columns.  A lane's columns are contiguous
// in Y as [P][Q] and go out of registers in 32-byte stores.  Y [M][N] takes P = A; the
// transposed Y [N][M] takes P = B (the tokens) once there are tokens enough to fill lanes, and
// P = A with Y written as [Q][P] (a warp's lanes along M) for a few.
//
// A persistent CTA walks tiles of 128 rows of P by BN rows of Q.  Warps:
//   0      copies: per stage of 256 of the depth, TMA boxes of P and Q (128-byte rows, 128-byte
//          swizzle) and the chunks of their scales
//   1      MMA: scales to tensor memory, then up to four products a stage
//   2..9   epilogue: 32 lanes of the accumulator and half of its columns each, 32 or 64 columns
//          at a time, through a tile in shared memory, so that Y is written in whole 128-byte
//          lines
// What bounds it, measured at 4096 x 4096 x 16384 (pairs): NV takes 115.6 us, MX 104.0, and copies of
// this kernel with parts left out 109 and 103.7 (no copies of scales), 109 and 90.7 (no loads), 90 and
// 83.5 (neither).  A stage of 256 x 256 x 256 is 542 cycles of products at the nominal rate and takes
// 830 (NV) and 740 (MX): the instructions that issue it, the 12 (6) scale copies among them, and 39 (36)
// KB a stage into each SM's shared memory bind together.  At 11008 x 4096 x 4096 with SiLU the tensor
// cores are busy for 44% of the time: a pair has one accumulator, and between two tiles it changes hands.
// The scales of a stage wait in a slot of tensor-memory columns, which is written again only
// after the products that read it are done (the commit that frees their stage).  With few
// tiles a cluster shares one tile's depth (SPLIT): each CTA leaves its partial sums in its own
// shared memory, and each adds a share of the columns over all of them in rank order, so that
// the result does not depend on timing.  Every wait is bounded (ptx.cuh); after one runs out
// the CTA stops, drains what it issued and returns.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include <mutex>
#include <type_traits>

#include "fp4.cuh"
#include "hinm_internal.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace hinm {
namespace {

constexpr int kStageDepth = 256;  // of the depth in one stage: 128-byte rows

// One side of the product.
struct Side {
  const uint8_t* scales;
  int tiles, chunks;        // scale tiles of one matrix; chunks of a tile
  int rows;                 // of one matrix
  int batched;              // one matrix for each expert
  int ragged;               // its rows are the ragged tokens
};

struct MmArgs {
  Side p, q;
  const float* ga;  // tensor scales: of A (a_batched: one for each expert) and B, or null
  const float* gb;
  const float* bias;  // per row of A, for each expert
  const int32_t* offsets;
  void* Y;
  long long ldy, y_batch;  // elements
  int a_batched, a_rows;
  int depth, groups, ragged;
  int pt, qt;       // tiles of P and Q (of the side that is not ragged, and of both else)
  int steps;        // products of 64 over the whole depth (unless ragged depth)
  int split;        // CTAs that share a tile's depth
  int dtype, act;
  int q_major;      // Y is [Q][P]: lanes along a row of Y
  int bias_q;       // the bias goes along Q
  int align;        // of Y's rows: a power of two, 32 at most
  int* status;
};

constexpr int kMaxSplit = 8;
constexpr int kEpiWarps = 8;
constexpr int kEpiCols = 16;  // columns that an epilogue warp takes at a time
constexpr int kEpiTile = 32 * 128;  // its staging tile: 32 rows of 128 bytes
constexpr int kEpiBytes = kEpiWarps * kEpiTile;

template <int FMT, int BN, bool PAIR>
struct MmCfg {
  static constexpr int kChunkDepth = 4 * fp4_block(FMT);
  static constexpr int kChunks = kStageDepth / kChunkDepth;  // scale chunks a stage
  static constexpr int kQTiles = BN > 128 ? 2 : 1;           // scale tiles of a Q tile
  // rows of one copy of Q: a tile takes as many as it has rows for; few tokens cost few bytes
  static constexpr int kQBox = PAIR ? BN / 2 : BN == 64 ? 16 : 64;
  static constexpr int kPBytes = 128 * 128;
  static constexpr int kPRows = PAIR ? 256 : 128;            // rows of a P tile
  static constexpr int kQBytes = (PAIR ? BN / 2 : BN) * 128; // a pair holds half of Q in each CTA
  static constexpr int kSfTile = kChunks * kFp4ChunkBytes;
  static constexpr int kSfBytes = (1 + kQTiles) * kSfTile;
  static constexpr int kStageBytes = kPBytes + kQBytes + kSfBytes;
  static constexpr int kAccBufs = BN <= 192 ? 2 : 1;
  static constexpr int kAccCols = BN;
  static constexpr int kSfCols = kChunks * 4 * (1 + kQTiles);
  // 1024 for alignment, 256 of barriers, the table of groups
  static constexpr size_t kOtherBytes = 1024 + kEpiBytes + 256 + (kFp4MaxGroups + 1) * 4;
  static constexpr int kStagesRaw = (int)((227 * 1024 - kOtherBytes) / kStageBytes);
  static constexpr int kStages = kStagesRaw > 8 ? 8 : kStagesRaw;
  static constexpr int kSlotsRaw = (512 - kAccBufs * kAccCols) / kSfCols;
  static constexpr int kSlots = kSlotsRaw > kStages ? kStages : kSlotsRaw;
  static_assert(kStages >= 2 && kSlots >= 2, "stages");
  static constexpr size_t kSmemBytes = (size_t)kStages * kStageBytes + kOtherBytes;
};
constexpr int kMmThreads = 64 + 32 * kEpiWarps;

// One tile of work.
struct Tile {
  int e;                       // expert, 0 without groups
  int p_row, q_row;            // first rows among all stored rows of P and Q
  int p_len, q_len;            // rows that count
  int p_out, q_out;            // their places in Y
  int p_tile, q_tile;          // scale tiles of the first rows
  int q_shift;                 // place of Q's first row in its scale tile (0 or 64)
  int k0;                      // first stored depth
  int steps;                   // products of 64
};

// cum: ragged rows: tiles of the ragged side before each group
// PR: rows of a P tile (128, or 256 of which rank 1 of a pair takes the upper half)
template <int BN, int PR>
__device__ __forceinline__ Tile tile_of(const MmArgs& a, const int* cum, int t, int pr) {
  Tile r;
  r.e = 0;
  r.k0 = 0;
  r.steps = a.steps;
  int pi, qi;  // tile indexes of P and Q
  int o = 0, end = 0;
  if (a.ragged == HINM_RAGGED_ROWS) {
    // tiles of one ragged tile stay together: its tokens are read once
    const int other = a.p.ragged ? a.qt : a.pt;
    const int u = t / other, v = t - u * other;
    int lo = 0, hi = a.groups - 1;  // the last group with cum[e] <= u: empty ones share a start
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (cum[mid] <= u) lo = mid;
      else hi = mid - 1;
    }
    r.e = lo;
    pi = a.p.ragged ? u - cum[lo] : v;
    qi = a.p.ragged ? v : u - cum[lo];
    o = __ldg(a.offsets + lo);
    end = __ldg(a.offsets + lo + 1);
  } else {
    if (a.ragged == HINM_RAGGED_DEPTH) {
      const int per = a.pt * a.qt;
      r.e = t / per;
      t -= r.e * per;
      o = __ldg(a.offsets + r.e);
      end = __ldg(a.offsets + r.e + 1);
      r.k0 = (int)fp4_group_tile(o, r.e) * kFp4DepthPad;
      r.steps = (end - o + kFp4DepthPad - 1) / kFp4DepthPad * 2;
    }
    qi = t / a.pt;
    pi = t - qi * a.pt;
  }
  const int p = pi * PR + pr * 128, q = qi * BN;
  r.q_shift = q % kFp4RowTile;
  if (a.p.ragged) {
    r.p_row = r.p_out = o + p;
    r.p_len = min(128, end - r.p_row);
    r.p_tile = (int)fp4_group_tile(o, r.e) + p / 128;
  } else {
    const int m = a.p.batched ? r.e : 0;
    r.p_row = m * a.p.rows + p;
    r.p_out = p;
    r.p_len = min(128, a.p.rows - p);
    r.p_tile = m * a.p.tiles + p / 128;
  }
  if (a.q.ragged) {
    r.q_row = r.q_out = o + q;
    r.q_len = min(BN, end - r.q_row);
    r.q_tile = (int)fp4_group_tile(o, r.e) + q / kFp4RowTile;
  } else {
    const int m = a.q.batched ? r.e : 0;
    r.q_row = m * a.q.rows + q;
    r.q_out = q;
    r.q_len = min(BN, a.q.rows - q);
    r.q_tile = m * a.q.tiles + q / kFp4RowTile;
  }
  return r;
}

// SiLU(x) = x / (1 + e^-x).  For outputs in 32 bits: h = e^(-x/2) is taken as 2^hi (1 + lo ln 2), where
// hi + lo is -x log2(e) / 2 with the constant in two parts and the product's residual, so that its error
// does not grow with |x|: 2^hi is 2^-22 off and two roundings follow, h^2 is off by twice that, the
// reciprocal by 2^-23, and with the sum's and the product's roundings SiLU(x) is within 2^-20 of itself.
// The fraction is scaled by 2^-32, so that nothing overflows before SiLU(x) is below 2^-149.
constexpr float kSiluHalf = -0.72134752f, kSiluRest = -9.6298149e-9f;
constexpr float kTwo32 = 2.3283064365386963e-10f;  // 2^-32
__device__ __forceinline__ float silu(float x) {
  const float y = fminf(x, 128.0f);  // (an infinity has no residual)
  const float hi = y * kSiluHalf;
  const float lo = fmaf(y, kSiluRest, fmaf(y, kSiluHalf, -hi));
  const float h = ptx::ex2(hi) * fmaf(lo, 0.69314718f, 1.0f);
  return x * (ptx::rcp(fmaf(h * kTwo32, h, kTwo32)) * kTwo32);
}
// Two at once, in packed instructions: 4096 x 4096 x 512 25.8 us, one by one 30.5.  (Where the columns are
// held in registers, the pairs' kernel, they cost more than they save: 11008 x 4096 x 4096 105 us, one by
// one 100, with the quick exponential 95.5.)
__device__ __forceinline__ void silu2(float& xa, float& xb) {
  using ptx::F2;
  const F2 y(fminf(xa, 128.0f), fminf(xb, 128.0f));
  const F2 half(kSiluHalf, kSiluHalf), two32(kTwo32, kTwo32);
  const F2 hi = ptx::mul2(y, half);
  const F2 lo = ptx::fma2(y, F2(kSiluRest, kSiluRest),
                          ptx::fma2(y, half, ptx::mul2(hi, F2(-1.0f, -1.0f))));
  float a, b;
  hi.get(a, b);
  const F2 h = ptx::mul2(F2(ptx::ex2(a), ptx::ex2(b)),
                         ptx::fma2(lo, F2(0.69314718f, 0.69314718f), F2(1.0f, 1.0f)));
  ptx::fma2(ptx::mul2(h, two32), h, two32).get(a, b);
  ptx::mul2(F2(xa, xb), ptx::mul2(F2(ptx::rcp(a), ptx::rcp(b)), two32)).get(xa, xb);
}
// For outputs in 16 bits the error may grow with |x|: (20 + 1.4 |x|) 2^-24 of SiLU(x), which is less
// than an eightieth of what the store rounds as long as SiLU(x) is not 0 there.  (Scaled by 2^-16 for
// the same reason.  11008 x 4096 x 4096 86.3 us, as above 91.9.)
__device__ __forceinline__ float silu_quick(float x) {
  constexpr float k16 = 1.52587890625e-5f;  // 2^-16
  return x * (ptx::rcp(ptx::ex2(fmaf(x, -1.4426950408889634f, -16.0f)) + k16) * k16);
}
// GELU(x) = x Phi(x), Phi(-a) = erfc(a / sqrt 2) / 2 = e^(-a^2/2) w(t), t = 1 / (1 + 0.3 a): without a
// difference of nearly equal numbers for either sign (1 + erf(x / sqrt 2) has none of its digits right
// from -5.6 on).  An exponential times a polynomial in t is the form of Hastings (Approximations for
// Digital Computers, 1955); the coefficients are a fit of their own, in relative error over a <= 14.5
// (2^-24; 2^-21 as evaluated in fp32).  The exponential is the square of h = 2^(-a^2 log2(e) / 4), which
// is normal as long as GELU(x) is; with its argument's roundings the error is within (z^2 + 16) 2^-23 of
// GELU(z), in the tail twice what half a step of z makes.  Two at once, in packed instructions: 11008 x
// 4096 x 4096 bf16 92 us, one by one 107, with erff 120, with erfcf 256.  (One by one, fp32 products of
// short depth without any activation also took 4 to 6% longer: the registers that the kernel gives this
// part go short elsewhere.)
__device__ __forceinline__ void gelu2(float& xa, float& xb) {
  using ptx::F2;
  constexpr float kW[9] = {0.03840738907456398f,  -0.16930744051933289f, 0.22895173728466034f,
                           -0.07683960348367691f, 0.14276523888111115f,  0.09458588063716888f,
                           0.12194526195526123f,  0.11948420852422714f,  7.3723608693399e-06f};
  const F2 a(fabsf(xa), fabsf(xb));
  float u, v;
  ptx::fma2(a, F2(0.3f, 0.3f), F2(1.0f, 1.0f)).get(u, v);
  const F2 t(ptx::rcp(u), ptx::rcp(v));
  F2 w(kW[0], kW[0]);
#pragma unroll
  for (int i = 1; i < 9; ++i) w = ptx::fma2(w, t, F2(kW[i], kW[i]));
  ptx::mul2(ptx::mul2(a, a), F2(-0.36067376022224085f, -0.36067376022224085f)).get(u, v);
  const F2 h(ptx::ex2(u), ptx::ex2(v));
  ptx::mul2(ptx::mul2(w, h), h).get(u, v);
  xa *= xa < 0.0f ? u : 1.0f - u;
  xb *= xb < 0.0f ? v : 1.0f - v;
}
// PRECISE: for outputs in 32 bits.
template <int ACT, bool PRECISE>
__device__ __forceinline__ float activate(float x) {
  if constexpr (ACT == HINM_ACT_RELU) return ptx::max_nan(x, 0.0f);  // NaN stays NaN
  if constexpr (ACT == HINM_ACT_SILU) {
    return PRECISE ? silu(x) : silu_quick(x);
  }
  if constexpr (ACT == HINM_ACT_GELU) {
    float other = x;
    gelu2(x, other);
  }
  return x;
}
template <bool PRECISE>
__device__ __forceinline__ float activate(float x, int act) {
  switch (act) {
    case HINM_ACT_RELU: return activate<HINM_ACT_RELU, PRECISE>(x);
    case HINM_ACT_SILU: return activate<HINM_ACT_SILU, PRECISE>(x);
    case HINM_ACT_GELU: return activate<HINM_ACT_GELU, PRECISE>(x);
    default: return x;
  }
}
// a lane's columns; the kind of activation is asked once for all of them
template <int ACT, bool PRECISE, bool PAIRS = false>
__device__ __forceinline__ void activate_all(float (&y)[kEpiCols]) {
  if constexpr (ACT == HINM_ACT_SILU && PRECISE && PAIRS) {
#pragma unroll
    for (int i = 0; i < kEpiCols; i += 2) silu2(y[i], y[i + 1]);
  } else if constexpr (ACT == HINM_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < kEpiCols; i += 2) gelu2(y[i], y[i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < kEpiCols; ++i) y[i] = activate<ACT, PRECISE>(y[i]);
  }
}

__device__ __forceinline__ void store_one(void* Y, int dtype, long long at, float v) {
  if (dtype == HINM_DTYPE_F32) reinterpret_cast<float*>(Y)[at] = v;
  else if (dtype == HINM_DTYPE_BF16)
    reinterpret_cast<__nv_bfloat16*>(Y)[at] = __float2bfloat16_rn(v);
  else reinterpret_cast<__half*>(Y)[at] = __float2half_rn(v);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The power of two (32 at most) that the addresses of Y's elements `at`, `at + ldy`, ... are multiples
// of.
__device__ __forceinline__ int align_of(const MmArgs& a, long long at) {
  const int bits = (int)(at * (a.dtype == HINM_DTYPE_F32 ? 4 : 2)) | a.align;
  return min(32, bits & -bits);
}

// The tensor-core instructions, of one CTA or of a pair.
template <bool PAIR>
__device__ __forceinline__ void scale_copy(uint32_t taddr, uint64_t desc) {
  if constexpr (PAIR) ptx::tc_cp_32x128b_x4_pair(taddr, desc);
  else ptx::tc_cp_32x128b_x4(taddr, desc);
}
template <bool PAIR>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (PAIR) ptx::tc_commit_pair(bar);
  else ptx::tc_commit(bar);
}
template <int FMT, bool PAIR>
__device__ __forceinline__ void product(uint32_t acc, uint64_t pd, uint64_t qd, uint32_t idesc,
                                        uint32_t sfp, uint32_t sfq, uint32_t more) {
  if constexpr (FMT == HINM_FP4_NV && PAIR)
    ptx::mma_fp4_block16_pair(acc, pd, qd, idesc, sfp, sfq, more);
  else if constexpr (FMT == HINM_FP4_NV)
    ptx::mma_fp4_block16(acc, pd, qd, idesc, sfp, sfq, more);
  else if constexpr (PAIR)
    ptx::mma_fp4_block32_pair(acc, pd, qd, idesc, sfp, sfq, more);
  else
    ptx::mma_fp4_block32(acc, pd, qd, idesc, sfp, sfq, more);
}

// The warp's staging tile holds 32 rows of up to 128 bytes of Y in 16-byte pieces, piece p of row
// r at place p ^ (r & 7): neither a lane's writes to its row nor the reads of whole rows meet in a
// bank.
__device__ __forceinline__ uint32_t piece(uint32_t tile, int r, int p) {
  return tile + r * 128 + ((p ^ (r & 7)) << 4);
}

// The staging tile's first n columns of `rows` rows to Y, W bytes a lane: as many rows at a time as
// 32 lanes hold 128 bytes of (narrower stores the less Y's rows are aligned).
template <class Word>
__device__ __forceinline__ void write_units(uint32_t tile, int lane, int rows, int bytes, char* y0,
                                            long long pitch) {
  constexpr int W = (int)sizeof(Word);
  constexpr int kLanes = 128 / W < 32 ? 128 / W : 32;  // lanes that write one row
  constexpr int kRows = 32 / kLanes;
  const int r0 = lane / kLanes;
#pragma unroll 1
  for (int at = lane % kLanes * W; at < bytes; at += kLanes * W) {
#pragma unroll 1
    for (int i = 0; i < 32 / kRows && i * kRows < rows; i += 8) {
      Word v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int r = (i + j) * kRows + r0;
        if (i + j < 32 / kRows)
          v[j] = *reinterpret_cast<const Word*>(__cvta_shared_to_generic(
              piece(tile, r, at / 16) + at % 16));
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int r = (i + j) * kRows + r0;
        if (i + j < 32 / kRows && r < rows) *reinterpret_cast<Word*>(y0 + r * pitch + at) = v[j];
      }
    }
  }
}
__device__ __forceinline__ void write_tile(const MmArgs& a, uint32_t tile, int lane, int rows,
                                           int n, long long at0) {
  const int es = a.dtype == HINM_DTYPE_F32 ? 4 : 2;
  const int bytes = n * es, unit = align_of(a, at0) | (bytes & 15 ? bytes : 16);
  char* y0 = reinterpret_cast<char*>(a.Y) + at0 * es;
  const long long pitch = a.ldy * es;
  const int low = unit & -unit;  // the largest power of two that divides rows' places and lengths
  if (low >= 16) write_units<uint4>(tile, lane, rows, bytes, y0, pitch);
  else if (low == 8) write_units<uint2>(tile, lane, rows, bytes, y0, pitch);
  else if (low == 4) write_units<uint32_t>(tile, lane, rows, bytes, y0, pitch);
  else write_units<uint16_t>(tile, lane, rows, bytes, y0, pitch);
}

// N columns of the accumulator into registers (zero: there were no products).
template <int N>
__device__ __forceinline__ void read_columns(uint32_t acc, bool zero, uint32_t (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 32) {
    if (!zero) {
      ptx::tmem_ld_32x32b_x32(acc + i, reinterpret_cast<uint32_t(&)[32]>(v[i]));
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[i + j] = 0;
    }
  }
  ptx::tmem_ld_wait();
}

// What goes with a warp's columns of one tile.
struct Columns {
  float alpha, bias_row;
  const float* bias_cols;
  uint32_t tile;  // the warp's staging tile
  int lane;       // brings row `lane`
  int rows, cols; // how many count
  long long at0;  // element 0 of row 0 in Y
};

// PC columns (64 or 128 bytes of Y), from column `col` on, into the staging tile.
template <int DT, int PC, bool BIASQ, bool LINES, bool HELD, bool ACTS>
__device__ __forceinline__ void stage_columns(const MmArgs& a, const Columns& c, int col,
                                              const uint32_t* v) {
  constexpr int es = DT == HINM_DTYPE_F32 ? 4 : 2;
  const uint32_t in = c.tile + c.lane * 128 + ((c.lane & 7) << 4);  // this lane's row (piece())
#pragma unroll
  for (int h = 0; h < PC; h += kEpiCols) {
    float f[kEpiCols];
#pragma unroll
    for (int i = 0; i < kEpiCols; ++i)
      f[i] = fmaf(__uint_as_float(v[h + i]), c.alpha,
                  BIASQ ? __ldg(c.bias_cols + (LINES ? col + h + i : min(col + h + i, c.cols - 1)))
                        : c.bias_row);
    constexpr bool kPrecise = DT == HINM_DTYPE_F32;
    if (!ACTS || a.act == HINM_ACT_NONE) {
    } else if (a.act == HINM_ACT_RELU) activate_all<HINM_ACT_RELU, kPrecise>(f);
    else if (a.act == HINM_ACT_SILU) activate_all<HINM_ACT_SILU, kPrecise, !HELD>(f);
    else if (a.act == HINM_ACT_GELU) activate_all<HINM_ACT_GELU, kPrecise>(f);
#pragma unroll
    for (int i = 0; i < kEpiCols * es / 16; ++i) {
      uint32_t u[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        u[j] = DT == HINM_DTYPE_F32    ? __float_as_uint(f[4 * i + j])
               : DT == HINM_DTYPE_BF16 ? pack_bf16(f[8 * i + 2 * j], f[8 * i + 2 * j + 1])
                                       : pack_f16(f[8 * i + 2 * j], f[8 * i + 2 * j + 1]);
      ptx::st_shared_v4(in ^ (uint32_t)(h * es + 16 * i), u[0], u[1], u[2], u[3]);
    }
  }
}

// COLS columns that all count, of rows that are 32-byte aligned.  HOLD (one accumulator): all are
// read first, and `done` is called, so that the accumulator is free while they are worked on (pairs
// at 11008 x 4096 x 4096: 86.8 us, else 89.5; with two accumulators it costs registers for nothing:
// 4096 x 4096 x 1024 in 128 x 192 tiles 18.4 us, else 17.1).
template <int DT, int COLS, bool BIASQ, bool HOLD, bool ACTS, class Done>
__device__ __forceinline__ void write_lines(const MmArgs& a, uint32_t acc, bool zero,
                                            const Columns& c, Done done) {
  constexpr int es = DT == HINM_DTYPE_F32 ? 4 : 2;
  constexpr int PC = DT != HINM_DTYPE_F32 && COLS % 64 == 0 ? 64 : 32;
  constexpr int kLanes = PC * es / 32;  // lanes that write one row, 32 bytes each
  constexpr int kRows = 32 / kLanes;    // rows of one store
  uint32_t v[HOLD ? COLS : PC];
  if constexpr (HOLD) {
    read_columns<COLS>(acc, zero, v);
    done();
  }
  // what this lane writes out: its row's number mod 8 does not change from store to store
  const int r0 = c.lane / kLanes, p0 = (c.lane % kLanes) * 2;
  const uint32_t out = c.tile + r0 * 128 + ((p0 ^ (r0 & 7)) << 4);
  const long long pitch = a.ldy * es;
  char* yr = reinterpret_cast<char*>(a.Y) + c.at0 * es + r0 * pitch + p0 * 16;
#pragma unroll
  for (int col = 0; col < COLS; col += PC) {
    if constexpr (!HOLD) {
      read_columns<PC>(acc + col, zero, v);
      if (col + PC >= COLS) done();
    }
    stage_columns<DT, PC, BIASQ, true, HOLD, ACTS>(a, c, col, HOLD ? v + col : v);
    __syncwarp();
    char* yo = yr + col * es;
#pragma unroll
    for (int i = 0; i < 32 / kRows; ++i) {
      if (r0 + i * kRows < c.rows) {
        const uint4 u = ptx::ld_shared_v4(out + i * kRows * 128);
        const uint4 w = ptx::ld_shared_v4((out ^ 16) + i * kRows * 128);
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(yo), "r"(u.x),
                     "r"(u.y), "r"(u.z), "r"(u.w), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w)
                     : "memory");
      }
      yo += kRows * pitch;
    }
    __syncwarp();
  }
}

// Any columns and rows: read as they are worked on.  (The kernels of pairs, with write_lines' held columns,
// already keep 116 bytes of a thread, and 132 with the activations, outside of their 168 registers.)
template <int DT, int COLS, bool BIASQ, bool ACTS, class Done>
__device__ __forceinline__ void write_any(const MmArgs& a, uint32_t acc, bool zero,
                                          const Columns& c, Done done) {
  constexpr int PC = DT != HINM_DTYPE_F32 && COLS % 64 == 0 ? 64 : 32;
#pragma unroll 1
  for (int col = 0; col < c.cols; col += PC) {
    uint32_t v[PC];
    read_columns<PC>(acc + col, zero, v);
    if (col + PC >= c.cols) done();
    stage_columns<DT, PC, BIASQ, false, false, ACTS>(a, c, col, v);
    __syncwarp();
    write_tile(a, c.tile, c.lane, c.rows, min(PC, c.cols - col), c.at0 + col);
    __syncwarp();
  }
}

// Four consecutive elements of Y, n of them real, from element `at` on.
__device__ __forceinline__ void store_four(const MmArgs& a, const float (&y)[4], int n,
                                           long long at) {
  const int es = a.dtype == HINM_DTYPE_F32 ? 4 : 2;
  if (n >= 4 && a.align >= 16 && (at * es) % (4 * es) == 0) {
    if (a.dtype == HINM_DTYPE_F32)
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.Y) + at) =
          make_float4(y[0], y[1], y[2], y[3]);
    else
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.Y) + at) =
          a.dtype == HINM_DTYPE_BF16
              ? make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]))
              : make_uint2(pack_f16(y[0], y[1]), pack_f16(y[2], y[3]));
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q < n) store_one(a.Y, a.dtype, at + q, y[q]);
  }
}

// ACTS: with the activations' code.  The two larger tiles have a kernel without it for products that take
// none, since what it asks for in registers costs the rest: 16 experts' weight gradients of 2048 x 1024,
// 8111 tokens, 38.5 us, with it 40.6; a prompt's 16 products of 4096 x 2048 77.0 and 78.2.
template <int FMT, int BN, bool SPLIT, bool PAIR, bool ACTS>
__global__ void __launch_bounds__(kMmThreads, 1)
    fp4_mm_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                  const __grid_constant__ CUtensorMap tmSp, const __grid_constant__ CUtensorMap tmSq,
                  const MmArgs a) {
  static_assert(!(SPLIT && PAIR), "a cluster has one use");
  using C = MmCfg<FMT, BN, PAIR>;
  extern __shared__ uint8_t smem_raw[];
  if constexpr (PAIR) ptx::enter_dependent();
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* epi_smem = smem + C::kStages * C::kStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(epi_smem + kEpiBytes);
  // [0,S) full, [S,2S) empty, 2S+{0,1} accumulator full, 2S+{2,3} accumulator empty, 2S+4 drain
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * C::kStages + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* bad_flag = reinterpret_cast<volatile int*>(tmem_slot + 2);
  int* cum = reinterpret_cast<int*>(epi_smem + kEpiBytes + 256);
  // the same in every lane, and known to be
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  auto full_bar = [&](int s) { return ptx::smem_u32(bars + s); };
  auto empty_bar = [&](int s) { return ptx::smem_u32(bars + C::kStages + s); };
  auto accf_bar = [&](int b) { return ptx::smem_u32(bars + 2 * C::kStages + b); };
  auto acce_bar = [&](int b) { return ptx::smem_u32(bars + 2 * C::kStages + 2 + b); };
  const uint32_t drain_bar = ptx::smem_u32(bars + 2 * C::kStages + 4);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      ptx::mbar_init(full_bar(s), 1);
      ptx::mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(accf_bar(b), 1);
      ptx::mbar_init(acce_bar(b), (PAIR ? 2 : 1) * kEpiWarps);
    }
    ptx::mbar_init(drain_bar, 1);
    *abort_flag = 0;
    *bad_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      ptx::tmem_alloc_pair(ptx::smem_u32(tmem_slot), 512);
    } else {
      ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
      ptx::tmem_relinquish();
    }
  }
  if (lane == 0) {
    if (warp == 2) ptx::prefetch_map(&tmP);
    if (warp == 3) ptx::prefetch_map(&tmQ);
    if (PAIR && warp == 4) ptx::prefetch_map(&tmSp);
    if (PAIR && warp == 5) ptx::prefetch_map(&tmSq);
  }
  // What is above touches no global memory: it runs while the stream's previous kernel ends.
  if constexpr (!PAIR) ptx::enter_dependent();
  if (warp == 0) {
    if (a.ragged != HINM_RAGGED_NONE) {
      // offsets that decrease or leave the matrix are reported, and nothing is computed
      const int limit = a.ragged == HINM_RAGGED_DEPTH ? a.depth : a.p.ragged ? a.p.rows : a.q.rows;
      const int per = a.p.ragged ? C::kPRows : BN;
      int before = 0;
      bool bad = false;
      for (int base = 0; base < a.groups; base += 32) {
        const int e = base + lane;
        const int o = e < a.groups ? __ldg(a.offsets + e) : 0;
        const int end = e < a.groups ? __ldg(a.offsets + e + 1) : 0;
        bad |= o < 0 || end < o || end > limit;
        const int n = end > o ? (end - o + per - 1) / per : 0;
        int sum = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int up = __shfl_up_sync(0xFFFFFFFFu, sum, d);
          if (lane >= d) sum += up;
        }
        if (e < a.groups) cum[e] = before + sum - n;
        before += __shfl_sync(0xFFFFFFFFu, sum, 31);
      }
      bad = __any_sync(0xFFFFFFFFu, bad);
      if (lane == 0) {
        cum[a.groups] = before;
        if (bad) {
          *bad_flag = 1;
          ptx::record_status(a.status, HINM_ERR_INVALID_ARG);
        }
      }
    }
    __syncwarp();
  }
  ptx::tc_fence_before();
  if constexpr (PAIR) {
    ptx::cluster_sync();  // the barriers of both CTAs stand
  } else if (warp == 0) {
    // the copies need nothing of the other warps: they start while tensor memory is allocated
    asm volatile("barrier.cta.arrive 1, %0;" ::"n"(kMmThreads) : "memory");
  } else {
    asm volatile("barrier.cta.sync 1, %0;" ::"n"(kMmThreads) : "memory");
  }
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;  // not read by warp 0
  int tiles = a.pt * a.qt;
  if (a.ragged == HINM_RAGGED_ROWS) tiles = cum[a.groups] * (a.p.ragged ? a.qt : a.pt);
  if (a.ragged == HINM_RAGGED_DEPTH) tiles = a.groups * a.pt * a.qt;
  if (*bad_flag) tiles = 0;
  // SPLIT, Y as [P][Q]: row pitch of the partial sums, an odd number of 16-byte pieces
  constexpr int kPartRow = BN + 4;
  static_assert(!SPLIT || 128 * kPartRow * 4 <= C::kStages * C::kStageBytes, "partial sums");
  constexpr uint32_t kSfCol0 = C::kAccBufs * C::kAccCols;
  // SPLIT: a cluster takes one tile, rank r the stages [n r / split, n (r + 1) / split)
  // PAIR: a cluster of two takes a tile of 256 rows of P, rank r rows 128 r .. 128 r + 127
  const int first = SPLIT ? (int)blockIdx.x / a.split : PAIR ? (int)blockIdx.x / 2 : (int)blockIdx.x;
  const int step = SPLIT ? 0x40000000 : PAIR ? (int)gridDim.x / 2 : (int)gridDim.x;
  const int rank = SPLIT ? (int)blockIdx.x % a.split : PAIR ? (int)blockIdx.x % 2 : 0;
  auto tile_at = [&](int t) { return tile_of<BN, C::kPRows>(a, cum, t, PAIR ? rank : 0); };
  // columns of a tile's products: a pair's halves are whole groups of 16
  auto mma_n = [](int q_len) { return PAIR ? (q_len + 31) & ~31 : (q_len + 15) & ~15; };
  auto stage_range = [&](int steps, int& s0, int& s1) {
    const int n = (steps + 3) / 4;
    s0 = SPLIT ? n * rank / a.split : 0;
    s1 = SPLIT ? n * (rank + 1) / a.split : n;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ copies
    if (lane == 0) {
      uint32_t it = 0;
      bool stop = false;
      for (int t = first; t < tiles && !stop; t += step) {
        const Tile w = tile_at(t);
        const int c0 = w.k0 / C::kChunkDepth;
        const uint8_t* sp =
            a.p.scales + ((long long)w.p_tile * a.p.chunks + c0) * kFp4ChunkBytes;
        const uint8_t* sq =
            a.q.scales + ((long long)w.q_tile * a.q.chunks + c0) * kFp4ChunkBytes;
        const bool two = C::kQTiles == 2 && w.q_shift + w.q_len > kFp4RowTile;
        const int qb = (w.q_len + C::kQBox - 1) / C::kQBox;
        int s0, s1;
        stage_range(w.steps, s0, s1);
        for (int st = s0; st < s1; ++st, ++it) {
          const int s = it % C::kStages;
          if (!ptx::mbar_wait(empty_bar(s), ((it / C::kStages) & 1) ^ 1, a.status, abort_flag)) {
            stop = true;
            break;
          }
          const int left = min(4, w.steps - 4 * st);
          const uint32_t sf = (uint32_t)(left * 64 / C::kChunkDepth) * kFp4ChunkBytes;
          const uint32_t P_s = ptx::smem_u32(smem + s * C::kStageBytes);
          const uint32_t Q_s = P_s + C::kPBytes, S_s = Q_s + C::kQBytes;
          if constexpr (PAIR) {
            // whole stages in both CTAs (what a partial tile does not need goes unread), all
            // completing on rank 0's barrier; scales as boxes of the stage's chunks
            const uint32_t bar = ptx::mapa_shared(full_bar(s), 0);
            if (rank == 0) ptx::mbar_arrive_expect_tx(full_bar(s), 2 * C::kStageBytes);
            const int x = w.k0 / 2 + st * 128, q_row = w.q_row + rank * (mma_n(w.q_len) / 2);
            const int c = c0 + st * C::kChunks;
            ptx::tma_load_2d_pair(P_s, &tmP, x, w.p_row, bar);
            ptx::tma_load_2d_pair(Q_s, &tmQ, x, q_row, bar);
            ptx::tma_load_2d_pair(S_s, &tmSp, 0, w.p_tile * a.p.chunks + c, bar);
            for (int j = 0; j < C::kQTiles; ++j)
              ptx::tma_load_2d_pair(S_s + (1 + j) * C::kSfTile, &tmSq, 0,
                                    (w.q_tile + j) * a.q.chunks + c, bar);
            continue;
          }
          ptx::mbar_arrive_expect_tx(full_bar(s), C::kPBytes + (uint32_t)qb * (C::kQBox * 128) +
                                                      sf * (two ? 3 : 2));
          const int x = w.k0 / 2 + st * 128;
          ptx::tma_load_2d(P_s, &tmP, x, w.p_row, full_bar(s));
          for (int b = 0; b < qb; ++b)
            ptx::tma_load_2d(Q_s + b * C::kQBox * 128, &tmQ, x, w.q_row + b * C::kQBox, full_bar(s));
          const long long at = (long long)st * C::kSfTile;
          ptx::bulk_g2s(S_s, sp + at, sf, full_bar(s));
          ptx::bulk_g2s(S_s + C::kSfTile, sq + at, sf, full_bar(s));
          if (two)
            ptx::bulk_g2s(S_s + 2 * C::kSfTile, sq + (long long)a.q.chunks * kFp4ChunkBytes + at, sf,
                          full_bar(s));
        }
      }
      if (*abort_flag && !(PAIR && rank != 0)) {
        for (uint32_t k = it > (uint32_t)C::kStages ? it - C::kStages : 0u; k < it; ++k)
          ptx::mbar_wait(full_bar(k % C::kStages), (k / C::kStages) & 1, a.status, nullptr);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    // The whole warp walks the stages and one lane issues: a stage is 4 products and up to 12
    // scale copies in some 500 cycles, so what is issued between them counts.  (With loops and
    // descriptors made in the branch of one lane, 8192^3 took 678 us; in this form, 359.)
    uint32_t it = 0, lu = 0;
    bool stop = false;
    // descriptors of stage 0: their upper words do not change, the address field of the lower
    // counts 16 bytes
    const uint32_t base = ptx::smem_u32(smem);
    const uint64_t pd0 = ptx::smem_desc(base, 16, 1024, 2);
    const uint64_t qd0 = ptx::smem_desc(base + C::kPBytes, 16, 1024, 2);
    // scales: 32 rows of 16 bytes, core matrices of 8 rows 128 bytes apart
    const uint64_t sd0 = ptx::smem_desc(base + C::kPBytes + C::kQBytes, 16, 128, 0);
    const int mine = PAIR && rank != 0 ? 0 : tiles;  // rank 0 of a pair issues for both
    for (int t = first; t < mine && !stop; t += step, ++lu) {
      const Tile w = tile_at(t);
      const int b = (int)(lu % C::kAccBufs);
      bool ok = ptx::mbar_wait(acce_bar(b), ((lu / C::kAccBufs) & 1) ^ 1, a.status, abort_flag);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      ptx::tc_fence_after();
      const uint32_t acc = tmem + b * C::kAccCols;
      const uint32_t n = mma_n(w.q_len), q_shift = w.q_shift / 32;
      const uint32_t id0 = ptx::idesc_fp4(C::kPRows, n, FMT == HINM_FP4_MX, 0);
      const uint32_t id2 = ptx::idesc_fp4(C::kPRows, n, FMT == HINM_FP4_MX, 2);
      const bool two =
          __any_sync(0xFFFFFFFFu, C::kQTiles == 2 && w.q_shift + w.q_len > kFp4RowTile);
      int s0, s1;
      stage_range(w.steps, s0, s1);
      for (int st = s0; st < s1; ++st, ++it) {
        const uint32_t s = it % C::kStages;
        ok = ptx::mbar_wait(full_bar(s), (it / C::kStages) & 1, a.status, abort_flag);
        if (C::kSlots < C::kStages && it >= (uint32_t)C::kSlots) {
          // the products that read this slot's scales are done
          const uint32_t old = it - C::kSlots;
          ok = ok && ptx::mbar_wait(empty_bar(old % C::kStages), (old / C::kStages) & 1, a.status,
                                    abort_flag);
        }
        if (!__all_sync(0xFFFFFFFFu, ok)) {
          stop = true;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t off = s * (C::kStageBytes / 16);
        const uint64_t pd = pd0 + off, qd = qd0 + off, sd = sd0 + off;
        const uint32_t sfp = tmem + kSfCol0 + (it % C::kSlots) * C::kSfCols;
        const uint32_t sfq = sfp + 4 * C::kChunks;
        const uint32_t sfq_mma = sfq + q_shift;
        const int left = min(4, w.steps - 4 * st);
        const uint32_t more = st > s0;
        if (ptx::elect_one()) {
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c) {
            if (c * (C::kChunkDepth / 64) < left) {
              scale_copy<PAIR>(sfp + 4 * c, sd + c * (kFp4ChunkBytes / 16));
              scale_copy<PAIR>(sfq + 4 * C::kQTiles * c,
                               sd + (C::kSfTile + c * kFp4ChunkBytes) / 16);
              if (two)
                scale_copy<PAIR>(sfq + 4 * C::kQTiles * c + 4,
                                 sd + (2 * C::kSfTile + c * kFp4ChunkBytes) / 16);
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k < left) {
              if constexpr (FMT == HINM_FP4_NV)
                product<FMT, PAIR>(acc, pd + 2 * k, qd + 2 * k, id0, sfp + 4 * k,
                                   sfq_mma + 4 * C::kQTiles * k, k > 0 ? 1u : more);
              else
                product<FMT, PAIR>(acc, pd + 2 * k, qd + 2 * k, (k & 1) ? id2 : id0,
                                   sfp + 4 * (k / 2), sfq_mma + 4 * C::kQTiles * (k / 2),
                                   k > 0 ? 1u : more);
            }
          }
          commit<PAIR>(empty_bar(s));
        }
        __syncwarp();
      }
      if (stop) break;
      if (ptx::elect_one()) commit<PAIR>(accf_bar(b));
      __syncwarp();
    }
    // Rank 1 of a pair issues nothing: it comes to the drain at once, and a wait there would last, and
    // be limited, for the whole kernel.  The epilogue's waits span a tile each, and behind its last tile
    // only the drain's own commit is left.
    if (PAIR && rank != 0) asm volatile("barrier.cta.sync 2, %0;" ::"n"(32 + 32 * kEpiWarps) : "memory");
    if (ptx::elect_one()) {
      if (!PAIR || rank == 0) commit<PAIR>(drain_bar);  // the last commit that reaches rank 1
      ptx::mbar_wait(drain_bar, 0, a.status, nullptr);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int quad = warp & 3, part = (warp - 2) >> 2;  // warps 2..5 and 6..9
    constexpr int kOwn = BN / (kEpiWarps / 4);  // columns of this warp
    static_assert(kOwn % kEpiCols == 0, "columns");
    const int row = quad * 32 + lane;
    // this warp has read what it needs of accumulator b
    auto release = [&](int b) {
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) ptx::mbar_arrive_cluster_relaxed(ptx::mapa_shared(acce_bar(b), 0));
        else ptx::mbar_arrive(acce_bar(b));
      }
    };
    uint32_t lu = 0;
    for (int t = first; t < tiles; t += step, ++lu) {
      const Tile w = tile_at(t);
      const int b = (int)(lu % C::kAccBufs);
      // (loaded while the products run)
      int s0, s1;
      stage_range(w.steps, s0, s1);
      const int m = a.a_batched ? w.e : 0;
      const float alpha = (a.ga ? __ldg(a.ga + m) : 1.0f) * (a.gb ? __ldg(a.gb) : 1.0f);
      const float* bias = a.bias ? a.bias + (long long)m * a.a_rows : nullptr;
      const bool mine = row < w.p_len;
      const float bias_p = bias && !a.bias_q && mine ? __ldg(bias + w.p_out + row) : 0.0f;
      bool ok = true;  // one lane asks, so that the waiting warps take few issue slots
      if (lane == 0) ok = ptx::mbar_wait(accf_bar(b), (lu / C::kAccBufs) & 1, a.status, abort_flag);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      ptx::tc_fence_after();
      const long long y0 = a.ragged == HINM_RAGGED_DEPTH ? w.e * a.y_batch : 0;
      const int col0 = part * kOwn, col1 = min(w.q_len, col0 + kOwn);
      const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(b * C::kAccCols);
      if constexpr (!SPLIT) {
        if (!a.q_major && col0 < col1) {
          const Columns cw{alpha,
                           bias_p,
                           bias && a.bias_q ? bias + w.q_out + col0 : nullptr,
                           ptx::smem_u32(epi_smem + (warp - 2) * kEpiTile),
                           lane,
                           w.p_len - quad * 32,
                           col1 - col0,
                           y0 + (long long)(w.p_out + quad * 32) * a.ldy + w.q_out + col0};
          const bool lines = cw.cols == kOwn && align_of(a, cw.at0) == 32;
          auto done = [&] { release(b); };
          auto write = [&](auto dt) {
            constexpr int DT = decltype(dt)::value;
            if (cw.bias_cols) {
              if (lines) write_lines<DT, kOwn, true, C::kAccBufs == 1, ACTS>(a, lanes + col0, s1 == s0, cw, done);
              else write_any<DT, kOwn, true, ACTS>(a, lanes + col0, s1 == s0, cw, done);
            } else {
              if (lines) write_lines<DT, kOwn, false, C::kAccBufs == 1, ACTS>(a, lanes + col0, s1 == s0, cw, done);
              else write_any<DT, kOwn, false, ACTS>(a, lanes + col0, s1 == s0, cw, done);
            }
          };
          if (a.dtype == HINM_DTYPE_BF16) write(std::integral_constant<int, HINM_DTYPE_BF16>{});
          else if (a.dtype == HINM_DTYPE_F16) write(std::integral_constant<int, HINM_DTYPE_F16>{});
          else write(std::integral_constant<int, HINM_DTYPE_F32>{});
          continue;
        }
      }
      uint32_t next[kEpiCols];
      if (col0 < col1 && s1 > s0) {
        ptx::tmem_ld_16(lanes + col0, next);
        ptx::tmem_ld_wait();
      }
#pragma unroll 1
      for (int col = col0; col < col1; col += kEpiCols) {
        uint32_t v[kEpiCols];
#pragma unroll
        for (int i = 0; i < kEpiCols; ++i) v[i] = s1 > s0 ? next[i] : 0u;  // no depth: zeros
        const bool last = col + kEpiCols >= col1;
        // the next columns arrive while these are worked on
        if (!last && s1 > s0) ptx::tmem_ld_16(lanes + col + kEpiCols, next);
        if (last) release(b);
        const int n = min(kEpiCols, w.q_len - col);
        if constexpr (SPLIT) {
          // partial sums to this CTA's stages, which its products are done with, in Y's order
          if (a.q_major) {
            float* part_sums = reinterpret_cast<float*>(smem) + col * 128 + row;
#pragma unroll
            for (int i = 0; i < kEpiCols; ++i)
              if (i < n) part_sums[i * 128] = __uint_as_float(v[i]);
          } else {
            uint4* part_sums = reinterpret_cast<uint4*>(smem + (row * kPartRow + col) * 4);
#pragma unroll
            for (int i = 0; i < kEpiCols / 4; ++i)
              part_sums[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          }
        } else {
          // Y as [Q][P] (then the bias goes along P)
          float y[kEpiCols];
#pragma unroll
          for (int i = 0; i < kEpiCols; ++i) y[i] = fmaf(__uint_as_float(v[i]), alpha, bias_p);
          if (a.act == HINM_ACT_RELU) activate_all<HINM_ACT_RELU, true>(y);
          else if (a.act == HINM_ACT_SILU) activate_all<HINM_ACT_SILU, true>(y);
          else if (a.act == HINM_ACT_GELU) activate_all<HINM_ACT_GELU, true>(y);
#pragma unroll
          for (int i = 0; i < kEpiCols; ++i)
            if (i < n && mine)
              store_one(a.Y, a.dtype,
                        y0 + (long long)(w.q_out + col + i) * a.ldy + w.p_out + row, y[i]);
        }
        if (!last && s1 > s0) ptx::tmem_ld_wait();
      }
      if (col0 >= col1) release(b);  // none of the columns
    }
    if (PAIR && rank != 0) asm volatile("barrier.cta.arrive 2, %0;" ::"n"(32 + 32 * kEpiWarps) : "memory");
  }
  if constexpr (SPLIT) {
    ptx::cluster_sync();  // every CTA's partial sums are in its shared memory
    if (first < tiles && !*abort_flag) {
      const Tile w = tile_at(first);
      const int m = a.a_batched ? w.e : 0;
      const float alpha = (a.ga ? __ldg(a.ga + m) : 1.0f) * (a.gb ? __ldg(a.gb) : 1.0f);
      const float* bias = a.bias ? a.bias + (long long)m * a.a_rows : nullptr;
      const long long y0 = a.ragged == HINM_RAGGED_DEPTH ? w.e * a.y_batch : 0;
      // groups of 4 along Y's rows, shared out over the ranks: rows of Y are P's 128 for a
      // column (q_major), else a row's columns
      const int inner = a.q_major ? 32 : (w.q_len + 3) / 4;
      const int outer = a.q_major ? w.q_len : w.p_len;
      const int o0 = outer * rank / a.split, groups = (outer * (rank + 1) / a.split - o0) * inner;
      const uint32_t part = ptx::smem_u32(smem);
      for (int i = threadIdx.x; i < groups; i += kMmThreads) {
        const int o = o0 + i / inner, j = i % inner * 4;
        const uint32_t at = part + (uint32_t)(o * (a.q_major ? 128 : kPartRow) + j) * 4;
        float4 v[kMaxSplit];
#pragma unroll
        for (int r = 0; r < kMaxSplit; ++r) {
          v[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (r < a.split) v[r] = ptx::ld_cluster_v4(ptx::mapa_shared(at, r));
        }
        float y[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
        for (int r = 1; r < kMaxSplit; ++r) {
          if (r < a.split) {
            y[0] = __fadd_rn(y[0], v[r].x);
            y[1] = __fadd_rn(y[1], v[r].y);
            y[2] = __fadd_rn(y[2], v[r].z);
            y[3] = __fadd_rn(y[3], v[r].w);
          }
        }
        const int n = min(4, (a.q_major ? w.p_len : w.q_len) - j);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int prow = w.p_out + (a.q_major ? j + q : o), qcol = w.q_out + (a.q_major ? o : j + q);
          const float bi = bias && q < n ? __ldg(bias + (a.bias_q ? qcol : prow)) : 0.0f;
          y[q] = activate<true>(fmaf(y[q], alpha, bi), a.act);
        }
        const long long out = y0 + (a.q_major ? (long long)(w.q_out + o) * a.ldy + w.p_out + j
                                              : (long long)(w.p_out + o) * a.ldy + w.q_out + j);
        store_four(a, y, n, out);
      }
    }
    ptx::cluster_sync();  // nobody reads this CTA's shared memory any more
  }
  ptx::tc_fence_before();
  if constexpr (PAIR) ptx::cluster_sync();  // nothing of the other CTA's is in flight here
  else __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    if constexpr (PAIR) ptx::tmem_dealloc_pair(tmem, 512);
    else ptx::tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ host side
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// The stored values as bytes: `rows` rows of `pitch`; boxes of 128 bytes by box_rows, zeros past
// the last row or byte.
bool make_map(CUtensorMap* m, const uint8_t* values, long long rows, long long pitch,
              int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)pitch, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)pitch};
  cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(values), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale chunks as rows of 512 bytes, boxes of a stage's chunks, zeros past the last.
bool make_scale_map(CUtensorMap* m, const uint8_t* scales, long long chunks, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {kFp4ChunkBytes / 4, (cuuint64_t)chunks};
  cuuint64_t strides[1] = {kFp4ChunkBytes};
  cuuint32_t box[2] = {kFp4ChunkBytes / 4, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t*>(scales), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int num_sms() {
  static int n = 0;
  if (n == 0) {
    int dev = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (n <= 0) n = 148;
  }
  return n;
}

struct Maps {
  CUtensorMap p, q, sp, sq;  // values; scales (pairs)
};

template <int FMT, int BN, bool SPLIT, bool PAIR, bool ACTS>
cudaError_t run(MmArgs a, const Maps& m, long long tiles, cudaStream_t s) {
  using C = MmCfg<FMT, BN, PAIR>;
  auto kernel = fp4_mm_kernel<FMT, BN, SPLIT, PAIR, ACTS>;
  cudaError_t e = set_max_dynamic_smem((const void*)kernel, (int)C::kSmemBytes);
  if (e != cudaSuccess) return e;
  if constexpr (!SPLIT && !PAIR) {
    const int grid = tiles < num_sms() ? (int)tiles : num_sms();
    return launch_kernel(kernel, grid, kMmThreads, C::kSmemBytes, s, nullptr, m.p, m.q, m.sp, m.sq,
                         a);
  } else {
    cudaLaunchAttribute cluster;
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = PAIR ? 2u : (unsigned)a.split;
    cluster.val.clusterDim.y = 1;
    cluster.val.clusterDim.z = 1;
    const long long grid = !PAIR ? tiles * a.split : 2 * (tiles < num_sms() / 2 ? tiles : num_sms() / 2);
    return launch_kernel(kernel, (unsigned)grid, kMmThreads, C::kSmemBytes, s, &cluster, m.p, m.q,
                         m.sp, m.sq, a);
  }
}

// How a product is cut: the rows of a Q tile, pairs of CTAs (256 rows of P) or not, and how many
// CTAs share a tile's depth.
struct Plan {
  int bn, pair, split;
};

// The cheapest cut by a model of the kernel's time: rounds of tiles over the SMs, a round being
// the stages of a tile at the rate that the copies from L2 allow, and what a tile costs besides.
// Measured on B200 (4096 x 4096, depths 256 to 16384; us a stage of 256 of the depth and us a tile
// besides): pair 256 x 256 0.40 and 2.1, 128 x 192 0.465 and 0.95, 128 x 128 0.42 and 0.7, 128 x 64
// 0.45 and 0.6; the last tile's columns are written after everything else, 0.011 a column.  So at
// depth 1024 128 x 192 takes 17.0 us and pairs 17.7, at 4096 45.0 and 35.9, at 16384 156 and 115.
// Sharing a tile's depth costs 1.5 us and 0.03 a column (partial sums through the cluster): 4096
// rows of depth 4096 by 1 column 7.1 us shared by four and 9.5 not, by 256 columns 13.1 shared by
// two and 10.4 not.
// A stage costs the same whatever the number of columns that are real, and few tokens over much depth
// take 128 columns (from 11008 x 8192 on) or pairs (32000 x 32768): right for 32 and 64 tokens (11008 x
// 8192 MX 14.9 and 14.7 us, in 64 columns 17.4 and 19.8) and about even for 16, but a single token loses
// where tiles go round several times (32000 x 8192 NV 39.7 us, in 64 columns 30.7; at 11008 x 8192 15.7
// and 16.2).
// p, q: rows of P and Q, in `groups` ragged parts when given (tokens: p_ragged or not).
Plan make_plan(long long p, long long q, long long depth, int p_groups, int q_groups, int times,
               int sms) {
  const Plan cut[4] = {{256, 1, 1}, {192, 0, 1}, {128, 0, 1}, {64, 0, 1}};
  const double stage_us[4] = {0.40, 0.465, 0.42, 0.45}, tile_us[4] = {2.1, 0.95, 0.7, 0.6};
  Plan best = cut[0];
  double best_us = 1e30;
  const long long stages = (depth + kStageDepth - 1) / kStageDepth;
  for (int i = 0; i < 4; ++i) {
    const long long pr = cut[i].pair ? 256 : 128, bn = cut[i].bn;
    // ragged: as if the groups had the same size
    const long long pt = p_groups ? p_groups * ((p + p_groups * pr - 1) / (p_groups * pr)) : (p + pr - 1) / pr;
    const long long qt = q_groups ? q_groups * ((q + q_groups * bn - 1) / (q_groups * bn)) : (q + bn - 1) / bn;
    const long long tiles = pt * qt * times;
    const long long units = cut[i].pair ? sms / 2 : sms;
    for (int split = 1; split <= (bn <= 128 ? kMaxSplit : 1); ++split) {
      if (split > 1 && (tiles * split > units || stages < 2 * split)) break;
      const double us = (double)((tiles * split + units - 1) / units) *
                        ((double)((stages + split - 1) / split) * stage_us[i] + tile_us[i] +
                         (split > 1 ? 1.5 + 0.03 * (double)(q < bn ? q : bn) : 0.0)) +
                        0.011 * (double)bn;
      if (us < best_us) {
        best_us = us;
        best = cut[i];
        best.split = split;
      }
    }
  }
  return best;
}

// Which side takes the accumulator's lanes, and the cut: both of the shapes alone.
struct Choice {
  bool swap;  // the tokens in the lanes
  Plan plan;
};
Choice choose(const hinm_fp4& A, const hinm_fp4& B, bool transposed) {
  const bool by_rows = B.ragged == HINM_RAGGED_ROWS, by_depth = B.ragged == HINM_RAGGED_DEPTH;
  const long long n = by_rows ? ((long long)B.rows + B.groups - 1) / B.groups : B.rows;
  Choice c;
  c.swap = transposed && n > 64;
  const int groups = by_rows ? B.groups : 0;
  c.plan = make_plan(c.swap ? B.rows : A.rows, c.swap ? A.rows : B.rows,
                     by_depth ? B.depth / B.groups : B.depth, c.swap ? groups : 0,
                     c.swap ? 0 : groups, by_depth ? B.groups : 1, num_sms());
  return c;
}

template <int FMT, int BN, bool PAIR>
cudaError_t launch_tiles(MmArgs a, const Maps& m, const Plan& p, cudaStream_t s) {
  constexpr int PR = MmCfg<FMT, BN, PAIR>::kPRows;
  a.pt = (a.p.rows + PR - 1) / PR;
  a.qt = (a.q.rows + BN - 1) / BN;
  // ragged rows: no more tiles than full ones and one partial for each group
  const long long tiles = a.p.ragged   ? ((long long)a.p.rows / PR + a.groups) * a.qt
                          : a.q.ragged ? ((long long)a.q.rows / BN + a.groups) * a.pt
                          : (long long)a.pt * a.qt *
                                (a.ragged == HINM_RAGGED_DEPTH ? a.groups : 1);
  if (tiles > 0x3FFFFFFFll) return cudaErrorInvalidValue;
  a.split = p.split;
  if constexpr (BN <= 128 && !PAIR) {
    if (p.split > 1) return run<FMT, BN, true, false, true>(a, m, tiles, s);
  }
  if constexpr (BN > 128) {
    if (a.act == HINM_ACT_NONE) return run<FMT, BN, false, PAIR, false>(a, m, tiles, s);
  }
  return run<FMT, BN, false, PAIR, true>(a, m, tiles, s);
}

template <int FMT>
cudaError_t pick(MmArgs a, const hinm_fp4& A, const hinm_fp4& B, bool transposed,
                 cudaStream_t s) {
  const Fp4Geom ga = fp4_geom(A.rows, A.depth, A.ragged, A.groups);
  const Fp4Geom gb = fp4_geom(B.rows, B.depth, B.ragged, B.groups);
  if (A.batch * ga.row_tiles * ga.chunks(FMT) > 0x7FFFFFFF || gb.row_tiles * gb.chunks(FMT) > 0x7FFFFFFF)
    return cudaErrorInvalidValue;
  const Side sa{A.scales, (int)ga.row_tiles, (int)ga.chunks(FMT), A.rows,
                a.ragged == HINM_RAGGED_ROWS ? 1 : 0, 0};
  const Side sb{B.scales, (int)gb.row_tiles, (int)gb.chunks(FMT), B.rows, 0,
                a.ragged == HINM_RAGGED_ROWS ? 1 : 0};
  a.steps = (int)(ga.depth_pad / 64);
  const Choice choice = choose(A, B, transposed);
  const bool swap = choice.swap;
  const Plan p = choice.plan;
  a.p = swap ? sb : sa;
  a.q = swap ? sa : sb;
  a.bias_q = swap;
  a.q_major = transposed && !swap;
  Maps m{};
  const int q_box = p.pair ? p.bn / 2 : p.bn == 64 ? 16 : 64;  // MmCfg::kQBox
  if (!make_map(swap ? &m.q : &m.p, A.values, (long long)A.batch * A.rows, ga.pitch(),
                swap ? q_box : 128) ||
      !make_map(swap ? &m.p : &m.q, B.values, B.rows, gb.pitch(), swap ? 128 : q_box))
    return cudaErrorInvalidValue;
  if (p.pair) {
    constexpr int kBox = kStageDepth / (4 * fp4_block(FMT));
    if (!make_scale_map(swap ? &m.sq : &m.sp, A.scales, A.batch * ga.row_tiles * ga.chunks(FMT), kBox) ||
        !make_scale_map(swap ? &m.sp : &m.sq, B.scales, gb.row_tiles * gb.chunks(FMT), kBox))
      return cudaErrorInvalidValue;
    return launch_tiles<FMT, 256, true>(a, m, p, s);
  }
  if (p.bn == 64) return launch_tiles<FMT, 64, false>(a, m, p, s);
  if (p.bn == 128) return launch_tiles<FMT, 128, false>(a, m, p, s);
  return launch_tiles<FMT, 192, false>(a, m, p, s);
}

}  // namespace

Fp4Cut fp4_cut(const hinm_fp4& A, const hinm_fp4& B, bool transposed) {
  const Choice c = choose(A, B, transposed);
  return Fp4Cut{c.plan.bn, c.plan.pair, c.plan.split, c.swap ? 1 : 0};
}

cudaError_t launch_fp4_matmul(const hinm_fp4& A, const hinm_fp4& B, const Fp4Out& o, int* status,
                              cudaStream_t s) {
  MmArgs a{};
  a.ga = A.tensor_scale;
  a.gb = B.tensor_scale;
  a.bias = o.bias;
  a.offsets = B.offsets;
  a.Y = o.Y;
  a.ldy = o.ldy;
  a.y_batch = o.batch_stride;
  a.a_batched = A.batch > 1;
  a.a_rows = A.rows;
  a.depth = B.depth;
  a.groups = B.groups;
  a.ragged = B.ragged;
  a.dtype = o.dtype;
  a.act = o.act;
  const long long es = o.dtype == HINM_DTYPE_F32 ? 4 : 2;
  const unsigned long long bits =
      reinterpret_cast<uintptr_t>(o.Y) | (uintptr_t)(o.ldy * es) | (uintptr_t)(o.batch_stride * es);
  a.align = (int)((bits | 32) & (~(bits | 32) + 1));
  a.status = status;
  return A.format == HINM_FP4_NV ? pick<HINM_FP4_NV>(a, A, B, o.transposed != 0, s)
                                 : pick<HINM_FP4_MX>(a, A, B, o.transposed != 0, s);
}

}  // namespace hinm
