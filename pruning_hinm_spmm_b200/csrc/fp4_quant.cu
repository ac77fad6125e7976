// b1. Microscaled 4-bit quantisation (hinm.h, section b1): the tensor scale, the quantiser
// and the way back.
//
//   NV: x' = fl32(x fl32(1/g)), s = e4m3(max |x'| / 6),               code = e2m1(x' / s)
//   MX: s = 2^(floor(log2 max |x|) - 2),                              code = e2m1(x / s)
//
// Every rounding is to nearest, ties to even, decided on the exact quotient.  MX divides by
// a power of two, which is exact.  NV: x' / s is taken as q0 = x' r with r = fl32(1 / s), one
// exact residual by fused multiply-add and one correction (Markstein, IBM J. Res. Dev. 34,
// 1990): the correctly rounded quotient.  Rounding to 24 bits cannot move a quotient onto a
// border between two codes: s has 4 significant bits and a border at most 3, so border * s is
// an fp32 number, x' differs from it by at least one unit in its last place, and the quotient
// from the border by more than half a unit (by a whole representable step below 0.25).
//
// A bf16 element costs 2 bytes in and 0.5 + 1/16 (NV) or 0.5 + 1/32 (MX) bytes out; at 11008 x 4096
// the kernels take 1.2 to 1.5 times as long as these bytes at the rate of a copy (NV along the rows
// 23.4 us for 17.6 of bytes, with a mask 27.7 for 18.5, down the columns 26.7; MX 21.4 and 21.9 for
// 17.4).  What holds them besides DRAM is the arithmetic of an element: with a mask along the rows the
// issue slots are 59% taken (DRAM 39%), down the columns registers leave a quarter of the warps.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp4.cuh"
#include "hinm_internal.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace hinm {
namespace {

using ptx::F2;
using ptx::fma2;
using ptx::mul2;

// ------------------------------------------------------------------ elements
template <int DT>
struct Elem;
template <>
struct Elem<HINM_DTYPE_BF16> {
  using T = uint16_t;
  static __device__ T of(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
  static __device__ void unpack(uint32_t w, float& a, float& b) {
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xFFFF0000u);
  }
};
template <>
struct Elem<HINM_DTYPE_F16> {
  using T = uint16_t;
  static __device__ T of(float v) { return __half_as_ushort(__float2half_rn(v)); }
  static __device__ void unpack(uint32_t w, float& a, float& b) {
    a = __half2float(__ushort_as_half((unsigned short)(w & 0xFFFF)));
    b = __half2float(__ushort_as_half((unsigned short)(w >> 16)));
  }
};
template <>
struct Elem<HINM_DTYPE_F32> {
  using T = uint32_t;
  static __device__ T of(float v) { return __float_as_uint(v); }
};

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// ------------------------------------------------------------------ codes
// e2m1 (round to nearest even, saturating at 6) of 8 values, the first in the lowest bits
__device__ __forceinline__ uint32_t e2m1x8(const float* q) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return r;
}

// e4m3 (round to nearest even, saturating at 448) of a >= 0
__device__ __forceinline__ uint32_t e4m3_of(float a) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(a));
  return r & 0xFFu;
}
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)code));
  return __half2float(__ushort_as_half((unsigned short)(h2 & 0xFFFF)));
}

// The 127 scales of NV and their reciprocals, in shared memory: a block needs one of each, and
// takes them from here instead of working them out (a decoding and a reciprocal for 16 elements
// were a third of the NV quantiser's instructions).
struct ScaleTable {
  float2 v[128];
};
template <int FMT>
__device__ __forceinline__ void fill(ScaleTable& t) {
  if constexpr (FMT == HINM_FP4_NV) {
    if (threadIdx.x < 128) {
      const float s = e4m3_value(threadIdx.x);
      t.v[threadIdx.x] = make_float2(s, threadIdx.x ? __frcp_rn(s) : 0.0f);  // scale 0: codes 0
    }
    __syncthreads();
  }
}

// A block's scale byte from the bits of its largest magnitude (NV: already over g), and what its
// codes are made with: q = x r, or (NV) the correctly rounded x / s from r = fl32(1 / s).  A block
// with a value that is not finite (the largest of all as bits) gets the scale NaN and codes of
// zero, so that whatever reads it is NaN.
struct BlockScale {
  uint32_t code;
  float s, r;
  bool finite;
};
template <int FMT>
__device__ __forceinline__ BlockScale block_scale(const ScaleTable& t, uint32_t am) {
  BlockScale b;
  b.finite = am < 0x7F800000u;
  if constexpr (FMT == HINM_FP4_NV) {
    // max / 6, correctly rounded: product with fl32(1/6) and one residual, as for the codes
    const float a = __uint_as_float(am), sixth = 1.0f / 6.0f;
    const float q0 = __fmul_rn(a, sixth);
    b.code = b.finite ? e4m3_of(__fmaf_rn(__fmaf_rn(-6.0f, q0, a), sixth, q0)) : 0x7Fu;
    const float2 v = t.v[b.code];
    b.s = v.x;
    b.r = v.y;
  } else {
    const int e = (int)(am >> 23) - 2;  // the largest's exponent less that of 4 (6 = 1.5 * 4)
    b.code = e > 0 ? (uint32_t)e : 0u;
    b.r = __uint_as_float((254u - b.code) << 23);
    b.s = 0.0f;
    if (!b.finite) b.code = 0xFFu;
  }
  return b;
}
// The codes of 8 values x; NV: of 8 values -x, over g, so that the residual t s - x is one fused
// operation and a zero keeps its sign (t = x r, q = t - (t s - x) r).
template <int FMT>
__device__ __forceinline__ uint32_t encode8(const F2 (&x)[4], const BlockScale& b) {
  float q[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    F2 t = mul2(x[i], FMT == HINM_FP4_NV ? F2(-b.r, -b.r) : F2(b.r, b.r));
    if constexpr (FMT == HINM_FP4_NV) t = fma2(fma2(t, F2(b.s, b.s), x[i]), F2(-b.r, -b.r), t);
    t.get(q[2 * i], q[2 * i + 1]);
  }
  return b.finite ? e2m1x8(q) : 0u;
}

// One block's codes (B / 8 words) and its scale byte.  inv_g: fl32(1 / g) (NV).
template <int FMT, int B>
__device__ __forceinline__ uint32_t encode_block(const ScaleTable& t, float (&v)[B], float inv_g,
                                                 uint32_t (&w)[B / 8]) {
  uint32_t am = 0;
#pragma unroll
  for (int i = 0; i < B; ++i) {
    if constexpr (FMT == HINM_FP4_NV) v[i] = __fmul_rn(v[i], -inv_g);
    am = max(am, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  }
  const BlockScale b = block_scale<FMT>(t, am);
#pragma unroll
  for (int i = 0; i < B / 8; ++i) {
    const F2 x[4] = {F2(v[8 * i], v[8 * i + 1]), F2(v[8 * i + 2], v[8 * i + 3]),
                     F2(v[8 * i + 4], v[8 * i + 5]), F2(v[8 * i + 6], v[8 * i + 7])};
    w[i] = encode8<FMT>(x, b);
  }
  return b.code;
}

// The bits of the larger magnitude in the two halves of a packed maximum, as fp32 (NV: over g).
template <int DT, int FMT>
__device__ __forceinline__ uint32_t widest(uint32_t m, float inv_g) {
  const uint32_t h = max(m & 0xFFFFu, m >> 16);
  float f, other;
  Elem<DT>::unpack(h, f, other);
  if constexpr (FMT == HINM_FP4_NV) f = __fmul_rn(f, inv_g);
  return __float_as_uint(f);
}
// 8 packed 16-bit elements as pairs (NV: over g)
template <int DT, int FMT>
__device__ __forceinline__ uint32_t encode_words(const uint32_t (&u)[4], float inv_g,
                                                 const BlockScale& b) {
  float l[4], h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) Elem<DT>::unpack(u[i], l[i], h[i]);
  F2 x[4] = {F2(l[0], h[0]), F2(l[1], h[1]), F2(l[2], h[2]), F2(l[3], h[3])};
  if constexpr (FMT == HINM_FP4_NV) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = mul2(x[i], F2(-inv_g, -inv_g));
  }
  return encode8<FMT>(x, b);
}

template <int FMT>
__device__ __forceinline__ float scale_value(uint32_t code) {
  if constexpr (FMT == HINM_FP4_NV) return e4m3_value(code);
  // 2^(code - 127): code 0 is the subnormal 2^-127, code 255 NaN
  return __uint_as_float(code == 255u ? 0x7FC00000u : code ? code << 23 : 0x00400000u);
}

// The values of the 8 codes of a word over s and g: fl32(code s g), code * s exact.
__device__ __forceinline__ void decode8(uint32_t w, float s, float g, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    mul2(mul2(F2(f.x, f.y), F2(s, s)), F2(g, g)).get(v[2 * i], v[2 * i + 1]);
  }
}
// Two values as 16-bit elements of a word; 8 in 4 words.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (DT == HINM_DTYPE_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <int DT>
__device__ __forceinline__ void pack8(const float (&v)[8], uint32_t (&u)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) u[i] = pack2<DT>(v[2 * i], v[2 * i + 1]);
}

// Number of groups whose start lies at or before p, less one: the group that p falls in.
// key(e) is nondecreasing for valid offsets; any values give an answer in [0, groups).
template <class Key>
__device__ __forceinline__ int group_of(int groups, long long p, Key key) {
  int lo = 0, hi = groups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (key(mid) <= p) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

struct QArgs {
  void* data;  // source or destination elements
  long long ld, batch_stride;
  const uint32_t* bits;  // mask words of the source's rows, or null
  uint8_t* values;
  uint8_t* scales;
  const float* g;  // [batch] or null
  const int32_t* offsets;
  int rows, depth, ragged, groups;
  int vec;  // rows are aligned to 32 or 16 bytes, or 0
  long long pitch, row_tiles, chunks, nblk;  // nblk: blocks of the stored depth
  int early;  // let the stream's next kernel begin its set-up (few blocks)
  int* status;
};

// Offsets that decrease or leave the dimension are reported by a launch's first block.  (The places
// below are looked up by searches that take nondecreasing offsets for granted: with others a group may
// never be found, so what they come across is no check.  They only keep every access inside.)
__device__ __forceinline__ void check_offsets(const int32_t* offsets, int groups, int limit,
                                              int* status) {
  if ((blockIdx.x | blockIdx.y | blockIdx.z) != 0) return;
  bool bad = false;
  for (int i = threadIdx.x; i < groups; i += blockDim.x) {
    const int o = __ldg(offsets + i), end = __ldg(offsets + i + 1);
    bad |= o < 0 || end < o || end > limit;
  }
  if (bad) ptx::record_status(status, HINM_ERR_INVALID_ARG);
}
// As a call, so that the kernels around it are compiled as without it: in line, 11008 x 4096 bf16 MX
// down the columns took 26.0 us instead of 22.0.  (The maximum's kernel has it in line: called, 5.3 us
// instead of 5.0 at 8192 x 1024.)
__device__ __noinline__ void check_offsets_called(const int32_t* offsets, int groups, int limit,
                                                  int* status) {
  check_offsets(offsets, groups, limit, status);
}
__device__ __forceinline__ void check_offsets(const QArgs& a) {
  if (a.ragged != HINM_RAGGED_NONE)
    check_offsets_called(a.offsets, a.groups, a.ragged == HINM_RAGGED_ROWS ? a.rows : a.depth,
                         a.status);
}

// Where the scales of a row of ragged group e (-1: before the first) lie: its tile and its place in
// it.  false: the row is in no group.
__device__ __forceinline__ bool place_in(const QArgs& a, int row, int e, long long& tile, int& at) {
  if (e < 0) return false;
  const int o = __ldg(a.offsets + e), end = __ldg(a.offsets + e + 1);
  if (row < o || row >= end) return false;
  tile = fp4_group_tile(o, e) + (row - o) / kFp4RowTile;
  at = (row - o) % kFp4RowTile;
  return o >= 0 && tile < a.row_tiles;
}

// The same for any stored row, its group looked for.
__device__ __forceinline__ bool row_place(const QArgs& a, int row, long long& tile, int& at) {
  if (a.ragged != HINM_RAGGED_ROWS) {
    tile = row / kFp4RowTile;
    at = row % kFp4RowTile;
    return true;
  }
  // the last of several groups that start at one row is the one that may hold it
  return place_in(a, row,
                  group_of(a.groups, row, [&](int i) { return (long long)__ldg(a.offsets + i); }),
                  tile, at);
}

// The last of the groups that start at or before each of N rows of a warp (the same rows in every
// lane; row_place finds one row's with a chain of loads, this takes 32 groups a load).
template <int N>
__device__ __forceinline__ void groups_of_rows(const QArgs& a, int row0, int step, int (&e)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) e[j] = -1;
  const int lane = threadIdx.x & 31;
  for (int base = 0; base < a.groups; base += 32) {
    const int i = base + lane;
    const int o = i < a.groups ? __ldg(a.offsets + i) : 0x7FFFFFFF;
#pragma unroll
    for (int j = 0; j < N; ++j) e[j] += __popc(__ballot_sync(0xFFFFFFFFu, o <= row0 + step * j));
  }
}
// Where the stored depth p (a multiple of a block) comes from: the first source position and
// how many of the `count` positions are real.  false: p is in no group's stored range.
__device__ __forceinline__ bool depth_place(const QArgs& a, long long p, int count, int& src,
                                            int& real) {
  if (a.ragged != HINM_RAGGED_DEPTH) {
    src = (int)p;
    const long long left = a.depth - p;
    real = left <= 0 ? 0 : left < count ? (int)left : count;
    return true;
  }
  const long long step = p / kFp4DepthPad;
  const int e = group_of(a.groups, step, [&](int i) {
    return fp4_group_tile(__ldg(a.offsets + i), i);
  });
  const int o = __ldg(a.offsets + e), end = __ldg(a.offsets + e + 1);
  const long long local = p - fp4_group_tile(o, e) * kFp4DepthPad;
  if (o < 0 || end > a.depth || end < o) return false;
  const long long n = end - o;
  if (local < 0 || local >= (n + kFp4DepthPad - 1) / kFp4DepthPad * kFp4DepthPad) return false;
  const long long left = n - local;
  src = (int)(o + local);
  real = left <= 0 ? 0 : left < count ? (int)left : count;
  return true;
}

// ------------------------------------------------------------------ depth along the source's rows
// A warp takes 32 consecutive blocks of one row (a lane a block), and four rows 32 apart at once:
// their scales for four blocks of depth are 16 contiguous bytes of a chunk.  All four rows' loads
// are issued before the first is used.
constexpr int kQWarps = 8;

// 32 aligned bytes: a lane's half of a block or a whole one, a sector of its own.
__device__ __forceinline__ void load32(const void* p, uint32_t* u) {
  asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]),
                 "=r"(u[6]), "=r"(u[7])
               : "l"(p));
}
__device__ __forceinline__ void store32(void* p, const uint32_t* u) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(u[0]),
               "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
               : "memory");
}

// Keeps the elements of a 16-bit pair whose bits (0 and 1) are set: each bit moved to a byte's sign,
// which the permutation copies over the element's bits.
__device__ __forceinline__ uint32_t masked(uint32_t u, uint32_t bits2) {
  uint32_t m;
  asm("prmt.b32 %0, %1, %2, 0xCC88;" : "=r"(m) : "r"(bits2 << 7), "r"(bits2 << 6));
  return u & m;
}

// The elements of 16 bytes whose bits are set.
template <int DT>
__device__ __forceinline__ uint4 masked_piece(const uint4& t, uint32_t k) {
  if constexpr (DT == HINM_DTYPE_F32)
    return make_uint4(k & 1u ? t.x : 0u, k & 2u ? t.y : 0u, k & 4u ? t.z : 0u, k & 8u ? t.w : 0u);
  else
    return make_uint4(masked(t.x, k), masked(t.y, k >> 2), masked(t.z, k >> 4), masked(t.w, k >> 6));
}

template <int DT, int FMT, bool VEC, bool RAGGED>
__global__ void __launch_bounds__(kQWarps * 32) quant_rows_kernel(const QArgs a) {
  __shared__ ScaleTable table;
  fill<FMT>(table);
  ptx::enter_dependent();
  if (a.early) ptx::launch_dependents();
  check_offsets(a);
  constexpr int B = fp4_block(FMT);
  using T = typename Elem<DT>::T;
  constexpr bool k16 = sizeof(T) == 2;
  constexpr int kWords = B * (int)sizeof(T) / 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kRead = kWords + (VEC ? 0 : 4);  // words read of a block
  const long long batch = blockIdx.z;
  const long long blk = (long long)blockIdx.y * 32 + lane;
  const int row0 = ((int)blockIdx.x >> 2) * kFp4RowTile + ((int)blockIdx.x & 3) * kQWarps + warp;
  const T* src = reinterpret_cast<const T*>(a.data) + batch * a.batch_stride;
  const uintptr_t lo = reinterpret_cast<uintptr_t>(src);
  const uintptr_t hi = lo + ((unsigned long long)(a.rows - 1) * a.ld + a.depth) * sizeof(T);
  const float inv_g = FMT == HINM_FP4_NV && a.g ? __frcp_rn(__ldg(a.g + batch)) : 1.0f;
  int k = 0, real = 0;
  const bool mine = blk < a.nblk && depth_place(a, blk * B, B, k, real);
  const bool chunk_ok = __shfl_sync(0xFFFFFFFFu, mine, lane & ~3);
  long long tile[4];
  int at[4];
  bool placed[4] = {true, true, true, true};
  if constexpr (RAGGED) {
    int e[4];
    groups_of_rows<4>(a, row0, 32, e);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      placed[j] = row0 + 32 * j < a.rows && place_in(a, row0 + 32 * j, e[j], tile[j], at[j]);
  }
  // (blocks of 32 fp32 values: two rows at once, to stay in registers)
  constexpr int kAtOnce = kWords > 16 ? 2 : 4;
  uint32_t word[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j0 = 0; j0 < 4; j0 += kAtOnce) {
    uint32_t u[kAtOnce][kRead], keep[kAtOnce];
    int shift[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int row = row0 + 32 * (j0 + j);
#pragma unroll
      for (int i = 0; i < kRead; ++i) u[j][i] = 0;
      shift[j] = 0;
      keep[j] = 0xFFFFFFFFu;
      if (row >= a.rows || real <= 0 || !placed[j0 + j]) continue;
      const T* p = src + (long long)row * a.ld;
      if (a.bits)
        keep[j] = __ldg(a.bits + (batch * a.rows + row) * ((a.depth + 31) / 32) + k / 32);
      p += k;
      // (rows that are not aligned: the aligned 16-byte pieces around the block, unless they reach
      // out of the matrix)
      const uintptr_t at0 = reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)15;
      if (VEC && real == B) {
        if (a.vec == 32) {
#pragma unroll
          for (int i = 0; i < kWords; i += 8) load32(p + i * 4 / (int)sizeof(T), &u[j][i]);
        } else {
#pragma unroll
          for (int i = 0; i < kWords; i += 4) {
            const uint4 t = __ldg(reinterpret_cast<const uint4*>(p) + i / 4);
            u[j][i] = t.x;
            u[j][i + 1] = t.y;
            u[j][i + 2] = t.z;
            u[j][i + 3] = t.w;
          }
        }
      } else if (!VEC && real == B && at0 >= lo && at0 + 4 * kRead <= hi) {
        shift[j] = (int)(reinterpret_cast<uintptr_t>(p) & 15);
#pragma unroll
        for (int i = 0; i < kRead; i += 4) {
          const uint4 t = __ldg(reinterpret_cast<const uint4*>(at0) + i / 4);
          u[j][i] = t.x;
          u[j][i + 1] = t.y;
          u[j][i + 2] = t.z;
          u[j][i + 3] = t.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < B; ++i) {
          if (i < real) {
            if constexpr (k16) u[j][i / 2] |= (uint32_t)__ldg(p + i) << (16 * (i & 1));
            else u[j][i] = __ldg(p + i);
          }
        }
      }
    }
    if constexpr (!VEC) {  // the block's words out of what was read
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        if (shift[j] & 8) {
#pragma unroll
          for (int i = 0; i + 2 < kRead; ++i) u[j][i] = u[j][i + 2];
        }
        if (shift[j] & 4) {
#pragma unroll
          for (int i = 0; i + 1 < kRead; ++i) u[j][i] = u[j][i + 1];
        }
        if (k16 && (shift[j] & 2)) {
#pragma unroll
          for (int i = 0; i < kWords; ++i) u[j][i] = __funnelshift_r(u[j][i], u[j][i + 1], 16);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int row = row0 + 32 * (j0 + j);
      if (row >= a.rows) break;
      uint32_t code = 0;
      if (mine) {
        uint32_t w[B / 8];
        if (a.bits) {
          // (shifted here: where it is loaded, the shift would wait for each row's word in turn;
          // 11008 x 4096 bf16 NV 35.4 us, this way 28.4)
          const uint32_t bits = keep[j] >> (k % 32);
#pragma unroll
          for (int i = 0; i < kWords; ++i) {
            if constexpr (k16) u[j][i] = masked(u[j][i], bits >> (2 * i));
            else u[j][i] = (bits >> i) & 1u ? u[j][i] : 0u;
          }
        }
        if constexpr (k16) {
          uint32_t m = 0;
#pragma unroll
          for (int i = 0; i < kWords; ++i) m = max_u16x2(m, u[j][i] & 0x7FFF7FFFu);
          const BlockScale b = block_scale<FMT>(table, widest<DT, FMT>(m, inv_g));
          code = b.code;
#pragma unroll
          for (int i = 0; i < B / 8; ++i)
            w[i] = encode_words<DT, FMT>(reinterpret_cast<const uint32_t(&)[4]>(u[j][4 * i]), inv_g, b);
        } else {
          float v[B];
#pragma unroll
          for (int i = 0; i < B; ++i) v[i] = __uint_as_float(u[j][i]);
          code = encode_block<FMT, B>(table, v, inv_g, w);
        }
        if (placed[j0 + j]) {  // a row of no group keeps what it holds
          uint8_t* out = a.values + (batch * a.rows + row) * a.pitch + blk * (B / 2);
          if constexpr (FMT == HINM_FP4_NV) *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
          else *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      uint32_t four = code << (8 * (lane & 3));  // the chunk's four scales of this row
      four |= __shfl_xor_sync(0xFFFFFFFFu, four, 1);
      four |= __shfl_xor_sync(0xFFFFFFFFu, four, 2);
      word[j0 + j] = four;
    }
  }
  if ((lane & 3) != 0 || !chunk_ok) return;
  const long long chunk = blk / 4;
  if constexpr (!RAGGED) {
    if (row0 >= a.rows) return;
    uint32_t* s = reinterpret_cast<uint32_t*>(
        a.scales + ((batch * a.row_tiles + row0 / kFp4RowTile) * a.chunks + chunk) * kFp4ChunkBytes +
        (row0 % 32) * 16);
    if (row0 + 96 < a.rows) {
      *reinterpret_cast<uint4*>(s) = make_uint4(word[0], word[1], word[2], word[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (row0 + 32 * j < a.rows) s[j] = word[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (placed[j])
        *reinterpret_cast<uint32_t*>(a.scales + (tile[j] * a.chunks + chunk) * kFp4ChunkBytes +
                                     (at[j] % 32) * 16 + (at[j] / 32) * 4) = word[j];
    }
  }
}

// ------------------------------------------------------------------ depth along the source's columns
constexpr int kQDepth = 64;  // of the depth that a warp takes
constexpr int kQThreads = 128;

// The 16 bytes at p, which is aligned to its elements only, in two steps, so that a thread's loads
// need not wait for one another.  Of 16-bit elements: the one or two aligned pieces around them, and
// then the bytes out of these; of 32-bit ones, or where the pieces reach out of [lo, hi): the
// elements inside it.
struct Around {
  uint4 x, y;
  int shift;  // bytes of x before the first element
};
template <class T>
__device__ __forceinline__ Around load_around(const T* p, uintptr_t lo, uintptr_t hi) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)15;
  Around r{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0),
           (int)(reinterpret_cast<uintptr_t>(p) & 15)};
  if (sizeof(T) == 2 && at >= lo && at + (r.shift ? 32 : 16) <= hi) {
    r.x = __ldg(reinterpret_cast<const uint4*>(at));
    if (r.shift) r.y = __ldg(reinterpret_cast<const uint4*>(at) + 1);
  } else {
    r.shift = 0;
    uint32_t u[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16 / (int)sizeof(T); ++i) {
      if (reinterpret_cast<uintptr_t>(p + i) + sizeof(T) <= hi) {
        if constexpr (sizeof(T) == 2) u[i / 2] |= (uint32_t)__ldg(p + i) << (16 * (i & 1));
        else u[i] = __ldg(p + i);
      }
    }
    r.x = make_uint4(u[0], u[1], u[2], u[3]);
  }
  return r;
}
__device__ __forceinline__ uint4 piece_of(const Around& r) {
  uint32_t u[8] = {r.x.x, r.x.y, r.x.z, r.x.w, r.y.x, r.y.y, r.y.z, r.y.w};
  if (r.shift & 8) {
#pragma unroll
    for (int i = 0; i < 6; ++i) u[i] = u[i + 2];
  }
  if (r.shift & 4) {
#pragma unroll
    for (int i = 0; i < 5; ++i) u[i] = u[i + 1];
  }
  if (r.shift & 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = __funnelshift_r(u[i], u[i + 1], 16);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// Rows as 16-byte pieces: a thread takes one piece's columns (8 of 16 bits, 4 of 32)
// and 16 of the depth, a warp 8 pieces and 64 of the depth, lane = 4 * piece + depth part: the loads
// of a row part are 128 contiguous bytes, and the 8 bytes that four lanes write for a column are one
// sector.  A block of 32 lies in two neighbouring lanes.  (Two columns and 64 of the depth a thread,
// with 4-byte loads, took 22.6 us at 4096 x 4096 bf16 NV and 33.6 us MX; this takes 11.2 and 8.9.)
// ALIGNED: rows are aligned and of whole pieces.
// Blocks an SM, which bound a thread's registers: 16-bit elements five (11008 x 4096 bf16 NV 26.7 us,
// with a mask 32.0, although both keep 16 to 32 bytes of a thread outside of its 96 registers; with four
// and three blocks, as many registers as are wanted, 28.5 and 37.7), rows that start anywhere four
// (3598 x 10954 bf16 NV 33.7 us and, spilling 40 bytes, 44.6; with five 36.9 and 60.1); fp32 six (8192 x
// 8192 NV 50 us, else 58), but with a mask's 16 bytes beside the elements five (11008 x 4096 NV 43.5 us,
// with six 73.8).
template <int DT, int FMT, bool MASK, bool ALIGNED>
__global__ void __launch_bounds__(kQThreads, DT == HINM_DTYPE_F32 ? (MASK ? 5 : 6) : ALIGNED ? 5 : 4)
    quant_pieces_kernel(const QArgs a) {
  __shared__ ScaleTable table;
  fill<FMT>(table);
  ptx::enter_dependent();
  if (a.early) ptx::launch_dependents();
  check_offsets(a);
  constexpr int B = fp4_block(FMT);
  using T = typename Elem<DT>::T;
  constexpr bool k16 = sizeof(T) == 2;
  constexpr int kCols = 16 / (int)sizeof(T);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long batch = blockIdx.z;
  const int part = lane & 3;
  const int c0 = ((int)blockIdx.x * (kQThreads / 32) + warp) * 8 * kCols + (lane >> 2) * kCols;
  const long long p0 = (long long)blockIdx.y * kQDepth;
  const float inv_g = FMT == HINM_FP4_NV && a.g ? __frcp_rn(__ldg(a.g + batch)) : 1.0f;
  int k = 0, real = 0;
  // the four lanes of a piece go on together, and the 64 lie in one group or none
  const uint32_t live = __ballot_sync(0xFFFFFFFFu, c0 < a.rows);
  if (c0 >= a.rows || !depth_place(a, p0, kQDepth, k, real)) return;
  const T* src = reinterpret_cast<const T*>(a.data) + batch * a.batch_stride + c0;
  const uintptr_t lo = reinterpret_cast<uintptr_t>(src - c0);
  const uintptr_t hi = lo + ((unsigned long long)(a.depth - 1) * a.ld + a.rows) * sizeof(T);
  uint32_t u[16][4];
  uint8_t keep[MASK ? 16 : 1];  // the byte of the mask that holds the piece's columns
  // rows that a thread loads before it uses the first; rows that are not aligned bring two pieces
  // each (3598 x 10954 bf16 NV, row by row 72.0 us, four at a time 38.8, eight 34.2; MX with a mask
  // 74.9, 46.5 and 54.9)
  constexpr int kRows = ALIGNED || !k16 ? 16 : MASK && FMT == HINM_FP4_MX ? 4 : 8;
#pragma unroll
  for (int i0 = 0; i0 < 16; i0 += kRows) {
    Around t[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int i = i0 + j, d = part * 16 + i;
      t[j] = Around{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0), 0};
      if (MASK) keep[i] = 0;
      if (d < real) {
        const T* p = src + (long long)(k + d) * a.ld;
        if constexpr (ALIGNED) t[j].x = __ldg(reinterpret_cast<const uint4*>(p));
        else t[j] = load_around(p, lo, hi);
        if constexpr (MASK)
          keep[i] = __ldg(reinterpret_cast<const uint8_t*>(
                              a.bits + (batch * a.depth + k + d) * ((a.rows + 31) / 32)) + c0 / 8);
      }
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const uint4 w = ALIGNED || !k16 ? t[j].x : piece_of(t[j]);
      u[i0 + j][0] = w.x;
      u[i0 + j][1] = w.y;
      u[i0 + j][2] = w.z;
      u[i0 + j][3] = w.w;
    }
  }
  // (where a piece is loaded, its mask would make each load wait for the one before: 11008 x 4096
  // bf16 NV 72.1 us, this way 37.7, in the blocks above 32.6)
  if constexpr (MASK) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint4 t = masked_piece<DT>(make_uint4(u[i][0], u[i][1], u[i][2], u[i][3]),
                                       (uint32_t)keep[i] >> (c0 % 8));
      u[i][0] = t.x;
      u[i][1] = t.y;
      u[i][2] = t.z;
      u[i][3] = t.w;
    }
  }
  uint32_t am[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if constexpr (k16) am[c] = max_u16x2(am[c], u[i][c] & 0x7FFF7FFFu);
      else am[c] = max(am[c], u[i][c] & 0x7FFFFFFFu);
    }
  }
  if constexpr (FMT == HINM_FP4_MX) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t other = __shfl_xor_sync(live, am[c], 1);
      if constexpr (k16) am[c] = max_u16x2(am[c], other);
      else am[c] = max(am[c], other);
    }
  }
  uint32_t code[kCols];
#pragma unroll
  for (int c = 0; c < kCols; ++c) {
    uint32_t w[2];
    if constexpr (k16) {
      const uint32_t m = c & 1 ? am[c / 2] >> 16 : am[c / 2] & 0xFFFFu;
      const BlockScale b = block_scale<FMT>(table, widest<DT, FMT>(m, inv_g));
      code[c] = b.code;
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // the column's elements in pairs
        uint32_t e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          e[i] = __byte_perm(u[8 * h + 2 * i][c / 2], u[8 * h + 2 * i + 1][c / 2],
                             c & 1 ? 0x7632 : 0x5410);
        w[h] = encode_words<DT, FMT>(e, inv_g, b);
      }
    } else {
      // (the largest over g is the largest of the elements over g: rounding keeps the order)
      float top = __uint_as_float(am[c]);
      if constexpr (FMT == HINM_FP4_NV) top = __fmul_rn(top, inv_g);
      const BlockScale b = block_scale<FMT>(table, __float_as_uint(top));
      code[c] = b.code;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(u[8 * h + i][c]);
        F2 x[4] = {F2(f[0], f[1]), F2(f[2], f[3]), F2(f[4], f[5]), F2(f[6], f[7])};
        if constexpr (FMT == HINM_FP4_NV) {
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = mul2(x[i], F2(-inv_g, -inv_g));
        }
        w[h] = encode8<FMT>(x, b);
      }
    }
    const int row = c0 + c;
    long long tile;
    int at;
    if ((ALIGNED || row < a.rows) && (a.ragged != HINM_RAGGED_ROWS || row_place(a, row, tile, at)))
      *reinterpret_cast<uint2*>(a.values + (batch * a.rows + row) * a.pitch + p0 / 2 + part * 8) =
          make_uint2(w[0], w[1]);
  }
  // four lanes' bytes of four columns -> lane `part` holds the word of column 4 h + part
#pragma unroll
  for (int h = 0; h < kCols / 4; ++h) {
    uint32_t word = 0;
    const uint32_t mine = code[4 * h] | code[4 * h + 1] << 8 | code[4 * h + 2] << 16 |
                          code[4 * h + 3] << 24;  // this part's bytes of four columns
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t from = __shfl_sync(live, mine, (lane & ~3) + q);
      word |= ((from >> (8 * part)) & 0xFFu) << (8 * q);
    }
    const int row = c0 + 4 * h + part;
    long long tile;
    int at;
    if ((!ALIGNED && row >= a.rows) || !row_place(a, row, tile, at)) continue;
    uint8_t* s = a.scales +
                 ((batch * a.row_tiles + tile) * a.chunks + p0 / (4 * B)) * kFp4ChunkBytes +
                 (at % 32) * 16 + (at / 32) * 4;
    if constexpr (FMT == HINM_FP4_NV)
      *reinterpret_cast<uint32_t*>(s) = word;
    else  // each scale stands in two lanes; the 64 of the depth are half of a chunk
      *reinterpret_cast<uint16_t*>(s + (p0 / kQDepth % 2) * 2) =
          (uint16_t)((word & 0xFFu) | (word >> 8 & 0xFF00u));
  }
}

// ------------------------------------------------------------------ back
// value = fl32(code s g): code * s has at most 6 significant bits, so the only rounding in
// fp32 is that of the product with g (none when g is a power of two).
// Rows that are not aligned, in a warp's own shared memory: lane l's block of n elements starts at
// l * kPitch (16 bytes more than the block, so that lanes do not meet in a bank), and 32 consecutive
// elements go to memory at a time.  (A lane's block element by element touches 32 lines at a time:
// 4883 x 3382 bf16 NV took 112 us, this way 21.)
template <class T, int B>
struct Staged {
  static constexpr int kPitch = B * (int)sizeof(T) + 16;
  static constexpr int kBytes = 32 * kPitch;
  // Element i of the warp's 32 B, its place in shared memory, and where in the row it lies (k and
  // real: each lane's first position and how many count).  false: it does not count.
  static __device__ __forceinline__ bool at(int i, int k, int real, int& place, int& col) {
    const int from = i / B, e = i % B;
    place = from * kPitch + e * (int)sizeof(T);
    col = __shfl_sync(0xFFFFFFFFu, k, from) + e;
    return e < __shfl_sync(0xFFFFFFFFu, real, from);
  }
};

template <int DT, int FMT, bool VEC>
__global__ void __launch_bounds__(kQWarps * 32) dequant_rows_kernel(const QArgs a) {
  ptx::enter_dependent();
  if (a.early) ptx::launch_dependents();
  check_offsets(a);
  constexpr int B = fp4_block(FMT);
  using T = typename Elem<DT>::T;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  using S = Staged<T, B>;
  __shared__ __align__(16) uint8_t staged[VEC ? 16 : kQWarps * S::kBytes];
  uint8_t* mine = staged + (VEC ? 0 : warp * S::kBytes);
  const long long batch = blockIdx.z;
  const long long blk = (long long)blockIdx.y * 32 + lane;
  const int row0 = ((int)blockIdx.x >> 2) * kFp4RowTile + ((int)blockIdx.x & 3) * kQWarps + warp;
  T* dst = reinterpret_cast<T*>(a.data) + batch * a.batch_stride;
  const float g = FMT == HINM_FP4_NV && a.g ? __ldg(a.g + batch) : 1.0f;
  int k = 0, real = 0;
  if (blk >= a.nblk || !depth_place(a, blk * B, B, k, real)) real = 0;
  if (VEC && real == 0) return;
  uint32_t w[4][B / 8], code[4];
  bool here[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int row = row0 + 32 * j;
    long long tile;
    int at;
    here[j] = row < a.rows && row_place(a, row, tile, at);
    code[j] = 0;
#pragma unroll
    for (int i = 0; i < B / 8; ++i) w[j][i] = 0;
    if (!here[j] || real == 0) continue;
    const uint8_t* in = a.values + (batch * a.rows + row) * a.pitch + blk * (B / 2);
    if constexpr (B == 16) {
      const uint2 t = __ldg(reinterpret_cast<const uint2*>(in));
      w[j][0] = t.x;
      w[j][1] = t.y;
    } else {
      const uint4 t = __ldg(reinterpret_cast<const uint4*>(in));
      w[j][0] = t.x;
      w[j][1] = t.y;
      w[j][2] = t.z;
      w[j][3] = t.w;
    }
    code[j] = __ldg(a.scales + ((batch * a.row_tiles + tile) * a.chunks + blk / 4) * kFp4ChunkBytes +
                    (at % 32) * 16 + (at / 32) * 4 + blk % 4);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (!here[j]) continue;
    const float s = scale_value<FMT>(code[j]);
    T* row = dst + (long long)(row0 + 32 * j) * a.ld;
#pragma unroll
    for (int i = 0; i < B / 16; ++i) {
      float v[16];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        decode8(w[j][2 * i + h], s, g, reinterpret_cast<float(&)[8]>(v[8 * h]));
      constexpr int kOut = 4 * (int)sizeof(T);  // words of 16 elements
      if (!VEC || real == B) {
        uint32_t u[kOut];
        if constexpr (sizeof(T) == 2) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            pack8<DT>(reinterpret_cast<const float(&)[8]>(v[8 * h]),
                      reinterpret_cast<uint32_t(&)[4]>(u[4 * h]));
        } else {
#pragma unroll
          for (int q = 0; q < 16; ++q) u[q] = __float_as_uint(v[q]);
        }
        T* to = VEC ? row + k + 16 * i
                    : reinterpret_cast<T*>(mine + lane * S::kPitch + i * 4 * kOut);
        if (VEC && a.vec == 32) {
#pragma unroll
          for (int q = 0; q < kOut; q += 8) store32(reinterpret_cast<uint32_t*>(to) + q, u + q);
        } else {
#pragma unroll
          for (int q = 0; q < kOut / 4; ++q)
            reinterpret_cast<uint4*>(to)[q] =
                make_uint4(u[4 * q], u[4 * q + 1], u[4 * q + 2], u[4 * q + 3]);
        }
      } else {
#pragma unroll
        for (int q = 0; q < 16; ++q)
          if (16 * i + q < real) row[k + 16 * i + q] = Elem<DT>::of(v[q]);
      }
    }
    if constexpr (!VEC) {
      __syncwarp();
#pragma unroll 8
      for (int i = lane; i < 32 * B; i += 32) {
        int place, col;
        const bool there = S::at(i, k, real, place, col);
        if (there) row[col] = *reinterpret_cast<const T*>(mine + place);
      }
      __syncwarp();
    }
  }
}

// The way back for what quant_pieces_kernel takes: the same share of a thread.
// (Five blocks an SM for MX, with 44 bytes of a thread outside of its registers: 8192 x 8192 bf16 37.6 us
// instead of 39.6; NV, which would keep more there, 46.9 instead of 37.5.)
template <int DT, int FMT>
__global__ void __launch_bounds__(kQThreads, FMT == HINM_FP4_MX ? 5 : 1) dequant_pieces_kernel(const QArgs a) {
  ptx::enter_dependent();
  if (a.early) ptx::launch_dependents();
  check_offsets(a);
  constexpr int B = fp4_block(FMT);
  using T = typename Elem<DT>::T;
  constexpr int kCols = 16 / (int)sizeof(T);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long batch = blockIdx.z;
  const int part = lane & 3;
  const int c0 = ((int)blockIdx.x * (kQThreads / 32) + warp) * 8 * kCols + (lane >> 2) * kCols;
  const long long p0 = (long long)blockIdx.y * kQDepth;
  const float g = FMT == HINM_FP4_NV && a.g ? __ldg(a.g + batch) : 1.0f;
  int k = 0, real = 0;
  if (c0 >= a.rows || !depth_place(a, p0, kQDepth, k, real)) return;
  uint32_t there = 0;  // the columns that are in a group
  uint2 w[kCols];
  uint32_t code[kCols];
#pragma unroll
  for (int c = 0; c < kCols; ++c) {
    const int row = c0 + c;
    long long tile;
    int at;
    w[c] = make_uint2(0, 0);
    code[c] = 0;
    if (!row_place(a, row, tile, at)) continue;
    there |= 1u << c;
    w[c] = __ldg(reinterpret_cast<const uint2*>(a.values + (batch * a.rows + row) * a.pitch +
                                                p0 / 2 + part * 8));
    code[c] = __ldg(a.scales +
                    ((batch * a.row_tiles + tile) * a.chunks + p0 / (4 * B)) * kFp4ChunkBytes +
                    (at % 32) * 16 + (at / 32) * 4 + (p0 / B + part * 16 / B) % 4);
  }
  uint32_t u[16][4];  // 16 of the depth, the piece's columns
#pragma unroll
  for (int c = 0; c < kCols; c += 8 / (int)sizeof(T) / 2) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[8];
      decode8(h ? w[c].y : w[c].x, scale_value<FMT>(code[c]), g, v);
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) u[8 * h + i][c] = __float_as_uint(v[i]);
      } else {
        float x[8];
        decode8(h ? w[c + 1].y : w[c + 1].x, scale_value<FMT>(code[c + 1]), g, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[8 * h + i][c / 2] = pack2<DT>(v[i], x[i]);
      }
    }
  }
  T* dst = reinterpret_cast<T*>(a.data) + batch * a.batch_stride + c0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int d = part * 16 + i;
    if (d >= real) continue;
    T* at = dst + (long long)(k + d) * a.ld;
    if (there == (1u << kCols) - 1) {
      *reinterpret_cast<uint4*>(at) = make_uint4(u[i][0], u[i][1], u[i][2], u[i][3]);
    } else {
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        if (!(there >> c & 1u)) continue;
        if constexpr (sizeof(T) == 4) at[c] = u[i][c];
        else at[c] = (T)(u[i][c / 2] >> (16 * (c & 1)));
      }
    }
  }
}

// A thread takes a column (a stored row) and 64 of the depth.
template <int DT, int FMT>
__global__ void __launch_bounds__(kQThreads) dequant_cols_kernel(const QArgs a) {
  ptx::enter_dependent();
  if (a.early) ptx::launch_dependents();
  check_offsets(a);
  constexpr int B = fp4_block(FMT);
  using T = typename Elem<DT>::T;
  const long long batch = blockIdx.z;
  const int row = (int)blockIdx.x * kQThreads + (int)threadIdx.x;
  const long long p = (long long)blockIdx.y * kQDepth;
  const float g = FMT == HINM_FP4_NV && a.g ? __ldg(a.g + batch) : 1.0f;
  int k = 0, real = 0, at = 0;
  long long tile = 0;
  if (row >= a.rows || !depth_place(a, p, kQDepth, k, real) || !row_place(a, row, tile, at)) return;
  const uint4* in =
      reinterpret_cast<const uint4*>(a.values + (batch * a.rows + row) * a.pitch + p / 2);
  const uint4 t0 = __ldg(in), t1 = __ldg(in + 1);
  const uint32_t w[8] = {t0.x, t0.y, t0.z, t0.w, t1.x, t1.y, t1.z, t1.w};
  const uint8_t* s = a.scales +
                     ((batch * a.row_tiles + tile) * a.chunks + p / (4 * B)) * kFp4ChunkBytes +
                     (at % 32) * 16 + (at / 32) * 4;
  const uint32_t sc = FMT == HINM_FP4_NV
                          ? __ldg(reinterpret_cast<const uint32_t*>(s))
                          : __ldg(reinterpret_cast<const uint16_t*>(s + (p / kQDepth % 2) * 2));
  T* dst = reinterpret_cast<T*>(a.data) + batch * a.batch_stride + row;
#pragma unroll
  for (int i = 0; i < kQDepth / 8; ++i) {
    float x[8];
    decode8(w[i], scale_value<FMT>((sc >> (8 * (8 * i / B))) & 0xFFu), g, x);
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (8 * i + q < real) dst[(long long)(k + 8 * i + q) * a.ld] = Elem<DT>::of(x[q]);
  }
}

// ------------------------------------------------------------------ tensor scale
// g = the smallest power of two with max |x| <= 6 * 448 g, for each matrix of the batch.  It
// grows with max |x|, so every block takes the power for its own maximum and the largest wins
// (an integer maximum of positive floats' bits, in any order the same).  scale_out starts
// at 0; 2^-126 stands for a matrix of zeros.
__device__ __forceinline__ uint32_t pow2_scale_bits(uint32_t am) {
  // am = m 2^E, 2688 = 1.3125 * 2^11: the exponent is E - 11 when m <= 1.3125, else E - 10
  const int e = (int)(am >> 23) - ((am & 0x7FFFFFu) <= 0x280000u ? 11 : 10);
  return (uint32_t)(e < 1 ? 1 : e) << 23;
}

struct AmaxArgs {
  const void* src;
  long long ld, batch_stride;
  const uint32_t* bits;
  const int32_t* offsets;  // ragged: only positions in [offsets[0], offsets[groups]) count
  int rows, cols, groups, along_rows;  // along_rows: the ragged dimension is the rows
  int vec;   // rows of whole 16-byte pieces
  int one;   // one block a matrix: it writes the scale itself
  int early;
  uint32_t* out;
  int* status;
};

// The largest magnitude's bits (of the element type) in the 16 bytes t; with FINITE, of the finite
// ones.
template <int DT, bool FINITE>
__device__ __forceinline__ uint32_t widest16(uint32_t m, const uint4& t) {
  const uint32_t u[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == HINM_DTYPE_F32) {
      const uint32_t b = u[i] & 0x7FFFFFFFu;
      m = max(m, FINITE && b >= 0x7F800000u ? 0u : b);
    } else {
      constexpr uint32_t kInf = DT == HINM_DTYPE_BF16 ? 0x7F80u : 0x7C00u;
      uint32_t b = u[i] & 0x7FFF7FFFu;
      if constexpr (FINITE) {
        if ((b & 0xFFFFu) >= kInf) b &= 0xFFFF0000u;
        if ((b >> 16) >= kInf) b &= 0xFFFFu;
      }
      m = max_u16x2(m, b);
    }
  }
  return m;
}
constexpr int kAhead = 4;  // pieces of 16 bytes that a thread loads before it uses the first

template <int DT>
__device__ __forceinline__ uint32_t infinite(uint32_t m) {  // some magnitude is not finite
  if constexpr (DT == HINM_DTYPE_F32) return m >= 0x7F800000u;
  constexpr uint32_t kInf = DT == HINM_DTYPE_BF16 ? 0x7F80u : 0x7C00u;
  return (m & 0xFFFFu) >= kInf || (m >> 16) >= kInf;
}

// This thread's share of a matrix: rows without gaps (ld == cols) as one run of memory.
template <int DT, bool FINITE>
__device__ __forceinline__ uint32_t amax_share(const AmaxArgs& a, long long batch, int r0, int r1,
                                               int c0, int c1) {
  using T = typename Elem<DT>::T;
  constexpr int kPer = 16 / (int)sizeof(T);
  const T* src = reinterpret_cast<const T*>(a.src) + batch * a.batch_stride;
  const long long tid = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long threads = (long long)gridDim.x * blockDim.x;
  const long long words = (a.cols + 31) / 32;
  uint32_t m = 0;
  if (a.ld == a.cols && c0 == 0 && c1 == a.cols && (!a.bits || (a.vec && a.cols % 32 == 0))) {
    const T* first = src + (long long)r0 * a.cols;
    const long long all = (long long)(r1 - r0) * a.cols;
    // elements before the first whole piece (none where rows are aligned) and behind the last
    const long long head =
        min(all, (long long)((16 - reinterpret_cast<uintptr_t>(first) % 16) % 16 / sizeof(T)));
    const uint4* p = reinterpret_cast<const uint4*>(first + head);
    const long long n = (all - head) / kPer, tail = head + n * kPer;
    if (tid < head) m = widest16<DT, FINITE>(m, make_uint4(__ldg(first + tid), 0, 0, 0));
    if (tid < all - tail) m = widest16<DT, FINITE>(m, make_uint4(__ldg(first + tail + tid), 0, 0, 0));
    // whole words of mask a row: the bits run along with the elements, kPer of them a piece
    const uint8_t* bits =
        a.bits ? reinterpret_cast<const uint8_t*>(a.bits + (batch * a.rows + r0) * words) : nullptr;
    for (long long i = tid; i < n; i += kAhead * threads) {
      uint4 t[kAhead];
      uint32_t k[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const long long at = i + j * threads;
        t[j] = make_uint4(0, 0, 0, 0);
        k[j] = 0;
        if (at < n) {
          t[j] = __ldg(p + at);
          if (bits) k[j] = __ldg(bits + at * kPer / 8);
        }
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        m = widest16<DT, FINITE>(
            m, bits ? masked_piece<DT>(t[j], k[j] >> ((i + j * threads) * kPer % 8)) : t[j]);
    }
    return m;
  }
  // rows apart, or not whole pieces: a row's pieces (its elements where they are not aligned), one
  // after the other over all rows
  const bool pieces = a.vec && c0 == 0 && c1 == a.cols;
  const int per = pieces ? a.cols / kPer : c1 - c0;
  const long long total = (long long)(r1 - r0) * per;
  for (long long i = tid; i < total; i += kAhead * threads) {
    uint4 t[kAhead];
    uint32_t k[kAhead];
    int at_bit[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const long long at = i + j * threads;
      t[j] = make_uint4(0, 0, 0, 0);
      k[j] = 0xFFFFFFFFu;
      at_bit[j] = 0;
      if (at >= total) continue;
      const long long row = total < 0x7FFFFFFF ? (uint32_t)at / (uint32_t)per : at / per;
      const int unit = (int)(at - row * per);
      const int col = pieces ? unit * kPer : c0 + unit;
      const T* p = src + (r0 + row) * a.ld + col;
      if (a.bits) k[j] = __ldg(a.bits + (batch * a.rows + r0 + row) * words + col / 32);
      at_bit[j] = col % 32;
      if (pieces) t[j] = __ldg(reinterpret_cast<const uint4*>(p));
      else t[j].x = __ldg(p);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      m = widest16<DT, FINITE>(m, a.bits ? masked_piece<DT>(t[j], k[j] >> at_bit[j]) : t[j]);
  }
  return m;
}

// (A kernel and not a memset, so that the next kernel's launch overlaps it.)
__global__ void __launch_bounds__(256) zero_kernel(uint32_t* out, int n) {
  ptx::enter_dependent();
  ptx::launch_dependents();
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < n) out[i] = 0;
}

template <int DT>
__global__ void __launch_bounds__(256) amax_kernel(const AmaxArgs a) {
  ptx::enter_dependent();
  if (a.early) ptx::launch_dependents();
  const long long batch = blockIdx.y;
  int r0 = 0, r1 = a.rows, c0 = 0, c1 = a.cols;
  if (a.offsets) {
    check_offsets(a.offsets, a.groups, a.along_rows ? a.rows : a.cols, a.status);
    const int lo = max(0, __ldg(a.offsets)), hi = __ldg(a.offsets + a.groups);
    if (a.along_rows) {
      r0 = min(lo, a.rows);
      r1 = max(r0, min(r1, hi));
    } else {
      c0 = min(lo, a.cols);
      c1 = max(c0, min(c1, hi));
    }
  }
  uint32_t m = amax_share<DT, false>(a, batch, r0, r1, c0, c1);
  if (infinite<DT>(m)) m = amax_share<DT, true>(a, batch, r0, r1, c0, c1);  // once more without
  if constexpr (sizeof(typename Elem<DT>::T) == 2)
    m = widest<DT, HINM_FP4_MX>(m, 1.0f);  // as fp32 bits
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  __shared__ uint32_t part[8];
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max(m, part[i]);
    if (a.one) a.out[batch] = pow2_scale_bits(m);
    else atomicMax(a.out + batch, pow2_scale_bits(m));
  }
}

// ------------------------------------------------------------------ host side
QArgs q_args(void* data, long long ld, long long batch_stride, const uint32_t* bits,
             const hinm_fp4& q, int* status) {
  const Fp4Geom g = fp4_geom(q.rows, q.depth, q.ragged, q.groups);
  QArgs a{};
  a.data = data;
  a.ld = ld;
  a.batch_stride = batch_stride;
  a.bits = bits;
  a.values = q.values;
  a.scales = q.scales;
  a.g = q.tensor_scale;
  a.offsets = q.offsets;
  a.rows = q.rows;
  a.depth = q.depth;
  a.ragged = q.ragged;
  a.groups = q.groups;
  a.pitch = g.pitch();
  a.row_tiles = g.row_tiles;
  a.chunks = g.chunks(q.format);
  a.nblk = g.depth_pad / fp4_block(q.format);
  a.status = status;
  return a;
}

bool multiple(const void* p, long long ld, long long batch_stride, int batch, int esize, int to) {
  return (reinterpret_cast<uintptr_t>(p) % to) == 0 && (ld * esize) % to == 0 &&
         (batch == 1 || (batch_stride * esize) % to == 0);
}

// Fewer blocks than would fill the SMs: the next kernel's set-up then fits beside them.
bool few(dim3 grid) { return (long long)grid.x * grid.y * grid.z <= 148; }

template <int DT, int FMT>
cudaError_t run_quant(QArgs a, int axis, int batch, bool back, cudaStream_t s) {
  constexpr int es = (int)sizeof(typename Elem<DT>::T);
  const bool vec = multiple(a.data, a.ld, a.batch_stride, batch, es, 16);
  if (axis == 1) {
    // the blocks of a ragged depth start at any element
    a.vec = a.ragged == HINM_RAGGED_DEPTH || !vec                    ? 0
            : multiple(a.data, a.ld, a.batch_stride, batch, es, 32) ? 32
                                                                     : 16;
    const dim3 grid((unsigned)((a.rows + kFp4RowTile - 1) / kFp4RowTile * 4),
                    (unsigned)((a.nblk + 31) / 32), (unsigned)batch);
    a.early = few(grid);
    if (back)
      return a.vec ? launch_kernel(dequant_rows_kernel<DT, FMT, true>, grid, kQWarps * 32, 0, s,
                                   nullptr, a)
                   : launch_kernel(dequant_rows_kernel<DT, FMT, false>, grid, kQWarps * 32, 0, s,
                                   nullptr, a);
    auto kernel = a.ragged == HINM_RAGGED_ROWS
                      ? (a.vec ? quant_rows_kernel<DT, FMT, true, true>
                               : quant_rows_kernel<DT, FMT, false, true>)
                      : (a.vec ? quant_rows_kernel<DT, FMT, true, false>
                               : quant_rows_kernel<DT, FMT, false, false>);
    return launch_kernel(kernel, grid, kQWarps * 32, 0, s, nullptr, a);
  }
  const unsigned ny = (unsigned)(a.nblk * fp4_block(FMT) / kQDepth);
  constexpr int kCols = 16 / es;
  const int per = kQThreads / 32 * 8 * kCols;
  const dim3 pieces((unsigned)((a.rows + per - 1) / per), ny, (unsigned)batch);
  const bool whole = vec && a.rows % kCols == 0;
  if (!back || whole) {
    a.early = few(pieces);
    auto kernel = back      ? dequant_pieces_kernel<DT, FMT>
                  : !a.bits ? (whole ? quant_pieces_kernel<DT, FMT, false, true>
                                     : quant_pieces_kernel<DT, FMT, false, false>)
                            : (whole ? quant_pieces_kernel<DT, FMT, true, true>
                                     : quant_pieces_kernel<DT, FMT, true, false>);
    return launch_kernel(kernel, pieces, kQThreads, 0, s, nullptr, a);
  }
  // back into other rows: element by element, a column a thread
  const dim3 grid((unsigned)((a.rows + kQThreads - 1) / kQThreads), ny, (unsigned)batch);
  a.early = few(grid);
  return launch_kernel(dequant_cols_kernel<DT, FMT>, grid, kQThreads, 0, s, nullptr, a);
}

cudaError_t dispatch(const QArgs& a, int dtype, int format, int axis, int batch, bool back,
                     cudaStream_t s) {
  const bool nv = format == HINM_FP4_NV;
  switch (dtype) {
    case HINM_DTYPE_BF16:
      return nv ? run_quant<HINM_DTYPE_BF16, HINM_FP4_NV>(a, axis, batch, back, s)
                : run_quant<HINM_DTYPE_BF16, HINM_FP4_MX>(a, axis, batch, back, s);
    case HINM_DTYPE_F16:
      return nv ? run_quant<HINM_DTYPE_F16, HINM_FP4_NV>(a, axis, batch, back, s)
                : run_quant<HINM_DTYPE_F16, HINM_FP4_MX>(a, axis, batch, back, s);
    default:
      return nv ? run_quant<HINM_DTYPE_F32, HINM_FP4_NV>(a, axis, batch, back, s)
                : run_quant<HINM_DTYPE_F32, HINM_FP4_MX>(a, axis, batch, back, s);
  }
}

}  // namespace

cudaError_t launch_fp4_quantize(const void* src, int dtype, long long ld, long long batch_stride,
                                int axis, const uint32_t* bits, const hinm_fp4& q, int* status,
                                cudaStream_t s) {
  return dispatch(q_args(const_cast<void*>(src), ld, batch_stride, bits, q, status), dtype,
                  q.format, axis, q.batch, false, s);
}

cudaError_t launch_fp4_dequantize(const hinm_fp4& q, int axis, void* dst, int dtype, long long ld,
                                  long long batch_stride, int* status, cudaStream_t s) {
  return dispatch(q_args(dst, ld, batch_stride, nullptr, q, status), dtype, q.format, axis,
                  q.batch, true, s);
}

cudaError_t launch_fp4_tensor_scale(const void* src, int dtype, long long ld,
                                    long long batch_stride, int axis, const uint32_t* bits,
                                    const hinm_fp4& q, int* status, cudaStream_t s) {
  AmaxArgs a{};
  a.status = status;
  a.src = src;
  a.ld = ld;
  a.batch_stride = batch_stride;
  a.bits = bits;
  a.offsets = q.ragged == HINM_RAGGED_NONE ? nullptr : q.offsets;
  a.rows = axis == 1 ? q.rows : q.depth;
  a.cols = axis == 1 ? q.depth : q.rows;
  a.groups = q.groups;
  a.along_rows = (q.ragged == HINM_RAGGED_ROWS) == (axis == 1);
  a.out = reinterpret_cast<uint32_t*>(q.tensor_scale);
  const int es = dtype == HINM_DTYPE_F32 ? 4 : 2;
  a.vec = a.cols * es % 16 == 0 && multiple(src, ld, batch_stride, q.batch, es, 16);
  // kAhead pieces of 16 bytes a thread; one block a matrix (of up to 64 KB) needs no other's maximum
  // and no starting value.  Larger ones have several whatever their number: 296 x 2048 x 2048 bf16
  // 340 us, with one block each 441 (296 x 512 x 512: 26 and 32; 512 x 256 x 512: 25 and 23).
  const long long pieces = (long long)a.rows * a.cols * es / 16;
  long long blocks = (pieces + 256 * kAhead - 1) / (256 * kAhead);
  a.one = blocks <= 4;
  if (blocks * q.batch > 148 * 8) blocks = (148 * 8 + q.batch - 1) / q.batch;
  if (a.one) blocks = 1;
  else if (cudaError_t e = launch_kernel(zero_kernel, dim3((unsigned)((q.batch + 255) / 256)), 256, 0,
                                         s, nullptr, a.out, q.batch);
           e != cudaSuccess)
    return e;
  const dim3 grid((unsigned)blocks, (unsigned)q.batch);
  a.early = few(grid);
  switch (dtype) {
    case HINM_DTYPE_BF16:
      return launch_kernel(amax_kernel<HINM_DTYPE_BF16>, grid, 256, 0, s, nullptr, a);
    case HINM_DTYPE_F16:
      return launch_kernel(amax_kernel<HINM_DTYPE_F16>, grid, 256, 0, s, nullptr, a);
    default:
      return launch_kernel(amax_kernel<HINM_DTYPE_F32>, grid, 256, 0, s, nullptr, a);
  }
}

}  // namespace hinm
