// b1. Microscaled 4-bit quantisation (hinm.h, section b1): the tensor scale, the quantiser
// and the way back.
//
//   NV: x' = fl32(x / g) (x times fl32(1/g)), s = e4m3(max |x'| / 6), code = e2m1(x' / s)
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
// The kernels are bound by DRAM: a bf16 element costs 2 bytes in and 0.5 + 1/16 (NV) or
// 0.5 + 1/32 (MX) bytes out.
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

// ------------------------------------------------------------------ elements
template <int DT>
struct Elem;
template <>
struct Elem<HINM_DTYPE_BF16> {
  using T = uint16_t;
  static __device__ float load(const T* p) { return __uint_as_float((uint32_t)__ldg(p) << 16); }
  static __device__ T of(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
  static __device__ void unpack(uint32_t w, float& a, float& b) {
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xFFFF0000u);
  }
};
template <>
struct Elem<HINM_DTYPE_F16> {
  using T = uint16_t;
  static __device__ float load(const T* p) { return __half2float(__ushort_as_half(__ldg(p))); }
  static __device__ T of(float v) { return __half_as_ushort(__float2half_rn(v)); }
  static __device__ void unpack(uint32_t w, float& a, float& b) {
    a = __half2float(__ushort_as_half((unsigned short)(w & 0xFFFF)));
    b = __half2float(__ushort_as_half((unsigned short)(w >> 16)));
  }
};
template <>
struct Elem<HINM_DTYPE_F32> {
  using T = uint32_t;
  static __device__ float load(const T* p) { return __uint_as_float(__ldg(p)); }
  static __device__ T of(float v) { return __float_as_uint(v); }
};

// n (<= B) consecutive elements into v, zeros behind them.  vec: p is 16-byte aligned.
template <int DT, int B>
__device__ __forceinline__ void load_run(const typename Elem<DT>::T* p, int n, bool vec,
                                         float (&v)[B]) {
  if (vec && n == B) {
    constexpr int kPer = 16 / sizeof(typename Elem<DT>::T);
    uint4 w[B / kPer];
#pragma unroll
    for (int i = 0; i < B / kPer; ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
#pragma unroll
    for (int i = 0; i < B / kPer; ++i) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(typename Elem<DT>::T) == 2)
          Elem<DT>::unpack(u[j], v[i * kPer + 2 * j], v[i * kPer + 2 * j + 1]);
        else
          v[i * kPer + j] = __uint_as_float(u[j]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < B; ++i) v[i] = i < n ? Elem<DT>::load(p + i) : 0.0f;
  }
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

// One block's codes (B / 8 words) and its scale byte.  A block with a value that is not
// finite (NV: after the division by g) gets the scale NaN and codes of zero, so that whatever
// reads it is NaN.  inv_g: fl32(1 / g) (NV).
template <int FMT, int B>
__device__ __forceinline__ uint32_t encode_block(float (&v)[B], float inv_g, uint32_t (&w)[B / 8]) {
  uint32_t am = 0;  // largest magnitude's bits: NaN and infinities are the largest of all
#pragma unroll
  for (int i = 0; i < B; ++i) {
    if constexpr (FMT == HINM_FP4_NV) v[i] = __fmul_rn(v[i], inv_g);
    am = max(am, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  }
  if (am >= 0x7F800000u) {
#pragma unroll
    for (int i = 0; i < B / 8; ++i) w[i] = 0;
    return FMT == HINM_FP4_NV ? 0x7Fu : 0xFFu;
  }
  uint32_t code;
  if constexpr (FMT == HINM_FP4_NV) {
    code = e4m3_of(__fdiv_rn(__uint_as_float(am), 6.0f));
    const float s = e4m3_value(code);
    const float r = code ? __frcp_rn(s) : 0.0f;  // scale 0: every code is 0
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const float q0 = __fmul_rn(v[i], r);
      v[i] = __fmaf_rn(__fmaf_rn(-q0, s, v[i]), r, q0);
    }
  } else {
    const int e = (int)(am >> 23) - 2;  // exponent of the largest less that of 4 = 2^2 (6 = 1.5 * 2^2)
    code = e > 0 ? (uint32_t)e : 0u;
    const float r = __uint_as_float((254u - code) << 23);
#pragma unroll
    for (int i = 0; i < B; ++i) v[i] = __fmul_rn(v[i], r);
  }
#pragma unroll
  for (int i = 0; i < B / 8; ++i) w[i] = e2m1x8(v + 8 * i);
  return code;
}

template <int FMT>
__device__ __forceinline__ float scale_value(uint32_t code) {
  if constexpr (FMT == HINM_FP4_NV) return e4m3_value(code);
  // 2^(code - 127): code 0 is the subnormal 2^-127, code 255 NaN
  return __uint_as_float(code == 255u ? 0x7FC00000u : code ? code << 23 : 0x00400000u);
}

// Value of the e2m1 code in the low 4 bits of c.
__device__ __forceinline__ float e2m1_value(uint32_t c) {
  const uint32_t e = (c >> 1) & 3u, m = c & 1u;
  const float a = e ? __uint_as_float(((126u + e) << 23) | (m << 22)) : 0.5f * (float)m;
  return (c & 8u) ? -a : a;
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
  int rows, depth, ragged, groups, vec;
  long long pitch, row_tiles, chunks, nblk;  // nblk: blocks of the stored depth
  int early;  // let the stream's next kernel begin its set-up (few blocks)
  int* status;
};

// Where a stored row's scales lie: its tile and its place in it.  false: the row is in no group.
__device__ __forceinline__ bool row_place(const QArgs& a, int row, long long& tile, int& at) {
  if (a.ragged != HINM_RAGGED_ROWS) {
    tile = row / kFp4RowTile;
    at = row % kFp4RowTile;
    return true;
  }
  // the last of several groups that start at one row is the one that may hold it
  const int e = group_of(a.groups, row, [&](int i) { return (long long)__ldg(a.offsets + i); });
  const int o = __ldg(a.offsets + e), end = __ldg(a.offsets + e + 1);
  if (row < o || row >= end) return false;
  tile = fp4_group_tile(o, e) + (row - o) / kFp4RowTile;
  at = (row - o) % kFp4RowTile;
  if (o < 0 || tile >= a.row_tiles) {
    ptx::record_status(a.status, HINM_ERR_INVALID_ARG);
    return false;
  }
  return true;
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
  if (o < 0 || end > a.depth || end < o) {
    ptx::record_status(a.status, HINM_ERR_INVALID_ARG);
    return false;
  }
  const long long n = end - o;
  if (local < 0 || local >= (n + kFp4DepthPad - 1) / kFp4DepthPad * kFp4DepthPad) return false;
  const long long left = n - local;
  src = (int)(o + local);
  real = left <= 0 ? 0 : left < count ? (int)left : count;
  return true;
}

// ------------------------------------------------------------------ depth along the source's rows
// A warp takes 32 consecutive blocks of one row (a lane a block), and four rows 32 apart in
// turn: their scales for four blocks of depth are 16 contiguous bytes of a chunk.
constexpr int kQWarps = 8;

template <int DT, int FMT>
__global__ void __launch_bounds__(kQWarps * 32) quant_rows_kernel(const QArgs a) {
  ptx::enter_dependent();
  if (a.early) ptx::launch_dependents();
  constexpr int B = fp4_block(FMT);
  using T = typename Elem<DT>::T;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long batch = blockIdx.z;
  const long long blk = (long long)blockIdx.y * 32 + lane;
  const int row0 = ((int)blockIdx.x >> 2) * kFp4RowTile + ((int)blockIdx.x & 3) * kQWarps + warp;
  const T* src = reinterpret_cast<const T*>(a.data) + batch * a.batch_stride;
  const float inv_g = FMT == HINM_FP4_NV && a.g ? __frcp_rn(__ldg(a.g + batch)) : 1.0f;
  int k = 0, real = 0;
  const bool mine = blk < a.nblk && depth_place(a, blk * B, B, k, real);
  const bool chunk_ok = __shfl_sync(0xFFFFFFFFu, mine, lane & ~3);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int row = row0 + 32 * j;
    if (row >= a.rows) break;
    long long tile;
    int at;
    if (!row_place(a, row, tile, at)) continue;
    uint32_t code = 0;
    if (mine) {
      float v[B];
      load_run<DT, B>(src + (long long)row * a.ld + k, real, a.vec, v);
      if (a.bits && real > 0) {
        const long long words = (a.depth + 31) / 32;
        const uint32_t m =
            __ldg(a.bits + (batch * a.rows + row) * words + k / 32) >> (k % 32);
#pragma unroll
        for (int i = 0; i < B; ++i)
          if (!((m >> i) & 1u)) v[i] = 0.0f;
      }
      uint32_t w[B / 8];
      code = encode_block<FMT, B>(v, inv_g, w);
      uint8_t* out = a.values + (batch * a.rows + row) * a.pitch + blk * (B / 2);
      if constexpr (FMT == HINM_FP4_NV) *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
      else *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    uint32_t word = code << (8 * (lane & 3));  // the chunk's four scales in one word
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 1);
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2);
    if ((lane & 3) == 0 && chunk_ok)
      *reinterpret_cast<uint32_t*>(a.scales +
                                   ((batch * a.row_tiles + tile) * a.chunks + blk / 4) *
                                       kFp4ChunkBytes +
                                   (at % 32) * 16 + (at / 32) * 4) = word;
  }
}

// ------------------------------------------------------------------ depth along the source's columns
// A thread takes V columns of the source (V stored rows) and 64 of the depth: 32 bytes of
// values, one whole sector, for each.
constexpr int kQDepth = 64;
constexpr int kQThreads = 128;

template <int DT, int FMT, int V>
__global__ void __launch_bounds__(kQThreads) quant_cols_kernel(const QArgs a) {
  ptx::enter_dependent();
  if (a.early) ptx::launch_dependents();
  constexpr int B = fp4_block(FMT);
  using T = typename Elem<DT>::T;
  const long long batch = blockIdx.z;
  const int c0 = ((int)blockIdx.x * kQThreads + (int)threadIdx.x) * V;
  const long long p = (long long)blockIdx.y * kQDepth;
  const float inv_g = FMT == HINM_FP4_NV && a.g ? __frcp_rn(__ldg(a.g + batch)) : 1.0f;
  int k = 0, real = 0;
  if (c0 >= a.rows || !depth_place(a, p, kQDepth, k, real)) return;
  const T* src = reinterpret_cast<const T*>(a.data) + batch * a.batch_stride + c0;
  uint32_t w[V][kQDepth / 8];
  uint32_t sc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) sc[v] = 0;
#pragma unroll
  for (int b = 0; b < kQDepth / B; ++b) {
    float x[V][B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int d = b * B + i;
#pragma unroll
      for (int v = 0; v < V; ++v) x[v][i] = 0.0f;
      if (d < real) {
        const T* at = src + (long long)(k + d) * a.ld;
        if constexpr (V == 2 && sizeof(T) == 2) {
          Elem<DT>::unpack(__ldg(reinterpret_cast<const uint32_t*>(at)), x[0][i], x[1][i]);
        } else if constexpr (V == 2) {
          const uint2 t = __ldg(reinterpret_cast<const uint2*>(at));
          x[0][i] = __uint_as_float(t.x);
          x[1][i] = __uint_as_float(t.y);
        } else {
          x[0][i] = Elem<DT>::load(at);
        }
        if (a.bits) {
          const long long words = (a.rows + 31) / 32;
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const uint32_t m = __ldg(a.bits + (batch * a.depth + k + d) * words + (c0 + v) / 32);
            if (!((m >> ((c0 + v) % 32)) & 1u)) x[v][i] = 0.0f;
          }
        }
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      uint32_t t[B / 8];
      sc[v] |= encode_block<FMT, B>(x[v], inv_g, t) << (8 * b);
#pragma unroll
      for (int i = 0; i < B / 8; ++i) w[v][b * (B / 8) + i] = t[i];
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int row = c0 + v;
    long long tile;
    int at;
    if (row >= a.rows || !row_place(a, row, tile, at)) continue;
    uint4* out = reinterpret_cast<uint4*>(a.values + (batch * a.rows + row) * a.pitch + p / 2);
    out[0] = make_uint4(w[v][0], w[v][1], w[v][2], w[v][3]);
    out[1] = make_uint4(w[v][4], w[v][5], w[v][6], w[v][7]);
    uint8_t* s = a.scales +
                 ((batch * a.row_tiles + tile) * a.chunks + p / (4 * B)) * kFp4ChunkBytes +
                 (at % 32) * 16 + (at / 32) * 4;
    if constexpr (FMT == HINM_FP4_NV) *reinterpret_cast<uint32_t*>(s) = sc[v];
    else *reinterpret_cast<uint16_t*>(s + (p / kQDepth % 2) * 2) = (uint16_t)sc[v];
  }
}

// ------------------------------------------------------------------ back
// value = fl32(code s g): code * s has at most 6 significant bits, so the only rounding in
// fp32 is that of the product with g (none when g is a power of two).
template <int DT, int FMT>
__global__ void __launch_bounds__(kQWarps * 32) dequant_rows_kernel(const QArgs a) {
  ptx::enter_dependent();
  if (a.early) ptx::launch_dependents();
  constexpr int B = fp4_block(FMT);
  using T = typename Elem<DT>::T;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long batch = blockIdx.z;
  const long long blk = (long long)blockIdx.y * 32 + lane;
  const int row0 = ((int)blockIdx.x >> 2) * kFp4RowTile + ((int)blockIdx.x & 3) * kQWarps + warp;
  T* dst = reinterpret_cast<T*>(a.data) + batch * a.batch_stride;
  const float g = FMT == HINM_FP4_NV && a.g ? __ldg(a.g + batch) : 1.0f;
  int k = 0, real = 0;
  if (blk >= a.nblk || !depth_place(a, blk * B, B, k, real) || real == 0) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int row = row0 + 32 * j;
    if (row >= a.rows) break;
    long long tile;
    int at;
    if (!row_place(a, row, tile, at)) continue;
    const uint8_t* in = a.values + (batch * a.rows + row) * a.pitch + blk * (B / 2);
    uint32_t w[B / 8];
#pragma unroll
    for (int i = 0; i < B / 8; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(in) + i);
    const float s = scale_value<FMT>(
        __ldg(a.scales + ((batch * a.row_tiles + tile) * a.chunks + blk / 4) * kFp4ChunkBytes +
              (at % 32) * 16 + (at / 32) * 4 + blk % 4));
    T o[B];
#pragma unroll
    for (int i = 0; i < B; ++i)
      o[i] = Elem<DT>::of(__fmul_rn(__fmul_rn(e2m1_value(w[i / 8] >> (4 * (i % 8))), s), g));
    T* out = dst + (long long)row * a.ld + k;
    if (a.vec && real == B) {
      constexpr int kPer = 16 / sizeof(T);
#pragma unroll
      for (int i = 0; i < B / kPer; ++i) {
        uint32_t u[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if constexpr (sizeof(T) == 2)
            u[q] = (uint32_t)o[i * kPer + 2 * q] | ((uint32_t)o[i * kPer + 2 * q + 1] << 16);
          else
            u[q] = o[i * kPer + q];
        }
        reinterpret_cast<uint4*>(out)[i] = make_uint4(u[0], u[1], u[2], u[3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < B; ++i)
        if (i < real) out[i] = o[i];
    }
  }
}

template <int DT, int FMT, int V>
__global__ void __launch_bounds__(kQThreads) dequant_cols_kernel(const QArgs a) {
  ptx::enter_dependent();
  if (a.early) ptx::launch_dependents();
  constexpr int B = fp4_block(FMT);
  using T = typename Elem<DT>::T;
  const long long batch = blockIdx.z;
  const int c0 = ((int)blockIdx.x * kQThreads + (int)threadIdx.x) * V;
  const long long p = (long long)blockIdx.y * kQDepth;
  const float g = FMT == HINM_FP4_NV && a.g ? __ldg(a.g + batch) : 1.0f;
  int k = 0, real = 0;
  if (c0 >= a.rows || !depth_place(a, p, kQDepth, k, real)) return;
  T* dst = reinterpret_cast<T*>(a.data) + batch * a.batch_stride + c0;
  uint32_t w[V][kQDepth / 8];
  uint32_t sc[V];
  bool ok[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int row = c0 + v;
    long long tile = 0;
    int at = 0;
    ok[v] = row < a.rows && row_place(a, row, tile, at);
    sc[v] = 0;
#pragma unroll
    for (int i = 0; i < kQDepth / 8; ++i) w[v][i] = 0;
    if (!ok[v]) continue;
    const uint4* in =
        reinterpret_cast<const uint4*>(a.values + (batch * a.rows + row) * a.pitch + p / 2);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 t = __ldg(in + i);
      w[v][4 * i] = t.x;
      w[v][4 * i + 1] = t.y;
      w[v][4 * i + 2] = t.z;
      w[v][4 * i + 3] = t.w;
    }
    const uint8_t* s = a.scales +
                       ((batch * a.row_tiles + tile) * a.chunks + p / (4 * B)) * kFp4ChunkBytes +
                       (at % 32) * 16 + (at / 32) * 4;
    if constexpr (FMT == HINM_FP4_NV) sc[v] = __ldg(reinterpret_cast<const uint32_t*>(s));
    else sc[v] = __ldg(reinterpret_cast<const uint16_t*>(s + (p / kQDepth % 2) * 2));
  }
#pragma unroll
  for (int d = 0; d < kQDepth; ++d) {
    if (d >= real) break;
    T o[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
      o[v] = Elem<DT>::of(
          __fmul_rn(__fmul_rn(e2m1_value(w[v][d / 8] >> (4 * (d % 8))),
                              scale_value<FMT>((sc[v] >> (8 * (d / B))) & 0xFFu)), g));
    T* at = dst + (long long)(k + d) * a.ld;
    if (V == 2 && ok[0] && ok[V - 1]) {
      if constexpr (sizeof(T) == 2)
        *reinterpret_cast<uint32_t*>(at) = (uint32_t)o[0] | ((uint32_t)o[V - 1] << 16);
      else
        *reinterpret_cast<uint2*>(at) = make_uint2(o[0], o[V - 1]);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (ok[v]) at[v] = o[v];
    }
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
  int rows, cols, groups, along_rows, vec;  // along_rows: the ragged dimension is the rows
  uint32_t* out;
  int early;
};

template <int DT>
__global__ void __launch_bounds__(256) amax_kernel(const AmaxArgs a) {
  ptx::enter_dependent();
  if (a.early) ptx::launch_dependents();
  using T = typename Elem<DT>::T;
  constexpr int kRun = 16;
  const long long batch = blockIdx.y;
  int r0 = 0, r1 = a.rows, c0 = 0, c1 = a.cols;
  if (a.offsets) {
    const int lo = max(0, __ldg(a.offsets)), hi = __ldg(a.offsets + a.groups);
    if (a.along_rows) {
      r0 = lo;
      r1 = min(r1, hi);
    } else {
      c0 = lo;
      c1 = min(c1, hi);
    }
  }
  const T* src = reinterpret_cast<const T*>(a.src) + batch * a.batch_stride;
  const int runs = (a.cols + kRun - 1) / kRun;
  const long long total = (long long)max(0, r1 - r0) * runs;
  const long long words = (a.cols + 31) / 32;
  uint32_t am = 0;
  for (long long t = (long long)blockIdx.x * 256 + threadIdx.x; t < total;
       t += (long long)gridDim.x * 256) {
    const int row = r0 + (int)(t / runs), col = (int)(t % runs) * kRun;
    float v[kRun];
    load_run<DT, kRun>(src + (long long)row * a.ld + col, min(kRun, a.cols - col), a.vec, v);
    uint32_t keep = 0xFFFFu;
    if (a.bits) keep = __ldg(a.bits + (batch * a.rows + row) * words + col / 32) >> (col % 32);
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const uint32_t b = __float_as_uint(v[i]) & 0x7FFFFFFFu;
      if (b < 0x7F800000u && ((keep >> i) & 1u) && col + i >= c0 && col + i < c1) am = max(am, b);
    }
  }
  am = __reduce_max_sync(0xFFFFFFFFu, am);
  __shared__ uint32_t part[8];
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = am;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 1; i < 8; ++i) am = max(am, part[i]);
    atomicMax(a.out + batch, pow2_scale_bits(am));
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
  if (axis == 1) {
    // 16-byte accesses; the blocks of a ragged depth start at any element
    a.vec = a.ragged != HINM_RAGGED_DEPTH && multiple(a.data, a.ld, a.batch_stride, batch, es, 16);
    const dim3 grid((unsigned)((a.rows + kFp4RowTile - 1) / kFp4RowTile * 4),
                    (unsigned)((a.nblk + 31) / 32), (unsigned)batch);
    a.early = few(grid);
    return back ? launch_kernel(dequant_rows_kernel<DT, FMT>, grid, kQWarps * 32, 0, s, nullptr, a)
                : launch_kernel(quant_rows_kernel<DT, FMT>, grid, kQWarps * 32, 0, s, nullptr, a);
  }
  // two columns a thread where every pair of them is one aligned load
  const bool two = a.rows % 2 == 0 && multiple(a.data, a.ld, a.batch_stride, batch, es, 2 * es);
  const int per = kQThreads * (two ? 2 : 1);
  const dim3 grid((unsigned)((a.rows + per - 1) / per),
                  (unsigned)(a.nblk * fp4_block(FMT) / kQDepth), (unsigned)batch);
  a.early = few(grid);
  if (two)
    return back ? launch_kernel(dequant_cols_kernel<DT, FMT, 2>, grid, kQThreads, 0, s, nullptr, a)
                : launch_kernel(quant_cols_kernel<DT, FMT, 2>, grid, kQThreads, 0, s, nullptr, a);
  return back ? launch_kernel(dequant_cols_kernel<DT, FMT, 1>, grid, kQThreads, 0, s, nullptr, a)
              : launch_kernel(quant_cols_kernel<DT, FMT, 1>, grid, kQThreads, 0, s, nullptr, a);
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
                                    const hinm_fp4& q, cudaStream_t s) {
  AmaxArgs a{};
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
  a.vec = multiple(src, ld, batch_stride, q.batch, dtype == HINM_DTYPE_F32 ? 4 : 2, 16);
  cudaError_t e = cudaMemsetAsync(q.tensor_scale, 0, (size_t)q.batch * 4, s);
  if (e != cudaSuccess) return e;
  const long long runs = (long long)a.rows * ((a.cols + 15) / 16);
  long long blocks = (runs + 256 * 4 - 1) / (256 * 4);
  if (blocks > 148 * 8) blocks = 148 * 8;
  if (blocks < 1) blocks = 1;
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
