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
// A persistent CTA walks tiles of 128 rows of A by BN rows of B.  Warps:
//   0      copies: per stage of 256 of the depth, TMA boxes of A and B (128-byte rows, 128-byte
//          swizzle) and the chunks of their scales
//   1      MMA: scales to tensor memory, then up to four products a stage
//   2..5   epilogue: 32 lanes of the accumulator each
// A stage's scales have tensor-memory columns of their own, which are written again only after
// the stage's products are done (the same commit that frees its shared memory).  Every wait is
// bounded (ptx.cuh); after one runs out the CTA stops, drains what it issued and returns.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include <mutex>

#include "fp4.cuh"
#include "hinm_internal.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace hinm {
namespace {

constexpr int kStageDepth = 256;  // of the depth in one stage: 128-byte rows

struct MmArgs {
  const uint8_t* sa;  // scales of A and B
  const uint8_t* sb;
  const float* ga;  // tensor scales (A: one a matrix), or null
  const float* gb;
  const float* bias;
  const int32_t* offsets;
  void* Y;
  long long ldy, y_batch;          // elements
  long long a_tiles, a_chunks;     // scale tiles of one matrix of A; chunks of a tile
  long long b_tiles, b_chunks;     // scale tiles of all of B
  int M, N, depth, groups, ragged, mt, nt;  // tiles of M; of N (unless ragged rows)
  int steps;                       // products of 64 over the whole depth (unless ragged depth)
  int dtype, transposed, act;
  int* status;
};

template <int FMT, int BN>
struct MmCfg {
  static constexpr int kChunkDepth = 4 * fp4_block(FMT);
  static constexpr int kChunks = kStageDepth / kChunkDepth;  // scale chunks a stage
  static constexpr int kBTiles = BN > 128 ? 2 : 1;           // scale tiles of a B tile
  static constexpr int kABytes = 128 * 128;
  static constexpr int kBBytes = BN * 128;
  static constexpr int kSfTile = kChunks * kFp4ChunkBytes;
  static constexpr int kSfBytes = (1 + kBTiles) * kSfTile;
  static constexpr int kStageBytes = kABytes + kBBytes + kSfBytes;
  static constexpr int kSfCols = kChunks * 4 * (1 + kBTiles);
  static constexpr int kAccBufs = BN <= 128 ? 2 : 1;
  static constexpr int kAccCols = BN;
  static constexpr int kStagesSmem = 221 * 1024 / kStageBytes;
  static constexpr int kStagesTmem = (512 - kAccBufs * kAccCols) / kSfCols;
  static constexpr int kStagesRaw = kStagesSmem < kStagesTmem ? kStagesSmem : kStagesTmem;
  static constexpr int kStages = kStagesRaw > 8 ? 8 : kStagesRaw;
  static_assert(kStages >= 2, "stages");
  static_assert(kAccBufs * kAccCols + kStages * kSfCols <= 512, "tensor memory");
  static constexpr size_t kSmemBytes = 1024 + (size_t)kStages * kStageBytes + 256 +
                                       (kFp4MaxGroups + 1) * 4;
};
constexpr int kMmThreads = 192;

// One tile of work.
struct Tile {
  int e;         // expert (matrix of A's batch), 0 without groups
  int m0;        // first row of A
  int n0, nlen;  // first row of B (its own row number) and how many rows count
  long long sb_tile;  // scale tile of B's first row
  int sb_shift;  // place of that row in the tile (0 or 64)
  long long k0;  // first stored depth
  int steps;     // products of 64
};

// cum: ragged rows: B tiles before each group
template <int BN>
__device__ __forceinline__ Tile tile_of(const MmArgs& a, const int* cum, int t) {
  Tile r;
  r.k0 = 0;
  r.steps = a.steps;
  const int m = t % a.mt, u = t / a.mt;
  r.m0 = m * 128;
  if (a.ragged == HINM_RAGGED_ROWS) {
    int lo = 0, hi = a.groups - 1;  // the last group with cum[e] <= u: empty ones share a start
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (cum[mid] <= u) lo = mid;
      else hi = mid - 1;
    }
    const int o = __ldg(a.offsets + lo), end = __ldg(a.offsets + lo + 1);
    const int j = (u - cum[lo]) * BN;
    r.e = lo;
    r.n0 = o + j;
    r.nlen = min(BN, end - r.n0);
    r.sb_tile = fp4_group_tile(o, lo) + j / kFp4RowTile;
    r.sb_shift = j % kFp4RowTile;
  } else {
    r.e = u / a.nt;
    r.n0 = (u - r.e * a.nt) * BN;
    r.nlen = min(BN, a.N - r.n0);
    r.sb_tile = r.n0 / kFp4RowTile;
    r.sb_shift = r.n0 % kFp4RowTile;
    if (a.ragged == HINM_RAGGED_DEPTH) {
      const int o = __ldg(a.offsets + r.e), end = __ldg(a.offsets + r.e + 1);
      r.k0 = fp4_group_tile(o, r.e) * kFp4DepthPad;
      r.steps = (end - o + kFp4DepthPad - 1) / kFp4DepthPad * 2;
    }
  }
  return r;
}

__device__ __forceinline__ float activate(float x, int act) {
  if (act == HINM_ACT_RELU) return fmaxf(x, 0.0f);
  if (act == HINM_ACT_SILU) return x / (1.0f + expf(-x));
  if (act == HINM_ACT_GELU) return 0.5f * x * (1.0f + erff(x * 0.70710678118654752f));
  return x;
}

__device__ __forceinline__ void store_one(const MmArgs& a, long long at, float v) {
  if (a.dtype == HINM_DTYPE_F32) reinterpret_cast<float*>(a.Y)[at] = v;
  else if (a.dtype == HINM_DTYPE_BF16)
    reinterpret_cast<__nv_bfloat16*>(a.Y)[at] = __float2bfloat16_rn(v);
  else reinterpret_cast<__half*>(a.Y)[at] = __float2half_rn(v);
}

template <int FMT, int BN>
__global__ void __launch_bounds__(kMmThreads, 1)
    fp4_mm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                  const MmArgs a) {
  using C = MmCfg<FMT, BN>;
  extern __shared__ uint8_t smem_raw[];
  ptx::enter_dependent();
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStageBytes);
  // [0,S) full, [S,2S) empty, 2S+{0,1} accumulator full, 2S+{2,3} accumulator empty, 2S+4 drain
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * C::kStages + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* bad_flag = reinterpret_cast<volatile int*>(tmem_slot + 2);
  int* cum = reinterpret_cast<int*>(smem + C::kStages * C::kStageBytes + 256);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
      ptx::mbar_init(acce_bar(b), 4);
    }
    ptx::mbar_init(drain_bar, 1);
    *abort_flag = 0;
    *bad_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish();
  }
  __syncthreads();
  // offsets that decrease or leave the matrix are reported, and nothing is computed
  if (a.ragged != HINM_RAGGED_NONE) {
    const int limit = a.ragged == HINM_RAGGED_ROWS ? a.N : a.depth;
    for (int e = threadIdx.x; e < a.groups; e += kMmThreads) {
      const int o = __ldg(a.offsets + e), end = __ldg(a.offsets + e + 1);
      if (o < 0 || end < o || end > limit) *bad_flag = 1;
    }
    if (a.ragged == HINM_RAGGED_ROWS && warp == 0) {
      int before = 0;
      for (int base = 0; base < a.groups; base += 32) {
        const int e = base + lane;
        int n = e < a.groups ? __ldg(a.offsets + e + 1) - __ldg(a.offsets + e) : 0;
        n = n > 0 ? (n + BN - 1) / BN : 0;
        int sum = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int up = __shfl_up_sync(0xFFFFFFFFu, sum, d);
          if (lane >= d) sum += up;
        }
        if (e < a.groups) cum[e] = before + sum - n;
        before += __shfl_sync(0xFFFFFFFFu, sum, 31);
      }
      if (lane == 0) cum[a.groups] = before;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  int tiles = a.ragged == HINM_RAGGED_ROWS   ? cum[a.groups] * a.mt
              : a.ragged == HINM_RAGGED_DEPTH ? a.groups * a.nt * a.mt
                                              : a.nt * a.mt;
  if (*bad_flag) {
    if (threadIdx.x == 0) ptx::record_status(a.status, HINM_ERR_INVALID_ARG);
    tiles = 0;
  }
  const uint32_t sf_col0 = C::kAccBufs * C::kAccCols;

  if (warp == 0) {
    // ------------------------------------------------------------ copies
    if (lane == 0) {
      uint32_t it = 0;
      bool stop = false;
      for (int t = blockIdx.x; t < tiles && !stop; t += gridDim.x) {
        const Tile w = tile_of<BN>(a, cum, t);
        const int batch = a.ragged == HINM_RAGGED_DEPTH ? 0 : w.e;  // matrix of A
        const uint8_t* sa = a.sa + ((batch * a.a_tiles + w.m0 / 128) * a.a_chunks +
                                    w.k0 / C::kChunkDepth) * kFp4ChunkBytes;
        const uint8_t* sb = a.sb + (w.sb_tile * a.b_chunks + w.k0 / C::kChunkDepth) * kFp4ChunkBytes;
        const int a_row = batch * a.M + w.m0;
        const bool two = C::kBTiles == 2 && w.nlen > 128;  // B's second scale tile exists
        for (int st = 0; st < w.steps; st += 4, ++it) {
          const int s = it % C::kStages;
          if (!ptx::mbar_wait(empty_bar(s), ((it / C::kStages) & 1) ^ 1, a.status, abort_flag)) {
            stop = true;
            break;
          }
          const int left = min(4, w.steps - st);
          const uint32_t sf = (uint32_t)(left * 64 / C::kChunkDepth) * kFp4ChunkBytes;
          const uint32_t A_s = ptx::smem_u32(smem + s * C::kStageBytes);
          const uint32_t B_s = A_s + C::kABytes, S_s = B_s + C::kBBytes;
          ptx::mbar_arrive_expect_tx(full_bar(s), C::kABytes + C::kBBytes + sf * (two ? 3 : 2));
          const int x = (int)(w.k0 / 2) + st * 32;
          ptx::tma_load_2d(A_s, &tmA, x, a_row, full_bar(s));
          ptx::tma_load_2d(B_s, &tmB, x, w.n0, full_bar(s));
          const long long at = (long long)(st * 64 / C::kChunkDepth) * kFp4ChunkBytes;
          ptx::bulk_g2s(S_s, sa + at, sf, full_bar(s));
          ptx::bulk_g2s(S_s + C::kSfTile, sb + at, sf, full_bar(s));
          if (two)
            ptx::bulk_g2s(S_s + 2 * C::kSfTile, sb + a.b_chunks * kFp4ChunkBytes + at, sf,
                          full_bar(s));
        }
      }
      if (*abort_flag) {
        for (uint32_t k = it > (uint32_t)C::kStages ? it - C::kStages : 0u; k < it; ++k)
          ptx::mbar_wait(full_bar(k % C::kStages), (k / C::kStages) & 1, a.status, nullptr);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    if (lane == 0) {
      uint32_t it = 0, lu = 0;
      bool stop = false;
      for (int t = blockIdx.x; t < tiles && !stop; t += gridDim.x, ++lu) {
        const Tile w = tile_of<BN>(a, cum, t);
        const int b = (int)(lu % C::kAccBufs);
        if (!ptx::mbar_wait(acce_bar(b), ((lu / C::kAccBufs) & 1) ^ 1, a.status, abort_flag)) break;
        ptx::tc_fence_after();
        const uint32_t acc = tmem + b * C::kAccCols;
        const int n = (w.nlen + 15) & ~15;
        const uint32_t id0 = ptx::idesc_fp4(n, FMT == HINM_FP4_MX, 0);
        const uint32_t id2 = ptx::idesc_fp4(n, FMT == HINM_FP4_MX, 2);
        const int tb = w.nlen > 128 ? 2 : 1;
        for (int st = 0; st < w.steps; st += 4, ++it) {
          const int s = it % C::kStages;
          if (!ptx::mbar_wait(full_bar(s), (it / C::kStages) & 1, a.status, abort_flag)) {
            stop = true;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t A_s = ptx::smem_u32(smem + s * C::kStageBytes);
          const uint32_t B_s = A_s + C::kABytes, S_s = B_s + C::kBBytes;
          const uint32_t sf = tmem + sf_col0 + s * C::kSfCols;
          const int left = min(4, w.steps - st);
          const int chunks = left * 64 / C::kChunkDepth;
          for (int c = 0; c < chunks; ++c) {
            // 32 rows of 16 bytes: core matrices of 8 rows, 128 bytes apart
            ptx::tc_cp_32x128b_x4(sf + 4 * c,
                                  ptx::smem_desc(S_s + c * kFp4ChunkBytes, 16, 128, 0));
            for (int j = 0; j < tb; ++j)
              ptx::tc_cp_32x128b_x4(
                  sf + 4 * C::kChunks + 4 * C::kBTiles * c + 4 * j,
                  ptx::smem_desc(S_s + (1 + j) * C::kSfTile + c * kFp4ChunkBytes, 16, 128, 0));
          }
          const uint32_t sfb = sf + 4 * C::kChunks + w.sb_shift / 32;
          for (int k = 0; k < left; ++k) {
            const uint64_t ad = ptx::smem_desc(A_s + 32 * k, 16, 1024, 2);
            const uint64_t bd = ptx::smem_desc(B_s + 32 * k, 16, 1024, 2);
            if constexpr (FMT == HINM_FP4_NV)
              ptx::mma_fp4_block16(acc, ad, bd, id0, sf + 4 * k, sfb + 4 * C::kBTiles * k,
                                   (st | k) ? 1u : 0u);
            else
              ptx::mma_fp4_block32(acc, ad, bd, (k & 1) ? id2 : id0, sf + 4 * (k / 2),
                                   sfb + 4 * C::kBTiles * (k / 2), (st | k) ? 1u : 0u);
          }
          ptx::tc_commit(empty_bar(s));
        }
        if (stop) break;
        ptx::tc_commit(accf_bar(b));
      }
      ptx::tc_commit(drain_bar);
      ptx::mbar_wait(drain_bar, 0, a.status, nullptr);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    uint32_t lu = 0;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++lu) {
      const Tile w = tile_of<BN>(a, cum, t);
      const int b = (int)(lu % C::kAccBufs);
      bool ok = ptx::mbar_wait(accf_bar(b), (lu / C::kAccBufs) & 1, a.status, abort_flag);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      ptx::tc_fence_after();
      const int m = w.m0 + q * 32 + lane;
      const int batch = a.ragged == HINM_RAGGED_DEPTH ? 0 : w.e;  // matrix of A
      const float alpha = (a.ga ? __ldg(a.ga + batch) : 1.0f) * (a.gb ? __ldg(a.gb) : 1.0f);
      const float bias =
          a.bias && m < a.M ? __ldg(a.bias + (long long)batch * a.M + m) : 0.0f;
      const long long y0 = a.ragged == HINM_RAGGED_DEPTH ? w.e * a.y_batch : 0;
      for (int col = 0; col < w.nlen; col += 32) {
        uint32_t v[32];
        if (w.steps > 0) {
          const uint32_t at = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * C::kAccCols + col);
          ptx::tmem_ld_32x32b_x32(at, v);
          ptx::tmem_ld_wait();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0;
        }
        if (m < a.M) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (col + i < w.nlen) {
              const float y = activate(fmaf(__uint_as_float(v[i]), alpha, bias), a.act);
              const long long n = w.n0 + col + i;
              store_one(a, y0 + (a.transposed ? n * a.ldy + m : (long long)m * a.ldy + n), y);
            }
          }
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(acce_bar(b));
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
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

template <int FMT, int BN>
cudaError_t run(MmArgs a, const hinm_fp4& A, const hinm_fp4& B, cudaStream_t s) {
  using C = MmCfg<FMT, BN>;
  cudaError_t e = set_max_dynamic_smem((const void*)fp4_mm_kernel<FMT, BN>, (int)C::kSmemBytes);
  if (e != cudaSuccess) return e;
  const Fp4Geom ga = fp4_geom(A.rows, A.depth, A.ragged, A.groups);
  const Fp4Geom gb = fp4_geom(B.rows, B.depth, B.ragged, B.groups);
  CUtensorMap ma, mb;
  if (!make_map(&ma, A.values, (long long)A.batch * A.rows, ga.pitch(), 128) ||
      !make_map(&mb, B.values, B.rows, gb.pitch(), BN))
    return cudaErrorInvalidValue;
  a.a_tiles = ga.row_tiles;
  a.a_chunks = ga.chunks(FMT);
  a.b_tiles = gb.row_tiles;
  a.b_chunks = gb.chunks(FMT);
  a.steps = (int)(ga.depth_pad / 64);
  a.mt = (A.rows + 127) / 128;
  a.nt = (B.rows + BN - 1) / BN;
  // ragged rows: no more column tiles than full ones and one partial for each group
  const long long nt = a.ragged == HINM_RAGGED_ROWS    ? (long long)B.rows / BN + a.groups
                       : a.ragged == HINM_RAGGED_DEPTH ? (long long)a.nt * a.groups
                                                       : a.nt;
  const long long tiles = nt * a.mt;
  if (tiles > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  const int grid = tiles < num_sms() ? (int)tiles : num_sms();
  return launch_kernel(fp4_mm_kernel<FMT, BN>, grid, kMmThreads, C::kSmemBytes, s, nullptr, ma, mb,
                       a);
}

template <int FMT>
cudaError_t pick(const MmArgs& a, const hinm_fp4& A, const hinm_fp4& B, cudaStream_t s) {
  const int n = a.ragged == HINM_RAGGED_ROWS ? (B.rows + a.groups - 1) / a.groups : B.rows;
  if (n <= 64) return run<FMT, 64>(a, A, B, s);
  if (n <= 128) return run<FMT, 128>(a, A, B, s);
  return run<FMT, 256>(a, A, B, s);
}

}  // namespace

cudaError_t launch_fp4_matmul(const hinm_fp4& A, const hinm_fp4& B, const Fp4Out& o, int* status,
                              cudaStream_t s) {
  MmArgs a{};
  a.sa = A.scales;
  a.sb = B.scales;
  a.ga = A.tensor_scale;
  a.gb = B.tensor_scale;
  a.bias = o.bias;
  a.offsets = B.offsets;
  a.Y = o.Y;
  a.ldy = o.ldy;
  a.y_batch = o.batch_stride;
  a.M = A.rows;
  a.N = B.rows;
  a.depth = B.depth;
  a.groups = B.groups;
  a.ragged = B.ragged;
  a.dtype = o.dtype;
  a.transposed = o.transposed;
  a.act = o.act;
  a.status = status;
  return A.format == HINM_FP4_NV ? pick<HINM_FP4_NV>(a, A, B, s) : pick<HINM_FP4_MX>(a, A, B, s);
}

}  // namespace hinm
