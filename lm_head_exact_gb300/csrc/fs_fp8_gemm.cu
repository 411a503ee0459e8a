// Product of two 8-bit matrices with a scale for each block of 128 elements of
// k, and the sampler over an 8-bit head:
//
//   out[i, j] = sum_b sa[i, b] sb[j, b] (sum_{k in block b} a[i, k] b[j, k])
//
// Mapping: a tile is 128 rows of a (MMA M, TMEM lanes) by kBN rows of b (MMA N).
// A stage of the TMA ring is one block of 128 elements of k: 128 bytes a row,
// one swizzle row, four tcgen05.mma kind::f8f6f4 of 32.  The tensor cores' sum of
// a block, in fp32, is one of several TMEM buffers in turn; eight epilogue
// warps multiply it by the block's scales and add it to registers while the next
// block is multiplied.  (Scales are any fp32 numbers, so the hardware's
// power-of-two block scales do not serve; and a sum of 128 products in TMEM,
// where additions are cut and not rounded, is short enough to lose nothing
// visible: the blocks are added in registers, to nearest.)
//
// With few tiles the k axis is split over the CTAs of a cluster; each leaves its
// partial tile in its own shared memory, and every CTA adds a part of the
// columns over all of them, in their order.
#include <cuda.h>

#include <algorithm>

#include "fs_epilogue.cuh"
#include "fs_finish.cuh"
#include "fs_fp8.cuh"
#include "fs_fp8.h"
#include "fs_fp8_ptx.cuh"
#include "fs_internal.h"
#include "fs_tmap.h"

namespace fs {
namespace {

using namespace sm100;

constexpr int kBM = 128;
constexpr int kBK = 128;                       // elements and bytes of a row in a stage
constexpr int kATile = kBM * kBK;
constexpr int kEpiWarps = 8;                   // 4 lane quarters x 2 column parts
constexpr int kProducerWarp = kEpiWarps;
constexpr int kMmaWarp = kEpiWarps + 1;
constexpr int kThreads = (kEpiWarps + 2) * 32;
constexpr int kPitch = 33;                     // words of a staged row of 32
constexpr int kStagingBytes = kEpiWarps * 32 * kPitch * 4;
constexpr int kBarBytes = 512;
constexpr int kSmemLimit = 232448;
constexpr int kMaxSplits = 8;

template <int kBN>
struct Shape {
  static constexpr int kStageBytes = kATile + kBN * kBK;
  static constexpr int kFit = (kSmemLimit - 1024 - kBarBytes - kStagingBytes) / kStageBytes;
  static constexpr int kStages = kFit < 8 ? kFit : 8;
  static constexpr int kBufs = kBN == 256 ? 2 : 4;
  static constexpr int kPart = kBN / 2;                   // columns of an epilogue warp
  static constexpr int kSmem = kStages * kStageBytes + kStagingBytes + kBarBytes + 1024;
};
static_assert((2 * 8 + 2 * 4 + 1) * 8 + 16 <= kBarBytes, "barriers fit");
static_assert(kBM * 257 * 4 <= Shape<256>::kStages * Shape<256>::kStageBytes, "a partial tile fits the stages");

struct Scales {
  const float* at;
  int64_t s_row, s_col;
};

struct Args {
  int64_t m, n;
  int n_kb, n_mt, n_tiles, splits;
  int box_a;                 // rows of a that a stage loads
  Scales sa, sb;
  uint32_t a_e5m2, b_e5m2;
  void* out;
  int out_type;
  int64_t out_stride;
  Problem p;                 // sampling
  Finish f;
  int* err;
};

__device__ __forceinline__ uint32_t pair_word(int type, float lo, float hi) {
  if (type == FS_TYPE_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void store_one(const Args& a, int64_t row, int64_t col, float v) {
  const int64_t at = row * a.out_stride + col;
  if (a.out_type == FS_TYPE_F32)
    static_cast<float*>(a.out)[at] = v;
  else if (a.out_type == FS_TYPE_BF16)
    static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(a.out)[at] = __float2half_rn(v);
}

// A warp's 32 rows x kPart columns of the output, through its staging area so
// that a store covers whole lines of one row.
template <int kPart>
__device__ __forceinline__ void store_part(const Args& a, const float (&acc)[kPart], uint32_t* stage, int64_t row0,
                                           int64_t col0) {
  const int lane = threadIdx.x & 31;
  const int rows = static_cast<int>(min(static_cast<int64_t>(32), a.m - row0));
  if (a.out_type == FS_TYPE_F32) {
#pragma unroll
    for (int c = 0; c < kPart; c += 32) {
      if (col0 + c >= a.n) break;
#pragma unroll
      for (int j = 0; j < 32; ++j) stage[lane * kPitch + j] = __float_as_uint(acc[c + j]);
      __syncwarp();
      if (col0 + c + lane < a.n) {
        float* dst = static_cast<float*>(a.out) + row0 * a.out_stride + col0 + c + lane;
#pragma unroll 4
        for (int i = 0; i < rows; ++i, dst += a.out_stride) *dst = __uint_as_float(stage[i * kPitch + lane]);
      }
      __syncwarp();
    }
    return;
  }
  constexpr int kWide = kPart < 64 ? kPart : 64;          // columns of a pass, two a word
  const bool whole = (reinterpret_cast<uintptr_t>(a.out) & 3) == 0 && (a.out_stride & 1) == 0;
#pragma unroll
  for (int c = 0; c < kPart; c += kWide) {
    if (col0 + c >= a.n) break;
#pragma unroll
    for (int j = 0; j < kWide / 2; ++j) stage[lane * kPitch + j] = pair_word(a.out_type, acc[c + 2 * j], acc[c + 2 * j + 1]);
    __syncwarp();
    const int64_t col = col0 + c + 2 * lane;
    if (lane < kWide / 2 && col < a.n) {
      uint16_t* dst = static_cast<uint16_t*>(a.out) + row0 * a.out_stride + col;
      if (whole && col + 1 < a.n) {
#pragma unroll 4
        for (int i = 0; i < rows; ++i, dst += a.out_stride) *reinterpret_cast<uint32_t*>(dst) = stage[i * kPitch + lane];
      } else {
        for (int i = 0; i < rows; ++i, dst += a.out_stride) {
          const uint32_t w = stage[i * kPitch + lane];
          dst[0] = static_cast<uint16_t>(w);
          if (col + 1 < a.n) dst[1] = static_cast<uint16_t>(w >> 16);
        }
      }
    }
    __syncwarp();
  }
}

// kRowScale: b has a scale for each of its rows, else for 128 of them.
template <int kBN, bool kSample, bool kRowScale, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
fp8_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b, const Args a) {
  using S = Shape<kBN>;
  constexpr int kStages = S::kStages, kBufs = S::kBufs, kPart = S::kPart;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint32_t* staging = reinterpret_cast<uint32_t*>(smem + kStages * S::kStageBytes);
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + kStages * S::kStageBytes + kStagingBytes);
  uint64_t* empty_bar = full_bar + kStages;
  uint64_t* tfull_bar = empty_bar + kStages;
  uint64_t* tempty_bar = tfull_bar + kBufs;
  uint64_t* drain_bar = tempty_bar + kBufs;
  uint32_t* tmem_base_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_base_slot + 1);
  int* last_flag = reinterpret_cast<int*>(tmem_base_slot + 2);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int split = kSplit ? static_cast<int>(cluster_ctarank()) : 0;
  const int splits = kSplit ? a.splits : 1;
  const int k0 = kSplit ? static_cast<int>(static_cast<int64_t>(a.n_kb) * split / splits) : 0;
  const int k1 = kSplit ? static_cast<int>(static_cast<int64_t>(a.n_kb) * (split + 1) / splits) : a.n_kb;
  const int first = kSplit ? blockIdx.x / splits : blockIdx.x;
  const int step = kSplit ? a.n_tiles : gridDim.x;        // (a cluster takes one tile)

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&tfull_bar[i], 1);
      mbar_init(&tempty_bar[i], kEpiWarps);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kProducerWarp && lane == 0) {
    tma_prefetch_desc(&tmap_a);
    tma_prefetch_desc(&tmap_b);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_base_slot, kBufs * kBN);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_base_slot;
  pdl_launch_dependents();

  if (warp == kProducerWarp) {
    // -------------------------------------------------------------- TMA producer
    pdl_wait();
    const uint32_t elected = elect_one();
    // b is read once per row tile of a, and those run side by side; a by every
    // column tile
    const uint64_t pol_a = policy_evict_last(), pol_b = a.n_mt > 1 ? policy_evict_normal() : policy_evict_first();
    const uint32_t full0 = smem_u32(full_bar), empty0 = smem_u32(empty_bar), smem0 = smem_u32(smem);
    const uint32_t bytes = a.box_a * kBK + kBN * kBK;
    int stage = 0;
    uint32_t phase = 0;
    int64_t n_issued = 0;
    bool ok = true;
    for (int t = first; ok && t < a.n_tiles; t += step) {
      const int m0 = t % a.n_mt * kBM, n0 = t / a.n_mt * kBN;
      for (int kb = k0; kb < k1; ++kb) {
        ok = mbar_wait_warp(empty0 + stage * 8, phase ^ 1, a.err, abort_flag);
        if (!ok) break;
        const uint32_t dst = smem0 + stage * S::kStageBytes, full = full0 + stage * 8;
        mbar_arrive_expect_tx_if(elected, full, bytes);
        tma_load_2d_if(elected, dst, &tmap_a, full, kb * kBK, m0, pol_a);
        tma_load_2d_if(elected, dst + kATile, &tmap_b, full, kb * kBK, n0, pol_b);
        ++n_issued;
        if (++stage == kStages) { stage = 0; phase ^= 1; }
      }
    }
    if (!ok) {                                             // leave only after the loads in flight have landed
      volatile int no_abort = 0;
      for (int64_t i = max(static_cast<int64_t>(0), n_issued - kStages); i < n_issued; ++i)
        mbar_wait_warp(full0 + static_cast<uint32_t>(i % kStages) * 8, static_cast<uint32_t>((i / kStages) & 1), a.err,
                       &no_abort);
    }
  } else if (warp == kMmaWarp) {
    // -------------------------------------------------------------- MMA issuer
    const uint32_t elected = elect_one();
    const uint32_t idesc = idesc_fp8_f32(a.a_e5m2, a.b_e5m2, kBM, kBN);
    const uint64_t a_desc0 = smem_desc_k128(smem_u32(smem)), b_desc0 = smem_desc_k128(smem_u32(smem) + kATile);
    const uint32_t full0 = smem_u32(full_bar), empty0 = smem_u32(empty_bar);
    const uint32_t tfull0 = smem_u32(tfull_bar), tempty0 = smem_u32(tempty_bar);
    int stage = 0, buf = 0;
    uint32_t phase = 0, buf_phase = 0;
    bool ok = true;
    for (int t = first; ok && t < a.n_tiles; t += step) {
      for (int kb = k0; kb < k1; ++kb) {
        ok = mbar_wait_warp(tempty0 + buf * 8, buf_phase ^ 1, a.err, abort_flag) &&
             mbar_wait_warp(full0 + stage * 8, phase, a.err, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint64_t a_desc = a_desc0 + stage * (S::kStageBytes >> 4);
        const uint64_t b_desc = b_desc0 + stage * (S::kStageBytes >> 4);
#pragma unroll
        for (int k = 0; k < kBK / 32; ++k)
          mma_fp8_if(elected, tmem_base + buf * kBN, a_desc + k * 2, b_desc + k * 2, idesc, k > 0);
        mma_commit_if(elected, empty0 + stage * 8);
        mma_commit_if(elected, tfull0 + buf * 8);
        if (++stage == kStages) { stage = 0; phase ^= 1; }
        if (++buf == kBufs) { buf = 0; buf_phase ^= 1; }
      }
    }
    if (!ok) {
      mma_commit_if(elected, smem_u32(drain_bar));
      volatile int no_abort = 0;
      mbar_wait_warp(smem_u32(drain_bar), 0, a.err, &no_abort);
    }
  } else {
    // -------------------------------------------------------------- epilogue
    const int quad = warp & 3;                             // TMEM lane quarter
    const int part = warp >> 2;
    uint32_t* stage = staging + warp * 32 * kPitch;
    float* row_scales = reinterpret_cast<float*>(stage);   // kRowScale: of this warp's columns, in the present block
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + part * kPart;
    pdl_wait();
    int buf = 0;
    uint32_t buf_phase = 0;
    bool ok = true;
    // sampling
    Best best = best_none();
    RowScan scan;
    bool active = false;
    int64_t batch_row = -1;
    const int64_t col_blocks = (a.n + kQuantBlock - 1) / kQuantBlock;
    for (int t = first; t < a.n_tiles; t += step) {
      const int64_t row0 = static_cast<int64_t>(t % a.n_mt) * kBM + quad * 32;
      const int64_t col0 = static_cast<int64_t>(t / a.n_mt) * kBN + part * kPart;
      const bool live = row0 < a.m && col0 < a.n;          // this warp has something to add up
      const bool row_ok = row0 + lane < a.m;
      const float* sa = a.sa.at + (row0 + lane) * a.sa.s_row;
      const float* sb = a.sb.at + col0 / kQuantBlock * a.sb.s_row;
      const bool sb_ok = col0 / kQuantBlock < col_blocks;
      if constexpr (kSample) {
        if (row0 + lane != batch_row) {
          if (batch_row >= 0 && batch_row < a.m) push_candidate(a.f, batch_row, best);
          best = best_none();
          batch_row = row0 + lane;
          const RowTemp rt = row_temp(row_ok ? a.p.temp[batch_row] : -1.0f);
          active = row_ok && rt.mode != kRowInvalid;
          scan.key = PhiloxKey{static_cast<uint32_t>(a.p.seed), static_cast<uint32_t>(a.p.seed >> 32)};
          scan.row = static_cast<uint32_t>(batch_row);
          scan.step_lo = static_cast<uint32_t>(a.p.step);
          scan.step_hi = static_cast<uint32_t>(a.p.step >> 32);
          scan.inv_t = rt.inv_t;
          scan.greedy = rt.mode == kRowGreedy;
          scan.bias_row = a.p.bias != nullptr ? a.p.bias + batch_row * a.p.bias_stride : nullptr;
        }
      }
      float acc[kPart];
#pragma unroll
      for (int c = 0; c < kPart; ++c) acc[c] = 0.0f;
      // the scales of a block are loaded a block ahead
      float sa_next = live && row_ok ? sa[k0 * a.sa.s_col] : 0.0f;
      float sb_next[kRowScale ? kPart / 32 : 1];
      auto load_sb = [&](int kb) {
        if constexpr (kRowScale) {
#pragma unroll
          for (int j = 0; j < kPart / 32; ++j) {
            const int64_t col = col0 + j * 32 + lane;
            sb_next[j] = col < a.n ? a.sb.at[col * a.sb.s_row + kb * a.sb.s_col] : 0.0f;
          }
        } else {
          sb_next[0] = sb_ok ? sb[kb * a.sb.s_col] : 0.0f;
        }
      };
      load_sb(k0);
      for (int kb = k0; kb < k1; ++kb) {
        float f = sa_next;
        if constexpr (kRowScale) {
          __syncwarp();
#pragma unroll
          for (int j = 0; j < kPart / 32; ++j) row_scales[j * 32 + lane] = sb_next[j];
          __syncwarp();
        } else {
          f *= sb_next[0];
        }
        if (kb + 1 < k1) {
          if (live && row_ok) sa_next = sa[(kb + 1) * a.sa.s_col];
          load_sb(kb + 1);
        }
        ok = mbar_wait(&tfull_bar[buf], buf_phase, a.err, abort_flag);
        if (!ok) break;
        __syncwarp();
        tc_fence_after();
        if (live) {
#pragma unroll
          for (int c = 0; c < kPart; c += 16) {
            uint32_t r[16];
            tmem_ld_16(lane_addr + buf * kBN + c, r);
            tmem_ld_wait_for(r);
            if constexpr (kRowScale) {
#pragma unroll
              for (int j = 0; j < 16; j += 4) {
                const float4 w = *reinterpret_cast<const float4*>(row_scales + c + j);
                acc[c + j + 0] = fmaf(__uint_as_float(r[j + 0]), f * w.x, acc[c + j + 0]);
                acc[c + j + 1] = fmaf(__uint_as_float(r[j + 1]), f * w.y, acc[c + j + 1]);
                acc[c + j + 2] = fmaf(__uint_as_float(r[j + 2]), f * w.z, acc[c + j + 2]);
                acc[c + j + 3] = fmaf(__uint_as_float(r[j + 3]), f * w.w, acc[c + j + 3]);
              }
            } else {
#pragma unroll
              for (int j = 0; j < 16; ++j) acc[c + j] = fmaf(__uint_as_float(r[j]), f, acc[c + j]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty_bar[buf]);
        if (++buf == kBufs) { buf = 0; buf_phase ^= 1; }
      }
      if (!ok) break;
      if constexpr (kRowScale) __syncwarp();               // the staging area is read no more
      if constexpr (kSplit) {
        // every load has landed and been multiplied: the stages hold the partial tile now
        float* red = reinterpret_cast<float*>(smem);
        if (live && row_ok) {
#pragma unroll
          for (int c = 0; c < kPart; ++c) red[(quad * 32 + lane) * (kBN + 1) + part * kPart + c] = acc[c];
        }
      } else if constexpr (kSample) {
        if (live && active) {
#pragma unroll 1
          for (int c = 0; c < kPart / 32; ++c) {           // one copy of the scan; the columns are selected
            uint32_t r[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              float v = acc[j];
#pragma unroll
              for (int h = 1; h < kPart / 32; ++h) v = c == h ? acc[h * 32 + j] : v;
              r[j] = __float_as_uint(v);
            }
            const int64_t v0 = col0 + c * 32;
            if (v0 >= a.n) break;
            if (scan.bias_row != nullptr)
              scan32<true>(r, v0, a.n, 0, scan, best);
            else
              scan32<false>(r, v0, a.n, 0, scan, best);
          }
        }
      } else if (live) {
        store_part<kPart>(a, acc, stage, row0, col0);
      }
    }
    if constexpr (kSample) {
      if (batch_row >= 0 && batch_row < a.m) push_candidate(a.f, batch_row, best);
      finish_grid<false>(a.f, a.m, threadIdx.x, kEpiWarps * 32, last_flag, named_bar1_and<kEpiWarps * 32>);
    }
  }

  if constexpr (kSplit) {
    __syncwarp();
    cluster_sync();                                        // every partial tile is there
    if (warp < kEpiWarps && *abort_flag == 0) {
      const int t = first;
      const int64_t row0 = static_cast<int64_t>(t % a.n_mt) * kBM, col0 = static_cast<int64_t>(t / a.n_mt) * kBN;
      const int rows = static_cast<int>(min(static_cast<int64_t>(kBM), a.m - row0));
      const int c0 = kBN * split / splits, cols = kBN * (split + 1) / splits - c0;
      const uint32_t red0 = smem_u32(smem);
      uint32_t peer[kMaxSplits];
#pragma unroll
      for (int s = 0; s < kMaxSplits; ++s) peer[s] = mapa_shared(red0, s < splits ? s : 0);
      for (int i = threadIdx.x; i < rows * cols; i += kEpiWarps * 32) {
        const int row = i / cols, col = c0 + i % cols;
        if (col0 + col >= a.n) continue;
        const uint32_t at = static_cast<uint32_t>(row * (kBN + 1) + col) * 4;
        float v[kMaxSplits];
#pragma unroll
        for (int s = 0; s < kMaxSplits; ++s) v[s] = s < splits ? ld_shared_cluster_f32(peer[s] + at) : 0.0f;
        float sum = v[0];
#pragma unroll
        for (int s = 1; s < kMaxSplits; ++s) sum += v[s];
        store_one(a, row0 + row, col0 + col, sum);
      }
    }
    __syncwarp();
    cluster_sync();                                        // nobody reads this CTA's shared memory any more
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem_base, kBufs * kBN);
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 152;
  }
  return sms > 0 ? sms : 152;
}

template <int kBN, bool kSample, bool kRowScale, bool kSplit>
cudaError_t launch(Args a, const Fp8Matrix& ma, const Fp8Matrix& mb, int64_t k, int grid, cudaStream_t stream) {
  CUtensorMap ta, tb;
  a.box_a = static_cast<int>(std::min<int64_t>(kBM, (a.m + 7) / 8 * 8));
  if (!encode_rows_u8(&ta, ma.q, a.m, k, ma.stride, kBK, a.box_a) || !encode_rows_u8(&tb, mb.q, a.n, k, mb.stride, kBK, kBN))
    return cudaErrorInvalidValue;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  constexpr auto kernel = fp8_kernel<kBN, kSample, kRowScale, kSplit>;
  if (e == cudaSuccess) e = raise_smem_limit<kernel>(dev, Shape<kBN>::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Shape<kBN>::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kSplit ? a.splits : 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kSplit ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, ta, tb, a);
}

// Tile width and split of a product.
struct Plan {
  int bn, splits;
};

Plan plan(int64_t m, int64_t n, int n_kb, int sms) {
  const int64_t n_mt = (m + kBM - 1) / kBM;
  Plan best{256, 1};
  double best_time = 1e300;
  for (const int bn : {256, 128, 64}) {
    const int64_t tiles = n_mt * ((n + bn - 1) / bn);
    const int splits = tiles >= sms ? 1 : static_cast<int>(std::min<int64_t>({kMaxSplits, n_kb, sms / tiles}));
    const double ctas = static_cast<double>(std::min<int64_t>(tiles * splits, sms));
    const double rounds = static_cast<double>((tiles + sms - 1) / sms);
    const double per_kb = std::max(2.4 * bn, bn * kBK / std::min(60.0, 3350.0 / ctas));      // clocks
    const double time = rounds * ((n_kb + splits - 1) / splits) * per_kb + (splits > 1 ? 1500.0 : 0.0);
    if (time < best_time) {
      best_time = time;
      best = Plan{bn, splits};
    }
  }
  return best;
}

template <int kBN>
cudaError_t launch_store(const Args& a, const Fp8Product& p, cudaStream_t stream) {
  const int grid = a.splits > 1 ? a.n_tiles * a.splits : std::min(a.n_tiles, sm_count());
  if (p.b.block_rows == 1)
    return a.splits > 1 ? launch<kBN, false, true, true>(a, p.a, p.b, p.k, grid, stream)
                        : launch<kBN, false, true, false>(a, p.a, p.b, p.k, grid, stream);
  return a.splits > 1 ? launch<kBN, false, false, true>(a, p.a, p.b, p.k, grid, stream)
                      : launch<kBN, false, false, false>(a, p.a, p.b, p.k, grid, stream);
}

Args common_args(const Fp8Matrix& a, const Fp8Matrix& b, int64_t m, int64_t n, int64_t k, int* err) {
  Args args{};
  args.m = m;
  args.n = n;
  args.n_kb = static_cast<int>(quant_blocks(k));
  args.n_mt = static_cast<int>((m + kBM - 1) / kBM);
  args.splits = 1;
  args.sa = Scales{a.scale, a.s_row, a.s_col};
  args.sb = Scales{b.scale, b.s_row, b.s_col};
  args.a_e5m2 = a.type == FS_TYPE_E5M2;
  args.b_e5m2 = b.type == FS_TYPE_E5M2;
  args.err = err;
  return args;
}

}  // namespace

cudaError_t launch_fp8_matmul(const Fp8Product& p, int* err, cudaStream_t stream) {
  Args a = common_args(p.a, p.b, p.m, p.n, p.k, err);
  const Plan s = plan(p.m, p.n, a.n_kb, sm_count());
  const int64_t tiles = a.n_mt * ((p.n + s.bn - 1) / s.bn);
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  a.n_tiles = static_cast<int>(tiles);
  a.splits = s.splits;
  a.out = p.out;
  a.out_type = p.out_type;
  a.out_stride = p.out_stride;
  switch (s.bn) {
    case 256: return launch_store<256>(a, p, stream);
    case 128: return launch_store<128>(a, p, stream);
    default: return launch_store<64>(a, p, stream);
  }
}

cudaError_t launch_fp8_sample(const Problem& p, const Fp8Matrix& h, const Fp8Matrix& W, int64_t k, const Finish& f,
                              int* err, cudaStream_t stream) {
  constexpr int kBN = 256;
  Args a = common_args(h, W, p.B, p.V_local, k, err);
  const int64_t n_nt = (p.V_local + kBN - 1) / kBN, tiles = a.n_mt * n_nt;
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  a.n_tiles = static_cast<int>(tiles);
  a.p = p;
  a.f = f;
  // as few CTAs as give each the same number of tiles; a multiple of the row
  // tiles, so that a CTA keeps its rows
  const int sms = sm_count();
  int grid = std::min(a.n_tiles, sms);
  if (a.n_mt <= sms) {
    const int64_t groups = sms / a.n_mt, per = (n_nt + groups - 1) / groups;
    grid = static_cast<int>((n_nt + per - 1) / per) * a.n_mt;
  }
  return W.block_rows == 1 ? launch<kBN, true, true, false>(a, h, W, k, grid, stream)
                           : launch<kBN, true, false, false>(a, h, W, k, grid, stream);
}

}  // namespace fs
