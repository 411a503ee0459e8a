// Product of two 8-bit matrices with a scale for each block of 128 elements of
// k, and the sampler over an 8-bit head:
//
//   out[i, j] = sum_b sa[i, b] sb[j, b] (sum_{k in block b} a[i, k] b[j, k])
//
// One persistent, warp-specialized kernel in three forms, by what lies on the
// MMA's M axis, that is on the TMEM lanes:
//
//   kThin  b (weights), with up to 64 rows of a (tokens) as columns: the product
//          is bound by reading b, nothing is padded, and every epilogue warp has its share
//   kWide  128 rows of a, 192 rows of b as columns
//   kPair  256 rows of a over a pair of CTAs (tcgen05 cta_group::2), 192 rows of b, of
//          which each CTA loads a half
//
// A stage of the TMA ring is one or two blocks of 128 elements of k: 128 bytes a
// row, one swizzle row, four tcgen05.mma kind::f8f6f4 of 32 each.  The tensor cores' sum of a
// block, in fp32, is one of several TMEM buffers in turn; epilogue warps multiply
// it by the block's scales and add it to registers while the next block is
// multiplied.  (Scales are any fp32 numbers, so the hardware's power-of-two block
// scales do not serve; and a sum of 128 products in TMEM, where additions are cut
// and not rounded, is short enough to lose nothing visible: the blocks are added
// in registers, to nearest.)
//
// What bounds it beyond few rows is the way of the sums through the epilogue, not
// the MMAs (a third of the cycles): by the times of the forms below, loading a
// column's sums of a lane quarter from TMEM takes 2 clocks and adding them up 2 more, and
// what hands a buffer over (barriers take 100 clocks to look at) some 300 a block, one
// after another; that one of these units is full is not shown.  kWide and kPair
// therefore take 192 columns, by twelve warps of a lane quarter and 64 columns (1000
// clocks a block; 256 columns by eight warps 1400, 128 by eight 800); kThin eight warps,
// with registers for two blocks' sums, so that one is loaded while the other is
// added up.  Where a tile has 64 columns or fewer, two groups of four warps take
// the tiles in turn, so that one tile's scan or stores overlap the next tile's
// sums.  A warp of its own brings the scales to shared memory ahead.
//
// With few tiles the k axis is split over the CTAs of a cluster; each leaves its
// partial tile in its own shared memory, and every CTA adds a part of it
// over all of them, in their order.
#pragma once

#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "fs_epilogue.cuh"
#include "fs_finish.cuh"
#include "fs_fp8.cuh"
#include "fs_fp8.h"
#include "fs_fp8_ptx.cuh"
#include "fs_internal.h"
#include "fs_tmap.h"

namespace fs {
namespace fp8 {

using namespace sm100;

enum Form : int { kThin, kWide, kPair };

constexpr int kLanes = 128;                    // rows on a CTA's lanes
constexpr int kBK = 128;                       // elements and bytes of a row in a stage
constexpr int kLTile = kLanes * kBK;
constexpr int kPitch = 33;                     // words of a staged row of 32
constexpr int kBarBytes = 1024;
constexpr int kSmemLimit = 232448;
constexpr int kMaxSplits = 8;

constexpr int kAhead = 4;                      // blocks whose scales are brought at a time
constexpr int kSlots = 2;                      // times that many

template <Form kForm, int kBN, bool kSample, bool kColScales>
struct Shape {
  static constexpr bool kSwap = kForm == kThin;
  static constexpr int kCtas = kForm == kPair ? 2 : 1;
  static constexpr int kTileL = kLanes * kCtas;
  static constexpr int kCLoad = kBN / kCtas;              // rows of the columns' operand a CTA loads
  static constexpr int kEpiWarps = kSwap ? 8 : 12;
  static constexpr int kThreads = (kEpiWarps + 4) * 32;
  // Registers of a thread at launch, and what the epilogue's warpgroups and the
  // last one (producer, MMA, scales) go on with.
  static constexpr int kLaunchRegs = kSwap ? 168 : 128, kEpiRegs = kSwap ? 232 : 160, kOtherRegs = kSwap ? 40 : 32;
  static_assert(kEpiWarps / 4 * kEpiRegs + kOtherRegs <= (kEpiWarps / 4 + 1) * kLaunchRegs,
                "no more than the block was launched with");
  static constexpr int kPairK = kSwap ? 2 : 1;            // blocks of k in a stage
  static constexpr bool kTwoBlocks = kSwap;               // registers for two blocks' sums
  static constexpr int kBlockBytes = kLTile + kCLoad * kBK;       // of a block of k in a stage
  static constexpr int kStageBytes = kPairK * kBlockBytes;
  static constexpr int kPart = kBN < 64 ? kBN : 64;       // columns of an epilogue warp
  static constexpr int kColParts = kBN / kPart;
  static constexpr int kGroups = kEpiWarps / 4 / kColParts;
  // Blocks of k that a TMEM buffer takes side by side: what hands a buffer over
  // is then done for several of them.
  static constexpr int kPer = !kSwap ? 1 : kBN <= 32 ? 4 : 2;
  static_assert(kPer % kPairK == 0, "a stage's blocks go into one buffer");
  static constexpr int kBufs = 512 / (kBN * kPer) < 8 ? 512 / (kBN * kPer) : 8;
  static constexpr int kTmemCols = 512;
  // Scales of a block: the lanes' (or one, of their tile), then the columns' (or
  // one for each part).
  static constexpr int kScaleWords = kLanes + (kColScales ? kBN : 4);
  static constexpr int kScaleBytes = kSlots * kAhead * kScaleWords * 4;
  static constexpr int kWarpWords = 32 * (kSwap || kSample ? kPitch : 32);  // of a warp's staging area (a box for TMA: whole KB)
  static constexpr int kStagingBytes = kEpiWarps * kWarpWords * 4;
  static constexpr int kKeyBytes = kSwap ? kBN * 8 : 0;
  static constexpr int kFit = (kSmemLimit - 1024 - kBarBytes - kStagingBytes - kScaleBytes - kKeyBytes) / kStageBytes;
  static constexpr int kStages = kFit < 10 ? kFit : 10;
  static constexpr int kSmem = kStages * kStageBytes + kStagingBytes + kScaleBytes + kKeyBytes + kBarBytes + 1024;
  static constexpr int kBars = 2 * kStages + 2 * kBufs + 2 * kSlots + kGroups + 1;
  static_assert(kBars * 8 + 16 <= kBarBytes, "barriers fit");
  static_assert(kLanes * (kBN + 1) * 4 + kBN * 4 <= kStages * kStageBytes, "a partial tile fits the stages");
};

struct Scales {
  const float* at;
  int64_t s_row, s_col;
  int shift;                 // of a row's number to its block's: 0 or 7
};

// The operands as the kernel sees them: l on the lanes, c as columns.
struct Args {
  int64_t l_rows, c_rows;    // kThin: (n, m), else (m, n)
  int n_kb, n_lt, n_ct, n_tiles, splits;
  int band;                  // column tiles of a band (0: see the kernel)
  int box_l, box_c;          // rows that a CTA loads into a stage
  Scales sl, sc;
  uint32_t l_e5m2, c_e5m2;
  void* out;
  int out_type;
  int64_t out_stride;
  int64_t tma_cols;          // of the output: a warp's columns that end up to here are stored by TMA
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

// 32 staged rows of 32 columns, column c of row r at c ^ r, to the output, whole
// rows of them by a store: outputs off 16-byte boundaries, and ends of rows.
__device__ __forceinline__ void store_rows(const Args& a, const float* stage, int64_t row0, int64_t col0) {
  const int lane = threadIdx.x & 31;
  const int rows = static_cast<int>(min(static_cast<int64_t>(32), a.l_rows - row0));
  const int cols = static_cast<int>(min(static_cast<int64_t>(32), a.c_rows - col0));
  if (a.out_type == FS_TYPE_F32) {
    float* dst = static_cast<float*>(a.out) + row0 * a.out_stride + col0 + lane;
    if (lane < cols) {
#pragma unroll 4
      for (int i = 0; i < rows; ++i, dst += a.out_stride) *dst = stage[i * 32 + (lane ^ i)];
    }
    return;
  }
  // two rows at a time, a lane two columns of one
  const int row = lane >> 4, col = 2 * (lane & 15);
  uint16_t* dst = static_cast<uint16_t*>(a.out) + (row0 + row) * a.out_stride + col0 + col;
  const bool whole = (reinterpret_cast<uintptr_t>(a.out) & 3) == 0 && (a.out_stride & 1) == 0 && (col0 & 1) == 0;
#pragma unroll 4
  for (int i = row; i < rows; i += 2, dst += 2 * a.out_stride) {
    const uint32_t w = pair_word(a.out_type, stage[i * 32 + (col ^ i)], stage[i * 32 + (col + 1 ^ i)]);
    if (whole && col + 1 < cols) {
      *reinterpret_cast<uint32_t*>(dst) = w;
    } else {
      if (col < cols) dst[0] = static_cast<uint16_t>(w);
      if (col + 1 < cols) dst[1] = static_cast<uint16_t>(w >> 16);
    }
  }
}

// A warp's sums, 32 rows x 64 columns, to the output by a TMA store, 128 bytes a
// row, that is on its way while the next tile's sums are added up.  (Stored by the
// warps, 32 columns at a time, a tile took 8500 clocks to leave.)  32-bit outputs take
// two turns.  The box lies swizzled, 16 bytes by 16, so that neither rows nor
// fragments (kFrag, see the kernel) meet bank conflicts.
template <typename T, bool kFrag>
__device__ __forceinline__ void store_tile(const CUtensorMap* out, const float (&acc)[64], uint8_t* box, int64_t row0, int64_t col0) {
  const int lane = threadIdx.x & 31;
  constexpr int kTurns = sizeof(T) / 2, kCols = 64 / kTurns;
  const auto word = [](float lo, float hi) {
    return pair_word(std::is_same<T, __half>::value ? FS_TYPE_F16 : FS_TYPE_BF16, lo, hi);
  };
#pragma unroll
  for (int turn = 0; turn < kTurns; ++turn) {
    if (lane == 0) sm100::bulk_wait_read();                // the box's last store has been read
    __syncwarp();
    if constexpr (kFrag) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (kTurns == 2 && q / 2 != turn) continue;
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const int row = 16 * (q & 1) + 8 * (i >> 1 & 1) + (lane >> 2);
          const int at = (32 * (q >> 1) - turn * kCols + 8 * (i >> 2) + 2 * (lane & 3)) * static_cast<int>(sizeof(T));
          uint8_t* dst = box + row * 128 + ((at >> 4 ^ (row & 7)) << 4) + (at & 15);
          const float lo = acc[16 * q + i], hi = acc[16 * q + i + 1];
          if constexpr (sizeof(T) == 4)
            *reinterpret_cast<float2*>(dst) = make_float2(lo, hi);
          else
            *reinterpret_cast<uint32_t*>(dst) = word(lo, hi);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint4 v;
        if constexpr (sizeof(T) == 4) {
          const float* from = acc + turn * kCols + 4 * j;
          v = make_uint4(__float_as_uint(from[0]), __float_as_uint(from[1]), __float_as_uint(from[2]), __float_as_uint(from[3]));
        } else {
          const float* from = acc + 8 * j;
          v = make_uint4(word(from[0], from[1]), word(from[2], from[3]), word(from[4], from[5]), word(from[6], from[7]));
        }
        *reinterpret_cast<uint4*>(box + lane * 128 + ((j ^ (lane & 7)) << 4)) = v;
      }
    }
    sm100::fence_async_shared();
    __syncwarp();
    if (lane == 0) {
      sm100::tma_store_2d(out, box, static_cast<int32_t>((col0 + turn * kCols) * sizeof(T)), static_cast<int32_t>(row0));
      sm100::bulk_commit();
    }
  }
}

// The best score that any CTA has pushed for a row so far.
__device__ __forceinline__ float best_so_far(const unsigned long long* key) {
  unsigned long long k;
  asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(k) : "l"(key) : "memory");
  return unpack_key(k).z;
}

// The sampling kernels' scan (fs_epilogue.cuh) of 32 staged logits of one row,
// ids v0 .. v0 + 31 (a multiple of 4 first), kStep words apart: the same scores in
// the same order, in a loop over the counters' quads.  (Unrolled, with and without
// bias, it made kernels of 200 KB, whose other parts then waited for instructions.)
//
// `bar`: a score that some id of the row has reached; only ids that reach it
// count.  A quad is left out where its largest scaled logit x and the largest noise
// do not, and, once its random words are there, where their noise does not: g(u) =
// -log(-log u) < bar - x where 1 - u >= exp(x - bar), as -log u >= 1 - u.  The
// margin is above all roundings: of x, of the difference and of the score (half an ulp
// of each, 2^-24 of |bar| + |x|), of g (2e-6) and of __expf (3e-6 of it); 1 - u is
// exact.  With the bar of all CTAs nearly every quad stops there, before its
// logarithms (256 rows x 4096 x 128256: 271 -> 226 us, of which the sums take 172).
template <int kStep>
__device__ __forceinline__ Best scan_staged(const float* at, int64_t v0, int64_t V, const RowScan& s, Best best, float bar) {
  const unsigned lanes = __activemask();
  bar = fmaxf(bar, best.z);
#pragma unroll 1
  for (int q = 0; q < 8; ++q, at += 4 * kStep, v0 += 4) {
    float x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = v0 + e < V ? at[e * kStep] : -INFINITY;
      if (s.bias_row != nullptr && v0 + e < V) x[e] += __ldg(s.bias_row + v0 + e);
    }
    const float most = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
    if (!__any_sync(lanes, (s.greedy ? most : fmaf(most, s.inv_t, kGumbelMax)) >= bar)) continue;
    const uint4 w = noise_words(s.key, static_cast<uint32_t>(v0 >> 2), s.row, s.step_lo, s.step_hi);
    const float scaled = most * s.inv_t, margin = fmaf(1e-6f, fabsf(bar) + fabsf(scaled), 1e-3f);
    const uint32_t top = max(max(w.x, w.y), max(w.z, w.w)) >> 9;
    const float rest = fmaf(static_cast<float>(0x7fffffu - top), 0x1p-23f, 0x1p-24f);     // 1 - u of the largest word
    if (!__any_sync(lanes, s.greedy || !(rest >= __expf(scaled - bar + margin)))) continue;
    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      keep_best(best, perturbed<false>(s, x[e], words[e], 0), static_cast<int32_t>(v0 + e));
    bar = fmaxf(bar, best.z);
  }
  return best;
}

// kColScales: the columns' operand has a scale for each of its rows, else for
// 128 of them, which a warp's columns share.  kLaneScales: the lanes' operand
// has one for each row, else a tile of lanes shares one.
//
// With scales by columns, sums are loaded in the matrix fragments' layout
// (tmem_ld_frag): a thread then needs the factors of a quarter of the columns. In
// whole lanes, where every thread needs them all, reading them took as much
// of shared memory's bandwidth as the operands do.
template <Form kForm, int kBN, bool kSample, bool kLaneScales, bool kColScales, bool kSplit>
__global__ void __launch_bounds__(Shape<kForm, kBN, kSample, kColScales>::kThreads, 1)
kernel(const __grid_constant__ CUtensorMap tmap_l, const __grid_constant__ CUtensorMap tmap_c,
       const __grid_constant__ CUtensorMap tmap_o, const Args a) {
  using S = Shape<kForm, kBN, kSample, kColScales>;
  constexpr bool kSwap = S::kSwap, kPairs = kForm == kPair;
  static_assert(kColScales || kLaneScales, "scales of a tile of lanes are folded into those of the columns");
  constexpr int kStages = S::kStages, kBufs = S::kBufs, kPart = S::kPart, kGroups = S::kGroups;
  constexpr int kPer = S::kPer, kPairK = S::kPairK, kEpiWarps = S::kEpiWarps;
  constexpr int kProducerWarp = kEpiWarps, kMmaWarp = kEpiWarps + 1, kScaleWarp = kEpiWarps + 2;
  constexpr int kGroupWarps = 4 * S::kColParts;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint32_t* staging = reinterpret_cast<uint32_t*>(smem + kStages * S::kStageBytes);
  float* scales = reinterpret_cast<float*>(smem + kStages * S::kStageBytes + S::kStagingBytes);   // [kSlots][kAhead][kScaleWords]
  uint8_t* tail = smem + kStages * S::kStageBytes + S::kStagingBytes + S::kScaleBytes;
  unsigned long long* keys = reinterpret_cast<unsigned long long*>(tail);
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(tail + S::kKeyBytes);
  uint64_t* empty_bar = full_bar + kStages;              // (kPairs: full and tempty are used in the even CTA)
  uint64_t* tfull_bar = empty_bar + kStages;
  uint64_t* tempty_bar = tfull_bar + kBufs;
  uint64_t* turn_bar = tempty_bar + kBufs;
  uint64_t* sfull_bar = turn_bar + kGroups;
  uint64_t* sempty_bar = sfull_bar + kSlots;
  uint64_t* drain_bar = sempty_bar + kSlots;
  uint32_t* tmem_base_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_base_slot + 1);
  int* last_flag = reinterpret_cast<int*>(tmem_base_slot + 2);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = kSplit || kPairs ? cluster_ctarank() : 0;
  const int half = kPairs ? static_cast<int>(rank & 1) : 0;      // of the pair; 0 issues the MMAs
  const uint32_t leader = rank - half;
  const int split = kSplit ? static_cast<int>(rank) / S::kCtas : 0;
  const int splits = kSplit ? a.splits : 1;
  const int k0 = kSplit ? static_cast<int>(static_cast<int64_t>(a.n_kb) * split / splits) : 0;
  const int k1 = kSplit ? static_cast<int>(static_cast<int64_t>(a.n_kb) * (split + 1) / splits) : a.n_kb;
  const int first = blockIdx.x / (S::kCtas * splits);
  const int step = kSplit ? a.n_tiles : gridDim.x / S::kCtas;    // (a cluster of splits takes one tile)
  // Tiles in bands of a.band column tiles: lane tiles one after another, the
  // band's column tiles fastest.  (Lane tiles fastest where band is 0.)
  const auto place = [&](int t, int* lt, int* ct) {
    if (a.band == 0) {
      *lt = t % a.n_lt;
      *ct = t / a.n_lt;
    } else {
      const int per = a.n_lt * a.band, b = t / per, in = t - b * per, width = min(a.band, a.n_ct - b * a.band);
      *lt = in / width;
      *ct = b * a.band + in % width;
    }
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&tfull_bar[i], 1);
      mbar_init(&tempty_bar[i], S::kCtas * kGroupWarps);
    }
    for (int i = 0; i < kGroups; ++i) mbar_init(&turn_bar[i], kGroupWarps);
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&sfull_bar[i], 32);
      mbar_init(&sempty_bar[i], kGroupWarps);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if constexpr (kSwap && kSample) {
    if (threadIdx.x < kBN) keys[threadIdx.x] = 0ull;
  }
  if (warp == kProducerWarp && lane == 0) {
    tma_prefetch_desc(&tmap_l);
    tma_prefetch_desc(&tmap_c);
  }
  if (warp == kMmaWarp) {
    if constexpr (kPairs) {
      tmem_alloc_pair(tmem_base_slot, S::kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_base_slot, S::kTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (kPairs) cluster_sync();                    // both CTAs' barriers exist before any cross-CTA signal
  tc_fence_after();
  const uint32_t tmem_base = *tmem_base_slot;

  // (the registers move within the roles' branches: code that both reach would
  // have to do with the fewer)
  if (warp >= kEpiWarps) {
    give_registers<S::kOtherRegs>();
    if (warp == kProducerWarp) {
      // ------------------------------------------------------------ TMA producer (both CTAs of a pair)
      pdl_wait();
      const uint32_t elected = elect_one();
      // a is read again by every tile of b; b by the tiles of a, side by side
      const uint64_t pol_a = policy_evict_last();
      const uint64_t pol_b = (kSwap ? a.n_ct : a.n_lt) > 1 ? policy_evict_normal() : policy_evict_first();
      const uint64_t pol_l = kSwap ? pol_b : pol_a, pol_c = kSwap ? pol_a : pol_b;
      const uint32_t full0 = smem_u32(full_bar), empty0 = smem_u32(empty_bar), smem0 = smem_u32(smem);
      const uint32_t leader0 = kPairs ? mapa_shared(full0, leader) : full0;
      const uint32_t bytes = S::kCtas * (a.box_l + a.box_c) * kBK;
      int stage = 0;
      uint32_t phase = 0;
      int64_t n_issued = 0;
      bool ok = true;
#pragma unroll 1
      for (int t = first; ok && t < a.n_tiles; t += step) {
        int lt, ct;
        place(t, &lt, &ct);
        const int l0 = lt * S::kTileL + half * kLanes, c0 = ct * kBN + half * S::kCLoad;
#pragma unroll 1
        for (int kb = k0; kb < k1; kb += kPairK) {
          ok = mbar_wait_warp(empty0 + stage * 8, phase ^ 1, a.err, abort_flag);
          if (!ok) break;
          const int blocks = min(kPairK, k1 - kb);
          if (half == 0) mbar_arrive_expect_tx_if(elected, full0 + stage * 8, blocks * bytes);
          uint32_t dst = smem0 + stage * S::kStageBytes;
#pragma unroll
          for (int i = 0; i < kPairK; ++i, dst += S::kBlockBytes) {
            if (i >= blocks) break;
            if constexpr (kPairs) {
              tma_load_2d_pair_if(elected, dst, &tmap_l, leader0 + stage * 8, (kb + i) * kBK, l0, pol_l);
              tma_load_2d_pair_if(elected, dst + kLTile, &tmap_c, leader0 + stage * 8, (kb + i) * kBK, c0, pol_c);
            } else {
              tma_load_2d_if(elected, dst, &tmap_l, full0 + stage * 8, (kb + i) * kBK, l0, pol_l);
              tma_load_2d_if(elected, dst + kLTile, &tmap_c, full0 + stage * 8, (kb + i) * kBK, c0, pol_c);
            }
          }
          ++n_issued;
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
      }
      if (!ok && half == 0) {                              // leave only after the loads in flight have landed
        volatile int no_abort = 0;
        for (int64_t i = max(static_cast<int64_t>(0), n_issued - kStages); i < n_issued; ++i)
          mbar_wait_warp(full0 + static_cast<uint32_t>(i % kStages) * 8, static_cast<uint32_t>((i / kStages) & 1), a.err,
                         &no_abort);
      }
    } else if (warp == kMmaWarp && half == 0) {
      // ------------------------------------------------------------ MMA issuer (of a pair: the even CTA)
      const uint32_t elected = elect_one();
      const uint32_t idesc = idesc_fp8_f32(a.l_e5m2, a.c_e5m2, S::kTileL, kBN);
      const uint16_t both = static_cast<uint16_t>(3u << leader);
      const uint64_t l_desc0 = smem_desc_k128(smem_u32(smem)), c_desc0 = smem_desc_k128(smem_u32(smem) + kLTile);
      const uint32_t full0 = smem_u32(full_bar), empty0 = smem_u32(empty_bar);
      const uint32_t tfull0 = smem_u32(tfull_bar), tempty0 = smem_u32(tempty_bar);
      int stage = 0, buf = 0;
      uint32_t phase = 0, buf_phase = 0, stage_seen = 0, buf_seen = 0;
      bool ok = true;
#pragma unroll 1
      for (int t = first; ok && t < a.n_tiles; t += step) {
#pragma unroll 1
        for (int kb = k0; kb < k1; kb += kPairK) {
          const int pos = (kb - k0) % kPer;                // within the buffer
          // (a barrier takes 100 clocks and more to look at: kThin looks at the next
          // ones before this stage's MMAs are issued, in the other forms the epilogue
          // waits for these MMAs)
          ok = (pos > 0 || (kSwap && __all_sync(0xffffffffu, buf_seen)) ||
                mbar_wait_warp(tempty0 + buf * 8, buf_phase ^ 1, a.err, abort_flag)) &&
               ((kSwap && __all_sync(0xffffffffu, stage_seen)) || mbar_wait_warp(full0 + stage * 8, phase, a.err, abort_flag));
          if (!ok) break;
          tc_fence_after();
          const int blocks = min(kPairK, k1 - kb);
          const bool last = pos + kPairK >= kPer || kb + kPairK >= k1;
          const uint64_t l_desc = l_desc0 + stage * (S::kStageBytes >> 4);
          const uint64_t c_desc = c_desc0 + stage * (S::kStageBytes >> 4);
          const uint32_t d_tmem = tmem_base + (buf * kPer + pos) * kBN;
          const uint32_t empty = empty0 + stage * 8, tfull = tfull0 + buf * 8;
          if (++stage == kStages) { stage = 0; phase ^= 1; }
          if (last && ++buf == kBufs) { buf = 0; buf_phase ^= 1; }
          if constexpr (kSwap) {
            stage_seen = mbar_test(full0 + stage * 8, phase);
            if (last) buf_seen = mbar_test(tempty0 + buf * 8, buf_phase ^ 1);
          }
#pragma unroll
          for (int i = 0; i < kPairK; ++i) {
            if (i >= blocks) break;
#pragma unroll
            for (int k = 0; k < kBK / 32; ++k) {
              constexpr int kNext = S::kBlockBytes >> 4;
              if constexpr (kPairs)
                mma_fp8_pair_if(elected, d_tmem + i * kBN, l_desc + i * kNext + k * 2, c_desc + i * kNext + k * 2, idesc, k > 0);
              else
                mma_fp8_if(elected, d_tmem + i * kBN, l_desc + i * kNext + k * 2, c_desc + i * kNext + k * 2, idesc, k > 0);
            }
          }
          if constexpr (kPairs) {
            mma_commit_pair_multicast_if(elected, empty, both);
            if (last) mma_commit_pair_multicast_if(elected, tfull, both);
          } else {
            mma_commit_if(elected, empty);
            if (last) mma_commit_if(elected, tfull);
          }
        }
      }
      if (!ok) {
        if constexpr (kPairs)
          mma_commit_pair_multicast_if(elected, smem_u32(drain_bar), static_cast<uint16_t>(1u << leader));
        else
          mma_commit_if(elected, smem_u32(drain_bar));
        volatile int no_abort = 0;
        mbar_wait_warp(smem_u32(drain_bar), 0, a.err, &no_abort);
      }
    } else if (warp == kScaleWarp) {
      // ------------------------------------------------------------ scales, kAhead blocks at a time
      pdl_wait();
      const uint32_t sfull0 = smem_u32(sfull_bar), sempty0 = smem_u32(sempty_bar);
      int slot = 0;
      uint32_t phase = 0;
      bool ok = true;
#pragma unroll 1
      for (int t = first; ok && t < a.n_tiles; t += step) {
        int lt, ct;
        place(t, &lt, &ct);
        const int64_t l0 = static_cast<int64_t>(lt) * S::kTileL + half * kLanes, c0 = static_cast<int64_t>(ct) * kBN;
        const int64_t l = kLaneScales ? l0 + lane : l0, c = kColScales ? c0 + lane : c0 + lane * kPart;
        const int l_left = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(kLanes), a.l_rows - l0)));
        const int c_left = static_cast<int>(min(static_cast<int64_t>(kBN), a.c_rows - c0));
        const float* sl = a.sl.at + (l >> a.sl.shift) * a.sl.s_row + k0 * a.sl.s_col;
        const float* sc = a.sc.at + (c >> a.sc.shift) * a.sc.s_row + k0 * a.sc.s_col;
        const int64_t l_step = 32 * a.sl.s_row, c_step = 32 * a.sc.s_row;
#pragma unroll 1
        for (int kb = k0; kb < k1; kb += kAhead) {
          ok = mbar_wait_warp(sempty0 + slot * 8, phase ^ 1, a.err, abort_flag);
          if (!ok) break;
          float* dst = scales + slot * kAhead * S::kScaleWords + lane;
#pragma unroll 1
          for (int i = 0; i < min(kAhead, k1 - kb); ++i, sl += a.sl.s_col, sc += a.sc.s_col, dst += S::kScaleWords) {
            if constexpr (kLaneScales) {
#pragma unroll
              for (int j = 0; j < kLanes / 32; ++j)
                if (j * 32 + lane < l_left) copy_async_f32(dst + j * 32, sl + j * l_step);
            } else {
              if (lane == 0 && l_left > 0) copy_async_f32(dst, sl);
            }
            if constexpr (kColScales) {
#pragma unroll
              for (int j = 0; j < (kBN + 31) / 32; ++j)
                if (j * 32 + lane < c_left) copy_async_f32(dst + kLanes + j * 32, sc + j * c_step);
            } else {
              if (lane * kPart < c_left) copy_async_f32(dst + kLanes, sc);
            }
          }
          copy_async_arrive(sfull0 + slot * 8);
          if (++slot == kSlots) { slot = 0; phase ^= 1; }
        }
      }
      copy_async_wait();
    }
  } else {
    // -------------------------------------------------------------- epilogue
    take_registers<S::kEpiRegs>();
    const int quad = warp & 3;                             // TMEM lane quarter
    const int part = (warp >> 2) % S::kColParts;           // columns
    const int group = (warp >> 2) / S::kColParts;          // every kGroups-th tile
    float* stage = reinterpret_cast<float*>(staging + warp * S::kWarpWords);
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + part * kPart;
    const uint32_t tempty0 = kPairs ? mapa_shared(smem_u32(tempty_bar), leader) : smem_u32(tempty_bar);
    const uint32_t sempty0 = smem_u32(sempty_bar);
    const int n_k = k1 - k0, n_use = (n_k + kPer - 1) / kPer, n_fill = (n_k + kAhead - 1) / kAhead;
    pdl_wait();
    if (kSample && warp == 0) pdl_launch_dependents();     // (see pdl_wait_then_launch; nothing else fits beside this block)
    // Columns of a TMEM load, its registers, and the loads of a block.  In
    // fragments, load q holds lanes 16 (q % 2) .. of 32 columns from 32 (q / 2) on:
    // register i lies in row 16 (q % 2) + 8 (i / 2 % 2) + lane / 4 and column
    // 32 (q / 2) + 8 (i / 4) + 2 (lane % 4) + i % 2.
    constexpr int kCols = kPart < 32 ? kPart : 32;
    constexpr int kRegs = kColScales ? kCols / 2 : kCols;
    constexpr int kLoads = kPart / kRegs;
    const auto frag_row = [&](int q, int i) { return 16 * (q & 1) + 8 * (i >> 1 & 1) + (lane >> 2); };
    const auto frag_col = [&](int q, int i) { return kCols * (q >> 1) + 8 * (i >> 2) + 2 * (lane & 3) + (i & 1); };
    bool ok = true;
    uint32_t turn_phase = 0;
    // sampling: the rows that this thread scans, 32 apart, and what it found
    constexpr int kScans = kSwap ? (kPart + 31) / 32 : 1;
    Best best[kScans];
    RowTemp temps[kScans];
    int64_t scan_row = -1;
    auto begin_rows = [&](int64_t row) {
#pragma unroll
      for (int i = 0; i < kScans; ++i) {
        best[i] = best_none();
        temps[i] = row_temp(row + 32 * i < a.p.B ? a.p.temp[row + 32 * i] : -1.0f);
      }
      scan_row = row;
    };
    if constexpr (kSample && kSwap) begin_rows(lane);
    int tile = group;                                      // of this CTA's, in order
#pragma unroll 1
    for (int t = first + group * step; t < a.n_tiles; t += kGroups * step, tile += kGroups) {
      int lt, ct;
      place(t, &lt, &ct);
      const int64_t l0 = static_cast<int64_t>(lt) * S::kTileL + half * kLanes + quad * 32;
      const int64_t c0 = static_cast<int64_t>(ct) * kBN + part * kPart;
      const bool live = l0 < a.l_rows && c0 < a.c_rows;    // this warp has something to add up
      const bool lane_ok = l0 + lane < a.l_rows;
      if constexpr (kSample && !kSwap) {
        if (l0 + lane != scan_row) {
          if (scan_row >= 0 && scan_row < a.p.B) push_candidate(a.f, scan_row, best[0]);
          begin_rows(l0 + lane);
        }
      }
      if (kGroups > 1 && tile > 0) {                       // the group before has taken the last tile's sums
        ok = mbar_wait(&turn_bar[group], turn_phase, a.err, abort_flag);
        if (!ok) break;
        turn_phase ^= 1;
      }
      f32x2 sum[kLoads * kRegs / 2];                       // columns by twos
#pragma unroll
      for (int c = 0; c < kLoads * kRegs / 2; ++c) sum[c] = 0ull;
      uint32_t use = static_cast<uint32_t>(tile) * n_use, fill = static_cast<uint32_t>(tile) * n_fill;
      uint32_t sums[S::kTwoBlocks ? 2 : 1][kLoads][kRegs];     // of two blocks, in turn, or of one
      // Waits for block kb's sums and scales and begins to load the sums.
      auto begin = [&](int kb, uint32_t (&r)[kLoads][kRegs]) {
        const int pos = (kb - k0) % kPer;
        if ((kb - k0) % kAhead == 0) {
          const uint32_t n = static_cast<uint32_t>(tile) * n_fill + (kb - k0) / kAhead;
          if (!mbar_wait(&sfull_bar[n % kSlots], (n / kSlots) & 1, a.err, abort_flag)) return false;
        }
        if (pos == 0) {
          if (!mbar_wait(&tfull_bar[use % kBufs], (use / kBufs) & 1, a.err, abort_flag)) return false;
          __syncwarp();
          tc_fence_after();
        }
        if (live) {
          const uint32_t from = lane_addr + (use % kBufs * kPer + pos) * kBN;
#pragma unroll
          for (int q = 0; q < kLoads; ++q) {
            if constexpr (kColScales)
              tmem_ld_frag(from + (static_cast<uint32_t>(q & 1) << 20) + kCols * (q >> 1), r[q]);
            else
              tmem_ld_32(from + kCols * q, r[q]);
          }
        }
        return true;
      };
      // Adds block kb's sums, while the next block's are loaded where there are registers for them.
      auto finish = [&](int kb, uint32_t (&r)[kLoads][kRegs], uint32_t (&r_next)[kLoads][kRegs]) {
        const int pos = (kb - k0) % kPer, at = (kb - k0) % kAhead;
        // the factors of this block: of the thread's rows and columns
        const float* lane_scales = scales + (fill % kSlots * kAhead + at) * S::kScaleWords;
        const float* col_scales = lane_scales + kLanes;
        float f[kLaneScales && kColScales ? 4 : 1];
        if constexpr (kLaneScales && kColScales) {
#pragma unroll
          for (int i = 0; i < 4; ++i) f[i] = lane_scales[quad * 32 + 8 * i + (lane >> 2)];
        } else if constexpr (kLaneScales) {
          f[0] = lane_scales[quad * 32 + lane] * col_scales[part];
        } else {
          f[0] = lane_scales[0];
        }
        if (live) {
#pragma unroll
          for (int q = 0; q < kLoads; ++q) tmem_ld_wait_for(r[q]);
        }
        if (pos == kPer - 1 || kb + 1 == k1) {             // the buffer's last block
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if constexpr (kPairs)
              mbar_arrive_tmem_cluster(tempty0 + use % kBufs * 8);
            else
              mbar_arrive_tmem(tempty0 + use % kBufs * 8);
          }
          ++use;
        }
        bool there = true;
        if (S::kTwoBlocks && kb + 1 < k1) there = begin(kb + 1, r_next);
        if (live) {
          f32x2 w[kColScales ? kCols / 8 : 1];
#pragma unroll
          for (int q = 0; q < kLoads; ++q) {
            if constexpr (kColScales) {
              if (q % 2 == 0) {
#pragma unroll
                for (int g = 0; g < kCols / 8; ++g) {
                  w[g] = *reinterpret_cast<const f32x2*>(col_scales + part * kPart + kCols * (q >> 1) + 8 * g + 2 * (lane & 3));
                  if constexpr (!kLaneScales) w[g] = mul2(w[g], pack2(f[0], f[0]));
                }
              }
            }
#pragma unroll
            for (int i = 0; i < kRegs; i += 2) {
              f32x2 by;
              if constexpr (!kColScales) {
                by = pack2(f[0], f[0]);
              } else if constexpr (kLaneScales) {
                const float row = f[2 * (q & 1) + (i >> 1 & 1)];
                by = mul2(w[i >> 2], pack2(row, row));
              } else {
                by = w[i >> 2];
              }
              f32x2& s = sum[(q * kRegs + i) / 2];
              s = fma2(pack2(__uint_as_float(r[q][i]), __uint_as_float(r[q][i + 1])), by, s);
            }
          }
        }
        if (at == kAhead - 1 || kb + 1 == k1) {            // this slot's scales are done with
          __syncwarp();
          if (lane == 0) mbar_arrive(&sempty_bar[fill % kSlots]);
          ++fill;
        }
        if (!S::kTwoBlocks && kb + 1 < k1) there = begin(kb + 1, r_next);
        return there;
      };
      ok = begin(k0, sums[0]);
#pragma unroll 1
      for (int kb = k0; ok && kb < k1; kb += S::kTwoBlocks ? 2 : 1) {
        ok = finish(kb, sums[0], sums[S::kTwoBlocks ? 1 : 0]);
        if (S::kTwoBlocks && ok && kb + 1 < k1) ok = finish(kb + 1, sums[S::kTwoBlocks ? 1 : 0], sums[0]);
      }
      if (!ok) break;
      __syncwarp();
      if (kGroups > 1 && lane == 0) mbar_arrive(&turn_bar[(group + 1) % kGroups]);
      float acc[kLoads * kRegs];
#pragma unroll
      for (int c = 0; c < kLoads * kRegs / 2; ++c) {
        const float2 v = unpack2(sum[c]);
        acc[2 * c] = v.x;
        acc[2 * c + 1] = v.y;
      }
      if constexpr (kSplit) {
        // every load has landed and been multiplied: the stages hold the partial tile now
        float* red = reinterpret_cast<float*>(smem);
        if (live) {
#pragma unroll
          for (int q = 0; q < kLoads; ++q)
#pragma unroll
            for (int i = 0; i < kRegs; ++i) {
              const int row = quad * 32 + (kColScales ? frag_row(q, i) : lane);
              const int col = part * kPart + (kColScales ? frag_col(q, i) : q * kCols + i);
              red[kSwap ? col * (kLanes + 1) + row : row * (kBN + 1) + col] = acc[q * kRegs + i];
            }
        }
      } else if (live && !kSample && !kSwap && c0 + kPart <= a.tma_cols) {
        if constexpr (!kSample && !kSwap) {
          if (a.out_type == FS_TYPE_F32)
            store_tile<float, kColScales>(&tmap_o, acc, reinterpret_cast<uint8_t*>(stage), l0, c0);
          else if (a.out_type == FS_TYPE_BF16)
            store_tile<__nv_bfloat16, kColScales>(&tmap_o, acc, reinterpret_cast<uint8_t*>(stage), l0, c0);
          else
            store_tile<__half, kColScales>(&tmap_o, acc, reinterpret_cast<uint8_t*>(stage), l0, c0);
        }
      } else if (live) {
        if constexpr (!kSample && !kSwap) {
          if (lane == 0) bulk_wait_read();
          __syncwarp();
        }
        // 32 rows x 32 columns at a time through the staging area: a lane then scans
        // a row (with kSwap, where lanes are vocabulary ids, a column), or a store
        // covers whole rows of the output
        // (one copy of the code: the columns are selected)
#pragma unroll 1
        for (int c = 0; c < kPart; c += 32) {
          if (c0 + c >= a.c_rows) break;
          float bar = -INFINITY;
          if constexpr (kSample) {
            if (scan_row + (kSwap ? c : 0) < a.p.B) bar = best_so_far(a.f.keys + scan_row + (kSwap ? c : 0));
          }
#pragma unroll
          for (int j = 0; j < (kPart < 32 ? kPart : 32); ++j) {
            constexpr int kNext = kPart > 32 ? 32 : 0;     // in acc, of the other 32 columns
            const float v = c == 0 ? acc[j] : acc[j + kNext];
            const int q = kColScales ? j / kRegs : 0, i = j % kRegs;
            const int row = kColScales ? frag_row(q, i) : lane, col = kColScales ? frag_col(q, i) : i;
            stage[kSample ? row * kPitch + col : kSwap ? col * kPitch + row : row * 32 + (col ^ row)] = v;
          }
          __syncwarp();
          if constexpr (kSample) {
            const int64_t row = scan_row + (kSwap ? c : 0);
            const RowTemp rt = c == 0 ? temps[0] : temps[kScans - 1];
            if (row < a.p.B && rt.mode != kRowInvalid && !(kSwap && lane >= kPart)) {
              RowScan scan;
              scan.key = PhiloxKey{static_cast<uint32_t>(a.p.seed), static_cast<uint32_t>(a.p.seed >> 32)};
              scan.row = static_cast<uint32_t>(row);
              scan.step_lo = static_cast<uint32_t>(a.p.step);
              scan.step_hi = static_cast<uint32_t>(a.p.step >> 32);
              scan.inv_t = rt.inv_t;
              scan.greedy = rt.mode == kRowGreedy;
              scan.bias_row = a.p.bias != nullptr ? a.p.bias + row * a.p.bias_stride : nullptr;
              const int64_t v0 = kSwap ? l0 : c0 + c;
              const Best b = scan_staged<kSwap ? kPitch : 1>(stage + (kSwap ? lane : lane * kPitch), v0, a.p.V_local, scan,
                                                             c == 0 ? best[0] : best[kScans - 1], bar);
              if (c == 0 || kScans == 1) best[0] = b; else best[kScans - 1] = b;
              if (b.z > bar) {                             // for the other warps' scans
                const unsigned long long key = pack_key(b.z, b.id);
                if (!kSwap || atomicMax(keys + row, key) < key) atomicMax(a.f.keys + row, key);
              }
            }
          } else if constexpr (kSwap) {
            // lanes lie along a row of the output
            const int cols = static_cast<int>(min(static_cast<int64_t>(kCols), a.c_rows - c0 - c));
            if (lane_ok) {
#pragma unroll 4
              for (int j = 0; j < cols; ++j) store_one(a, c0 + c + j, l0 + lane, stage[j * kPitch + lane]);
            }
          } else {
            store_rows(a, stage, l0, c0 + c);
          }
          __syncwarp();
        }
      }
    }
    if constexpr (!kSample && !kSwap && !kSplit) {
      if (lane == 0) bulk_wait();
    }
    if constexpr (kSample) {
      if constexpr (kSwap) {
        // the CTA's warps first: few rows would otherwise gather all warps' candidates
#pragma unroll
        for (int i = 0; i < kScans; ++i)
          if (scan_row + 32 * i < a.p.B && lane < kPart && best[i].id != kNoId)
            atomicMax(keys + scan_row + 32 * i, pack_key(best[i].z, best[i].id));
        named_bar1_and<kEpiWarps * 32>(true);
        if (threadIdx.x < kBN && threadIdx.x < a.p.B && keys[threadIdx.x] != 0ull)
          atomicMax(a.f.keys + threadIdx.x, keys[threadIdx.x]);
      } else {
        if (scan_row >= 0 && scan_row < a.p.B) push_candidate(a.f, scan_row, best[0]);
      }
      finish_grid<false>(a.f, a.p.B, threadIdx.x, kEpiWarps * 32, last_flag, named_bar1_and<kEpiWarps * 32>);
    }
  }

  if constexpr (kSplit) {
    __syncwarp();
    cluster_sync();                                        // every partial tile is there
    if (warp < kEpiWarps && *abort_flag == 0) {
      int lt, ct;
      place(first, &lt, &ct);
      const int64_t l0 = static_cast<int64_t>(lt) * S::kTileL + half * kLanes, c0 = static_cast<int64_t>(ct) * kBN;
      const int l_rows = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(kLanes), a.l_rows - l0)));
      const int c_rows = static_cast<int>(min(static_cast<int64_t>(kBN), a.c_rows - c0));
      // this CTA's part: of the axis along which the output's rows run
      const int along = kSwap ? l_rows : c_rows, across = kSwap ? c_rows : l_rows;
      const int from = along * split / splits, span = along * (split + 1) / splits - from;
      const uint32_t red0 = smem_u32(smem);
      uint32_t peer[kMaxSplits];
#pragma unroll
      for (int s = 0; s < kMaxSplits; ++s) peer[s] = mapa_shared(red0, s < splits ? s * S::kCtas + half : rank);
#pragma unroll 1
      for (int i = threadIdx.x; i < span * across; i += kEpiWarps * 32) {
        const int row = i / span, col = from + i % span;
        const uint32_t at = static_cast<uint32_t>(row * (kSwap ? kLanes + 1 : kBN + 1) + col) * 4;
        float v[kMaxSplits];
#pragma unroll
        for (int s = 0; s < kMaxSplits; ++s) v[s] = s < splits ? ld_shared_cluster_f32(peer[s] + at) : 0.0f;
        float sum = v[0];
#pragma unroll
        for (int s = 1; s < kMaxSplits; ++s) sum += v[s];
        store_one(a, (kSwap ? c0 : l0) + row, (kSwap ? l0 : c0) + col, sum);
      }
    }
    __syncwarp();
  }
  // teardown: no CTA leaves (or frees TMEM) while the pair's MMAs, the peer's
  // signals or its reads may still touch it
  tc_fence_before();
  __syncthreads();
  if constexpr (kSplit || kPairs) cluster_sync();
  tc_fence_after();
  if (warp == kMmaWarp) {
    if constexpr (kPairs)
      tmem_dealloc_pair(tmem_base, S::kTmemCols);
    else
      tmem_dealloc(tmem_base, S::kTmemCols);
  }
}

int sm_count();

// a [m, k], b [n, k]; `ctas`: CTAs (of kPair: pairs), or clusters of splits.
template <Form kForm, int kBN, bool kSample, bool kLaneScales, bool kColScales, bool kSplit>
cudaError_t launch(Args a, const Fp8Matrix& ma, const Fp8Matrix& mb, int64_t m, int64_t n, int64_t k, int ctas,
                   cudaStream_t stream) {
  using S = Shape<kForm, kBN, kSample, kColScales>;
  constexpr bool kSwap = S::kSwap;
  const Fp8Matrix& l = kSwap ? mb : ma;
  const Fp8Matrix& c = kSwap ? ma : mb;
  a.l_rows = kSwap ? n : m;
  a.c_rows = kSwap ? m : n;
  a.sl = Scales{l.scale, l.s_row, l.s_col, l.block_rows == 1 ? 0 : 7};
  a.sc = Scales{c.scale, c.s_row, c.s_col, c.block_rows == 1 ? 0 : 7};
  a.l_e5m2 = l.type == FS_TYPE_E5M2;
  a.c_e5m2 = c.type == FS_TYPE_E5M2;
  a.box_l = static_cast<int>(std::min<int64_t>(kLanes, (a.l_rows + 7) / 8 * 8));
  a.box_c = static_cast<int>(std::min<int64_t>(S::kCLoad, (a.c_rows + 7) / 8 * 8));
  CUtensorMap tl, tc;
  if (!encode_rows_u8(&tl, l.q, a.l_rows, k, l.stride, kBK, a.box_l) || !encode_rows_u8(&tc, c.q, a.c_rows, k, c.stride, kBK, a.box_c))
    return cudaErrorInvalidValue;
  CUtensorMap to = tc;                                     // (of the output, where it is used)
  if constexpr (!kSample && !kSwap && !kSplit) {
    const int64_t width = a.out_type == FS_TYPE_F32 ? 4 : 2;
    // (a TMA store leaves out what lies behind the last column by 16 bytes, not by
    // elements: rows that end within 16 have their last columns stored by the warps)
    if (reinterpret_cast<uintptr_t>(a.out) % 16 == 0 && a.out_stride * width % 16 == 0 && n * width <= INT32_MAX - 1024 &&
        encode_rows_u8(&to, a.out, m, n * width, a.out_stride * width, 128, 32))
      a.tma_cols = n * width % 16 == 0 ? INT64_MAX : n;
  }
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  constexpr auto fn = kernel<kForm, kBN, kSample, kLaneScales, kColScales, kSplit>;
  if (e == cudaSuccess) e = raise_smem_limit<fn>(dev, S::kSmem);
  if (e == cudaSuccess) {
    // a warpgroup's rise would wait for ever in a kernel compiled with fewer
    // (only an answer is kept: a query that failed is made again by the next call)
    static std::atomic<int> known{0};
    int regs = known.load(std::memory_order_relaxed);
    if (regs == 0) {
      cudaFuncAttributes attr = {};
      e = cudaFuncGetAttributes(&attr, fn);
      if (e != cudaSuccess) return e;
      known.store(regs = attr.numRegs, std::memory_order_relaxed);
    }
    if (regs != S::kLaunchRegs) return cudaErrorInvalidDeviceFunction;
  }
  if (e != cudaSuccess) return e;
  const int cluster = S::kCtas * (kSplit ? a.splits : 1);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas * cluster));
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, fn, tl, tc, to, a);
}

// Tiles of a launch; false where their number passes 31 bits.
inline bool set_tiles(Args* a, int64_t l_rows, int64_t c_rows, int tile_l, int bn, int band) {
  const int64_t n_lt = (l_rows + tile_l - 1) / tile_l, n_ct = (c_rows + bn - 1) / bn;
  if (n_lt * n_ct > INT32_MAX / 2) return false;
  a->n_lt = static_cast<int>(n_lt);
  a->n_ct = static_cast<int>(n_ct);
  a->n_tiles = static_cast<int>(n_lt * n_ct);
  a->band = band;
  return true;
}

// Columns of a thin tile: as few as hold a's rows.
constexpr int64_t kThinMaxRows = 64;
inline int thin_columns(int64_t m) { return m <= 16 ? 16 : m <= 32 ? 32 : 64; }

}  // namespace fp8
}  // namespace fs
