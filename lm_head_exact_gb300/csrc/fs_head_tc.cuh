// Tensor-core engine of the training operators of the LM head: one persistent,
// warp-specialized kernel over pairs of CTAs (tcgen05 cta_group::2) for the
// four products
//
//   kLse  x^T  = W h^T          each tile reduced to its columns' sums of exp
//   kDs   ds^T from x^T         the same product, written as bf16 ds
//   kDh   grad_h^T = W^T ds^T   split along the vocabulary, fp32 partials
//   kDw   grad_W = ds^T h
//
// The axis that a tile's epilogue stores along lies on the MMA's M axis, that
// is on the 32 lanes of a warp (vocabulary ids of x and ds, the model width of
// grad_h), so it loads and stores whole lines; and the tokens lie on N, whose
// size is any multiple of 16, so a batch of 517 tokens runs as 3 x 176 columns
// instead of 3 x 256 rows.  grad_W has the model width on N: its rows go
// through shared memory and leave by TMA.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "fs_head_ptx.cuh"
#include "fs_tmap.h"
#include "fs_train.h"

namespace fs {
namespace head {

using namespace sm100;

enum Kind : int { kLse, kDs, kDh, kDw };

constexpr int kTileM = 256;              // rows of a pair's tile, 128 a CTA
constexpr int kMaxN = 256;               // columns of a pair's tile
constexpr int kBK = 64;
constexpr int kATile = 128 * kBK * 2;    // bytes of A a CTA loads per stage
constexpr int kMaxStages = 12;
constexpr int kEpiWarps = 16;            // 4 lane quarters x 4 column parts
constexpr int kParts = 4;
constexpr int kPartCols = kMaxN / kParts;
constexpr int kProducerWarp = kEpiWarps;
constexpr int kMmaWarp = kEpiWarps + 1;
constexpr int kThreads = (kEpiWarps + 2) * 32;
constexpr uint16_t kPairMask = 0x3;

constexpr bool a_mn_major(Kind k) { return k == kDh || k == kDw; }
constexpr bool b_mn_major(Kind k) { return k == kDw; }

// Shared memory behind the stages: barriers, then the epilogue's arrays.
constexpr int kBarBytes = (2 * kMaxStages + 5) * 8 + 24;
constexpr int epi_arrays(Kind k) { return k == kLse ? 1 : k == kDs ? 3 : 0; }    // of kPartCols floats a warp
constexpr int epi_bytes(Kind k) { return epi_arrays(k) * kEpiWarps * kPartCols * 4; }
// The tensor cores add to an accumulator in TMEM by cutting, not rounding: each
// of the d / 16 additions of a logit loses half a step of the running sum on
// average, always toward zero, which for d = 4096 shrinks x by 5e-6 and moves
// lse by 1e-6 of itself.  So logits are accumulated sub_blocks k blocks of 64
// products at a time and the pieces are added in registers, rounding to
// nearest: 16 blocks for up to 256 tokens, one column tile, where the head's way
// from HBM hides it (2e-7 of lse at any d; 8 blocks halve that and cost 10 of
// 165 us), and 32 beyond (4e-7), where smaller pieces end sooner than the
// epilogue of the tile before (528 rows of a 4096 x 128256 head: 350 us with
// 32, 405 with 16).  The gradients, rounded to 8 bits in the end, take their
// whole sums.
constexpr int sub_blocks(int64_t n) { return n <= 256 ? 16 : 32; }
constexpr int kWhole = 0x7fffffff;
// kDw: a box of 32 vocabulary rows x 64 columns of bf16 a warp, on its way out.
constexpr int kBoxCols = 64;
constexpr int kBoxBytes = 32 * kBoxCols * 2;
constexpr int out_bytes(Kind k) { return k == kDw ? kEpiWarps * kBoxBytes : 0; }
constexpr int kSmemLimit = 232448;

// L2 priority of an operand.  One that is read once gives way first.  One that
// several tiles read must outlast the output written in between (grad_W of 528
// rows: 427 us with kStream, 363 with kNormal).  One of at most kKeepBytes is
// read again by the next launches (W by the backward pass, ds by both products)
// and gives way last: a training pass over 257 rows of a 520 x 32001 head takes
// 107 us so and 117 without.  A larger one would not be there any more, and
// would only stay in the way of what follows.
enum Keep : int { kStream, kNormal, kLong };
constexpr int64_t kKeepBytes = int64_t(48) << 20;

__device__ __forceinline__ uint64_t policy_of(Keep k) {
  return k == kStream ? policy_evict_first() : k == kNormal ? policy_evict_normal() : policy_evict_last();
}

struct Args {
  HeadProblem p;
  int64_t M, N;              // extents of this launch's product
  int bn;                    // columns of a tile (a multiple of 16, <= 256)
  int n_stages;
  int n_nt;                  // column tiles
  int n_mt;                  // row tiles
  int n_kb;                  // k blocks of the whole product
  int splits;                // kDh
  int sub;                   // k blocks that one accumulator takes
  int n_pairs;               // pairs of the grid
  Keep keep_a, keep_b;       // the operands' L2 priorities
  bool prefetch;             // kDw: bring the next tile's ds into L2 ahead
  // kLse
  LsePart* parts;            // [parts, n]
  float* own_x;              // [n]
  float* kept;               // nullable [n, kept_pitch]
  int64_t kept_pitch;
  // kDs
  const float* logp;
  const float* lse;
  const float* coef;
  __nv_bfloat16* ds;
  int64_t ds_pitch;
  int64_t v0;                // first vocabulary row of the chunk
  // kDh
  float* partials;
  bool add;
  // kDs writes, kDw reads: a token's own entry of ds, what rounding it to bf16
  // left over [n]; kDw: the tokens' ids (-1: no gradient) and h [n, N]
  float* rest;
  const int* own;
  const __nv_bfloat16* h;
  int* err;
};

// The tiles of one pair: every n_pairs-th of an order in which the tiles that
// run side by side share what is read from HBM.  kLse and kDs: the column tiles
// (tokens) of one row tile after another, so that W is read once.  kDh: one
// split after another, so that all pairs work on the same vocabulary rows at a
// time.  kDw: the column tiles (the model width) of one row tile after another,
// so that ds is read once.
//
// The order is a mixed-radix count (kDh: row tile, column tile, split; else
// column tile, row tile); a pair's step through it is split into
// digits once, so that moving on takes additions and carries.
template <Kind kKind>
struct Units {
  static constexpr bool kColsFirst = kKind != kDh;
  int lo, mid, hi;                             // the digits of the present tile
  int step_lo, step_mid, step_hi, n_lo, n_mid, n_hi;
  int n_kb, splits;

  __device__ __forceinline__ Units(const Args& a, int pair)
      : n_lo(kColsFirst ? a.n_nt : a.n_mt), n_mid(kColsFirst ? a.n_mt : a.n_nt), n_hi(a.splits), n_kb(a.n_kb), splits(a.splits) {
    lo = pair % n_lo;
    mid = pair / n_lo % n_mid;
    hi = pair / n_lo / n_mid;
    step_lo = a.n_pairs % n_lo;
    step_mid = a.n_pairs / n_lo % n_mid;
    step_hi = a.n_pairs / n_lo / n_mid;
  }
  __device__ __forceinline__ bool more() const { return hi < n_hi; }
  __device__ __forceinline__ void next() {
    lo += step_lo;
    mid += step_mid;
    hi += step_hi;
    if (lo >= n_lo) { lo -= n_lo; ++mid; }
    if (mid >= n_mid) { mid -= n_mid; ++hi; }
  }
  __device__ __forceinline__ int mt() const { return kColsFirst ? mid : lo; }
  __device__ __forceinline__ int nt() const { return kColsFirst ? lo : mid; }
  __device__ __forceinline__ int split() const { return hi; }
  __device__ __forceinline__ int k0() const {
    return kKind == kDh ? static_cast<int>(static_cast<int64_t>(n_kb) * hi / splits) : 0;
  }
  __device__ __forceinline__ int k1() const {
    return kKind == kDh ? static_cast<int>(static_cast<int64_t>(n_kb) * (hi + 1) / splits) : n_kb;
  }
};

// ---------------------------------------------------------------- logit epilogues
// Exponentials are __expf's, within some 2^-21 of their value where the result
// matters: a term of a row's sum, or an entry of ds that is rounded to 2^-8
// right after.  expf's further bits would be lost in the logits' own error, and
// its instructions are on every element.
constexpr float kLowest = -3.402823466e38f;  // the lowest finite value

// value(i) of 16 columns joined over the warp's lanes: lanes 2 i and 2 i + 1
// return column i.  16 shuffles instead of the 80 of 16 separate reductions:
// each step but the last sends the half of the values that the other lane
// keeps.
template <typename Join, typename Value>
__device__ __forceinline__ float join_columns(int lane, Join join, Value value) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool up = (lane & 16) != 0;
    const float lo = value(i), hi = value(i + 8);
    v[i] = join(up ? hi : lo, __shfl_xor_sync(0xffffffffu, up ? lo : hi, 16));
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) {
    const bool up = (lane & (2 * o)) != 0;
#pragma unroll
    for (int i = 0; i < o; ++i)
      v[i] = join(up ? v[i + o] : v[i], __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + o], 2 * o));
  }
  return join(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
}

// The largest value of a warp, in every lane; NaNs do not count.  One
// instruction on this GPU, at 0.84 clocks a warp (a shuffle takes 1.03).
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ LsePart lse_join(LsePart a, LsePart b) {
  const float m = fmaxf(a.m, b.m);
  return LsePart{m, a.s * __expf(a.m - m) + b.s * __expf(b.m - m)};
}

// A token's own entry of ds, c (1 - p), is the largest of its row, by far
// where the rest is spread over many entries, and its rounding to bf16 alone
// would then make the gradients' error half again as large as rounding the
// results does.  What the rounding leaves over is kept and added in fp32: rest
// W[id] to grad_h, rest h to row id of grad_W.  1 - p comes from logp: for a
// token that is nearly certain, 1 - exp(x - lse) would consist of the
// rounding of lse (at lse = 200 and p = 1 - 1e-4 it is off by 7%).
__device__ __forceinline__ __nv_bfloat16 own_ds_of(float logp, float coef, float& rest) {
  const float v = -coef * expm1f(logp);
  const __nv_bfloat16 r = __float2bfloat16_rn(v);
  rest = v - __bfloat162float(r);
  return r;
}

// ds of another token; rows without a gradient hold zeros whatever their
// logits are.
__device__ __forceinline__ __nv_bfloat16 ds_of(float x, float lse, float coef) {
  return __float2bfloat16_rn(coef == 0.0f ? 0.0f : -coef * __expf(x - lse));
}

// The tokens t whose own rows are among the 32 rows from m_warp on, in order,
// with the row's number; the whole warp looks at 128 tokens at a time and
// visits each one found together.  Tokens that share a row are visited one
// after another, 0.9 us each: where most of some ten thousand tokens have one
// id, or the vocabulary has fewer rows than that, this is what grad_W takes.
template <typename Visit>
__device__ __forceinline__ void each_own(const Args& a, int m_warp, Visit visit) {
  const int lane = threadIdx.x & 31;
  const int n = static_cast<int>(a.p.n), first = static_cast<int>(a.v0) + m_warp;
  for (int t0 = 0; t0 < n; t0 += 128) {
    int row[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int t = t0 + k * 32 + lane;
      row[k] = t >= 0 && t < n ? __ldg(a.own + t) - first : -1;     // (t may pass 2^31)
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t found = __ballot_sync(0xffffffffu, static_cast<unsigned>(row[k]) < 32u);
      while (found != 0) {
        const int src = __ffs(found) - 1;
        found &= found - 1;
        visit(t0 + k * 32 + src, __shfl_sync(0xffffffffu, row[k], src));
        __syncwarp();
      }
    }
    if (n - t0 <= 128) break;
  }
}

// 576 threads leave 96 registers each.  The epilogues of kLse and kDs hold 64
// logits and 8 part values and spill (kLse 232 bytes, with a bias 196; kDs 92 and
// 268; kDh 76, kDw 24), which is part of what bounds narrow heads, where an
// epilogue is longer than a tile's products.
template <Kind kKind, bool kBias>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
gemm_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
            const __grid_constant__ CUtensorMap tmap_out, const Args a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int b_tile = a.bn * kBK;                         // bytes: half of the columns, 2 bytes each
  const int stage_bytes = kATile + b_tile;
  uint8_t* out = smem + a.n_stages * stage_bytes;
  uint8_t* tail = out + out_bytes(kKind);
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(tail);               // used in the even CTA
  uint64_t* empty_bar = full_bar + kMaxStages;                          // both CTAs
  uint64_t* tfull_bar = empty_bar + kMaxStages;                         // both CTAs
  uint64_t* tempty_bar = tfull_bar + 2;                                 // used in the even CTA
  uint64_t* drain_bar = tempty_bar + 2;
  uint32_t* tmem_base_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_base_slot + 1);
  float* epi = reinterpret_cast<float*>(tail + kBarBytes);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();               // 0: issues the MMAs
  const int pair = blockIdx.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < a.n_stages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull_bar[i], 1);
      mbar_init(&tempty_bar[i], 2 * kEpiWarps);          // one arrival per epilogue warp of both CTAs
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
    tmem_alloc_pair(tmem_base_slot, 2 * kMaxN);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                                        // both CTAs' barriers exist before any cross-CTA signal
  tc_fence_after();
  const uint32_t tmem_base = *tmem_base_slot;

  if (warp == kProducerWarp) {
    // -------------------------------------------------------------- TMA producer (both CTAs)
    // As the MMA warp's, its loop is run by the whole warp: with one lane
    // running them, the two loops took 500 clocks for a k block, as long as a
    // tile of 256 columns multiplies and twice as long as one of 128.
    pdl_wait();
    const uint32_t elected = elect_one();
    const uint64_t pol_a = policy_of(a.keep_a), pol_b = policy_of(a.keep_b);
    const uint32_t full0 = smem_u32(full_bar), empty0 = smem_u32(empty_bar);
    const uint32_t leader0 = mapa_shared(full0, 0);
    const uint32_t smem0 = smem_u32(smem);
    int stage = 0;
    uint32_t phase = 0;
    int64_t n_issued = 0;
    bool ok = true;
    for (Units<kKind> u(a, pair); ok && u.more(); u.next()) {
      const int m0 = u.mt() * kTileM + static_cast<int>(rank) * 128;
      const int n0 = u.nt() * a.bn + static_cast<int>(rank) * (a.bn / 2);
      const int k1 = u.k1();
      if constexpr (kKind == kDw) {
        // The next tile's ds into L2 while this one is multiplied: the column
        // tiles that share it take a k block each in turn.
        if (a.prefetch) {
          Units<kKind> next = u;
          next.next();
          if (next.more() && elected) {
            const int m = next.mt() * kTileM + static_cast<int>(rank) * 128;
            for (int kb = next.nt(); kb < a.n_kb; kb += a.n_nt) {
              tma_prefetch_2d(&tmap_a, m, kb * kBK);
              tma_prefetch_2d(&tmap_a, m + 64, kb * kBK);
            }
          }
          __syncwarp();
        }
      }
      for (int kb = u.k0(); kb < k1; ++kb) {
        ok = mbar_wait_warp(empty0 + stage * 8, phase ^ 1, a.err, abort_flag);
        if (!ok) break;
        const uint32_t full = leader0 + stage * 8;
        const uint32_t dst = smem0 + stage * stage_bytes;
        if (rank == 0) mbar_arrive_expect_tx_if(elected, full0 + stage * 8, 2 * stage_bytes);
        if constexpr (a_mn_major(kKind)) {
          tma_load_2d_pair_if(elected, dst, &tmap_a, full, m0, kb * kBK, pol_a);
          tma_load_2d_pair_if(elected, dst + kATile / 2, &tmap_a, full, m0 + 64, kb * kBK, pol_a);
        } else {
          tma_load_2d_pair_if(elected, dst, &tmap_a, full, kb * kBK, m0, pol_a);
        }
        if constexpr (b_mn_major(kKind)) {
          tma_load_2d_pair_if(elected, dst + kATile, &tmap_b, full, n0, kb * kBK, pol_b);
          if (a.bn == kMaxN)
            tma_load_2d_pair_if(elected, dst + kATile + kATile / 2, &tmap_b, full, n0 + 64, kb * kBK, pol_b);
        } else {
          tma_load_2d_pair_if(elected, dst + kATile, &tmap_b, full, kb * kBK, n0, pol_b);
        }
        ++n_issued;
        if (++stage == a.n_stages) { stage = 0; phase ^= 1; }
      }
    }
    if (!ok && rank == 0) {                              // leave only after the loads in flight have landed
      volatile int no_abort = 0;
      for (int64_t i = max(static_cast<int64_t>(0), n_issued - a.n_stages); i < n_issued; ++i)
        mbar_wait_warp(full0 + static_cast<uint32_t>(i % a.n_stages) * 8, static_cast<uint32_t>((i / a.n_stages) & 1), a.err,
                       &no_abort);
    }
  } else if (warp == kMmaWarp) {
    // -------------------------------------------------------------- MMA issuer (even CTA only)
    // The whole warp runs the loop and one elected lane issues.  A stage's
    // descriptors are the first stage's plus a multiple of its size.
    if (rank == 0) {
      const uint32_t elected = elect_one();
      const uint32_t idesc = idesc_bf16_f32(kTileM, static_cast<uint32_t>(a.bn)) |
                             (a_mn_major(kKind) ? kIdescMnMajorA : 0u) | (b_mn_major(kKind) ? kIdescMnMajorB : 0u);
      const uint32_t smem0 = smem_u32(smem);
      const uint64_t a_desc0 = a_mn_major(kKind) ? smem_desc_mn128(smem0) : smem_desc_k128(smem0);
      const uint64_t b_desc0 = b_mn_major(kKind) ? smem_desc_mn128(smem0 + kATile) : smem_desc_k128(smem0 + kATile);
      const uint32_t full0 = smem_u32(full_bar), empty0 = smem_u32(empty_bar);
      const uint32_t stage_step = static_cast<uint32_t>(stage_bytes) >> 4;
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int use = 0;                                       // accumulators taken so far, in turn
      for (Units<kKind> u(a, pair); ok && u.more(); u.next()) {
        const int k1 = u.k1();
        for (int kb0 = u.k0(), n_kb; ok && kb0 < k1; kb0 += n_kb, ++use) {
          n_kb = min(a.sub, k1 - kb0);
          const int acc = use & 1;
          ok = mbar_wait_warp(smem_u32(&tempty_bar[acc]), ((use >> 1) & 1) ^ 1, a.err, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + acc * kMaxN;
          for (int kb = 0; kb < n_kb; ++kb) {
            ok = mbar_wait_warp(full0 + stage * 8, phase, a.err, abort_flag);
            if (!ok) break;
            tc_fence_after();
            const uint64_t a_desc = a_desc0 + stage * stage_step;
            const uint64_t b_desc = b_desc0 + stage * stage_step;
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k)
              mma_bf16_pair_if(elected, d_tmem, a_desc + k * (a_mn_major(kKind) ? 128 : 2),
                               b_desc + k * (b_mn_major(kKind) ? 128 : 2), idesc, kb > 0 || k > 0);
            mma_commit_pair_multicast_if(elected, empty0 + stage * 8, kPairMask);   // frees the stage in both CTAs
            if (++stage == a.n_stages) { stage = 0; phase ^= 1; }
          }
          if (ok) mma_commit_pair_multicast_if(elected, smem_u32(&tfull_bar[acc]), kPairMask);
        }
      }
      if (!ok) {
        mma_commit_pair_multicast_if(elected, smem_u32(drain_bar), 0x1);
        volatile int no_abort = 0;
        mbar_wait_warp(smem_u32(drain_bar), 0, a.err, &no_abort);
      }
    }
  } else {
    // -------------------------------------------------------------- epilogue (both CTAs)
    const int quad = warp & 3;
    const int part = warp >> 2;
    const int part_cols = kKind == kDw ? kBoxCols : kKind == kDh ? (a.bn / kParts + 15) / 16 * 16 : (a.bn / kParts + 7) / 8 * 8;
    const int col0 = part * part_cols;
    const int cols = max(0, min(part_cols, a.bn - col0));
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + col0;
    pdl_wait();
    auto release = [&](int acc) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&tempty_bar[acc]), 0));
    };
    if constexpr (kKind == kLse || kKind == kDs) {
      // per warp: 1/T of its columns, and for kDs their lse and coefficients
      float* inv_t = epi + warp * epi_arrays(kKind) * kPartCols;
      float* second = inv_t + kPartCols;
      float* third = inv_t + 2 * kPartCols;
      constexpr int kGroups = kPartCols / 16;
      LsePart part[kGroups];                                     // of columns 16 k + lane / 2
#pragma unroll
      for (int k = 0; k < kGroups; ++k) part[k] = LsePart{kLowest, 0.0f};
      int id[2] = {-1, -1};                                      // tokens of columns lane and 32 + lane, as rows of A
      int nt = -1, use = 0;
      bool ok = cols > 0;
      for (Units<kKind> u(a, pair); u.more();) {
        const int mt = u.mt();
        const int64_t t_first = static_cast<int64_t>(u.nt()) * a.bn + col0;
        const int n_cols = static_cast<int>(min(static_cast<int64_t>(cols), a.N - t_first));   // that are tokens
        const int64_t m_warp = static_cast<int64_t>(mt) * kTileM + rank * 128 + quad * 32;
        const int64_t m = m_warp + lane;
        const bool row_ok = m < a.M;
        if (u.nt() != nt) {                                      // other tokens than before
          nt = u.nt();
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int c = k * 32 + lane;
            const int64_t t = t_first + c;
            const bool real = c < n_cols;
            inv_t[c] = real ? row_temp(a.p.temp[t]).inv_t : 0.0f;
            const int64_t own = real ? a.p.ids[t] - a.v0 : -1;
            id[k] = own >= 0 && own < a.M ? static_cast<int>(own) : -1;
            if constexpr (kKind == kDs) {
              second[c] = real ? a.lse[t] : 0.0f;
              third[c] = real ? a.coef[t] : 0.0f;
            }
          }
          __syncwarp();
        }
        // the logits start from the bias, whose loads then overlap the products
        float x[kPartCols];
#pragma unroll
        for (int c = 0; c < kPartCols; ++c) x[c] = 0.0f;
        if constexpr (kBias) {
          if (row_ok) {
            const float* b = a.p.bias + a.v0 + m;
            if (a.p.bias_stride == 0) {
              const float shared = __ldg(b);
#pragma unroll
              for (int c = 0; c < kPartCols; ++c) x[c] = shared;
            } else {
              b += t_first * a.p.bias_stride;
#pragma unroll
              for (int c = 0; c < kPartCols; ++c, b += a.p.bias_stride)
                if (c < n_cols) x[c] = __ldg(b);
            }
          }
        }
        for (int kb0 = 0; kb0 < a.n_kb; kb0 += a.sub, ++use) {
          const int acc = use & 1;
          if (!mbar_wait(&tfull_bar[acc], (use >> 1) & 1, a.err, abort_flag)) { ok = false; break; }
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < kPartCols; c += 8) {
            if (c >= cols) break;
            uint32_t r[8];
            tmem_ld_8(lane_addr + acc * kMaxN + c, r);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 8; ++j) x[c + j] += __uint_as_float(r[j]);
          }
          release(acc);
        }
        u.next();
        if (!ok) {                                               // a wait gave up, or this warp has no columns
          if (cols > 0) break;
          continue;
        }
#pragma unroll
        for (int c = 0; c < kPartCols; c += 4) {
          const float4 f = *reinterpret_cast<const float4*>(inv_t + c);
          x[c + 0] *= f.x;
          x[c + 1] *= f.y;
          x[c + 2] *= f.z;
          x[c + 3] *= f.w;
        }
        if (m_warp + 32 > a.M && !row_ok) {                      // a ragged last tile
#pragma unroll
          for (int c = 0; c < kPartCols; ++c) x[c] = -INFINITY;
        }
        if constexpr (kKind == kLse) {
          if (a.kept != nullptr && row_ok) {
            float* dst = a.kept + t_first * a.kept_pitch + m;
#pragma unroll
            for (int c = 0; c < kPartCols; ++c, dst += a.kept_pitch)
              if (c < n_cols) __stcs(dst, x[c]);
          }
          // of each column the largest x, then the sum of exp(x - largest)
#pragma unroll
          for (int k = 0; k < kGroups; ++k) {
            if (k * 16 >= n_cols) break;
            float mine = kLowest;                                // the largest x of this lane's column
            const float sum = join_columns(lane, [](float p, float q) { return p + q; }, [&](int c) {
              const float top = fmaxf(warp_max(x[k * 16 + c]), kLowest);
              if (lane >> 1 == c) mine = top;
              return __expf(x[k * 16 + c] - top);
            });
            part[k] = lse_join(part[k], LsePart{mine, sum});
          }
        } else if (row_ok) {
          __nv_bfloat16* dst = a.ds + t_first * a.ds_pitch + m;
#pragma unroll
          for (int c = 0; c < kPartCols; c += 4) {
            const float4 z = *reinterpret_cast<const float4*>(second + c);
            const float4 f = *reinterpret_cast<const float4*>(third + c);
            if (c + 0 < n_cols) dst[0] = ds_of(x[c + 0], z.x, f.x);
            if (c + 1 < n_cols) dst[a.ds_pitch] = ds_of(x[c + 1], z.y, f.y);
            if (c + 2 < n_cols) dst[2 * a.ds_pitch] = ds_of(x[c + 2], z.z, f.z);
            if (c + 3 < n_cols) dst[3 * a.ds_pitch] = ds_of(x[c + 3], z.w, f.w);
            dst += 4 * a.ds_pitch;
          }
        }
        // a token's own logit lies in few tiles: looked for by ballots
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t hits = __ballot_sync(0xffffffffu, static_cast<unsigned>(id[k] - static_cast<int>(m_warp)) < 32u);
          while (hits != 0) {
            const int c = k * 32 + __ffs(hits) - 1;
            hits &= hits - 1;
            const int own = __shfl_sync(0xffffffffu, id[k], c & 31) - static_cast<int>(m_warp);
            float mine = 0.0f;
            if constexpr (kKind == kLse) {
#pragma unroll
              for (int j = k * 32; j < k * 32 + 32; ++j) mine = j == c ? x[j] : mine;
            }
            if (lane == own) {
              if constexpr (kKind == kLse) {
                a.own_x[t_first + c] = mine;
              } else if (third[c] != 0.0f) {
                a.ds[(t_first + c) * a.ds_pitch + m] =
                    own_ds_of(a.logp[t_first + c], third[c], a.rest[t_first + c]);
              }
            }
          }
        }
        if constexpr (kKind == kLse) {
          // with one column tile the pair's tiles share a part, else each has its own
          if (a.n_nt > 1 || !u.more()) {
            const int64_t which = static_cast<int64_t>(a.n_nt > 1 ? mt : pair) * 8 + rank * 4 + quad;
#pragma unroll
            for (int k = 0; k < kGroups; ++k) {
              const int c = k * 16 + (lane >> 1);
              if (c < n_cols && (lane & 1) == 0) a.parts[which * a.N + t_first + c] = part[k];
              part[k] = LsePart{kLowest, 0.0f};
            }
          }
        }
      }
    } else {
      int use = 0;
      for (Units<kKind> u(a, pair); u.more(); u.next(), ++use) {
        const int acc = use & 1;
        const int m_warp = u.mt() * kTileM + static_cast<int>(rank) * 128 + quad * 32;
        // kDw: the tokens whose own rows these are, looked for while the tile
        // is still being multiplied; the first two are kept
        int hits = 0, hit_t[2] = {0, 0}, hit_row[2] = {-1, -1};
        if constexpr (kKind == kDw) {
          if (cols > 0) {
            each_own(a, m_warp, [&](int t, int row) {
              if (hits == 0) { hit_t[0] = t; hit_row[0] = row; }
              if (hits == 1) { hit_t[1] = t; hit_row[1] = row; }
              ++hits;
            });
          }
        }
        if (!mbar_wait(&tfull_bar[acc], (use >> 1) & 1, a.err, abort_flag)) break;
        tc_fence_after();
        const int64_t n_first = static_cast<int64_t>(u.nt()) * a.bn + col0;
        if constexpr (kKind == kDh) {
          const int64_t m = m_warp + lane;
          const bool row_ok = m < a.M;
#pragma unroll 1
          for (int c = 0; c < cols; c += 16) {
            uint32_t r[16];
            tmem_ld_16(lane_addr + acc * kMaxN + c, r);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int64_t n = n_first + c + j;
              if (n >= a.N || !row_ok) continue;
              const float y = __uint_as_float(r[j]);
              float* at = a.partials + (static_cast<int64_t>(u.split()) * a.N + n) * a.M + m;
              *at = a.add ? *at + y : y;
            }
          }
          release(acc);
        } else {
          // 32 rows x 64 columns, and what the rounding of the tokens' own
          // entries left over for these rows
          float x[kBoxCols];
#pragma unroll
          for (int c = 0; c < kBoxCols; c += 16) {
            if (c >= cols) break;
            uint32_t r[16];
            tmem_ld_16(lane_addr + acc * kMaxN + c, r);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) x[c + j] = __uint_as_float(r[j]);
          }
          release(acc);
          auto add_rest = [&](int t, int row) {
            if (row != lane) return;
            const float rest = a.rest[t];
            const uint4* h = reinterpret_cast<const uint4*>(a.h + t * a.N + n_first);
#pragma unroll
            for (int q = 0; q < kBoxCols / 8; ++q) {
              if (n_first + q * 8 >= a.N) break;
              const uint4 v = __ldg(h + q);
              const __nv_bfloat162* two = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 f = __bfloat1622float2(two[j]);
                x[q * 8 + 2 * j] = fmaf(rest, f.x, x[q * 8 + 2 * j]);
                x[q * 8 + 2 * j + 1] = fmaf(rest, f.y, x[q * 8 + 2 * j + 1]);
              }
            }
          };
          if (hits <= 2) {
            if (hits > 0) add_rest(hit_t[0], hit_row[0]);
            if (hits > 1) add_rest(hit_t[1], hit_row[1]);
          } else {
            each_own(a, m_warp, add_rest);
          }
          __syncwarp();
          // to the warp's box, its 16-byte pieces swizzled as the tensor map
          // says (no bank conflicts), then out by TMA
          uint8_t* box = out + warp * kBoxBytes;
          if (lane == 0) bulk_wait_read();                // the box's last store has been read
          __syncwarp();
#pragma unroll
          for (int q = 0; q < kBoxCols / 8; ++q) {
            uint4 v;
            uint32_t* w = &v.x;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const __nv_bfloat162 two = __floats2bfloat162_rn(x[q * 8 + 2 * j], x[q * 8 + 2 * j + 1]);
              w[j] = *reinterpret_cast<const uint32_t*>(&two);
            }
            *reinterpret_cast<uint4*>(box + lane * 128 + ((q ^ (lane & 7)) * 16)) = v;
          }
          fence_async_shared();
          __syncwarp();
          if (lane == 0 && cols > 0 && m_warp < a.M && n_first < a.N) {
            tma_store_2d(&tmap_out, box, static_cast<int32_t>(n_first), m_warp);
            bulk_commit();
          }
        }
      }
      if constexpr (kKind == kDw) {
        if (lane == 0) bulk_wait();
      }
    }
  }

  // The next kernel may start now, not earlier: its blocks, waiting beside this
  // one's, made this kernel 5% slower.
  pdl_launch_dependents();
  // ---- teardown: neither CTA leaves (or frees TMEM) while the pair's MMAs or
  // the peer's signals may still touch it
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc_pair(tmem_base, 2 * kMaxN);
}

}  // namespace head
}  // namespace fs
