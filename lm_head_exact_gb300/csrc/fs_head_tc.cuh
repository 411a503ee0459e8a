// Tensor-core engine of the training operators of the LM head: one persistent,
// warp-specialized kernel over pairs of CTAs (tcgen05 cta_group::2) for the
// four products
//
//   kLse  x^T  = W h^T          each tile reduced to its columns' sums of exp
//   kDs   ds^T from x^T         the same product, written as bf16 ds
//   kDh   grad_h^T = W^T ds^T   split along the vocabulary, fp32 partials
//   kDw   grad_W^T = h^T ds
//
// All are formed TRANSPOSED: the axis that is contiguous in memory (vocabulary
// ids of x and ds, the model width of the gradients) lies on the MMA's M axis,
// that is on the 32 lanes of a warp, so the epilogues load and store whole
// lines; and the tokens lie on N, whose size is any multiple of 16, so a batch
// of 517 tokens runs as 3 x 176 columns instead of 3 x 256 rows.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "fs_sm100.cuh"
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
constexpr int epi_bytes(Kind k) {
  return k == kLse ? (kMaxN + kEpiWarps * kPartCols) * 4 : k == kDs ? 3 * kMaxN * 4 : 0;
}
constexpr int kSmemLimit = 232448;

struct Args {
  HeadProblem p;
  int64_t M, N;              // extents of this launch's product
  int bn;                    // columns of a tile (a multiple of 16, <= 256)
  int n_stages;
  int n_nt;                  // column tiles
  int n_mt;                  // row tiles
  int n_kb;                  // k blocks of the whole product
  int splits;                // kDh
  int n_pairs;               // pairs of the grid
  int64_t t0, t_end;         // kLse / kDs: the tokens of this launch
  // kLse
  LsePart* parts;            // [n, n_parts]
  int64_t n_parts;
  float* own_x;              // [n]
  float* kept;               // nullable [n, kept_pitch]
  int64_t kept_pitch;
  // kDs
  const float* lse;
  const float* coef;
  __nv_bfloat16* ds;
  int64_t ds_pitch;
  int64_t v0;                // first vocabulary row of the chunk
  // kDh
  float* partials;
  bool add;
  // kDw
  __nv_bfloat16* grad_W;
  int* err;
};

// The tiles of one pair, in order.  kLse and kDs: a fixed column tile and
// every n_pairs / n_nt-th row tile, so that the pairs that share W rows run
// side by side and W comes from HBM once.  kDh: one split after another, so
// that all pairs work on the same vocabulary rows at a time.  kDw: the row
// tiles (the model width) of one column tile after another.
struct Unit {
  int mt, nt, k0, k1, split;
};

template <Kind kKind>
__device__ __forceinline__ bool unit_at(const Args& a, int pair, int i, Unit& u) {
  u.k0 = 0;
  u.k1 = a.n_kb;
  u.split = 0;
  if constexpr (kKind == kLse || kKind == kDs) {
    const int groups = a.n_pairs / a.n_nt;
    u.nt = pair % a.n_nt;
    u.mt = pair / a.n_nt + i * groups;
    return u.mt < a.n_mt;
  } else {
    const int64_t tiles = static_cast<int64_t>(a.n_mt) * a.n_nt;
    const int64_t at = pair + static_cast<int64_t>(i) * a.n_pairs;
    if (at >= tiles * a.splits) return false;
    u.split = static_cast<int>(at / tiles);
    const int64_t tile = at % tiles;
    u.mt = static_cast<int>(tile % a.n_mt);
    u.nt = static_cast<int>(tile / a.n_mt);
    if constexpr (kKind == kDh) {
      u.k0 = static_cast<int>(static_cast<int64_t>(a.n_kb) * u.split / a.splits);
      u.k1 = static_cast<int>(static_cast<int64_t>(a.n_kb) * (u.split + 1) / a.splits);
    }
    return true;
  }
}

// ---------------------------------------------------------------- kLse epilogue
// Each thread holds one vocabulary row of the tile and sums exp(x - ref) of
// its rows for each of its part's columns (tokens) in a register, over all
// tiles of the pair; lanes are added once, at the end.  ref, one per (warp,
// column), is the warp's largest x of the first tile that had any, and moves
// only when an x exceeds it by kSlack: the sums then stay within fp32's range
// (2^24 terms of e^20 at most) and a term is lost only where the term at ref
// outweighs it by far more than fp32 resolves.  So the common case is one
// fused multiply-add, one comparison, one exponential and one addition per
// logit, without a running maximum.
constexpr float kSlack = 20.0f;
constexpr float kUnset = -3.402823466e38f;   // the lowest finite value: an x of that value (a mask) counts as it should

struct LseState {
  float s[kPartCols];
};

// x of column c + j before the scaling.
template <bool kBias>
__device__ __forceinline__ float biased(const Args& a, uint32_t acc, int64_t t, int64_t v, bool row_ok) {
  float x = __uint_as_float(acc);
  if constexpr (kBias) {
    if (row_ok && t < a.t_end) x += __ldg(a.p.bias + t * a.p.bias_stride + v);
  }
  return x;
}

template <bool kBias>
__device__ __forceinline__ void lse_tile(const Args& a, LseState& st, const float* inv_t, float* ref, uint32_t taddr,
                                         int cols, int64_t t_first, int64_t v) {
  const bool row_ok = v < a.p.V;
#pragma unroll
  for (int c = 0; c < kPartCols; c += 8) {
    if (c >= cols) break;
    float d[8];
    float over = -INFINITY;
    {
      uint32_t r[8];
      tmem_ld_8(taddr + c, r);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t t = t_first + c + j;
        const float x = biased<kBias>(a, r[j], t, v, row_ok);
        if (a.kept != nullptr && row_ok && t < a.t_end) a.kept[t * a.kept_pitch + v] = x * inv_t[c + j];
        d[j] = row_ok ? fmaf(x, inv_t[c + j], -ref[c + j]) : -INFINITY;
        over = fmaxf(over, d[j]);
      }
    }
    if (__any_sync(0xffffffffu, over > kSlack)) {       // seldom: some ref moves
      uint32_t r[8];
      tmem_ld_8(taddr + c, r);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (!__any_sync(0xffffffffu, d[j] > kSlack)) continue;
        const float old = ref[c + j];
        const float x = row_ok ? biased<kBias>(a, r[j], t_first + c + j, v, row_ok) * inv_t[c + j] : -INFINITY;
        float top = x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        top = fminf(top, 3.402823466e38f);
        st.s[c + j] *= __expf(old - top);               // 0 from an unset ref
        d[j] = x - top;
        __syncwarp();
        if ((threadIdx.x & 31) == 0) ref[c + j] = top;
      }
      __syncwarp();
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) st.s[c + j] += __expf(d[j]);
  }
}

template <Kind kKind, bool kBias>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
gemm_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b, const Args a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int b_tile = a.bn * kBK;                         // bytes: half of the columns, 2 bytes each
  const int stage_bytes = kATile + b_tile;
  uint8_t* tail = smem + a.n_stages * stage_bytes;
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
  pdl_launch_dependents();
  const uint32_t tmem_base = *tmem_base_slot;

  if (warp == kProducerWarp) {
    // -------------------------------------------------------------- TMA producer (both CTAs)
    if (lane == 0) {
      pdl_wait();
      const uint64_t pol_a = kKind == kDw ? policy_evict_last() : policy_evict_first();
      const uint64_t pol_b = kKind == kDw ? policy_evict_first() : policy_evict_last();
      int stage = 0;
      uint32_t phase = 0;
      int64_t n_issued = 0;
      bool ok = true;
      Unit u;
      for (int i = 0; ok && unit_at<kKind>(a, pair, i, u); ++i) {
        const int m0 = u.mt * kTileM + static_cast<int>(rank) * 128;
        const int n0 = u.nt * a.bn + static_cast<int>(rank) * (a.bn / 2);
        for (int kb = u.k0; kb < u.k1; ++kb) {
          if (!mbar_wait(&empty_bar[stage], phase ^ 1, a.err, abort_flag)) { ok = false; break; }
          const uint32_t full = mapa_shared(smem_u32(&full_bar[stage]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&full_bar[stage], 2 * stage_bytes);
          uint8_t* dst = smem + stage * stage_bytes;
          if constexpr (a_mn_major(kKind)) {
            tma_load_2d_pair(dst, &tmap_a, full, m0, kb * kBK, pol_a);
            tma_load_2d_pair(dst + kATile / 2, &tmap_a, full, m0 + 64, kb * kBK, pol_a);
          } else {
            tma_load_2d_pair(dst, &tmap_a, full, kb * kBK, m0, pol_a);
          }
          if constexpr (b_mn_major(kKind)) {
            tma_load_2d_pair(dst + kATile, &tmap_b, full, n0, kb * kBK, pol_b);
            tma_load_2d_pair(dst + kATile + kATile / 2, &tmap_b, full, n0 + 64, kb * kBK, pol_b);
          } else {
            tma_load_2d_pair(dst + kATile, &tmap_b, full, kb * kBK, n0, pol_b);
          }
          ++n_issued;
          if (++stage == a.n_stages) { stage = 0; phase ^= 1; }
        }
      }
      if (!ok && rank == 0) {                            // leave only after the loads in flight have landed
        volatile int no_abort = 0;
        for (int64_t i = max(static_cast<int64_t>(0), n_issued - a.n_stages); i < n_issued; ++i)
          mbar_wait(&full_bar[i % a.n_stages], static_cast<uint32_t>((i / a.n_stages) & 1), a.err, &no_abort);
      }
    }
  } else if (warp == kMmaWarp) {
    // -------------------------------------------------------------- MMA issuer (even CTA only)
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = idesc_bf16_f32(kTileM, static_cast<uint32_t>(a.bn)) |
                             (a_mn_major(kKind) ? kIdescMnMajorA : 0u) | (b_mn_major(kKind) ? kIdescMnMajorB : 0u);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      Unit u;
      for (int i = 0; ok && unit_at<kKind>(a, pair, i, u); ++i) {
        const int acc = i & 1;
        if (!mbar_wait(&tempty_bar[acc], ((i >> 1) & 1) ^ 1, a.err, abort_flag)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * kMaxN;
        for (int kb = u.k0; kb < u.k1; ++kb) {
          if (!mbar_wait(&full_bar[stage], phase, a.err, abort_flag)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(smem + stage * stage_bytes);
          const uint32_t b_addr = a_addr + kATile;
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k)
            mma_bf16_pair(d_tmem,
                          a_mn_major(kKind) ? smem_desc_mn128(a_addr + k * 2048) : smem_desc_k128(a_addr + k * 32),
                          b_mn_major(kKind) ? smem_desc_mn128(b_addr + k * 2048) : smem_desc_k128(b_addr + k * 32),
                          idesc, kb > u.k0 || k > 0);
          mma_commit_pair_multicast(&empty_bar[stage], kPairMask);       // frees the stage in both CTAs
          if (++stage == a.n_stages) { stage = 0; phase ^= 1; }
        }
        if (ok) mma_commit_pair_multicast(&tfull_bar[acc], kPairMask);
      }
      if (!ok) {
        mma_commit_pair_multicast(drain_bar, 0x1);
        volatile int no_abort = 0;
        mbar_wait(drain_bar, 0, a.err, &no_abort);
      }
    }
  } else {
    // -------------------------------------------------------------- epilogue (both CTAs)
    const int quad = warp & 3;
    const int part = warp >> 2;
    const int part_cols = (a.bn / kParts + 15) / 16 * 16;  // columns of a part, whole loads of 16
    const int col0 = part * part_cols;
    const int cols = max(0, min(part_cols, a.bn - col0));
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + col0;
    pdl_wait();
    // kLse / kDs: the columns' constants, the same for all tiles of the pair
    const int64_t tile_t = a.t0 + static_cast<int64_t>(pair % a.n_nt) * a.bn;
    const int64_t t_first = tile_t + col0;
    float* ref = epi + kMaxN + warp * kPartCols;
    int64_t id[2] = {-1, -1};
    LseState st;
    if constexpr (kKind == kLse || kKind == kDs) {
      for (int c = threadIdx.x; c < a.bn; c += kEpiWarps * 32) {
        const int64_t t = tile_t + c;
        epi[c] = t < a.t_end ? row_temp(a.p.temp[t]).inv_t : 0.0f;
        if constexpr (kKind == kDs) {
          epi[kMaxN + c] = t < a.t_end ? a.lse[t] : 0.0f;
          epi[2 * kMaxN + c] = t < a.t_end ? a.coef[t] : 0.0f;
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int c = k * 32 + lane;
        if (c < cols && t_first + c < a.t_end) id[k] = a.p.ids[t_first + c];
        if constexpr (kKind == kDs) {
          if (id[k] >= 0) id[k] -= a.v0;
        }
      }
      if constexpr (kKind == kLse) {
#pragma unroll
        for (int c = 0; c < kPartCols; ++c) st.s[c] = 0.0f;
        for (int c = lane; c < kPartCols; c += 32) ref[c] = kUnset;
      }
      asm volatile("bar.sync 1, %0;" ::"n"(kEpiWarps * 32) : "memory");
    }
    Unit u;
    for (int i = 0; unit_at<kKind>(a, pair, i, u); ++i) {
      const int acc = i & 1;
      if (!mbar_wait(&tfull_bar[acc], (i >> 1) & 1, a.err, abort_flag)) break;
      tc_fence_after();
      const uint32_t taddr = lane_addr + acc * kMaxN;
      const int64_t m_warp = static_cast<int64_t>(u.mt) * kTileM + rank * 128 + quad * 32;
      const int64_t m = m_warp + lane;
      if constexpr (kKind == kLse || kKind == kDs) {
        if constexpr (kKind == kLse) {
          lse_tile<kBias>(a, st, epi + col0, ref, taddr, cols, t_first, m);
        } else {
          const bool row_ok = m < a.M;
#pragma unroll 1
          for (int c = 0; c < cols; c += 16) {
            uint32_t r[16];
            tmem_ld_16(taddr + c, r);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int64_t t = t_first + c + j;
              if (t >= a.t_end) break;
              float x = __uint_as_float(r[j]);
              if constexpr (kBias) {
                if (row_ok) x += __ldg(a.p.bias + t * a.p.bias_stride + a.v0 + m);
              }
              const int col = col0 + c + j;
              const float coef = epi[2 * kMaxN + col];
              const float p = __expf(fmaf(x, epi[col], -epi[kMaxN + col]));
              if (row_ok) a.ds[t * a.ds_pitch + m] = __float2bfloat16_rn(coef == 0.0f ? 0.0f : -coef * p);
            }
          }
        }
        // a token's own logit: in few tiles, so looked for by ballots
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t hits = __ballot_sync(0xffffffffu, id[k] >= m_warp && id[k] < m_warp + 32 && id[k] < a.M);
          while (hits != 0) {
            const int c = __ffs(hits) - 1;
            hits &= hits - 1;
            const int own = static_cast<int>(__shfl_sync(0xffffffffu, id[k], c) - m_warp);
            float x = __uint_as_float(tmem_ld_1(taddr + k * 32 + c));
            tmem_ld_wait();
            const int64_t t = t_first + k * 32 + c;
            const int col = col0 + k * 32 + c;
            if (lane == own) {
              if constexpr (kBias) x += __ldg(a.p.bias + t * a.p.bias_stride + a.v0 + m);
              if constexpr (kKind == kLse) {
                a.own_x[t] = x * epi[col];
              } else {
                const float coef = epi[2 * kMaxN + col];
                const float p = __expf(fmaf(x, epi[col], -epi[kMaxN + col]));
                if (coef != 0.0f) a.ds[t * a.ds_pitch + m] = __float2bfloat16_rn(coef * (1.0f - p));
              }
            }
          }
        }
      } else {
        const int64_t n_first = static_cast<int64_t>(u.nt) * a.bn + col0;
        const bool row_ok = m < a.M;
#pragma unroll 1
        for (int c = 0; c < cols; c += 16) {
          uint32_t r[16];
          tmem_ld_16(taddr + c, r);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int64_t n = n_first + c + j;
            if (n >= a.N || !row_ok) continue;
            const float y = __uint_as_float(r[j]);
            if constexpr (kKind == kDh) {
              float* at = a.partials + (static_cast<int64_t>(u.split) * a.N + n) * a.M + m;
              *at = a.add ? *at + y : y;
            } else {
              a.grad_W[(a.v0 + n) * a.M + m] = __float2bfloat16_rn(y);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&tempty_bar[acc]), 0));
    }
    if constexpr (kKind == kLse) {
      // the warp's lanes added: one part per (column, pair group, CTA, quarter)
      const int64_t which = static_cast<int64_t>(pair / a.n_nt) * 8 + rank * 4 + quad;
#pragma unroll
      for (int c = 0; c < kPartCols; ++c) {
        if (c >= cols) break;
        float s = st.s[c];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        const int64_t t = t_first + c;
        if (lane == (c & 31) && t < a.t_end) a.parts[t * a.n_parts + which] = LsePart{ref[c], s};
      }
    }
  }

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
