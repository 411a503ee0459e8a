// Token log-probabilities through the LM head and their gradients.
//
//   x = (h W^T + bias) / T,  lse = log sum exp x,  logp = x[id] - lse
//   ds = c (1[v = id] - exp(x - lse)),  c = g / T;  grad_h = ds W,  grad_W = ds^T h
//
// Forward: every tile of x is reduced on chip to one (max, sum of exp) per
// row; the parts are merged by a second, small launch.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "fs_head_tc.cuh"
#include "fs_train.h"

namespace fs {
namespace {

using head::lse_join;

// Merge of the parts [n_parts, n] of kMergeRows tokens a block.  Every thread
// joins every (kThreads / 4)th part of one token, 8 loads in flight and one
// rescaling for each 8 (one at a time took three times as long: the loads
// waited for the exponentials); then the block's threads are joined.  Blocks of
// 1024 threads where there are few, of 256 where there are enough (10 and 7 us
// for 528 tokens of 128256 words, 20 and 28 for 2048).
constexpr int kMergeRows = 4;

template <int kThreads>
__global__ void __launch_bounds__(kThreads) head_merge_kernel(const HeadProblem p, const LsePart* parts,
                                                              int64_t n_parts, const float* own_x, float* logp,
                                                              float* lse) {
  __shared__ LsePart warps[32][kMergeRows];
  constexpr int kSlices = kThreads / kMergeRows;
  const int row = threadIdx.x & (kMergeRows - 1);
  int64_t t = static_cast<int64_t>(blockIdx.x) * kMergeRows + row;
  pdl_launch_dependents();
  pdl_wait();
  LsePart part{head::kLowest, 0.0f};
  if (t < p.n) {
    for (int64_t i = threadIdx.x / kMergeRows; i < n_parts; i += 8 * kSlices) {
      LsePart v[8];
      float m = part.m;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[k] = LsePart{head::kLowest, 0.0f};
        if (i + k * kSlices < n_parts) v[k] = parts[(i + k * kSlices) * p.n + t];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) m = fmaxf(m, v[k].m);
      part.s *= __expf(part.m - m);
      part.m = m;
#pragma unroll
      for (int k = 0; k < 8; ++k) part.s += v[k].s * __expf(v[k].m - m);
    }
  }
#pragma unroll
  for (int o = 16; o >= kMergeRows; o >>= 1)
    part = lse_join(part, LsePart{__shfl_xor_sync(0xffffffffu, part.m, o), __shfl_xor_sync(0xffffffffu, part.s, o)});
  if ((threadIdx.x & 31) < kMergeRows) warps[threadIdx.x >> 5][row] = part;
  __syncthreads();
  // a warp for each token
  const int lane = threadIdx.x & 31;
  t = static_cast<int64_t>(blockIdx.x) * kMergeRows + (threadIdx.x >> 5);
  if (threadIdx.x >= 32 * kMergeRows || t >= p.n) return;
  part = lane < kThreads / 32 ? warps[lane][threadIdx.x >> 5] : LsePart{head::kLowest, 0.0f};
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    part = lse_join(part, LsePart{__shfl_xor_sync(0xffffffffu, part.m, o), __shfl_xor_sync(0xffffffffu, part.s, o)});
  if (lane != 0) return;
  const bool valid = row_temp(p.temp[t]).mode != kRowInvalid;
  const int64_t id = p.ids[t];
  float z = !valid || part.s == 0.0f ? -INFINITY : part.m + logf(part.s);
  if (valid && !(part.s < INFINITY)) z = NAN;           // a NaN or infinite logit
  lse[t] = z;
  float lp = 0.0f;
  if (valid && id >= 0 && id < p.V) {
    const float x = own_x[t];
    // not x - z: z is rounded to its own size, which for a token that is nearly
    // certain is all that x - z would hold (lse = 200: 8e-6); logf(s) is small
    lp = z != z ? NAN : x == -INFINITY ? -INFINITY : (x - part.m) - logf(part.s);
  }
  logp[t] = lp;
}

// A row's coefficient c = g / T, 0 where it carries no gradient.
__device__ __forceinline__ float row_coef(const HeadRows& r, const HeadProblem& p, int64_t t) {
  const RowTemp rt = row_temp(p.temp[t]);
  const int64_t id = p.ids[t];
  const float g = r.g[t];
  const bool live = rt.mode != kRowInvalid && id >= 0 && id < p.V && g != 0.0f && r.lse[t] != -INFINITY &&
                    r.logp[t] != -INFINITY;
  return live ? g * rt.inv_t : 0.0f;
}

// What the later launches need of a row, written by one block of 256 threads.
// (rest is written with the token's own entry of ds; rows without one have
// own = -1.)
__device__ __forceinline__ void write_row(const HeadRows& r, const HeadProblem& p, int64_t t, float coef) {
  if (threadIdx.x == 0) {
    r.coef[t] = coef;
    r.own[t] = coef != 0.0f ? static_cast<int>(p.ids[t]) : -1;
  }
  if (r.h_live == nullptr) return;
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.h) + t * p.d);
  uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(r.h_live) + t * p.d);
  for (int64_t i = threadIdx.x; i < p.d / 8; i += 256) dst[i] = coef != 0.0f ? src[i] : make_uint4(0, 0, 0, 0);
}

__global__ void __launch_bounds__(256) head_rows_kernel(const HeadProblem p, const HeadRows r) {
  pdl_launch_dependents();
  pdl_wait();
  write_row(r, p, blockIdx.x, row_coef(r, p, blockIdx.x));
}

// ds of vocabulary rows [v0, v0 + vc) from the kept logits: 4 bytes read and 2
// written per element, 8 elements a thread; the first piece's blocks write the
// rows besides.  The pitches are multiples of 64 elements and v0 of 256, so
// every group of 8 is aligned; columns in [vc, pitch) hold what the padding of
// `kept` gives and are never read.
__global__ void __launch_bounds__(256) head_ds_kept_kernel(const HeadProblem p, const HeadRows r, const float* kept,
                                                           int64_t kept_pitch, int64_t v0, __nv_bfloat16* ds,
                                                           int64_t pitch) {
  const int64_t t = blockIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  const float c = row_coef(r, p, t), z = r.lse[t];
  if (v0 == 0 && blockIdx.y == 0) write_row(r, p, t, c);
  const int64_t id = p.ids[t] - v0;
  const float* src = kept + t * kept_pitch + v0;
  __nv_bfloat16* dst = ds + t * pitch;
  const int64_t stride = static_cast<int64_t>(gridDim.y) * 256 * 8;
#pragma unroll 2
  for (int64_t v = (static_cast<int64_t>(blockIdx.y) * 256 + threadIdx.x) * 8; v < pitch; v += stride) {
    __align__(16) __nv_bfloat16 o[8];
    if (c == 0.0f) {
      *reinterpret_cast<uint4*>(o) = make_uint4(0, 0, 0, 0);
    } else {
      const float4 a = __ldcs(reinterpret_cast<const float4*>(src + v));
      const float4 b = __ldcs(reinterpret_cast<const float4*>(src + v + 4));
      const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = head::ds_of(x[j], z, c);
      if (id >= v && id < v + 8) {                       // the token's own entry is one of these
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (v + j == id) o[j] = head::own_ds_of(r.logp[t], c, r.rest[t]);
      }
    }
    *reinterpret_cast<uint4*>(dst + v) = *reinterpret_cast<uint4*>(o);
  }
}

// grad_h: the splits' partials added in their order, then what the rounding of
// the tokens' own entries left over, and rounded once.
__global__ void __launch_bounds__(256) head_dh_sum_kernel(const HeadProblem p, const float* partials, int64_t splits,
                                                          const int* own, const float* rest, __nv_bfloat16* grad_h) {
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;     // d is a multiple of 8
  pdl_launch_dependents();
  pdl_wait();
  if (i >= p.n * p.d) return;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const int64_t t = i / p.d;
  const int id = own[t];
  if (id >= 0) {                                        // else the row carries no gradient
    const uint2 raw = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.W) + id * p.d + (i - t * p.d)));
    const float r = rest[t];
#pragma unroll 4
    for (int64_t k = 0; k < splits; ++k) {
      const float4 x = __ldcs(reinterpret_cast<const float4*>(partials + k * p.n * p.d + i));
      s.x += x.x;
      s.y += x.y;
      s.z += x.z;
      s.w += x.w;
    }
    const float2 lo = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw.x));
    const float2 hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw.y));
    s.x = fmaf(r, lo.x, s.x);
    s.y = fmaf(r, lo.y, s.y);
    s.z = fmaf(r, hi.x, s.z);
    s.w = fmaf(r, hi.y, s.w);
  }
  __align__(8) __nv_bfloat16 o[4] = {__float2bfloat16_rn(s.x), __float2bfloat16_rn(s.y), __float2bfloat16_rn(s.z),
                                     __float2bfloat16_rn(s.w)};
  *reinterpret_cast<uint2*>(grad_h + i) = *reinterpret_cast<uint2*>(o);
}

// ---------------------------------------------------------------- launch geometry
// The products, and the small kernels that follow a small kernel, are launched
// as programmatic dependents: each waits for the one before it
// (griddepcontrol.wait) before it reads or writes global memory, so only its
// start-up overlaps.  The small kernels after a product are launched plainly:
// as dependents they slowed the next product's start down by more than they
// gained (scores of 257 rows, width 520: 37 and 43 us).
using head::Args;
using head::Kind;

constexpr int kBox = 64;                                 // columns of a TMA box: 128 bytes

// Columns of a tile for n tokens: as few tiles as 256 columns allow, all of
// one size.
struct ColumnTiles {
  int bn, count;
};

ColumnTiles column_tiles(int64_t n) {
  ColumnTiles c;
  const int64_t count = std::max<int64_t>(1, (n + head::kMaxN - 1) / head::kMaxN);
  c.bn = static_cast<int>(((n + count - 1) / count + 15) / 16 * 16);
  c.bn = std::max(c.bn, 16);
  c.count = static_cast<int>((n + c.bn - 1) / c.bn);
  return c;
}

int row_tiles(int64_t m) { return static_cast<int>((m + head::kTileM - 1) / head::kTileM); }
int k_blocks(int64_t k) { return static_cast<int>((k + head::kBK - 1) / head::kBK); }

template <Kind kKind>
int stages_for(int bn) {
  return std::min(head::kMaxStages,
                  (head::kSmemLimit - 1024 - head::kBarBytes - head::epi_bytes(kKind) - head::out_bytes(kKind)) /
                      (head::kATile + bn * head::kBK));
}

template <Kind kKind>
int smem_for(int bn) {
  return stages_for<kKind>(bn) * (head::kATile + bn * head::kBK) + head::kBarBytes + head::epi_bytes(kKind) +
         head::out_bytes(kKind) + 1024;
}

// Pairs that can be resident at once: a pair needs two SMs of one cluster
// group, so this can be below SMs / 2.
int resident_pairs() {
  static std::atomic<int> cached[64];                    // zero-initialized (static storage)
  int dev = -1, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 76;                                           // no device: sizes only
  }
  if (dev < 64 && cached[dev].load(std::memory_order_relaxed) > 0) return cached[dev].load(std::memory_order_relaxed);
  constexpr auto kernel = head::gemm_kernel<head::kDw, false>;
  int n = 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * (sms / 2)));
  cfg.blockDim = dim3(head::kThreads);
  cfg.dynamicSmemBytes = smem_for<head::kDw>(head::kMaxN);
  if (raise_smem_limit<kernel>(dev, smem_for<head::kDw>(head::kMaxN)) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    n = sms / 2;
  }
  n = std::max(1, std::min(n, sms / 2));
  if (dev < 64) cached[dev].store(n, std::memory_order_relaxed);
  return n;
}

template <Kind kKind, bool kBias>
cudaError_t launch(const Args& a, const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tout,
                   cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  const int smem = smem_for<kKind>(a.bn);
  if (e == cudaSuccess) e = raise_smem_limit<head::gemm_kernel<kKind, kBias>>(dev, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(head::gemm_kernel<kKind, kBias>, dim3(static_cast<unsigned>(2 * a.n_pairs)),
                       dim3(head::kThreads), smem, stream, true, ta, tb, tout, a);
}

// The priority of a bf16 operand that `readers` tiles read each part of.
head::Keep keep_of(int64_t elements, int readers) {
  return 2 * elements <= head::kKeepBytes ? head::kLong : readers > 1 ? head::kNormal : head::kStream;
}

int pairs_for(int64_t units) { return static_cast<int>(std::min<int64_t>(resident_pairs(), units)); }

// The product x^T = W h^T over vocabulary rows [v0, v0 + vc).
template <Kind kKind>
cudaError_t launch_logits(Args a, int64_t v0, int64_t vc, cudaStream_t stream) {
  const HeadProblem& p = a.p;
  const ColumnTiles c = column_tiles(p.n);
  CUtensorMap tw, th;
  if (!encode_rows_bf16(&tw, static_cast<const uint16_t*>(p.W) + v0 * p.d, vc, p.d, p.d, kBox, 128) ||
      !encode_rows_bf16(&th, p.h, p.n, p.d, p.d, kBox, c.bn / 2))
    return cudaErrorInvalidValue;
  a.M = vc;
  a.N = p.n;
  a.bn = c.bn;
  a.n_stages = stages_for<kKind>(c.bn);
  a.n_nt = c.count;
  a.n_mt = row_tiles(vc);
  a.n_kb = k_blocks(p.d);
  a.splits = 1;
  a.sub = head::sub_blocks(p.n);
  a.n_pairs = pairs_for(static_cast<int64_t>(a.n_mt) * a.n_nt);
  a.keep_a = keep_of(vc * p.d, a.n_nt);
  a.keep_b = keep_of(p.n * p.d, a.n_mt);
  a.v0 = v0;
  return p.bias != nullptr ? launch<kKind, true>(a, tw, th, tw, stream) : launch<kKind, false>(a, tw, th, tw, stream);
}

}  // namespace

// Eight parts (2 CTAs x 4 lane quarters) for each row tile, or, where one
// column tile takes all tokens, for each pair.
int64_t head_parts(int64_t n, int64_t V) {
  const int tiles = std::max(1, row_tiles(V));
  return 8 * static_cast<int64_t>(column_tiles(n).count > 1 ? tiles : pairs_for(tiles));
}

cudaError_t launch_head_parts(const HeadProblem& p, LsePart* parts, float* own_x, float* kept, int* err,
                              cudaStream_t stream) {
  Args a{};
  a.p = p;
  a.parts = parts;
  a.own_x = own_x;
  a.kept = kept;
  a.kept_pitch = padded_cols(p.V);
  a.err = err;
  return launch_logits<head::kLse>(a, 0, p.V, stream);
}

cudaError_t launch_head_merge(const HeadProblem& p, const LsePart* parts, int64_t n_parts, const float* own_x,
                              float* logp, float* lse, cudaStream_t stream) {
  const int64_t blocks = (p.n + kMergeRows - 1) / kMergeRows;
  const bool few = blocks <= 192;
  return launch_kernel(few ? head_merge_kernel<1024> : head_merge_kernel<256>, dim3(static_cast<unsigned>(blocks)),
                       dim3(few ? 1024 : 256), 0, stream, false, p, parts, n_parts, own_x, logp, lse);
}

cudaError_t launch_head_ds(const HeadProblem& p, const HeadRows& r, const float* kept, int64_t v0, int64_t vc, void* ds,
                           int* err, cudaStream_t stream) {
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(ds);
  const int64_t pitch = padded_cols(vc);
  if (kept != nullptr) {
    // a block of a large batch takes 8192 columns, so that reading the row's
    // scalars is paid for; a block of a small one 2048, so that there are enough
    const int64_t span = p.n * pitch >= (int64_t(1) << 24) ? 8192 : 2048;
    const int64_t blocks = std::min<int64_t>((pitch + span - 1) / span, 65535);
    return launch_kernel(head_ds_kept_kernel, dim3(static_cast<unsigned>(p.n), static_cast<unsigned>(blocks)),
                         dim3(256), 0, stream, true, p, r, kept, padded_cols(p.V), v0, out, pitch);
  }
  if (v0 == 0) {
    const cudaError_t e = launch_kernel(head_rows_kernel, dim3(static_cast<unsigned>(p.n)), dim3(256), 0, stream, true,
                                        p, r);
    if (e != cudaSuccess) return e;
  }
  Args a{};
  a.p = p;
  a.logp = r.logp;
  a.lse = r.lse;
  a.coef = r.coef;
  a.ds = out;
  a.ds_pitch = pitch;
  a.rest = r.rest;
  a.err = err;
  return launch_logits<head::kDs>(a, v0, vc, stream);
}

// Splits of grad_h's product along the vocabulary: its tiles alone (16 by the
// number of column tiles for a width of 4096) seldom fill the pairs evenly.
// Each count is rated by its rounds of pairs times the k blocks of a split
// (bn clocks per k block and 128 rows at the tensor rate, twice that for the
// pair's tile) plus the partials' way through memory and back.
int64_t head_dh_splits(int64_t n, int64_t d, int64_t vc) {
  const ColumnTiles c = column_tiles(n);
  const int64_t tiles = static_cast<int64_t>(row_tiles(d)) * c.count;
  const int64_t pairs = resident_pairs(), kb = k_blocks(vc);
  int64_t best = 1;
  double best_time = 1e300;
  for (int64_t s = 1; s <= std::min<int64_t>(kb, 32); ++s) {
    const double rounds = static_cast<double>((tiles * s + pairs - 1) / pairs);
    const double time = rounds * (static_cast<double>((kb + s - 1) / s) * std::max(c.bn, 64) * 1.1e-9 + 1.0e-6) +
                        static_cast<double>(s) * n * d * 8.0 / 6.0e12;
    if (time < best_time * 0.995) {
      best_time = time;
      best = s;
    }
  }
  return best;
}

cudaError_t launch_head_dh(const HeadProblem& p, const void* ds, int64_t v0, int64_t vc, int64_t splits, bool add,
                           float* partials, int* err, cudaStream_t stream) {
  const ColumnTiles c = column_tiles(p.n);
  CUtensorMap tw, ts;
  if (!encode_rows_bf16(&tw, static_cast<const uint16_t*>(p.W) + v0 * p.d, vc, p.d, p.d, kBox, head::kBK) ||
      !encode_rows_bf16(&ts, ds, p.n, vc, padded_cols(vc), kBox, c.bn / 2))
    return cudaErrorInvalidValue;
  Args a{};
  a.p = p;
  a.M = p.d;
  a.N = p.n;
  a.bn = c.bn;
  a.n_stages = stages_for<head::kDh>(c.bn);
  a.n_nt = c.count;
  a.n_mt = row_tiles(p.d);
  a.n_kb = k_blocks(vc);
  a.splits = static_cast<int>(std::min<int64_t>(splits, a.n_kb));
  a.sub = head::kWhole;
  a.n_pairs = pairs_for(static_cast<int64_t>(a.n_mt) * a.n_nt * a.splits);
  a.keep_a = keep_of(vc * p.d, a.n_nt);
  a.keep_b = keep_of(p.n * padded_cols(vc), a.n_mt);
  a.partials = partials;
  a.add = add;
  a.err = err;
  return launch<head::kDh, false>(a, tw, ts, tw, stream);
}

cudaError_t launch_head_dh_sum(const HeadProblem& p, const HeadRows& r, const float* partials, int64_t splits,
                               void* grad_h, cudaStream_t stream) {
  return launch_kernel(head_dh_sum_kernel, dim3(static_cast<unsigned>((p.n * p.d / 4 + 255) / 256)), dim3(256), 0,
                       stream, false, p, partials, splits, static_cast<const int*>(r.own), static_cast<const float*>(r.rest),
                       static_cast<__nv_bfloat16*>(grad_h));
}

cudaError_t launch_head_dw(const HeadProblem& p, const HeadRows& r, const void* ds, int64_t v0, int64_t vc,
                           void* grad_W, int* err, cudaStream_t stream) {
  Args a{};
  a.p = p;
  a.M = vc;
  a.N = p.d;
  a.bn = p.d <= 128 ? 128 : head::kMaxN;
  CUtensorMap th, ts, tg;
  if (!encode_rows_bf16(&ts, ds, p.n, vc, padded_cols(vc), kBox, head::kBK) ||
      !encode_rows_bf16(&th, r.h_live, p.n, p.d, p.d, kBox, head::kBK) ||
      !encode_rows_bf16(&tg, static_cast<uint16_t*>(grad_W) + v0 * p.d, vc, p.d, p.d, kBox, 32))
    return cudaErrorInvalidValue;
  a.n_stages = stages_for<head::kDw>(a.bn);
  a.n_nt = static_cast<int>((p.d + a.bn - 1) / a.bn);
  a.n_mt = row_tiles(vc);
  a.n_kb = k_blocks(p.n);
  a.splits = 1;
  a.sub = head::kWhole;
  a.n_pairs = pairs_for(static_cast<int64_t>(a.n_mt) * a.n_nt);
  a.keep_a = keep_of(p.n * padded_cols(vc), a.n_nt);
  a.keep_b = keep_of(p.n * p.d, a.n_mt);
  // With few k blocks a tile there is no time to wait for ds behind the writes
  // of a grad_W larger than L2 (256 tokens of 128256 x 4096: 305 us, with the
  // next tile's ds brought in ahead 271; 512: 375 and 366; a 32001 x 520 grad_W,
  // which stays in L2: 32 and 34).
  a.prefetch = a.n_kb <= 8 && 2 * vc * p.d > (int64_t(128) << 20);
  a.v0 = v0;
  a.rest = r.rest;
  a.own = r.own;
  a.h = static_cast<const __nv_bfloat16*>(r.h_live);
  a.err = err;
  return launch<head::kDw, false>(a, ts, th, tg, stream);
}

}  // namespace fs
