// Token log-probabilities through the LM head and their gradients.
//
//   x = (h W^T + bias) / T,  lse = log sum exp x,  logp = x[id] - lse
//   ds = c (1[v = id] - exp(x - lse)),  c = g / T;  grad_h = ds W,  grad_W = ds^T h
//
// Forward: every tile of x is reduced on chip to one (max, sum of exp) per
// row; the parts are merged by a second, small launch.
#include <cuda_bf16.h>

#include <algorithm>

#include "fs_train.h"

namespace fs {
namespace {

constexpr int kTile = 64;
constexpr int kStep = 16;

__device__ __forceinline__ LsePart lse_join(LsePart a, LsePart b) {
  if (b.s == 0.0f) return a;
  if (a.s == 0.0f) return b;
  const float m = fmaxf(a.m, b.m);
  return LsePart{m, a.s * expf(a.m - m) + b.s * expf(b.m - m)};
}

// acc[i][j] = sum_k A(m0 + ty + 16 i, k) B(n0 + tx + 16 j, k) over k in
// [0, K), with element (r, k) of an operand at r * row + k * col.
__device__ __forceinline__ void tile_product(const __nv_bfloat16* A, int64_t a_row, int64_t a_col, int64_t M,
                                             const __nv_bfloat16* B, int64_t b_row, int64_t b_col, int64_t N,
                                             int64_t k_begin, int64_t K, int64_t m0, int64_t n0, float (&acc)[4][4]) {
  __shared__ float sa[kStep][kTile + 1], sb[kStep][kTile + 1];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
  for (int64_t k0 = k_begin; k0 < K; k0 += kStep) {
    for (int e = threadIdx.x; e < kTile * kStep; e += 256) {
      int r = e / kStep, k = e % kStep;
      if (a_col != 1) { r = e % kTile; k = e / kTile; }
      sa[k][r] = m0 + r < M && k0 + k < K ? __bfloat162float(A[(m0 + r) * a_row + (k0 + k) * a_col]) : 0.0f;
      r = e / kStep, k = e % kStep;
      if (b_col != 1) { r = e % kTile; k = e / kTile; }
      sb[k][r] = n0 + r < N && k0 + k < K ? __bfloat162float(B[(n0 + r) * b_row + (k0 + k) * b_col]) : 0.0f;
    }
    __syncthreads();
    for (int k = 0; k < kStep; ++k)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][ty + 16 * i], sb[k][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
}

__device__ __forceinline__ float scaled(const HeadProblem& p, int64_t t, int64_t v, float dot, float inv_t) {
  if (p.bias != nullptr) dot += p.bias[t * p.bias_stride + v];
  return dot * inv_t;
}

__global__ void __launch_bounds__(256) head_parts_kernel(const HeadProblem p, LsePart* parts, int64_t n_parts,
                                                         float* own_x, float* kept, int64_t pitch) {
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kTile, n0 = static_cast<int64_t>(blockIdx.x) * kTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4];
  tile_product(static_cast<const __nv_bfloat16*>(p.h), p.d, 1, p.n, static_cast<const __nv_bfloat16*>(p.W), p.d, 1, p.V,
               0, p.d, m0, n0, acc);
  for (int i = 0; i < 4; ++i) {
    const int64_t t = m0 + ty + 16 * i;
    const bool row = t < p.n;
    const float inv_t = row ? row_temp(p.temp[t]).inv_t : 0.0f;
    const int64_t id = row ? p.ids[t] : -1;
    float x[4];
    LsePart part{-INFINITY, 0.0f};
    for (int j = 0; j < 4; ++j) {
      const int64_t v = n0 + tx + 16 * j;
      x[j] = -INFINITY;
      if (!row || v >= p.V) continue;
      x[j] = scaled(p, t, v, acc[i][j], inv_t);
      if (kept != nullptr) kept[t * pitch + v] = x[j];
      if (v == id) own_x[t] = x[j];
      if (x[j] == -INFINITY) continue;
      part = lse_join(part, LsePart{x[j], 1.0f});
    }
    for (int o = 8; o > 0; o >>= 1)
      part = lse_join(part, LsePart{__shfl_xor_sync(0xffffffffu, part.m, o), __shfl_xor_sync(0xffffffffu, part.s, o)});
    if (tx == 0 && row) parts[t * n_parts + blockIdx.x] = part;
  }
}

__global__ void __launch_bounds__(128) head_merge_kernel(const HeadProblem p, const LsePart* parts, int64_t n_parts,
                                                         const float* own_x, float* logp, float* lse) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (t >= p.n) return;
  LsePart part{-INFINITY, 0.0f};
  for (int64_t i = lane; i < n_parts; i += 32) part = lse_join(part, parts[t * n_parts + i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    part = lse_join(part, LsePart{__shfl_xor_sync(0xffffffffu, part.m, o), __shfl_xor_sync(0xffffffffu, part.s, o)});
  if (lane != 0) return;
  const bool valid = row_temp(p.temp[t]).mode != kRowInvalid;
  const int64_t id = p.ids[t];
  float z = !valid || part.s == 0.0f ? -INFINITY : part.m + logf(part.s);
  if (valid && part.m == INFINITY) z = NAN;
  lse[t] = z;
  float lp = 0.0f;
  if (valid && id >= 0 && id < p.V) {
    const float x = own_x[t];
    lp = x == -INFINITY ? -INFINITY : x - z;
  }
  logp[t] = lp;
}

__global__ void __launch_bounds__(256) head_rows_kernel(const HeadProblem p, const float* logp, const float* lse,
                                                        const float* g, float* coef, __nv_bfloat16* h_live) {
  const int64_t t = blockIdx.x;
  const RowTemp rt = row_temp(p.temp[t]);
  const int64_t id = p.ids[t];
  const bool live = rt.mode != kRowInvalid && id >= 0 && id < p.V && g[t] != 0.0f && lse[t] != -INFINITY &&
                    logp[t] != -INFINITY;
  if (threadIdx.x == 0) coef[t] = live ? g[t] * rt.inv_t : 0.0f;
  if (h_live == nullptr) return;
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.h) + t * p.d);
  uint4* dst = reinterpret_cast<uint4*>(h_live + t * p.d);
  for (int64_t i = threadIdx.x; i < p.d / 8; i += 256) dst[i] = live ? src[i] : make_uint4(0, 0, 0, 0);
}

__device__ __forceinline__ float ds_of(float x, float lse, float c, bool own) {
  return c == 0.0f ? 0.0f : c * ((own ? 1.0f : 0.0f) - expf(x - lse));
}

__global__ void __launch_bounds__(256) head_ds_kept_kernel(const HeadProblem p, const float* lse, const float* coef,
                                                           const float* kept, int64_t kept_pitch, int64_t v0,
                                                           int64_t vc, __nv_bfloat16* ds, int64_t pitch) {
  const int64_t t = blockIdx.x;
  const float c = coef[t], z = lse[t];
  const int64_t id = p.ids[t] - v0;
  for (int64_t v = static_cast<int64_t>(blockIdx.y) * 256 + threadIdx.x; v < vc; v += static_cast<int64_t>(gridDim.y) * 256)
    ds[t * pitch + v] = __float2bfloat16_rn(ds_of(kept[t * kept_pitch + v0 + v], z, c, v == id));
}

__global__ void __launch_bounds__(256) head_ds_kernel(const HeadProblem p, const float* lse, const float* coef,
                                                      int64_t v0, int64_t vc, __nv_bfloat16* ds, int64_t pitch) {
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kTile, n0 = static_cast<int64_t>(blockIdx.x) * kTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4];
  tile_product(static_cast<const __nv_bfloat16*>(p.h), p.d, 1, p.n,
               static_cast<const __nv_bfloat16*>(p.W) + v0 * p.d, p.d, 1, vc, 0, p.d, m0, n0, acc);
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t t = m0 + ty + 16 * i, v = n0 + tx + 16 * j;
      if (t >= p.n || v >= vc) continue;
      const float x = scaled(p, t, v0 + v, acc[i][j], row_temp(p.temp[t]).inv_t);
      ds[t * pitch + v] = __float2bfloat16_rn(ds_of(x, lse[t], coef[t], v0 + v == p.ids[t]));
    }
}

// partials[t, j] (+)= sum over [0, vc) of ds(t, v) W(v0 + v, j).
__global__ void __launch_bounds__(256) head_dh_kernel(const HeadProblem p, const __nv_bfloat16* ds, int64_t pitch,
                                                      int64_t v0, int64_t vc, bool add, float* partials) {
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kTile, n0 = static_cast<int64_t>(blockIdx.x) * kTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4];
  tile_product(ds, pitch, 1, p.n, static_cast<const __nv_bfloat16*>(p.W) + v0 * p.d, 1, p.d, p.d, 0, vc, m0, n0, acc);
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t t = m0 + ty + 16 * i, k = n0 + tx + 16 * j;
      if (t >= p.n || k >= p.d) continue;
      float* at = partials + t * p.d + k;
      *at = add ? *at + acc[i][j] : acc[i][j];
    }
}

__global__ void __launch_bounds__(256) head_dw_kernel(const HeadProblem p, const __nv_bfloat16* ds, int64_t pitch,
                                                      const __nv_bfloat16* h_live, int64_t v0, int64_t vc,
                                                      __nv_bfloat16* grad_W) {
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kTile, n0 = static_cast<int64_t>(blockIdx.x) * kTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4];
  tile_product(ds, 1, pitch, vc, h_live, 1, p.d, p.d, 0, p.n, m0, n0, acc);
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t v = m0 + ty + 16 * i, k = n0 + tx + 16 * j;
      if (v < vc && k < p.d) grad_W[(v0 + v) * p.d + k] = __float2bfloat16_rn(acc[i][j]);
    }
}

__global__ void __launch_bounds__(256) head_dh_sum_kernel(const HeadProblem p, const float* partials, int64_t splits,
                                                          const float* coef, __nv_bfloat16* grad_h) {
  const int64_t t = blockIdx.x;
  const bool live = coef[t] != 0.0f;
  for (int64_t k = threadIdx.x; k < p.d; k += 256) {
    float s = 0.0f;
    if (live)
      for (int64_t i = 0; i < splits; ++i) s += partials[(i * p.n + t) * p.d + k];
    grad_h[t * p.d + k] = __float2bfloat16_rn(s);
  }
}

unsigned tiles(int64_t n) { return static_cast<unsigned>((n + kTile - 1) / kTile); }

}  // namespace

int64_t head_parts(int64_t, int64_t V) { return std::max<int64_t>(1, tiles(V)); }

cudaError_t launch_head_parts(const HeadProblem& p, LsePart* parts, float* own_x, float* kept, int*,
                              cudaStream_t stream) {
  return launch_kernel(head_parts_kernel, dim3(tiles(p.V), tiles(p.n)), dim3(256), 0, stream, false, p, parts,
                       head_parts(p.n, p.V), own_x, kept, padded_cols(p.V));
}

cudaError_t launch_head_merge(const HeadProblem& p, const LsePart* parts, int64_t n_parts, const float* own_x,
                              float* logp, float* lse, cudaStream_t stream) {
  return launch_kernel(head_merge_kernel, dim3(static_cast<unsigned>((p.n + 3) / 4)), dim3(128), 0, stream, false, p,
                       parts, n_parts, own_x, logp, lse);
}

cudaError_t launch_head_rows(const HeadProblem& p, const float* logp, const float* lse, const float* g, float* coef,
                             void* h_live, cudaStream_t stream) {
  return launch_kernel(head_rows_kernel, dim3(static_cast<unsigned>(p.n)), dim3(256), 0, stream, false, p, logp, lse,
                       g, coef, static_cast<__nv_bfloat16*>(h_live));
}

cudaError_t launch_head_ds(const HeadProblem& p, const float* lse, const float* coef, const float* kept, int64_t v0,
                           int64_t vc, void* ds, int*, cudaStream_t stream) {
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(ds);
  if (kept != nullptr)
    return launch_kernel(head_ds_kept_kernel, dim3(static_cast<unsigned>(p.n), 64), dim3(256), 0, stream, false, p,
                         lse, coef, kept, padded_cols(p.V), v0, vc, out, padded_cols(vc));
  return launch_kernel(head_ds_kernel, dim3(tiles(vc), tiles(p.n)), dim3(256), 0, stream, false, p, lse, coef, v0, vc,
                       out, padded_cols(vc));
}

int64_t head_dh_splits(int64_t, int64_t, int64_t) { return 1; }

cudaError_t launch_head_dh(const HeadProblem& p, const void* ds, int64_t v0, int64_t vc, int64_t, bool add,
                           float* partials, int*, cudaStream_t stream) {
  return launch_kernel(head_dh_kernel, dim3(tiles(p.d), tiles(p.n)), dim3(256), 0, stream, false, p,
                       static_cast<const __nv_bfloat16*>(ds), padded_cols(vc), v0, vc, add, partials);
}

cudaError_t launch_head_dh_sum(const HeadProblem& p, const float* partials, int64_t splits, const float* coef,
                               void* grad_h, cudaStream_t stream) {
  return launch_kernel(head_dh_sum_kernel, dim3(static_cast<unsigned>(p.n)), dim3(256), 0, stream, false, p, partials,
                       splits, coef, static_cast<__nv_bfloat16*>(grad_h));
}

cudaError_t launch_head_dw(const HeadProblem& p, const void* ds, const void* h_live, int64_t v0, int64_t vc,
                           void* grad_W, int*, cudaStream_t stream) {
  return launch_kernel(head_dw_kernel, dim3(tiles(p.d), tiles(vc)), dim3(256), 0, stream, false, p,
                       static_cast<const __nv_bfloat16*>(ds), padded_cols(vc),
                       static_cast<const __nv_bfloat16*>(h_live), v0, vc, static_cast<__nv_bfloat16*>(grad_W));
}

}  // namespace fs
