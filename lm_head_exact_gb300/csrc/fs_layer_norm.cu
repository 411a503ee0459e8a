// Layer norm of rows and its backward pass.
//
//   y = xh w + b,  xh = (x - mean) rstd,  rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//   a = g w,  gx = rstd (a - mean(a) - xh mean(a xh)),  gw = sum g xh,  gb = sum g
//
// rms: without the mean (and without mean(a)).  Both passes are bound by
// memory: a row is read once and stays in registers, where its statistics are
// taken in two passes (the mean, then the squares about it, which cancel
// nothing), in fp32.  The forward pass can write the result in 8 bits with a
// scale for each 128 columns instead, from the fp32 values.
#include <algorithm>

#include "fs_fp8.cuh"
#include "fs_fp8.h"

namespace fs {
namespace {

constexpr int kSmallRow = 32;              // threads of a row that one warp takes
constexpr int kRowsPerBlock = 8;           // rows (warps) of a block of such

// kV elements from p (16-byte aligned where kV > 1).
template <typename T, int kV>
__device__ __forceinline__ void load_group(const T* p, float (&v)[kV]) {
  if constexpr (kV == 1) {
    v[0] = to_float<T>(*p);
  } else {
#pragma unroll
    for (int h = 0; h < kV; h += kVec<T>) {
      float part[kVec<T>];
      unpack<T>(*reinterpret_cast<const uint4*>(p + h), part);
#pragma unroll
      for (int j = 0; j < kVec<T>; ++j) v[h + j] = part[j];
    }
  }
}

template <typename T, int kV>
__device__ __forceinline__ void store_group(T* p, const float (&v)[kV]) {
  if constexpr (kV == 1)
    *p = from_float<T>(v[0]);
  else
    *reinterpret_cast<uint4*>(p) = pack<T>(v);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the threads of a row: a warp (kOneWarp), or the whole block through
// `parts` (32 floats, another set for each sum of a row).
template <bool kOneWarp>
__device__ __forceinline__ float row_sum(float v, float* parts) {
  v = warp_sum(v);
  if constexpr (kOneWarp) return v;
  if ((threadIdx.x & 31) == 0) parts[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum((threadIdx.x & 31) < (blockDim.x >> 5) ? parts[threadIdx.x & 31] : 0.0f);
}

// A row on `threads` threads: thread t holds the groups of kV columns
// i * threads + t.  kE elements a thread.
template <typename T, typename W, int kV, int kE, bool kOneWarp, int kQuantType>
__global__ void __launch_bounds__(kOneWarp ? kSmallRow* kRowsPerBlock : 1024) norm_kernel(const NormProblem p) {
  constexpr int kN = kE / kV;
  constexpr bool kQuant = kQuantType != 0;
  __shared__ float parts[2][32];
  // largest magnitudes of the blocks of 128 columns, as bits, where a block is not within half a warp or a warp
  constexpr bool kTops = kQuant && kV == 1;
  __shared__ int tops[kTops ? (kOneWarp ? kRowsPerBlock : 1) : 1][kTops ? (kOneWarp ? 8 : kNormMaxWidth / kQuantBlock) : 1];
  const int t = kOneWarp ? threadIdx.x & 31 : threadIdx.x;
  const int threads = kOneWarp ? 32 : blockDim.x;
  const int sub = kOneWarp ? threadIdx.x >> 5 : 0;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kOneWarp ? kRowsPerBlock : 1) + sub;
  const int d = static_cast<int>(p.d);
  pdl_launch_dependents();
  pdl_wait();
  if (kOneWarp && row >= p.n) return;                    // (no block barrier follows)
  const T* x = static_cast<const T*>(p.x) + row * p.x_stride;
  if constexpr (kTops) {
    for (int i = t; i < (d + kQuantBlock - 1) / kQuantBlock; i += threads) tops[sub][i] = 0;
    if constexpr (kOneWarp) __syncwarp(); else __syncthreads();
  }
  float v[kN][kV];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int c = (i * threads + t) * kV;
    if (c < d) {
      load_group<T, kV>(x + c, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < kV; ++j) v[i][j] = 0.0f;
    }
  }
  const float inv_d = 1.0f / static_cast<float>(d);
  float mean = 0.0f;
  if (!p.rms) {
#pragma unroll
    for (int i = 0; i < kN; ++i)
#pragma unroll
      for (int j = 0; j < kV; ++j) sum += v[i][j];
    mean = row_sum<kOneWarp>(sum, parts[0]) * inv_d;
  }
  float squares = 0.0f;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    if ((i * threads + t) * kV < d) {
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        v[i][j] -= mean;
        squares = fmaf(v[i][j], v[i][j], squares);
      }
    }
  }
  const float rstd = rsqrtf(row_sum<kOneWarp>(squares, parts[1]) * inv_d + p.eps);
  if (t == 0) {
    if (p.mean != nullptr) p.mean[row] = mean;
    if (p.rstd != nullptr) p.rstd[row] = rstd;
  }
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int c = (i * threads + t) * kV;
    if (!kQuant && c >= d) break;
    if (c >= d) {                                        // (zeros, which no block's largest value minds)
#pragma unroll
      for (int j = 0; j < kV; ++j) v[i][j] = 0.0f;
    } else {
      float w[kV], b[kV];
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        w[j] = 1.0f;
        b[j] = 0.0f;
      }
      if (p.weight != nullptr) load_group<W, kV>(static_cast<const W*>(p.weight) + c, w);
      if (p.bias != nullptr) load_group<W, kV>(static_cast<const W*>(p.bias) + c, b);
#pragma unroll
      for (int j = 0; j < kV; ++j) v[i][j] = fmaf(v[i][j] * rstd, w[j], b[j]);
    }
    if constexpr (!kQuant) {
      store_group<T, kV>(static_cast<T*>(p.y) + row * p.y_stride + c, v[i]);
    } else if constexpr (kV > 1) {
      // 128 columns are 16 lanes (8 elements each) or 32 (4 each)
      float top = 0.0f;
#pragma unroll
      for (int j = 0; j < kV; ++j) top = fmaxf(top, fabsf(v[i][j]));
#pragma unroll
      for (int o = 64 / kV; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const BlockScale s = block_scale(top, fp8_largest(kQuantType));
      if (c < d) {
        if (c % kQuantBlock == 0) p.scale[row * p.s_row + c / kQuantBlock * p.s_col] = s.scale;
        uint8_t* dst = static_cast<uint8_t*>(p.q) + row * p.q_stride + c;
        uint32_t o[kV / 4];
#pragma unroll
        for (int j = 0; j < kV; j += 4)
          o[j / 4] = fp8_quad<kQuantType>(v[i][j], v[i][j + 1], v[i][j + 2], v[i][j + 3], s.inverse);
        if constexpr (kV == 8)
          *reinterpret_cast<uint2*>(dst) = make_uint2(o[0], o[1]);
        else
          *reinterpret_cast<uint32_t*>(dst) = o[0];
      }
    } else {
      // 32 lanes lie within one block of 128 columns
      float top = fabsf(v[i][0]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int block = (i * threads + (t & ~31)) / kQuantBlock;
      if ((t & 31) == 0 && block * kQuantBlock < d) atomicMax(&tops[sub][block], __float_as_int(top));
    }
  }
  if constexpr (kTops) {
    if constexpr (kOneWarp) __syncwarp(); else __syncthreads();
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int c = i * threads + t;
      if (c >= d) break;
      const BlockScale s = block_scale(__int_as_float(tops[sub][c / kQuantBlock]), fp8_largest(kQuantType));
      if (c % kQuantBlock == 0) p.scale[row * p.s_row + c / kQuantBlock * p.s_col] = s.scale;
      static_cast<uint8_t*>(p.q)[row * p.q_stride + c] = fp8_one<kQuantType>(v[i][0], s.inverse);
    }
  }
}

// Backward: a block goes through rows blockIdx.x, + gridDim.x, ... (a warp each
// where rows are short) and keeps the columns' sums of g xh and g in registers;
// they leave as one partial sum a block, added by norm_sum_kernel in the order
// of the blocks, so that results do not depend on the run.
template <typename T, typename W, int kV, int kE, bool kOneWarp>
__global__ void __launch_bounds__(kOneWarp ? kSmallRow* kRowsPerBlock : (kE <= 16 ? 512 : 1024))
norm_grad_kernel(const NormGradProblem p) {
  constexpr int kN = kE / kV;
  __shared__ float parts[2][2][32];
  __shared__ float cols[kOneWarp ? 2 * 32 * kE : 1];
  const int t = kOneWarp ? threadIdx.x & 31 : threadIdx.x;
  const int threads = kOneWarp ? 32 : blockDim.x;
  const int sub = kOneWarp ? threadIdx.x >> 5 : 0;
  const int d = static_cast<int>(p.d);
  const float inv_d = 1.0f / static_cast<float>(d);
  const bool sums = p.gw != nullptr || p.gb != nullptr;
  pdl_launch_dependents();
  pdl_wait();
  float w[kN][kV], gw[kN][kV], gb[kN][kV];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int c = (i * threads + t) * kV;
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      gw[i][j] = gb[i][j] = 0.0f;
      w[i][j] = 1.0f;
    }
    if (p.weight != nullptr && c < d) load_group<W, kV>(static_cast<const W*>(p.weight) + c, w[i]);
  }
  int turn = 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kOneWarp ? kRowsPerBlock : 1);
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * (kOneWarp ? kRowsPerBlock : 1) + sub; row < p.n; row += step) {
    const T* x = static_cast<const T*>(p.x) + row * p.x_stride;
    const T* g = static_cast<const T*>(p.g) + row * p.g_stride;
    const float mean = p.rms ? 0.0f : p.mean[row], rstd = p.rstd[row];
    float xh[kN][kV], a[kN][kV];
    float sum_a = 0.0f, sum_ax = 0.0f;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int c = (i * threads + t) * kV;
      if (c < d) {
        load_group<T, kV>(x + c, xh[i]);
        load_group<T, kV>(g + c, a[i]);
      } else {
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          xh[i][j] = mean;
          a[i][j] = 0.0f;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) {
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        xh[i][j] = (xh[i][j] - mean) * rstd;
        gw[i][j] = fmaf(a[i][j], xh[i][j], gw[i][j]);
        gb[i][j] += a[i][j];
        a[i][j] *= w[i][j];
        sum_a += a[i][j];
        sum_ax = fmaf(a[i][j], xh[i][j], sum_ax);
      }
    }
    if (p.gx == nullptr) continue;
    sum_a = warp_sum(sum_a);
    sum_ax = warp_sum(sum_ax);
    if constexpr (!kOneWarp) {
      // (two sets in turn: a thread that is a row ahead does not overwrite what another still reads)
      if ((threadIdx.x & 31) == 0) {
        parts[turn][0][threadIdx.x >> 5] = sum_a;
        parts[turn][1][threadIdx.x >> 5] = sum_ax;
      }
      __syncthreads();
      const bool mine = (threadIdx.x & 31) < (blockDim.x >> 5);
      sum_a = warp_sum(mine ? parts[turn][0][threadIdx.x & 31] : 0.0f);
      sum_ax = warp_sum(mine ? parts[turn][1][threadIdx.x & 31] : 0.0f);
      turn ^= 1;
    }
    const float m_a = p.rms ? 0.0f : sum_a * inv_d, m_ax = sum_ax * inv_d;
    T* gx = static_cast<T*>(p.gx) + row * p.gx_stride;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int c = (i * threads + t) * kV;
      if (c >= d) break;
      float o[kV];
#pragma unroll
      for (int j = 0; j < kV; ++j) o[j] = rstd * (a[i][j] - m_a - xh[i][j] * m_ax);
      store_group<T, kV>(gx + c, o);
    }
  }
  if (!sums) return;
  float* out = p.partials + static_cast<int64_t>(blockIdx.x) * 2 * d;
  if constexpr (kOneWarp) {
    // the warps' sums, one after another
    for (int r = 0; r < kRowsPerBlock; ++r) {
      if (sub == r) {
#pragma unroll
        for (int i = 0; i < kN; ++i)
#pragma unroll
          for (int j = 0; j < kV; ++j) {
            const int at = (i * 32 + t) * kV + j;
            cols[at] = (r > 0 ? cols[at] : 0.0f) + gw[i][j];
            cols[32 * kE + at] = (r > 0 ? cols[32 * kE + at] : 0.0f) + gb[i][j];
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < d; c += blockDim.x) {
      out[c] = cols[c];
      out[d + c] = cols[32 * kE + c];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int c = (i * threads + t) * kV;
      if (c >= d) break;
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        out[c + j] = gw[i][j];
        out[d + c + j] = gb[i][j];
      }
    }
  }
}

// Sums over the blocks' partials: 32 columns a block of threads, 8 slices of the
// partials, joined in the order of the slices.
constexpr int kSumSlices = 16;

template <typename W>
__global__ void __launch_bounds__(32 * kSumSlices) norm_sum_kernel(const float* partials, int64_t blocks, int64_t d, W* gw,
                                                                   W* gb) {
  __shared__ float sums[kSumSlices][33];
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x % 32;     // of [gw, gb]
  const int slice = threadIdx.x / 32;
  pdl_launch_dependents();
  pdl_wait();
  float s = 0.0f;
  if (c < 2 * d) {
#pragma unroll 4
    for (int64_t b = slice; b < blocks; b += kSumSlices) s += partials[b * 2 * d + c];
  }
  sums[slice][threadIdx.x % 32] = s;
  __syncthreads();
  if (slice != 0 || c >= 2 * d) return;
  for (int k = 1; k < kSumSlices; ++k) s += sums[k][threadIdx.x];
  if (c < d) {
    if (gw != nullptr) gw[c] = from_float<W>(s);
  } else if (gb != nullptr) {
    gb[c - d] = from_float<W>(s);
  }
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Rows of up to 1024 columns are one warp's, of which a thread takes 8, 16 or
// 32 elements; wider ones a block's.
template <typename T, typename W, int kV, int kE, bool kOneWarp>
cudaError_t launch_norm_as(const NormProblem& p, int threads, cudaStream_t stream) {
  const int64_t grid = kOneWarp ? (p.n + kRowsPerBlock - 1) / kRowsPerBlock : p.n;
  const dim3 g(static_cast<unsigned>(grid)), b(kOneWarp ? kSmallRow * kRowsPerBlock : threads);
  if (p.q == nullptr) return launch_kernel(norm_kernel<T, W, kV, kE, kOneWarp, 0>, g, b, 0, stream, true, p);
  if (p.q_type == FS_TYPE_E5M2)
    return launch_kernel(norm_kernel<T, W, kV, kE, kOneWarp, FS_TYPE_E5M2>, g, b, 0, stream, true, p);
  return launch_kernel(norm_kernel<T, W, kV, kE, kOneWarp, FS_TYPE_E4M3>, g, b, 0, stream, true, p);
}

int threads_for(int64_t d, int elements) { return static_cast<int>((d + 32 * elements - 1) / (32 * elements)) * 32; }

template <typename T, typename W, int kV>
cudaError_t launch_norm_of(const NormProblem& p, cudaStream_t stream) {
  if (p.d <= 32 * 8) return launch_norm_as<T, W, kV, 8, true>(p, 32, stream);
  if (p.d <= 32 * 32 && p.n > 512) return launch_norm_as<T, W, kV, 32, true>(p, 32, stream);
  // few rows: more threads for each
  if (p.n <= 512 && p.d <= 1024 * 8) return launch_norm_as<T, W, kV, 8, false>(p, threads_for(p.d, 8), stream);
  return launch_norm_as<T, W, kV, 32, false>(p, threads_for(p.d, 32), stream);
}

template <typename T, typename W>
cudaError_t launch_norm_typed(const NormProblem& p, cudaStream_t stream) {
  constexpr int kV = kVec<T>;
  const int64_t size = sizeof(T);
  const bool vectors = p.d % kV == 0 && aligned16(p.x) && p.x_stride * size % 16 == 0 && aligned16(p.weight) &&
                       aligned16(p.bias) && (p.q != nullptr || (aligned16(p.y) && p.y_stride * size % 16 == 0));
  return vectors ? launch_norm_of<T, W, kV>(p, stream) : launch_norm_of<T, W, 1>(p, stream);
}

// Columns a thread of the backward pass takes, and the threads of a row.
struct GradShape {
  int elements, threads;      // threads 32: a warp a row
};

GradShape grad_shape(int64_t d) {
  if (d <= 256) return {8, 32};
  if (d <= 1024) return {32, 32};
  if (d <= 512 * 16) return {16, threads_for(d, 16)};
  return {32, threads_for(d, 32)};
}

template <typename T, typename W, int kV, int kE, bool kOneWarp>
cudaError_t launch_grad_as(const NormGradProblem& p, int threads, cudaStream_t stream) {
  const int64_t blocks = norm_grad_blocks(p.n, p.d);
  return launch_kernel(norm_grad_kernel<T, W, kV, kE, kOneWarp>, dim3(static_cast<unsigned>(blocks)),
                       dim3(kOneWarp ? kSmallRow * kRowsPerBlock : threads), 0, stream, true, p);
}

template <typename T, typename W, int kV>
cudaError_t launch_grad_of(const NormGradProblem& p, cudaStream_t stream) {
  const GradShape s = grad_shape(p.d);
  if (s.threads == 32)
    return s.elements == 8 ? launch_grad_as<T, W, kV, 8, true>(p, 32, stream) : launch_grad_as<T, W, kV, 32, true>(p, 32, stream);
  return s.elements == 16 ? launch_grad_as<T, W, kV, 16, false>(p, s.threads, stream)
                          : launch_grad_as<T, W, kV, 32, false>(p, s.threads, stream);
}

template <typename T, typename W>
cudaError_t launch_grad_typed(const NormGradProblem& p, cudaStream_t stream) {
  constexpr int kV = kVec<T>;
  const int64_t size = sizeof(T);
  const bool vectors = p.d % kV == 0 && aligned16(p.x) && p.x_stride * size % 16 == 0 && aligned16(p.weight) &&
                       aligned16(p.g) && p.g_stride * size % 16 == 0 && aligned16(p.gx) &&
                       (p.gx == nullptr || p.gx_stride * size % 16 == 0);
  cudaError_t e = vectors ? launch_grad_of<T, W, kV>(p, stream) : launch_grad_of<T, W, 1>(p, stream);
  if (e != cudaSuccess || (p.gw == nullptr && p.gb == nullptr)) return e;
  return launch_kernel(norm_sum_kernel<W>, dim3(static_cast<unsigned>((2 * p.d + 31) / 32)), dim3(32 * kSumSlices), 0, stream,
                       true, static_cast<const float*>(p.partials), norm_grad_blocks(p.n, p.d), p.d, static_cast<W*>(p.gw),
                       static_cast<W*>(p.gb));
}

// Calls f(element type, type of the weights).
template <typename F>
cudaError_t by_types(int x_type, int w_type, F f) {
  const bool same = x_type == w_type;
  if (x_type == FS_TYPE_BF16) return same ? f(__nv_bfloat16(), __nv_bfloat16()) : f(__nv_bfloat16(), float());
  if (x_type == FS_TYPE_F16) return same ? f(__half(), __half()) : f(__half(), float());
  return f(float(), float());
}

}  // namespace

cudaError_t launch_norm(const NormProblem& p, cudaStream_t stream) {
  return by_types(p.x_type, p.w_type, [&](auto x, auto w) { return launch_norm_typed<decltype(x), decltype(w)>(p, stream); });
}

int64_t norm_grad_blocks(int64_t n, int64_t d) {
  const int64_t rows = grad_shape(d).threads == 32 ? kRowsPerBlock : 1;
  return std::max<int64_t>(1, std::min<int64_t>((n + rows - 1) / rows, 304));
}

cudaError_t launch_norm_grad(const NormGradProblem& p, cudaStream_t stream) {
  return by_types(p.x_type, p.w_type, [&](auto x, auto w) { return launch_grad_typed<decltype(x), decltype(w)>(p, stream); });
}

}  // namespace fs
