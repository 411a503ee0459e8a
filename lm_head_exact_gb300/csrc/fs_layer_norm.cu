// Layer norm of rows and its backward pass.
//
//   y = xh w + b,  xh = (x - mean) rstd,  rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//   a = g w,  gx = rstd (a - mean(a) - xh mean(a xh)),  gw = sum g xh,  gb = sum g
//
// rms: without the mean (and without mean(a)).  Both passes are to be bound by
// memory: a row is read once and held by its threads, which take its statistics
// in two passes (the mean, then the squares about it, which cancel
// nothing), in fp32.  The forward pass can write the result in 8 bits with a
// scale for each 128 columns instead, from the fp32 values.
//
// Rows on 16-byte boundaries stay in registers (but for up to 72 bytes a thread),
// in the backward pass up to 8192 columns.  Other forms spill, bytes a thread: shifted
// rows of more than some 500 columns 270 to 430, single elements over a block 460 to
// 710, the backward pass of more than 8192 columns 1600 to 2450.  us, and what the
// bytes take:
//   16384 x 4097 forward 112, 40; into 8 bits 335, 30; backward 169, 59
//   4096 x 12288 backward 339, 45; 4096 x 16384 520, 59
#include <algorithm>

#include "fs_fp8.cuh"
#include "fs_fp8.h"
#include "fs_fp8_ptx.cuh"

namespace fs {
namespace {

constexpr int kSmallRow = 32;              // threads of a row that one warp takes
constexpr int kRowsPerBlock = 8;           // rows (warps) of a block of such

// kV elements as they lie in memory: 16 aligned bytes, or one element.
template <typename T, int kV>
struct Group {
  uint4 raw;
  __device__ __forceinline__ void load(const T* p) { raw = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&v)[kV]) const { unpack<T>(raw, v); }
};
template <typename T>
struct Group<T, 1> {
  T raw;
  __device__ __forceinline__ void load(const T* p) { raw = *p; }
  __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = to_float<T>(raw); }
};

// kV weights from p, with 16-byte loads where they are aligned.
template <typename W, int kV>
__device__ __forceinline__ void load_weights(const W* p, float (&v)[kV]) {
  if constexpr (kV < kVec<W>) {
#pragma unroll
    for (int j = 0; j < kV; ++j) v[j] = to_float<W>(p[j]);
  } else {
#pragma unroll
    for (int h = 0; h < kV; h += kVec<W>) {
      float part[kVec<W>];
      unpack<W>(*reinterpret_cast<const uint4*>(p + h), part);
#pragma unroll
      for (int j = 0; j < kVec<W>; ++j) v[h + j] = part[j];
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

// The same of a row's columns c .. c + kV - 1, of which only those in [0, d) exist.
template <typename T, int kV>
__device__ __forceinline__ void store_some(T* row, int c, int d, const float (&v)[kV]) {
  if (c >= 0 && c + kV <= d) {
    store_group<T, kV>(row + c, v);
  } else {
#pragma unroll
    for (int j = 0; j < kV; ++j)
      if (c + j >= 0 && c + j < d) row[c + j] = from_float<T>(v[j]);
  }
}
template <typename W, int kV>
__device__ __forceinline__ void load_some(const W* p, int c, int d, float otherwise, float (&v)[kV]) {
#pragma unroll
  for (int j = 0; j < kV; ++j) v[j] = c + j >= 0 && c + j < d ? to_float<W>(p[c + j]) : otherwise;
}

// Elements from a 16-byte boundary to p.
template <typename T>
__device__ __forceinline__ int shift_of(const T* p) {
  return static_cast<int>(reinterpret_cast<uintptr_t>(p) % 16 / sizeof(T));
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

constexpr int kRowsAhead = 608;            // that a block asks for: 4 for each SM of this GPU

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
  if constexpr (kQuant) pdl_wait_then_launch(); else pdl_wait();
  if (kOneWarp && row >= p.n) return;                    // (no block barrier follows)
  const T* x = static_cast<const T*>(p.x) + row * p.x_stride;
  // (to L2 while this row is summed up: 16384 x 4096 57.0 -> 53.0 us; 304 rows ahead the same, 2432 55.3)
  if constexpr (!kOneWarp && kV > 1) {
    if (t == 0 && row + kRowsAhead < p.n) sm100::bulk_prefetch(x + kRowsAhead * p.x_stride, d * sizeof(T));
  }
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
      Group<T, kV> g;
      g.load(x + c);
      g.get(v[i]);
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
      if (p.weight != nullptr) load_weights<W, kV>(static_cast<const W*>(p.weight) + c, w);
      if (p.bias != nullptr) load_weights<W, kV>(static_cast<const W*>(p.bias) + c, b);
#pragma unroll
      for (int j = 0; j < kV; ++j) v[i][j] = fmaf(v[i][j] * rstd, w[j], b[j]);
    }
    if constexpr (!kQuant) store_group<T, kV>(static_cast<T*>(p.y) + row * p.y_stride + c, v[i]);
  }
  if constexpr (kQuant && kV == 8) {
    // 128 columns are 16 lanes
    float top[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      top[i] = 0.0f;
#pragma unroll
      for (int j = 0; j < kV; ++j) top[i] = fmaxf(top[i], fabsf(v[i][j]));
    }
    const int lane = threadIdx.x & 31;
    const BlockScale s = spread_scale<kN>(top, lane, fp8_largest(kQuantType));
    constexpr int kEach = 16 / kN;                         // lanes that hold a group's scale
    const int mine = ((lane & 15) / kEach * threads + (t & ~15)) * kV;
    if (lane % kEach == 0 && mine < d) p.scale[row * p.s_row + mine / kQuantBlock * p.s_col] = s.scale;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int c = (i * threads + t) * kV;
      const float by = spread_get<kN>(s.inverse, i, lane);
      if (c < d)
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.q) + row * p.q_stride + c) =
            make_uint2(fp8_quad<kQuantType>(v[i][0], v[i][1], v[i][2], v[i][3], by),
                       fp8_quad<kQuantType>(v[i][4], v[i][5], v[i][6], v[i][7], by));
    }
  } else if constexpr (kQuant) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      // 32 lanes hold 128 columns, or lie within them
      const int c = (i * threads + t) * kV;
      float top = 0.0f;
#pragma unroll
      for (int j = 0; j < kV; ++j) top = fmaxf(top, fabsf(v[i][j]));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      if constexpr (kV == 4) {
        const BlockScale s = block_scale(top, fp8_largest(kQuantType));
        if (c < d) {
          if (c % kQuantBlock == 0) p.scale[row * p.s_row + c / kQuantBlock * p.s_col] = s.scale;
          *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.q) + row * p.q_stride + c) =
              fp8_quad<kQuantType>(v[i][0], v[i][1], v[i][2], v[i][3], s.inverse);
        }
      } else {
        const int block = (i * threads + (t & ~31)) / kQuantBlock;
        if ((t & 31) == 0 && block * kQuantBlock < d) atomicMax(&tops[sub][block], __float_as_int(top));
      }
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

// Rows that begin off a 16-byte boundary: a thread's groups begin at boundaries
// all the same, `shift` elements before its columns, and what lies outside the row is
// neither used nor written.  (An access never leaves the 16 bytes around an element
// of the row.)  Element by element, 16384 rows of 4097 took seven times as long as
// rows of 4096.  A block goes through rows whose numbers differ by multiples of
// 8, which share their shift, so that the weights' columns stay in registers.
template <typename T, typename W, int kE, bool kOneWarp>
__global__ void __launch_bounds__(kOneWarp ? kSmallRow* kRowsPerBlock : 1024) norm_shift_kernel(const NormProblem p) {
  constexpr int kV = kVec<T>, kN = kE / kV;
  __shared__ float parts[2][2][32];
  const int t = kOneWarp ? threadIdx.x & 31 : threadIdx.x;
  const int threads = kOneWarp ? 32 : blockDim.x;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kOneWarp ? kRowsPerBlock : 1) + (kOneWarp ? threadIdx.x >> 5 : 0);
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kOneWarp ? kRowsPerBlock : 1);
  const int d = static_cast<int>(p.d);
  const float inv_d = 1.0f / static_cast<float>(d);
  pdl_wait();
  if (kOneWarp && first >= p.n) return;                    // (no block barrier follows)
  const T* x = static_cast<const T*>(p.x) + first * p.x_stride;
  T* y = static_cast<T*>(p.y) + first * p.y_stride;
  const int shift = shift_of(x);
  float w[kN][kV], b[kN][kV];
  Group<T, kV> next[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int c = (i * threads + t) * kV - shift;
    if (p.weight != nullptr) {
      load_some<W, kV>(static_cast<const W*>(p.weight), c, d, 0.0f, w[i]);
    } else {
#pragma unroll
      for (int j = 0; j < kV; ++j) w[i][j] = 1.0f;
    }
    if (p.bias != nullptr) {
      load_some<W, kV>(static_cast<const W*>(p.bias), c, d, 0.0f, b[i]);
    } else {
#pragma unroll
      for (int j = 0; j < kV; ++j) b[i][j] = 0.0f;
    }
    if (c < d) next[i].load(x + c);
  }
  int turn = 0;
#pragma unroll 1
  for (int64_t row = first; row < p.n; row += step, y += step * p.y_stride, turn ^= 1) {
    float v[kN][kV];
    float sum = 0.0f;
    x += step * p.x_stride;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int c = (i * threads + t) * kV - shift;
      next[i].get(v[i]);
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        if (c + j < 0 || c + j >= d) v[i][j] = 0.0f;
        sum += v[i][j];
      }
      if (row + step < p.n && c < d) next[i].load(x + c);
    }
    const float mean = p.rms ? 0.0f : row_sum<kOneWarp>(sum, parts[turn][0]) * inv_d;
    float squares = 0.0f;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int c = (i * threads + t) * kV - shift;
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        v[i][j] = c + j < 0 || c + j >= d ? 0.0f : v[i][j] - mean;
        squares = fmaf(v[i][j], v[i][j], squares);
      }
    }
    const float rstd = rsqrtf(row_sum<kOneWarp>(squares, parts[turn][1]) * inv_d + p.eps);
    if (t == 0) {
      if (p.mean != nullptr) p.mean[row] = mean;
      if (p.rstd != nullptr) p.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int c = (i * threads + t) * kV - shift;
      if (c >= d) break;
#pragma unroll
      for (int j = 0; j < kV; ++j) v[i][j] = fmaf(v[i][j] * rstd, w[i][j], b[i][j]);
      store_some<T, kV>(y, c, d, v[i]);
    }
  }
}

// Backward: a block goes through rows blockIdx.x, + gridDim.x, ... (a warp each
// where rows are short) and keeps the columns' sums of g xh and g in registers;
// they leave as one partial sum a block, added by norm_sum_kernel in the order
// of the blocks, so that results do not depend on the run.
// The next row is on its way while a row is summed up.  kShift: see
// norm_shift_kernel.
template <typename T, typename W, int kV, int kE, bool kOneWarp, bool kShift>
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
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kOneWarp ? kRowsPerBlock : 1) + sub;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kOneWarp ? kRowsPerBlock : 1);
  pdl_wait();
  if (sums) pdl_launch_dependents();                       // (norm_sum_kernel, which waits first)
  const T* x = static_cast<const T*>(p.x) + first * p.x_stride;
  const T* g = static_cast<const T*>(p.g) + first * p.g_stride;
  const int shift = kShift ? shift_of(x) : 0;
  Group<T, kV> next_x[kN], next_g[kN];
  float w[kN][kV], gw[kN][kV], gb[kN][kV];
  float mean = 0.0f, rstd = 0.0f;
  if (first < p.n) {
    mean = p.rms ? 0.0f : p.mean[first];
    rstd = p.rstd[first];
  }
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int c = (i * threads + t) * kV - shift;
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      gw[i][j] = gb[i][j] = 0.0f;
      w[i][j] = 1.0f;
    }
    if (p.weight != nullptr && c < d) {
      if constexpr (kShift)
        load_some<W, kV>(static_cast<const W*>(p.weight), c, d, 0.0f, w[i]);
      else
        load_weights<W, kV>(static_cast<const W*>(p.weight) + c, w[i]);
    }
    if (first < p.n && c < d) {
      next_x[i].load(x + c);
      next_g[i].load(g + c);
    }
  }
  int turn = 0;
#pragma unroll 1
  for (int64_t row = first; row < p.n; row += step) {
    float xh[kN][kV], a[kN][kV];
    float sum_a = 0.0f, sum_ax = 0.0f;
    const float row_mean = mean, row_rstd = rstd;
    x += step * p.x_stride;
    g += step * p.g_stride;
    const bool more = row + step < p.n;
    if (more) {
      mean = p.rms ? 0.0f : p.mean[row + step];
      rstd = p.rstd[row + step];
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int c = (i * threads + t) * kV - shift;
      next_x[i].get(xh[i]);
      next_g[i].get(a[i]);
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        if (kShift ? c + j < 0 || c + j >= d : c >= d) {
          xh[i][j] = row_mean;
          a[i][j] = 0.0f;
        }
      }
      if (more && c < d) {
        next_x[i].load(x + c);
        next_g[i].load(g + c);
      }
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        xh[i][j] = (xh[i][j] - row_mean) * row_rstd;
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
      const int c = (i * threads + t) * kV - shift;
      if (c >= d) break;
      float o[kV];
#pragma unroll
      for (int j = 0; j < kV; ++j) o[j] = row_rstd * (a[i][j] - m_a - xh[i][j] * m_ax);
      if constexpr (kShift)
        store_some<T, kV>(gx, c, d, o);
      else
        store_group<T, kV>(gx + c, o);
    }
  }
  if (!sums) return;
  float* out = p.partials + static_cast<int64_t>(blockIdx.x) * 2 * d;
  if constexpr (kOneWarp) {
    // the warps' sums, one after another (a block's rows may have different shifts)
    for (int c = threadIdx.x; c < 2 * 32 * kE; c += blockDim.x) cols[c] = 0.0f;
    __syncthreads();
    for (int r = 0; r < kRowsPerBlock; ++r) {
      if (sub == r) {
#pragma unroll
        for (int i = 0; i < kN; ++i)
#pragma unroll
          for (int j = 0; j < kV; ++j) {
            const int c = (i * 32 + t) * kV - shift + j;
            if (c >= 0 && c < d) {
              cols[c] += gw[i][j];
              cols[32 * kE + c] += gb[i][j];
            }
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
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        const int c = (i * threads + t) * kV - shift + j;
        if (c >= 0 && c < d) {
          out[c] = gw[i][j];
          out[d + c] = gb[i][j];
        }
      }
    }
  }
}

// The backward pass of wide rows on 16-byte boundaries: rows of x and g come by bulk
// copies into a ring of shared memory, kRing rows ahead, so that enough of them are
// on their way whatever registers hold (16384 x 4096: 102 us with the next row in
// registers, and more of them spilled).  A block's one barrier a row, which its sums need
// anyway, says that the row's place may be filled again.
constexpr int kRing = 4;

template <typename T, typename W, int kE>
__global__ void __launch_bounds__(512) norm_grad_ring_kernel(const NormGradProblem p, int ring) {
  constexpr int kV = kVec<T>, kN = kE / kV;
  extern __shared__ __align__(128) uint8_t rows[];         // [ring][2][d] of T
  __shared__ float parts[2][2][32];
  __shared__ uint64_t full[kRing];
  __shared__ int abort_flag;
  const int t = threadIdx.x, threads = blockDim.x;
  const int d = static_cast<int>(p.d);
  const uint32_t bytes = static_cast<uint32_t>(d * sizeof(T));
  const float inv_d = 1.0f / static_cast<float>(d);
  if (t == 0) {
    for (int i = 0; i < ring; ++i) sm100::mbar_init(&full[i], 1);
    abort_flag = 0;
    sm100::fence_barrier_init();
  }
  __syncthreads();
  pdl_wait();
  if (p.gw != nullptr || p.gb != nullptr) pdl_launch_dependents();     // (norm_sum_kernel, which waits first)
  auto fill = [&](int64_t row, int slot) {
    if (row >= p.n) return;
    uint8_t* at = rows + static_cast<size_t>(slot) * 2 * bytes;
    sm100::mbar_arrive_expect_tx(&full[slot], 2 * bytes);
    sm100::bulk_load(at, static_cast<const T*>(p.x) + row * p.x_stride, bytes, &full[slot]);
    sm100::bulk_load(at + bytes, static_cast<const T*>(p.g) + row * p.g_stride, bytes, &full[slot]);
  };
  const int64_t step = gridDim.x;
  if (t == 0)
    for (int i = 0; i < ring; ++i) fill(blockIdx.x + i * step, i);
  float w[kN][kV], gw[kN][kV], gb[kN][kV];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int c = (i * threads + t) * kV;
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      gw[i][j] = gb[i][j] = 0.0f;
      w[i][j] = 1.0f;
    }
    if (p.weight != nullptr && c < d) load_weights<W, kV>(static_cast<const W*>(p.weight) + c, w[i]);
  }
  int turn = 0, slot = 0;
  uint32_t phase = 0;
  bool stopped = false;                                    // (thread 0 asks for no more rows)
  float next_mean = p.rms ? 0.0f : p.mean[blockIdx.x], next_rstd = p.rstd[blockIdx.x];
#pragma unroll 1
  for (int64_t row = blockIdx.x; row < p.n; row += step) {
    const float mean = next_mean, rstd = next_rstd;
    if (row + step < p.n) {                                // (a row ahead: the loads take as long as a row)
      next_mean = p.rms ? 0.0f : p.mean[row + step];
      next_rstd = p.rstd[row + step];
    }
    // (a wait that gives up leaves the error word set, and the block's further ones
    // do not wait: it goes on with whatever lies there, so that its barriers stay
    // whole.  Thread 0 then lets the rows on their way land and asks for no more.
    // All of it behind the first look at the barrier: 80.5 us with a flag of each
    // thread's own ahead of it, 79.2 so.)
    if (!sm100::mbar_try_wait(sm100::smem_u32(&full[slot]), phase)) {
      const bool given_up = *static_cast<volatile int*>(&abort_flag) != 0;
      if ((given_up || !sm100::mbar_wait(&full[slot], phase, p.err, &abort_flag)) && t == 0 && !stopped) {
        stopped = true;
        volatile int no_abort = 0;
        for (int i = 0, at = slot, of = phase; i < ring && row + i * step < p.n; ++i) {
          sm100::mbar_wait(&full[at], of, p.err, &no_abort);
          if (++at == ring) { at = 0; of ^= 1; }
        }
      }
    }
    const T* x = reinterpret_cast<const T*>(rows + static_cast<size_t>(slot) * 2 * bytes);
    const T* g = x + d;
    float xh[kN][kV], a[kN][kV];
    float sum_a = 0.0f, sum_ax = 0.0f;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int c = (i * threads + t) * kV;
      if (c < d) {
        unpack<T>(*reinterpret_cast<const uint4*>(x + c), xh[i]);
        unpack<T>(*reinterpret_cast<const uint4*>(g + c), a[i]);
      } else {
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          xh[i][j] = mean;
          a[i][j] = 0.0f;
        }
      }
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
    sum_a = warp_sum(sum_a);
    sum_ax = warp_sum(sum_ax);
    // (two sets in turn: a thread that is a row ahead does not overwrite what another still reads)
    if ((t & 31) == 0) {
      parts[turn][0][t >> 5] = sum_a;
      parts[turn][1][t >> 5] = sum_ax;
    }
    __syncthreads();
    if (t == 0 && !stopped) fill(row + ring * step, slot);
    if (++slot == ring) { slot = 0; phase ^= 1; }
    if (p.gx == nullptr) continue;
    const bool mine = (t & 31) < (threads >> 5);
    sum_a = warp_sum(mine ? parts[turn][0][t & 31] : 0.0f);
    sum_ax = warp_sum(mine ? parts[turn][1][t & 31] : 0.0f);
    turn ^= 1;
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
  if (p.gw == nullptr && p.gb == nullptr) return;
  float* out = p.partials + static_cast<int64_t>(blockIdx.x) * 2 * d;
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

// Sums over the blocks' partials: 32 columns a block of threads, 16 slices of the
// partials, joined in the order of the slices.
constexpr int kSumSlices = 16;

template <typename W>
__global__ void __launch_bounds__(32 * kSumSlices) norm_sum_kernel(const float* partials, int64_t blocks, int64_t d, W* gw,
                                                                   W* gb) {
  __shared__ float sums[kSumSlices][33];
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x % 32;     // of [gw, gb]
  const int slice = threadIdx.x / 32;
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

// Rows of up to 1024 columns (256 where there are up to 512 of them) are one
// warp's, wider ones a block's; a thread takes 8 or 32 elements.
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

// Whether rows of these tensors have the same shift, row by row.
template <typename T>
bool same_shift(const void* a, int64_t a_stride, const void* b, int64_t b_stride) {
  return (reinterpret_cast<uintptr_t>(a) - reinterpret_cast<uintptr_t>(b)) % 16 == 0 && (a_stride - b_stride) % kVec<T> == 0;
}

constexpr int kShiftElements = 16;         // of a row a thread takes where rows are shifted
constexpr int kShiftBlocks = 608;          // a multiple of 8: 4 blocks for each SM of this GPU

template <typename T, typename W>
cudaError_t launch_norm_typed(const NormProblem& p, cudaStream_t stream) {
  constexpr int kV = kVec<T>;
  const int64_t size = sizeof(T);
  const bool vectors = p.d % kV == 0 && aligned16(p.x) && p.x_stride * size % 16 == 0 && aligned16(p.weight) &&
                       aligned16(p.bias) && (p.q != nullptr || (aligned16(p.y) && p.y_stride * size % 16 == 0));
  if (vectors) return launch_norm_of<T, W, kV>(p, stream);
  const int64_t wide = p.d + kV;             // columns with the shift before them
  if (p.q == nullptr && wide <= 1024 * kShiftElements && same_shift<T>(p.x, p.x_stride, p.y, p.y_stride)) {
    if (wide <= 32 * kShiftElements)
      return launch_kernel(norm_shift_kernel<T, W, kShiftElements, true>,
                           dim3(static_cast<unsigned>(std::min<int64_t>((p.n + kRowsPerBlock - 1) / kRowsPerBlock, kShiftBlocks))),
                           dim3(kSmallRow * kRowsPerBlock), 0, stream, true, p);
    return launch_kernel(norm_shift_kernel<T, W, kShiftElements, false>,
                         dim3(static_cast<unsigned>(std::min<int64_t>(p.n, kShiftBlocks))),
                         dim3(threads_for(wide, kShiftElements)), 0, stream, true, p);
  }
  return launch_norm_of<T, W, 1>(p, stream);
}

// Columns a thread of the backward pass takes, and the threads of a row.
struct GradShape {
  int elements, threads;      // threads 32: a warp a row
};

GradShape grad_shape(int64_t width) {
  if (width <= 256) return {8, 32};
  if (width <= 1024) return {32, 32};
  if (width <= 512 * 16) return {16, threads_for(width, 16)};
  return {32, threads_for(width, 32)};
}

constexpr int64_t kGradBlocks = 304;       // a multiple of 8: 2 blocks for each SM of this GPU

template <typename T, typename W, int kV, int kE, bool kOneWarp, bool kShift>
cudaError_t launch_grad_as(const NormGradProblem& p, int threads, int64_t* blocks, cudaStream_t stream) {
  *blocks = std::min<int64_t>(kOneWarp ? (p.n + kRowsPerBlock - 1) / kRowsPerBlock : p.n, kGradBlocks);
  return launch_kernel(norm_grad_kernel<T, W, kV, kE, kOneWarp, kShift>, dim3(static_cast<unsigned>(*blocks)),
                       dim3(kOneWarp ? kSmallRow * kRowsPerBlock : threads), 0, stream, true, p);
}

template <typename T, typename W, int kV, bool kShift>
cudaError_t launch_grad_of(const NormGradProblem& p, int64_t* blocks, cudaStream_t stream) {
  const GradShape s = grad_shape(kShift ? p.d + kV : p.d);
  if (s.threads == 32)
    return s.elements == 8 ? launch_grad_as<T, W, kV, 8, true, kShift>(p, 32, blocks, stream)
                           : launch_grad_as<T, W, kV, 32, true, kShift>(p, 32, blocks, stream);
  return s.elements == 16 ? launch_grad_as<T, W, kV, 16, false, kShift>(p, s.threads, blocks, stream)
                          : launch_grad_as<T, W, kV, 32, false, kShift>(p, s.threads, blocks, stream);
}

// The ring takes whole rows of more than a warp's, where two of them fit.
constexpr int kRingBytes = 96 * 1024;      // a block's, of which two are on an SM

template <typename T, typename W>
cudaError_t launch_grad_ring(const NormGradProblem& p, int64_t* blocks, cudaStream_t stream) {
  const int bytes = static_cast<int>(2 * p.d * sizeof(T)), ring = std::min(kRing, kRingBytes / bytes);
  *blocks = std::min<int64_t>(p.n, kGradBlocks);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = raise_smem_limit<norm_grad_ring_kernel<T, W, 16>>(dev, kRingBytes);
  if (e != cudaSuccess) return e;
  return launch_kernel(norm_grad_ring_kernel<T, W, 16>, dim3(static_cast<unsigned>(*blocks)), dim3(threads_for(p.d, 16)),
                       ring * bytes, stream, true, p, ring);
}

template <typename T, typename W>
cudaError_t launch_grad_typed(const NormGradProblem& p, cudaStream_t stream) {
  constexpr int kV = kVec<T>;
  const int64_t size = sizeof(T);
  const bool vectors = p.d % kV == 0 && aligned16(p.x) && p.x_stride * size % 16 == 0 && aligned16(p.weight) &&
                       aligned16(p.g) && p.g_stride * size % 16 == 0 && aligned16(p.gx) &&
                       (p.gx == nullptr || p.gx_stride * size % 16 == 0);
  const bool shifted = p.d + kV <= kNormMaxWidth && same_shift<T>(p.x, p.x_stride, p.g, p.g_stride) &&
                       (p.gx == nullptr || same_shift<T>(p.x, p.x_stride, p.gx, p.gx_stride));
  int64_t blocks = 0;
  const bool ring = vectors && p.d > 1024 && p.d <= 512 * 16 && 4 * p.d * size <= kRingBytes && p.n > kGradBlocks;
  const cudaError_t e = ring      ? launch_grad_ring<T, W>(p, &blocks, stream)
                        : vectors ? launch_grad_of<T, W, kV, false>(p, &blocks, stream)
                        : shifted ? launch_grad_of<T, W, kV, true>(p, &blocks, stream)
                                  : launch_grad_of<T, W, 1, false>(p, &blocks, stream);
  if (e != cudaSuccess || (p.gw == nullptr && p.gb == nullptr)) return e;
  return launch_kernel(norm_sum_kernel<W>, dim3(static_cast<unsigned>((2 * p.d + 31) / 32)), dim3(32 * kSumSlices), 0, stream,
                       true, static_cast<const float*>(p.partials), blocks, p.d, static_cast<W*>(p.gw),
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

int64_t norm_grad_blocks(int64_t n) { return std::min(n, kGradBlocks); }

cudaError_t launch_norm_grad(const NormGradProblem& p, cudaStream_t stream) {
  return by_types(p.x_type, p.w_type, [&](auto x, auto w) { return launch_grad_typed<decltype(x), decltype(w)>(p, stream); });
}

}  // namespace fs
