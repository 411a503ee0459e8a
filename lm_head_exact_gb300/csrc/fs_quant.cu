// Quantising to 8 bits with a scale for each block of 128:
//
//   scale = max(amax / largest, 2^-100),  q = nearest even(x * (1 / scale))
//
// for blocks of 1 x 128 or 128 x 128 of the matrix or of its transpose.  What
// bounds it is memory: 2 (or 4) bytes read and 1 written per element, each
// once.  A block of 256 threads takes a tile of up to 128 rows x 128 columns into
// registers as it lies in memory, 8 elements of a row a thread and load, finds the
// blocks' largest values by shuffles (and through shared memory where a block
// spans the warps), and writes whole 128-byte lines; the transpose's bytes cross
// shared memory, swizzled so that neither side meets bank conflicts.
#include "fs_fp8.cuh"
#include "fs_fp8.h"

namespace fs {
namespace {

constexpr int kThreads = 256;
constexpr int kCols = 128;                 // of x a tile takes
constexpr int kGroup = 8;                  // elements of a row a thread takes at a time

// kRows rows a thread: a tile of 16 kRows rows.  Thread t holds columns
// 8 (t % 16) .. + 7 of rows kRows (t / 16) .. of the tile.
template <typename T, int kType, int kRows, bool kTranspose, bool kSquare>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const QuantProblem p, bool aligned) {
  constexpr bool kTile = kTranspose || kSquare;          // a whole 128 x 128 block is needed
  static_assert(!kTile || kRows == 8, "a tile of 128 rows");
  __shared__ __align__(16) Tops<T> tops[kSquare || kTranspose ? 8 : 1][kTranspose && !kSquare ? 16 : 1];
  __shared__ __align__(16) uint8_t bytes[kTranspose ? kCols * 128 : 16];
  const int lane = threadIdx.x & 31;
  const int col_in = (threadIdx.x & 15) * kGroup;
  const int row_in = (threadIdx.x >> 4) * kRows;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * kCols + col_in;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * 16 * kRows + row_in;
  pdl_wait_then_launch();
  Eight<T> v[kRows];
  const T* src = static_cast<const T*>(p.x) + r0 * p.x_stride + c0;
#pragma unroll
  for (int i = 0; i < kRows; ++i)
#pragma unroll
    for (int h = 0; h < 8 / kVec<T>; ++h) v[i].raw[h] = make_uint4(0u, 0u, 0u, 0u);
  if (aligned && c0 + kGroup <= p.cols) {
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (r0 + i < p.rows) {
#pragma unroll
        for (int h = 0; h < 8 / kVec<T>; ++h) v[i].raw[h] = reinterpret_cast<const uint4*>(src + i * p.x_stride)[h];
      }
  } else {
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int j = 0; j < kGroup; ++j)
        if (r0 + i < p.rows && c0 + j < p.cols) reinterpret_cast<T*>(v[i].raw)[j] = src[i * p.x_stride + j];
  }
  constexpr float kLargest = fp8_largest(kType);
  float inverse[kTranspose && !kSquare ? kGroup : kSquare ? 1 : kRows];
  if constexpr (kSquare || kTranspose) {
    Tops<T> top;
    top.clear();
#pragma unroll
    for (int i = 0; i < kRows; ++i) top.add(v[i]);
    top.join(16);
    if constexpr (kSquare) {
      float all[1] = {top.all()};
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) all[0] = fmaxf(all[0], __shfl_xor_sync(0xffffffffu, all[0], o));
      float* shared = reinterpret_cast<float*>(tops);
      if (lane == 0) shared[threadIdx.x >> 5] = all[0];
      __syncthreads();
#pragma unroll
      for (int w = 0; w < 8; ++w) all[0] = fmaxf(all[0], shared[w]);
      const BlockScale s = block_scale(all[0], kLargest);
      inverse[0] = s.inverse;
      if (threadIdx.x == 0)
        p.scale[(kTranspose ? blockIdx.x : blockIdx.y) * p.s_row + (kTranspose ? blockIdx.y : blockIdx.x) * p.s_col] = s.scale;
    } else {
      // the blocks lie along x's rows: one for each column of the tile
      if (lane < 16) tops[threadIdx.x >> 5][lane] = top;
      __syncthreads();
      float* scales = reinterpret_cast<float*>(bytes);   // (until the bytes are put down)
      if (threadIdx.x < kCols) {
        float m = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) m = fmaxf(m, tops[w][threadIdx.x >> 3].column(threadIdx.x & 7));
        const BlockScale s = block_scale(m, kLargest);
        scales[threadIdx.x] = s.inverse;
        const int64_t c = static_cast<int64_t>(blockIdx.x) * kCols + threadIdx.x;
        if (c < p.cols) p.scale[c * p.s_row + blockIdx.y * p.s_col] = s.scale;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kGroup; ++j) inverse[j] = scales[col_in + j];
      __syncthreads();
    }
  } else {
    float top[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      Tops<T> t;
      t.clear();
      t.add(v[i]);
      top[i] = t.all();
    }
    const BlockScale s = spread_scale<kRows>(top, lane, kLargest);
    constexpr int kEach = 16 / kRows;                      // lanes that hold a row's scale
    const int64_t row = r0 + (lane & 15) / kEach;
    if (lane % kEach == 0 && row < p.rows) p.scale[row * p.s_row + blockIdx.x * p.s_col] = s.scale;
#pragma unroll
    for (int i = 0; i < kRows; ++i) inverse[i] = spread_get<kRows>(s.inverse, i, lane);
  }
  uint8_t* q = static_cast<uint8_t*>(p.q);
  if constexpr (!kTranspose) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (r0 + i >= p.rows) break;
      const float by = inverse[kSquare ? 0 : i];
      const uint2 o = make_uint2(fp8_quad<kType>(v[i].value(0), v[i].value(1), v[i].value(2), v[i].value(3), by),
                                 fp8_quad<kType>(v[i].value(4), v[i].value(5), v[i].value(6), v[i].value(7), by));
      uint8_t* dst = q + (r0 + i) * p.q_stride + c0;
      if (c0 + kGroup <= p.cols) {
        *reinterpret_cast<uint2*>(dst) = o;
      } else {
        const uint8_t* e = reinterpret_cast<const uint8_t*>(&o);
#pragma unroll
        for (int j = 0; j < kGroup; ++j)
          if (c0 + j < p.cols) dst[j] = e[j];
      }
    }
  } else {
    // row c of the transposed tile: 16 groups of 8 bytes, group g at place
    // g ^ (c / 8), so that the 16 lanes of a store lie in different banks
#pragma unroll
    for (int j = 0; j < kGroup; ++j) {
      const float by = inverse[kSquare ? 0 : j];
      const int place = (threadIdx.x >> 4) ^ ((col_in >> 3) & 15);
      *reinterpret_cast<uint2*>(bytes + (col_in + j) * 128 + place * 8) =
          make_uint2(fp8_quad<kType>(v[0].value(j), v[1].value(j), v[2].value(j), v[3].value(j), by),
                     fp8_quad<kType>(v[4].value(j), v[5].value(j), v[6].value(j), v[7].value(j), by));
    }
    __syncthreads();
    const int64_t t0 = static_cast<int64_t>(blockIdx.y) * 128;            // first column of q's tile
#pragma unroll
    for (int k = 0; k < 4; ++k) {                                         // 128 rows x 8 pairs of groups
      const int at = k * kThreads + threadIdx.x;
      const int c = at >> 3, pair = at & 7;
      const int64_t col = static_cast<int64_t>(blockIdx.x) * kCols + c;
      if (col >= p.cols) break;
      const int turn = (c >> 3) & 15;
      uint4 o = *reinterpret_cast<const uint4*>(bytes + c * 128 + ((2 * pair ^ turn) & ~1) * 8);
      if (turn & 1) o = make_uint4(o.z, o.w, o.x, o.y);
      uint8_t* dst = q + col * p.q_stride + t0 + pair * 16;
      const int64_t left = p.rows - t0 - pair * 16;
      if (left >= 16) {
        *reinterpret_cast<uint4*>(dst) = o;
      } else {
        const uint8_t* e = reinterpret_cast<const uint8_t*>(&o);
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (j < left) dst[j] = e[j];
      }
    }
  }
}

template <typename T, int kType, int kRows, bool kTranspose, bool kSquare>
cudaError_t launch_tiles(const QuantProblem& p, cudaStream_t stream) {
  const bool aligned = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && p.x_stride * static_cast<int64_t>(sizeof(T)) % 16 == 0;
  const int64_t across = (p.cols + kCols - 1) / kCols, rows = 16 * kRows;
  // the grid's second axis ends at 65535 tiles
  const int64_t slice = 65535 * rows;
  for (int64_t r = 0; r < p.rows; r += slice) {
    QuantProblem s = p;
    s.rows = p.rows - r < slice ? p.rows - r : slice;
    s.x = static_cast<const T*>(p.x) + r * p.x_stride;
    s.q = static_cast<uint8_t*>(p.q) + (kTranspose ? r : r * p.q_stride);
    const int64_t block = kTranspose ? r / kQuantBlock * p.s_col : kSquare ? r / kQuantBlock * p.s_row : r * p.s_row;
    s.scale = p.scale + block;
    const cudaError_t e =
        launch_kernel(quantize_kernel<T, kType, kRows, kTranspose, kSquare>,
                      dim3(static_cast<unsigned>(across), static_cast<unsigned>((s.rows + rows - 1) / rows)), dim3(kThreads),
                      0, stream, true, s, aligned);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename T, int kType>
cudaError_t launch_typed(const QuantProblem& p, cudaStream_t stream) {
  const bool square = p.block_rows == kQuantBlock;
  if (p.transpose)
    return square ? launch_tiles<T, kType, 8, true, true>(p, stream) : launch_tiles<T, kType, 8, true, false>(p, stream);
  if (square) return launch_tiles<T, kType, 8, false, true>(p, stream);
  // few rows: one row a thread, so that there are more blocks of threads
  return p.rows * quant_blocks(p.cols) < 16384 ? launch_tiles<T, kType, 1, false, false>(p, stream)
                                               : launch_tiles<T, kType, 8, false, false>(p, stream);
}

template <typename T>
cudaError_t launch_from(const QuantProblem& p, cudaStream_t stream) {
  return p.q_type == FS_TYPE_E5M2 ? launch_typed<T, FS_TYPE_E5M2>(p, stream) : launch_typed<T, FS_TYPE_E4M3>(p, stream);
}

}  // namespace

cudaError_t launch_quantize(const QuantProblem& p, cudaStream_t stream) {
  switch (p.x_type) {
    case FS_TYPE_BF16: return launch_from<__nv_bfloat16>(p, stream);
    case FS_TYPE_F16: return launch_from<__half>(p, stream);
    default: return launch_from<float>(p, stream);
  }
}

}  // namespace fs
