// The global norm of many gradients and their scaling.
//
// Two launches: every block sums the squares (or takes the largest magnitude)
// of its chunks, the last block to finish turns the blocks' sums into the norm
// and the factor, and a second launch scales.  Bytes: every element is read
// twice and written once, except that the scaling launch walks the chunks from
// the last to the first, so what the first launch left in L2 is not read from
// HBM again.
//
// The tensors travel as a table in the kernel's parameters: no copy to the
// device, so the calls can be captured in a graph.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "fs_train.h"

namespace fs {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 16384;            // elements of one chunk: 32 KB of 16-bit, 64 KB of 32-bit

struct Entry {
  const void* g;
  void* o;
  int64_t n;
  int32_t first_chunk;                   // chunks of the tensors before it in this launch
  int32_t type;
};

template <int kEntries>
struct Table {
  Entry e[kEntries];
  int32_t n;
  int32_t chunks;
};

struct NormArgs {
  TrainScratch* scratch;
  float* norm;
  double max_norm;
  bool first, last;                      // of the launches that share one norm
};

template <int kEntries>
__device__ __forceinline__ const Entry& entry_of(const Table<kEntries>& t, int chunk) {
  int lo = 0, hi = t.n;                  // e[lo].first_chunk <= chunk < e[hi].first_chunk
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.e[mid].first_chunk <= chunk) lo = mid; else hi = mid;
  }
  return t.e[lo];
}

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float(float v) { return v; }
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float(float v) { return __float2half_rn(v); }

// 16 bytes as the elements they hold.
template <typename T>
union Pack {
  uint4 raw;
  T v[16 / sizeof(T)];
  __device__ Pack() {}
};

template <bool kMax>
__device__ __forceinline__ void accumulate(float& acc, float x) {
  if constexpr (kMax)
    acc = (x != x || acc != acc) ? NAN : fmaxf(acc, fabsf(x));
  else
    acc = fmaf(x, x, acc);
}

// Elements of [p, p + len) before the first 16-byte boundary.
template <typename T>
__device__ __forceinline__ int head_of(const T* p, int len) {
  return min(len, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / static_cast<int>(sizeof(T)));
}

// A thread's share of one chunk: the sum of its squares, or its largest
// magnitude (NaN if there is one).  Tensors that are views into a flat buffer
// begin anywhere: a few elements are taken one by one, so that the rest goes
// in 16-byte loads (one by one throughout, norm and scaling of 107 MB of fp32
// took 72 us instead of 45).
template <typename T, bool kMax>
__device__ __forceinline__ float chunk_norm(const T* g, int len) {
  constexpr int kPer = 16 / sizeof(T);
  float acc = 0.0f;
  const int head = head_of(g, len);
  if (static_cast<int>(threadIdx.x) < head) accumulate<kMax>(acc, to_float(g[threadIdx.x]));
  g += head;
  len -= head;
  const int packs = len / kPer;
  constexpr int kFlight = 8;             // loads written together (at 30 registers not all of them are in flight)
  for (int i = threadIdx.x; i < packs; i += kThreads * kFlight) {
    Pack<T> x[kFlight];
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const int at = i + k * kThreads;
      x[k].raw = at < packs ? reinterpret_cast<const uint4*>(g)[at] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < kFlight; ++k)
#pragma unroll
      for (int j = 0; j < kPer; ++j) accumulate<kMax>(acc, to_float(x[k].v[j]));
  }
  const int tail = packs * kPer + threadIdx.x;
  if (tail < len) accumulate<kMax>(acc, to_float(g[tail]));
  return acc;
}

template <bool kMax>
__device__ double join(double a, double b) {
  if constexpr (kMax) return (a != a || b != b) ? NAN : fmax(a, b);
  return a + b;
}

template <bool kMax>
__device__ double block_join(double v) {
  __shared__ double part[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = join<kMax>(v, __shfl_xor_sync(0xffffffffu, v, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int i = 1; i < kThreads / 32; ++i) v = join<kMax>(v, part[i]);
  __syncthreads();
  return v;                              // valid in thread 0
}

// Squares pass fp32's range for values above 1.8e19 and lose their last bits
// below 2^-126: a block whose sum shows either goes over its chunks once more,
// with the values scaled by a power of two (an infinity among them stays one).
// Rare, so in as little code as it takes: with wide loads, inlined or called,
// it changed the registers of the loop that every call runs (537 MB of bf16:
// 84 us, and 88 with such a call).
template <int kEntries>
__device__ __forceinline__ double squares_scaled(const Table<kEntries>& t, float scale) {
  double total = 0.0;
  for (int c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const Entry& e = entry_of(t, c);
    const int64_t at = static_cast<int64_t>(c - e.first_chunk) * kChunk;
    const int64_t end = min(at + kChunk, e.n);
    float acc = 0.0f;
#pragma unroll 1
    for (int64_t i = at + threadIdx.x; i < end; i += kThreads) {
      const float v = e.type == FS_TYPE_F32    ? static_cast<const float*>(e.g)[i]
                      : e.type == FS_TYPE_BF16 ? to_float(static_cast<const __nv_bfloat16*>(e.g)[i])
                                               : to_float(static_cast<const __half*>(e.g)[i]);
      accumulate<false>(acc, v * scale);
    }
    total += static_cast<double>(acc);
  }
  return total;
}

template <int kEntries, bool kMax>
__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ Table<kEntries> t, const NormArgs a) {
  __shared__ bool last;
  __shared__ float rescale;
  pdl_launch_dependents();
  double total = 0.0;
  for (int c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const Entry& e = entry_of(t, c);
    const int64_t at = static_cast<int64_t>(c - e.first_chunk) * kChunk;
    const int len = static_cast<int>(min(static_cast<int64_t>(kChunk), e.n - at));
    float v;
    if (e.type == FS_TYPE_F32)
      v = chunk_norm<float, kMax>(static_cast<const float*>(e.g) + at, len);
    else if (e.type == FS_TYPE_BF16)
      v = chunk_norm<__nv_bfloat16, kMax>(static_cast<const __nv_bfloat16*>(e.g) + at, len);
    else
      v = chunk_norm<__half, kMax>(static_cast<const __half*>(e.g) + at, len);
    total = join<kMax>(total, static_cast<double>(v));
  }
  total = block_join<kMax>(total);
  if constexpr (!kMax) {
    if (threadIdx.x == 0) rescale = total == INFINITY ? 0x1p-100f : total > 0.0 && total < 0x1p-90 ? 0x1p100f : 0.0f;
    __syncthreads();
    if (rescale != 0.0f)
      total = block_join<false>(squares_scaled(t, rescale)) * (rescale < 1.0f ? 0x1p200 : 0x1p-200);
  }
  if (threadIdx.x == 0) {
    double* mine = &a.scratch->sums[blockIdx.x][0];
    *mine = a.first ? total : join<kMax>(*mine, total);
    __threadfence();
    last = a.last && atomicAdd(&a.scratch->ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double v = 0.0;
  for (unsigned b = threadIdx.x; b < gridDim.x; b += kThreads) v = join<kMax>(v, __ldcg(&a.scratch->sums[b][0]));
  v = block_join<kMax>(v);
  if (threadIdx.x == 0) {
    const double norm = kMax ? v : sqrt(v);
    const double coef = a.max_norm / (norm + 1e-6);
    *a.norm = static_cast<float>(norm);
    // a norm that is not finite scales nothing; one that fp32 cannot hold is
    // finite here, and a factor below fp32's normal range is applied in two steps
    const bool scales = isfinite(norm) && coef < 1.0, small = scales && coef < 0x1p-126;
    a.scratch->first_coef = small ? 0x1p-64f : 1.0f;
    a.scratch->coef = scales ? static_cast<float>(small ? coef * 0x1p64 : coef) : 1.0f;
    a.scratch->ticket = 0;
  }
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const T* g, T* o, int len, float coef) {
  constexpr int kPer = 16 / sizeof(T);
  if (((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(o)) & 15) == 0) {
    const int head = head_of(g, len);
    if (static_cast<int>(threadIdx.x) < head) o[threadIdx.x] = from_float<T>(to_float(g[threadIdx.x]) * coef);
    g += head;
    o += head;
    len -= head;
    const int packs = len / kPer;
    constexpr int kFlight = 8;
    for (int i = threadIdx.x; i < packs; i += kThreads * kFlight) {
      Pack<T> x[kFlight];
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        const int at = i + k * kThreads;
        if (at < packs) x[k].raw = reinterpret_cast<const uint4*>(g)[at];
      }
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        const int at = i + k * kThreads;
        if (at >= packs) break;
#pragma unroll
        for (int j = 0; j < kPer; ++j) x[k].v[j] = from_float<T>(to_float(x[k].v[j]) * coef);
        reinterpret_cast<uint4*>(o)[at] = x[k].raw;
      }
    }
    const int tail = packs * kPer + threadIdx.x;
    if (tail < len) o[tail] = from_float<T>(to_float(g[tail]) * coef);
  } else {                               // no common 16-byte boundary
#pragma unroll 8
    for (int i = threadIdx.x; i < len; i += kThreads) o[i] = from_float<T>(to_float(g[i]) * coef);
  }
}

// The same by two factors, where their product is below fp32's normal range.
template <typename T>
__device__ __noinline__ void chunk_scale_twice(const T* g, T* o, int len, float first, float coef) {
  for (int i = threadIdx.x; i < len; i += kThreads) o[i] = from_float<T>(to_float(g[i]) * first * coef);
}

template <typename T>
__device__ __forceinline__ void chunk_scale_by(const Entry& e, int64_t at, int len, float first, float coef) {
  const T* g = static_cast<const T*>(e.g) + at;
  T* o = static_cast<T*>(e.o) + at;
  if (first == 1.0f)
    chunk_scale(g, o, len, coef);
  else
    chunk_scale_twice(g, o, len, first, coef);
}

template <int kEntries>
__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ Table<kEntries> t,
                                                         const TrainScratch* scratch) {
  pdl_wait();
  const float coef = *reinterpret_cast<const volatile float*>(&scratch->coef);
  const float first = *reinterpret_cast<const volatile float*>(&scratch->first_coef);
  for (int c = t.chunks - 1 - static_cast<int>(blockIdx.x); c >= 0; c -= gridDim.x) {
    const Entry& e = entry_of(t, c);
    if (coef == 1.0f && e.o == e.g) continue;          // in place and unchanged
    const int64_t at = static_cast<int64_t>(c - e.first_chunk) * kChunk;
    const int len = static_cast<int>(min(static_cast<int64_t>(kChunk), e.n - at));
    if (e.type == FS_TYPE_F32)
      chunk_scale_by<float>(e, at, len, first, coef);
    else if (e.type == FS_TYPE_BF16)
      chunk_scale_by<__nv_bfloat16>(e, at, len, first, coef);
    else
      chunk_scale_by<__half>(e, at, len, first, coef);
  }
}

// Kernel parameters hold up to 32,764 bytes: 640 tensors a launch (20 KB).
// Calls of up to 48 tensors take a table of 1.5 KB instead.
constexpr int kManyEntries = 640;
constexpr int kFewEntries = 48;
constexpr int kBlocksPerSm = 4;

template <int kEntries>
cudaError_t run(const void* const* grads, void* const* outs, const int64_t* sizes, const int* types, int n_tensors,
                double max_norm, bool use_max, float* norm, TrainScratch* scratch, int sms, cudaStream_t stream) {
  // tables of up to kEntries tensors and 2^30 chunks
  const int full_grid = std::min(kBlocksPerSm * sms, kTrainMaxBlocks);
  auto fill = [&](Table<kEntries>& t, int from) {
    t.n = 0;
    t.chunks = 0;
    int i = from;
    for (; i < n_tensors && t.n < kEntries; ++i) {
      if (sizes[i] == 0) continue;
      const int64_t chunks = (sizes[i] + kChunk - 1) / kChunk;
      if (t.n > 0 && t.chunks + chunks > (int64_t(1) << 30)) break;
      t.e[t.n++] = Entry{grads[i], outs != nullptr ? outs[i] : nullptr, sizes[i], t.chunks, types[i]};
      t.chunks += static_cast<int32_t>(chunks);
    }
    return i;
  };
  Table<kEntries> t;
  int from = 0;
  bool first = true, single = false;
  do {
    from = fill(t, from);
    const bool last = from == n_tensors;
    single = first && last;
    const int grid = single ? std::max(1, std::min(t.chunks, full_grid)) : full_grid;
    const NormArgs a{scratch, norm, max_norm, first, last};
    const cudaError_t e =
        launch_kernel(use_max ? norm_kernel<kEntries, true> : norm_kernel<kEntries, false>, dim3(grid),
                      dim3(kThreads), 0, stream, false, t, a);
    if (e != cudaSuccess) return e;
    first = false;
  } while (from < n_tensors);
  if (outs == nullptr) return cudaSuccess;
  from = 0;
  do {
    if (!single) from = fill(t, from); else from = n_tensors;
    if (t.chunks > 0) {
      const cudaError_t e = launch_kernel(scale_kernel<kEntries>, dim3(std::min(t.chunks, full_grid)),
                                          dim3(kThreads), 0, stream, single, t,
                                          static_cast<const TrainScratch*>(scratch));
      if (e != cudaSuccess) return e;
    }
  } while (from < n_tensors);
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_clip_grad_norm(const void* const* grads, void* const* outs, const int64_t* sizes, const int* types,
                                  int n_tensors, double max_norm, int norm_type, float* norm, TrainScratch* scratch,
                                  cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const bool use_max = norm_type == FS_NORM_MAX;
  // an infinite bound changes nothing in place: the norm alone
  bool in_place = outs != nullptr;
  for (int i = 0; in_place && i < n_tensors; ++i) in_place = sizes[i] == 0 || outs[i] == grads[i];
  if (in_place && std::isinf(max_norm)) outs = nullptr;
  return n_tensors <= kFewEntries
             ? run<kFewEntries>(grads, outs, sizes, types, n_tensors, max_norm, use_max, norm, scratch, sms, stream)
             : run<kManyEntries>(grads, outs, sizes, types, n_tensors, max_norm, use_max, norm, scratch, sms, stream);
}

}  // namespace fs
