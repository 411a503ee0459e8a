// Clipped policy loss with a KL penalty: the loss, its terms and its gradient
// with respect to the log-probabilities, in one pass over the tokens.
//
//   r = exp(logp - old), q = ref - logp, weight w of the token
//   loss += w (-min(r A, clip(r) A) + kl (e^q - 1 - q)),
//   grad  = w (-r A [not clipped] + kl (1 - e^q)).
//
// Each token is read once and its gradient written once (8 bytes in, up to 17
// with reference, advantage and mask by token, and 4 out).  The weights need the number of tokens that take part: with a mask or
// a mean over sequences a counting launch goes first, which reads the mask
// only (one byte a token).
#include <algorithm>

#include "fs_train.h"

namespace fs {
namespace {

constexpr int kThreads = 256;
constexpr int kCountThreads = 512;
constexpr int kFlush = 16;                      // rounds of 4 tokens a thread that stay in fp32
constexpr int kBlocksPerSm = 3;

__device__ __forceinline__ int bytes_set(uint32_t w) {
  return __popc(__vcmpne4(w, 0u) & 0x01010101u);
}

// Bytes that are not zero in mask[lo, hi), over the block's threads (each
// returns its own share).
__device__ long long count_range(const uint8_t* mask, int64_t lo, int64_t hi, int tid, int threads) {
  long long c = 0;
  const int64_t a = min(hi, lo + static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(mask + lo) & 15)) & 15));
  const int64_t b = a + (hi - a) / 16 * 16;
  for (int64_t i = lo + tid; i < a; i += threads) c += mask[i] != 0;
  for (int64_t i = a + static_cast<int64_t>(tid) * 16; i < b; i += static_cast<int64_t>(threads) * 16) {
    const uint4 w = *reinterpret_cast<const uint4*>(mask + i);
    c += bytes_set(w.x) + bytes_set(w.y) + bytes_set(w.z) + bytes_set(w.w);
  }
  for (int64_t i = b + tid; i < hi; i += threads) c += mask[i] != 0;
  return c;
}

template <int kBlock>
__device__ long long block_sum(long long v) {
  __shared__ long long part[kBlock / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
  for (int i = 0; i < kBlock / 32; ++i) v += part[i];
  __syncthreads();
  return v;
}

// Tokens that take part: of each sequence (a block each) and the number of
// sequences that have any, or of the whole batch.  Whole numbers, so the order
// of the atomic additions does not matter.
__global__ void __launch_bounds__(kCountThreads) policy_count_kernel(const PolicyProblem p) {
  pdl_launch_dependents();
  pdl_wait();
  if (p.mean == FS_MEAN_SEQUENCE) {
    for (int64_t s = blockIdx.x; s < p.n_seqs; s += gridDim.x) {
      int64_t lo = p.starts != nullptr ? p.starts[s] : s * p.row_len;
      int64_t hi = p.starts != nullptr ? p.starts[s + 1] : lo + p.row_len;
      lo = max(static_cast<int64_t>(0), min(lo, p.N));        // no read outside whatever the offsets hold
      hi = max(lo, min(hi, p.N));
      const long long c = p.mask == nullptr
                              ? hi - lo
                              : block_sum<kCountThreads>(count_range(p.mask, lo, hi, threadIdx.x, kCountThreads));
      if (threadIdx.x == 0) {
        p.counts[s] = static_cast<float>(c);              // (a sequence may pass 2^31 tokens)
        if (c > 0) atomicAdd(&p.scratch->count, 1ull);
      }
    }
  } else {
    const int64_t per = ((p.N + gridDim.x - 1) / gridDim.x + 15) / 16 * 16;
    const int64_t lo = min(p.N, static_cast<int64_t>(blockIdx.x) * per), hi = min(p.N, lo + per);
    const long long c = block_sum<kCountThreads>(count_range(p.mask, lo, hi, threadIdx.x, kCountThreads));
    if (threadIdx.x == 0 && c > 0) atomicAdd(&p.scratch->count, static_cast<unsigned long long>(c));
  }
}

// e^q - 1 - q (kl) and e^q - 1 (em1).  For small q the differences lose what
// they are made of (q = 0.01: 5e-5 of two terms near 0.01), so kl is summed from
// its Taylor series there -- the first term left out, q^10 / 10!, is below
// 2^-27 of q^2 / 2 for |q| <= 1/2 -- and em1 is q + kl.  Beyond, the
// differences keep all but 3 of their bits.
__device__ __forceinline__ void kl_terms(float q, float& kl, float& em1) {
  float s = 1.0f / 362880.0f;
  s = fmaf(s, q, 1.0f / 40320.0f);
  s = fmaf(s, q, 1.0f / 5040.0f);
  s = fmaf(s, q, 1.0f / 720.0f);
  s = fmaf(s, q, 1.0f / 120.0f);
  s = fmaf(s, q, 1.0f / 24.0f);
  s = fmaf(s, q, 1.0f / 6.0f);
  s = fmaf(s, q, 0.5f);
  kl = s * q * q;
  em1 = fmaf(s * q, q, q);
  if (!(fabsf(q) <= 0.5f)) {
    em1 = expf(q) - 1.0f;
    kl = em1 - q;
  }
}

// Whether a token of advantage A is clipped: logp - old above hi (A > 0) or
// below lo (A < 0).  The borders are held as sums of two fp32 numbers, x the
// nearest one.  Rounding keeps order, so the fp32 difference d decides unless
// it equals x; then its own rounding error (exact in fp32) is compared with y.
// FP64 instructions would decide the same, but they alone took 60 us for 4.2 M
// tokens.
__device__ __forceinline__ bool is_clipped(float A, float d, float logp, float old, float2 hi, float2 lo) {
  bool above = d > hi.x, below = d < lo.x;
  if (d == hi.x || d == lo.x) {
    const float v = logp - d;                   // d + err = logp - old, exactly
    const float err = (logp - (d + v)) + (v - old);
    above |= d == hi.x && err > hi.y;
    below |= d == lo.x && err < lo.y;
  }
  return A > 0.0f ? above : A < 0.0f && below;
}

// Sums of one thread over kFlush rounds, in fp32; they are added up in fp64.
struct Sums {
  float policy, kl, clipped;
};

struct Weights {
  float token;                  // FS_MEAN_TOKEN / FS_MEAN_NONE: the same for every token
  float seqs;                   // FS_MEAN_SEQUENCE: sequences that have tokens
};

// The sequence that token i belongs to: the last one that starts at or before
// it.  Always in [0, n_seqs), whatever the offsets hold.
__device__ __forceinline__ int64_t sequence_of(const PolicyProblem& p, int64_t i) {
  if (p.starts == nullptr)
    return p.N < (int64_t(1) << 31) ? static_cast<uint32_t>(i) / static_cast<uint32_t>(p.row_len) : i / p.row_len;
  int64_t lo = 0, hi = p.n_seqs;                // starts[lo] <= i < starts[hi]
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    if (p.starts[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

// What tokens [i, i + kVec) of one thread hold.
template <int kVec>
struct Loaded {
  float lp[kVec], old[kVec], ref[kVec], adv[kVec];
  bool on[kVec];

  __device__ __forceinline__ void load(const PolicyProblem& p, int64_t i) {
    if constexpr (kVec == 4) {
      const float4 a = __ldcs(reinterpret_cast<const float4*>(p.logp + i));
      const float4 b = __ldcs(reinterpret_cast<const float4*>(p.old_logp + i));
      float4 c = make_float4(0.0f, 0.0f, 0.0f, 0.0f), e = c;
      uchar4 m = make_uchar4(1, 1, 1, 1);
      if (p.ref_logp != nullptr) c = __ldcs(reinterpret_cast<const float4*>(p.ref_logp + i));
      if (!p.adv_per_seq) e = __ldcs(reinterpret_cast<const float4*>(p.adv + i));
      if (p.mask != nullptr) m = __ldcs(reinterpret_cast<const uchar4*>(p.mask + i));
      lp[0] = a.x; lp[1] = a.y; lp[2] = a.z; lp[3] = a.w;
      old[0] = b.x; old[1] = b.y; old[2] = b.z; old[3] = b.w;
      ref[0] = c.x; ref[1] = c.y; ref[2] = c.z; ref[3] = c.w;
      adv[0] = e.x; adv[1] = e.y; adv[2] = e.z; adv[3] = e.w;
      on[0] = m.x != 0; on[1] = m.y != 0; on[2] = m.z != 0; on[3] = m.w != 0;
    } else {
      lp[0] = p.logp[i];
      old[0] = p.old_logp[i];
      ref[0] = p.ref_logp != nullptr ? p.ref_logp[i] : 0.0f;
      adv[0] = p.adv_per_seq ? 0.0f : p.adv[i];
      on[0] = p.mask == nullptr || p.mask[i] != 0;
    }
  }
};

// Their terms and gradients.  Masked tokens go through the arithmetic like the
// others and are selected away (their values may be NaN): branches around them
// would split nearly every warp.
// kBySeq: something depends on the token's sequence (its advantage or weight).
template <int kVec, bool kBySeq>
__device__ __forceinline__ void tokens(const PolicyProblem& p, const Weights& w, int64_t i, const Loaded<kVec>& x,
                                       Sums& sums) {
  int64_t s = kBySeq ? sequence_of(p, i) : 0;
  int64_t end = 0;
  if (kBySeq) end = p.starts != nullptr ? p.starts[s + 1] : (s + 1) * p.row_len;
  float seq_adv = 0.0f, weight = w.token;
  auto enter = [&]() {
    if (p.adv_per_seq) seq_adv = p.adv[s];
    if (p.mean == FS_MEAN_SEQUENCE) weight = 1.0f / (p.counts[s] * w.seqs);
  };
  if (kBySeq) enter();
  float policy = 0.0f, kl = 0.0f, clipped = 0.0f, g[kVec];
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    while (kBySeq && i + j >= end && s + 1 < p.n_seqs) {       // into the next sequence that has tokens
      ++s;
      end = p.starts != nullptr ? p.starts[s + 1] : end + p.row_len;
      if (i + j < end) enter();
    }
    const float A = kBySeq && p.adv_per_seq ? seq_adv : x.adv[j];
    const float d = x.lp[j] - x.old[j];
    const bool cut = is_clipped(A, d, x.lp[j], x.old[j], p.log_hi, p.log_lo);
    float rA = expf(d) * A;
    if (d > 88.0f) {                             // where e^d may pass fp32's range and r A does not
      const float half = expf(0.5f * d);
      rA = A == 0.0f && d < INFINITY ? 0.0f : A * half * half;
    }
    const float term = cut ? (A > 0.0f ? p.hi : p.lo) * A : rA;
    policy = x.on[j] ? fmaf(-term, weight, policy) : policy;
    float grad = cut ? 0.0f : -rA;
    clipped += x.on[j] && cut ? weight : 0.0f;
    if (p.ref_logp != nullptr) {
      float estimate, em1;
      kl_terms(x.ref[j] - x.lp[j], estimate, em1);
      kl = x.on[j] ? fmaf(estimate, weight, kl) : kl;
      grad = p.kl_coef != 0.0f ? fmaf(-p.kl_coef, em1, grad) : grad;      // (em1 may be infinite)
    }
    g[j] = x.on[j] ? grad * weight : 0.0f;
  }
  sums.policy += policy;
  sums.kl += kl;
  sums.clipped += clipped;
  if constexpr (kVec == 4)
    __stcs(reinterpret_cast<float4*>(p.grad + i), make_float4(g[0], g[1], g[2], g[3]));
  else
    p.grad[i] = g[0];
}

// The block's sums of three values, added in fp64 in a fixed order: a warp for
// each value, 8 of them a lane and then the lanes as a tree.  FP64 additions
// are few and slow here, so the chain of 13 counts: one of 40 made the
// smallest call 4 us longer.
template <typename T>
__device__ void block_sums(const T (&mine)[3], double (&total)[3]) {
  __shared__ T all[3][kThreads];
  __shared__ double sum[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) all[k][threadIdx.x] = mine[k];
  __syncthreads();
  const int k = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (k < 3) {
    double v = 0.0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) v += static_cast<double>(all[k][lane + 32 * i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) sum[k] = v;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) total[k] = sum[k];
  __syncthreads();
}

template <bool kAligned, bool kBySeq>
__global__ void __launch_bounds__(kThreads) policy_loss_kernel(const PolicyProblem p, const bool counted) {
  __shared__ bool last;
  Sums sums{0.0f, 0.0f, 0.0f};
  double v[3] = {0.0, 0.0, 0.0}, t[3];
  constexpr int kVec = kAligned ? 4 : 1;
  const int64_t items = p.N / kVec;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
  int64_t k = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  Loaded<kVec> now, then;
  if (k < items) now.load(p, k * kVec);
  // The counting kernel starts after whatever wrote the inputs has ended, so
  // only its counts are waited for, with the first loads in flight.
  pdl_wait();
  Weights w{1.0f, 1.0f};
  const unsigned long long count = counted ? *reinterpret_cast<volatile unsigned long long*>(&p.scratch->count) : 0ull;
  if (p.mean == FS_MEAN_TOKEN) w.token = 1.0f / static_cast<float>(counted ? max(count, 1ull) : p.N);
  if (p.mean == FS_MEAN_SEQUENCE) w.seqs = static_cast<float>(count);
  if (kAligned && k < p.N - items * kVec) {      // the last few tokens
    Loaded<1> x;
    x.load(p, items * kVec + k);
    tokens<1, kBySeq>(p, w, items * kVec + k, x, sums);
  }
  for (int round = 1; k - threadIdx.x < items; k += stride, ++round) {
    if (k + stride < items) then.load(p, (k + stride) * kVec);     // in flight while this round computes
    if (k < items) tokens<kVec, kBySeq>(p, w, k * kVec, now, sums);
    now = then;
    if (round % kFlush == 0) {                   // long sums do not stay in fp32
      block_sums({sums.policy, sums.kl, sums.clipped}, t);
#pragma unroll
      for (int j = 0; j < 3; ++j) v[j] += t[j];
      sums = Sums{0.0f, 0.0f, 0.0f};
    }
  }
  block_sums({sums.policy, sums.kl, sums.clipped}, t);
#pragma unroll
  for (int k = 0; k < 3; ++k) t[k] += v[k];
  if (gridDim.x > 1) {
    if (threadIdx.x == 0) {
      double* mine = p.scratch->sums[blockIdx.x];
      for (int k = 0; k < 3; ++k) mine[k] = t[k];
      __threadfence();
      last = atomicAdd(&p.scratch->ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    // the block that finishes last adds the blocks' sums, in their order
    __threadfence();
    for (int k = 0; k < 3; ++k) v[k] = 0.0;
    for (unsigned b = threadIdx.x; b < gridDim.x; b += kThreads) {
#pragma unroll
      for (int k = 0; k < 3; ++k) v[k] += __ldcg(&p.scratch->sums[b][k]);
    }
    block_sums(v, t);
  }
  if (threadIdx.x == 0) {
    p.stats[0] = static_cast<float>(p.kl_coef != 0.0f ? t[0] + static_cast<double>(p.kl_coef) * t[1] : t[0]);
    p.stats[1] = static_cast<float>(t[0]);
    p.stats[2] = static_cast<float>(t[1]);
    p.stats[3] = static_cast<float>(t[2]);
    p.scratch->ticket = 0;
    p.scratch->count = 0;
  }
}

bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace

cudaError_t launch_policy_loss(const PolicyProblem& p, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const bool counted = p.mean == FS_MEAN_SEQUENCE || (p.mean == FS_MEAN_TOKEN && p.mask != nullptr);
  if (counted) {
    const int64_t want = p.mean == FS_MEAN_SEQUENCE ? p.n_seqs : (p.N + kCountThreads * 16 - 1) / (kCountThreads * 16);
    e = launch_kernel(policy_count_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(want, 4 * sms))),
                      dim3(kCountThreads), 0, stream, false, p);
    if (e != cudaSuccess) return e;
  }
  const bool vec = aligned_to(p.logp, 16) && aligned_to(p.old_logp, 16) && aligned_to(p.ref_logp, 16) &&
                   (p.adv_per_seq || aligned_to(p.adv, 16)) && aligned_to(p.mask, 4) && aligned_to(p.grad, 16);
  const int64_t items = vec ? (p.N + 3) / 4 : p.N;
  const int64_t blocks = std::min<int64_t>({(items + kThreads - 1) / kThreads, kBlocksPerSm * sms, kTrainMaxBlocks});
  const bool by_seq = p.adv_per_seq || p.mean == FS_MEAN_SEQUENCE;
  const auto kernel = vec ? (by_seq ? policy_loss_kernel<true, true> : policy_loss_kernel<true, false>)
                          : (by_seq ? policy_loss_kernel<false, true> : policy_loss_kernel<false, false>);
  if (counted && api_later_launch_fails())
    e = cudaErrorLaunchOutOfResources;
  else
    e = launch_kernel(kernel, dim3(static_cast<unsigned>(std::max<int64_t>(blocks, 1))), dim3(kThreads), 0, stream,
                      counted, p, counted);
  // The loss kernel would have left the count at zero for the next call.
  if (e != cudaSuccess && counted &&
      cudaMemsetAsync(&p.scratch->count, 0, sizeof(p.scratch->count), stream) != cudaSuccess)
    cudaGetLastError();
  return e;
}

}  // namespace fs
