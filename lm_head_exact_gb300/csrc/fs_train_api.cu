// C entry points of the training operators: argument checks, the layout of
// the caller's workspace, and the order of the launches.  Contracts:
// include/flashsample.h.
#include <algorithm>
#include <cmath>
#include <vector>

#include "flashsample.h"
#include "fs_api_util.h"
#include "fs_train.h"

namespace fs {
namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1024;
constexpr size_t kAlign = 256;
size_t aligned(size_t bytes) { return (bytes + kAlign - 1) / kAlign * kAlign; }

// A cursor over the caller's workspace (or, from nullptr, over its size).
struct Layout {
  size_t at = 0;
  template <typename T>
  T* take(void* base, size_t count) {
    T* p = reinterpret_cast<T*>(static_cast<char*>(base) + at);
    at += aligned(count * sizeof(T));
    return p;
  }
};

struct ForwardWorkspace {
  LsePart* parts;
  float* own_x;
  int64_t n_parts;
  size_t bytes;
};

ForwardWorkspace forward_workspace(void* base, int64_t n, int64_t V) {
  Layout l;
  ForwardWorkspace w;
  w.n_parts = head_parts(n, V);
  w.parts = l.take<LsePart>(base, static_cast<size_t>(n) * w.n_parts);
  w.own_x = l.take<float>(base, n);
  w.bytes = l.at;
  return w;
}

// ds is formed for as many vocabulary rows at a time as fit this many bytes:
// the whole vocabulary of a usual micro-batch (2048 rows of 128256 take
// 0.5 GB), a few pieces of a very large one.
constexpr int64_t kMaxDsBytes = int64_t(4) << 30;

int64_t ds_chunk(int64_t n, int64_t V) {
  const int64_t cols = std::max<int64_t>(256, kMaxDsBytes / 2 / std::max<int64_t>(n, 1) / 256 * 256);
  return std::min(cols, V);
}

struct BackwardWorkspace {
  float* coef;
  float* rest;
  int* own;
  uint16_t* h_live;
  uint16_t* ds;
  float* partials;
  int64_t chunk, splits;
  size_t bytes;
};

BackwardWorkspace backward_workspace(void* base, int64_t n, int64_t d, int64_t V) {
  Layout l;
  BackwardWorkspace w;
  w.chunk = ds_chunk(n, V);
  w.splits = head_dh_splits(n, d, w.chunk);
  w.coef = l.take<float>(base, n);
  w.rest = l.take<float>(base, n);
  w.own = l.take<int>(base, n);
  w.h_live = l.take<uint16_t>(base, static_cast<size_t>(n) * d);
  w.ds = l.take<uint16_t>(base, static_cast<size_t>(n) * padded_cols(w.chunk));
  w.partials = l.take<float>(base, static_cast<size_t>(w.splits) * n * d);
  w.bytes = l.at;
  return w;
}

// The memory that a call works in: the caller's, or the library's own block
// where that suffices.
fs_status find_workspace(void** workspace, size_t have, size_t need, cudaStream_t stream) {
  if (*workspace == nullptr && need <= FS_SMALL_WORKSPACE) {
    TrainScratch* scratch = nullptr;
    FS_API_TRY(api_train_scratch(stream, &scratch));
    *workspace = scratch->small;
    return FS_OK;
  }
  if (have < need) return api_fail(FS_ERR_INVALID_ARG, "workspace has %zu bytes, needs %zu", have, need);
  return api_check_array(*workspace, 16, "workspace");
}

// Sizes that the sampler takes, less the last few: tile coordinates, which may
// run past the end by a tile, stay within 31 bits.
fs_status check_sizes(int64_t n, int64_t d, int64_t V) {
  FS_API_TRY(api_check_shapes(n, d, V));
  if (n > kMaxRows || V > kMaxRows)
    return api_fail(FS_ERR_UNSUPPORTED, "n and V must be <= %lld", static_cast<long long>(kMaxRows));
  return FS_OK;
}

fs_status check_head(const HeadProblem& p) {
  FS_API_TRY(api_check_array(p.h, 16, "h"));
  FS_API_TRY(api_check_array(p.ids, 8, "ids"));
  FS_API_TRY(api_check_array(p.temp, 4, "temp"));
  if (p.V > 0) FS_API_TRY(api_check_array(p.W, 16, "W"));
  if (p.bias != nullptr) {
    if (p.bias_stride != 0 && p.bias_stride < p.V)
      return api_fail(FS_ERR_INVALID_ARG, "bias_row_stride must be 0 or >= V");
    FS_API_TRY(api_check_array(p.bias, 4, "bias"));
  }
  return FS_OK;
}

float2 two_floats(double v) {
  const float hi = static_cast<float>(v);
  return make_float2(hi, static_cast<float>(v - hi));
}

// No C++ exception leaves a C entry (the library's maps can run out of memory).
template <typename Body>
fs_status guarded(Body body) {
  try {
    return body();
  } catch (...) {
    return api_fail(FS_ERR_WORKSPACE, "out of host memory");
  }
}

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const char* x = static_cast<const char*>(a);
  const char* y = static_cast<const char*>(b);
  return na > 0 && nb > 0 && x < y + nb && y < x + na;
}

// Whether a tensor that fs_clip_grad_norm writes shares memory with another
// one: blocks scale in any order, so it would be scaled once or twice.
bool written_twice(const void* const* grads, void* const* outs, const int64_t* sizes, const int* types, int n,
                   bool scales) {
  struct Span {
    uintptr_t at, end;
    bool written;
  };
  std::vector<Span> spans;
  spans.reserve(2 * static_cast<size_t>(n));
  for (int i = 0; i < n; ++i) {
    const uintptr_t bytes = static_cast<uintptr_t>(sizes[i]) * (types[i] == FS_TYPE_F32 ? 4 : 2);
    const uintptr_t g = reinterpret_cast<uintptr_t>(grads[i]), o = reinterpret_cast<uintptr_t>(outs[i]);
    if (bytes == 0) continue;
    spans.push_back({g, g + bytes, scales && o == g});
    if (o != g) spans.push_back({o, o + bytes, true});
  }
  std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.at < b.at; });
  uintptr_t end = 0, written = 0;         // of the spans so far, and of the written ones
  for (const Span& s : spans) {
    if (s.at < (s.written ? end : written)) return true;
    end = std::max(end, s.end);
    if (s.written) written = std::max(written, s.end);
  }
  return false;
}

}  // namespace
}  // namespace fs

using namespace fs;

extern "C" {

size_t fs_token_logprobs_workspace_bytes(int64_t n, int64_t d, int64_t V) {
  return n <= 0 || d <= 0 || V < 0 ? 0 : forward_workspace(nullptr, n, V).bytes;
}

int64_t fs_logprob_buffer_elems(int64_t n, int64_t V) { return n <= 0 || V <= 0 ? 0 : n * padded_cols(V); }

fs_status fs_token_logprobs(const void* h, const void* W, int64_t n, int64_t d, int64_t V, const int64_t* ids,
                            const float* temp, const float* bias, int64_t bias_row_stride, float* logp, float* lse,
                            float* kept, void* workspace, size_t workspace_bytes, void* stream_) {
  api_begin();
  return guarded([&]() -> fs_status {
  FS_API_TRY(check_sizes(n, d, V));
  if (n == 0) return FS_OK;
  const HeadProblem p{h, W, n, d, V, ids, temp, bias, bias_row_stride};
  FS_API_TRY(check_head(p));
  FS_API_TRY(api_check_array(logp, 4, "logp"));
  FS_API_TRY(api_check_array(lse, 4, "lse"));
  if (kept != nullptr) FS_API_TRY(api_check_array(kept, 16, "kept"));
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const CallLock lock(stream);
  FS_API_TRY(find_workspace(&workspace, workspace_bytes, forward_workspace(nullptr, n, V).bytes, stream));
  const ForwardWorkspace w = forward_workspace(workspace, n, V);
  int* err = nullptr;
  FS_API_TRY(api_error_word(&err, stream));
  FS_API_TRY(api_check_launch());
  if (V > 0) FS_API_TRY(api_launched(launch_head_parts(p, w.parts, w.own_x, kept, err, stream), "scoring kernel launch"));
  return api_launched(launch_head_merge(p, w.parts, V > 0 ? w.n_parts : 0, w.own_x, logp, lse, stream),
                      "log-sum merge launch");
  });
}

size_t fs_token_logprobs_backward_workspace_bytes(int64_t n, int64_t d, int64_t V) {
  return n <= 0 || d <= 0 || V <= 0 ? 0 : backward_workspace(nullptr, n, d, V).bytes;
}

fs_status fs_token_logprobs_backward(const void* h, const void* W, int64_t n, int64_t d, int64_t V,
                                     const int64_t* ids, const float* temp, const float* bias,
                                     int64_t bias_row_stride, const float* logp, const float* lse,
                                     const float* grad_logp, const float* kept, void* grad_h, void* grad_W,
                                     void* workspace, size_t workspace_bytes, void* stream_) {
  api_begin();
  return guarded([&]() -> fs_status {
  FS_API_TRY(check_sizes(n, d, V));
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (grad_h != nullptr && n > 0) FS_API_TRY(api_check_array(grad_h, 16, "grad_h"));
  if (grad_W != nullptr && V > 0) FS_API_TRY(api_check_array(grad_W, 16, "grad_W"));
  if (n == 0 || V == 0) {                 // no logits: zero gradients
    if (grad_h != nullptr && n > 0)
      FS_API_TRY(api_launched(cudaMemsetAsync(grad_h, 0, static_cast<size_t>(n) * d * 2, stream), "zeroing grad_h"));
    if (grad_W != nullptr && V > 0)
      FS_API_TRY(api_launched(cudaMemsetAsync(grad_W, 0, static_cast<size_t>(V) * d * 2, stream), "zeroing grad_W"));
    return FS_OK;
  }
  const HeadProblem p{h, W, n, d, V, ids, temp, bias, bias_row_stride};
  FS_API_TRY(check_head(p));
  FS_API_TRY(api_check_array(logp, 4, "logp"));
  FS_API_TRY(api_check_array(lse, 4, "lse"));
  FS_API_TRY(api_check_array(grad_logp, 4, "grad_logp"));
  if (kept != nullptr) FS_API_TRY(api_check_array(kept, 16, "kept"));
  const size_t nd = static_cast<size_t>(n) * d * 2, vd = static_cast<size_t>(V) * d * 2;
  if ((grad_h != nullptr && (overlaps(grad_h, nd, h, nd) || overlaps(grad_h, nd, W, vd))) ||
      (grad_W != nullptr && (overlaps(grad_W, vd, h, nd) || overlaps(grad_W, vd, W, vd))) ||
      (grad_h != nullptr && grad_W != nullptr && overlaps(grad_h, nd, grad_W, vd)))
    return api_fail(FS_ERR_INVALID_ARG, "grad_h and grad_W must not overlap each other, h or W");
  if (grad_h == nullptr && grad_W == nullptr) return FS_OK;
  const CallLock lock(stream);
  FS_API_TRY(find_workspace(&workspace, workspace_bytes, backward_workspace(nullptr, n, d, V).bytes, stream));
  const BackwardWorkspace w = backward_workspace(workspace, n, d, V);
  int* err = nullptr;
  FS_API_TRY(api_error_word(&err, stream));
  FS_API_TRY(api_check_launch());
  const HeadRows r{logp, lse, grad_logp, w.coef, w.own, w.rest, grad_W != nullptr ? w.h_live : nullptr};
  for (int64_t v0 = 0; v0 < V; v0 += w.chunk) {
    const int64_t vc = std::min(w.chunk, V - v0);
    FS_API_TRY(api_launched(launch_head_ds(p, r, kept, v0, vc, w.ds, err, stream), "logit gradient launch"));
    if (grad_W != nullptr)
      FS_API_TRY(api_launched(launch_head_dw(p, r, w.ds, v0, vc, grad_W, err, stream), "grad_W launch"));
    if (grad_h != nullptr)
      FS_API_TRY(api_launched(launch_head_dh(p, w.ds, v0, vc, w.splits, v0 > 0, w.partials, err, stream),
                              "grad_h launch"));
  }
  if (grad_h != nullptr)
    FS_API_TRY(api_launched(launch_head_dh_sum(p, r, w.partials, w.splits, grad_h, stream), "grad_h sum launch"));
  return FS_OK;
  });
}

size_t fs_policy_loss_workspace_bytes(int64_t n_seqs) {
  return n_seqs <= 0 ? 0 : aligned(static_cast<size_t>(n_seqs) * sizeof(float));
}

fs_status fs_policy_loss(const float* logp, const float* old_logp, const float* ref_logp, const float* advantages,
                         int adv_per_seq, const uint8_t* mask, const int64_t* seq_starts, int64_t n_seqs, int64_t N,
                         double clip_low, double clip_high, double kl_coef, int mean, float* stats, float* grad,
                         void* workspace, size_t workspace_bytes, void* stream_) {
  api_begin();
  return guarded([&]() -> fs_status {
  if (N < 0 || n_seqs < 0) return api_fail(FS_ERR_INVALID_ARG, "need N >= 0 and n_seqs >= 0 (got %lld, %lld)",
                                           (long long)N, (long long)n_seqs);
  if (n_seqs >= (int64_t(1) << 31) || N >= (int64_t(1) << 40))
    return api_fail(FS_ERR_UNSUPPORTED, "n_seqs must be < 2^31 and N < 2^40");
  if (N > 0 && n_seqs == 0) return api_fail(FS_ERR_INVALID_ARG, "N > 0 tokens need n_seqs >= 1");
  if (seq_starts == nullptr && n_seqs > 0 && N % n_seqs != 0)
    return api_fail(FS_ERR_INVALID_ARG, "without seq_starts, N must be a multiple of n_seqs");
  if (!(clip_low >= 0.0 && clip_low < 1.0)) return api_fail(FS_ERR_INVALID_ARG, "clip_low must be in [0, 1)");
  if (!(clip_high >= 0.0) || std::isinf(clip_high))
    return api_fail(FS_ERR_INVALID_ARG, "clip_high must be finite and >= 0");
  if (!std::isfinite(kl_coef)) return api_fail(FS_ERR_INVALID_ARG, "kl_coef must be finite");
  if (ref_logp == nullptr && kl_coef != 0.0) return api_fail(FS_ERR_INVALID_ARG, "kl_coef needs ref_logp");
  if (mean < FS_MEAN_TOKEN || mean > FS_MEAN_NONE) return api_fail(FS_ERR_INVALID_ARG, "unknown mean %d", mean);
  if (adv_per_seq != 0 && adv_per_seq != 1) return api_fail(FS_ERR_INVALID_ARG, "adv_per_seq must be 0 or 1");
  FS_API_TRY(api_check_array(stats, 4, "stats"));
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (N == 0) return api_launched(cudaMemsetAsync(stats, 0, 4 * sizeof(float), stream), "zeroing stats");
  FS_API_TRY(api_check_array(logp, 4, "logp"));
  FS_API_TRY(api_check_array(old_logp, 4, "old_logp"));
  if (ref_logp != nullptr) FS_API_TRY(api_check_array(ref_logp, 4, "ref_logp"));
  FS_API_TRY(api_check_array(advantages, 4, "advantages"));
  if (mask != nullptr) FS_API_TRY(api_check_array(mask, 1, "mask"));
  if (seq_starts != nullptr) FS_API_TRY(api_check_array(seq_starts, 8, "seq_starts"));
  FS_API_TRY(api_check_array(grad, 4, "grad"));
  const CallLock lock(stream);
  if (mean == FS_MEAN_SEQUENCE)
    FS_API_TRY(find_workspace(&workspace, workspace_bytes, fs_policy_loss_workspace_bytes(n_seqs), stream));
  TrainScratch* scratch = nullptr;
  FS_API_TRY(api_train_scratch(stream, &scratch));
  FS_API_TRY(api_check_launch());
  PolicyProblem p{logp, old_logp, ref_logp, advantages, adv_per_seq == 1, mask, seq_starts, n_seqs, N / n_seqs, N};
  p.log_hi = two_floats(std::log1p(clip_high));
  p.log_lo = two_floats(std::log1p(-clip_low));
  p.hi = static_cast<float>(1.0 + clip_high);
  p.lo = static_cast<float>(1.0 - clip_low);
  p.kl_coef = static_cast<float>(kl_coef);
  p.mean = mean;
  p.stats = stats;
  p.grad = grad;
  p.counts = static_cast<float*>(workspace);
  p.scratch = scratch;
  return api_launched(launch_policy_loss(p, stream), "policy loss launch");
  });
}

fs_status fs_clip_grad_norm(const void* const* grads, void* const* outs, const int64_t* sizes, const int* types,
                            int n_tensors, double max_norm, int norm_type, float* norm, void* stream_) {
  api_begin();
  return guarded([&]() -> fs_status {
  if (n_tensors < 0) return api_fail(FS_ERR_INVALID_ARG, "need n_tensors >= 0 (got %d)", n_tensors);
  if (!(max_norm >= 0.0)) return api_fail(FS_ERR_INVALID_ARG, "max_norm must be >= 0 and not NaN");
  if (norm_type != FS_NORM_L2 && norm_type != FS_NORM_MAX)
    return api_fail(FS_ERR_INVALID_ARG, "unknown norm type %d", norm_type);
  if (n_tensors > 0 && (grads == nullptr || sizes == nullptr || types == nullptr))
    return api_fail(FS_ERR_INVALID_ARG, "grads, sizes or types is NULL");
  for (int i = 0; i < n_tensors; ++i) {
    if (sizes[i] < 0) return api_fail(FS_ERR_INVALID_ARG, "sizes[%d] is negative", i);
    if (sizes[i] >= (int64_t(1) << 40)) return api_fail(FS_ERR_UNSUPPORTED, "sizes[%d] must be < 2^40", i);
    if (types[i] < FS_TYPE_F32 || types[i] > FS_TYPE_F16)
      return api_fail(FS_ERR_INVALID_ARG, "unknown type %d of tensor %d", types[i], i);
  }
  if (outs != nullptr && written_twice(grads, outs, sizes, types, n_tensors, !std::isinf(max_norm)))
    return api_fail(FS_ERR_INVALID_ARG, "an output overlaps another tensor, or its gradient without being it");
  FS_API_TRY(api_check_array(norm, 4, "norm"));
  for (int i = 0; i < n_tensors; ++i) {
    if (sizes[i] == 0) continue;
    const size_t width = types[i] == FS_TYPE_F32 ? 4 : 2;
    FS_API_TRY(api_check_array(grads[i], width, "a gradient"));
    if (outs != nullptr && outs[i] != grads[i]) FS_API_TRY(api_check_array(outs[i], width, "an output"));
  }
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const CallLock lock(stream);
  TrainScratch* scratch = nullptr;
  FS_API_TRY(api_train_scratch(stream, &scratch));
  FS_API_TRY(api_check_launch());
  return api_launched(launch_clip_grad_norm(grads, outs, sizes, types, n_tensors, max_norm, norm_type, norm, scratch,
                                            stream),
                      "gradient norm launch");
  });
}

}  // extern "C"
