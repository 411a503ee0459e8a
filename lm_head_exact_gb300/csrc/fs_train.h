// Internals of the training operators: token log-probabilities through the
// LM head and their gradients, the policy loss, gradient clipping.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "fs_api_util.h"
#include "fs_internal.h"

namespace fs {

// One scoring problem: n rows of h against the V rows of W.
struct HeadProblem {
  const void* h;            // bf16 [n, d]
  const void* W;            // bf16 [V, d]
  int64_t n, d, V;
  const int64_t* ids;       // [n]
  const float* temp;        // [n]
  const float* bias;        // nullable, element (t, v) at bias[t * bias_stride + v]
  int64_t bias_stride;
};

// Row pitch, in elements, of kept logits and of ds: rows start on 128-byte
// boundaries whatever V is.
inline int64_t padded_cols(int64_t V) { return (V + 63) / 64 * 64; }

// (max, sum of exp(x - max)) of a part of a row's x.
struct __align__(8) LsePart {
  float m, s;
};

// Forward: every row's parts [head_parts, n] and its own token's x (written
// by whichever tile holds the token's id), kept logits on request; then the
// merge of the parts.
int64_t head_parts(int64_t n, int64_t V);
cudaError_t launch_head_parts(const HeadProblem& p, LsePart* parts, float* own_x, float* kept, int* err,
                              cudaStream_t stream);
cudaError_t launch_head_merge(const HeadProblem& p, const LsePart* parts, int64_t n_parts, const float* own_x,
                              float* logp, float* lse, cudaStream_t stream);

// Backward: what is known of the rows, and what launch_head_ds() leaves of them
// for the products.
struct HeadRows {
  const float* logp;
  const float* lse;
  const float* g;
  float* coef;              // [n] g / T, 0 for rows without a gradient
  int* own;                 // [n] their tokens' ids, -1 for rows without a gradient
  float* rest;              // [n] what rounding left over of the tokens' own entries of ds
  void* h_live;             // bf16 [n, d] h, those rows zeroed; nullable (no grad_W)
};

// ds of vocabulary rows [v0, v0 + vc) as bf16 [n, padded_cols(vc)], from kept
// logits or from h and W; the two products; and the sum of grad_h's split
// partials.
cudaError_t launch_head_ds(const HeadProblem& p, const HeadRows& r, const float* kept, int64_t v0, int64_t vc, void* ds,
                           int* err, cudaStream_t stream);
int64_t head_dh_splits(int64_t n, int64_t d, int64_t vc);
cudaError_t launch_head_dh(const HeadProblem& p, const void* ds, int64_t v0, int64_t vc, int64_t splits, bool add,
                           float* partials, int* err, cudaStream_t stream);
cudaError_t launch_head_dh_sum(const HeadProblem& p, const HeadRows& r, const float* partials, int64_t splits,
                               void* grad_h, cudaStream_t stream);
cudaError_t launch_head_dw(const HeadProblem& p, const HeadRows& r, const void* ds, int64_t v0, int64_t vc,
                           void* grad_W, int* err, cudaStream_t stream);

struct PolicyProblem {
  const float* logp;
  const float* old_logp;
  const float* ref_logp;        // nullable
  const float* adv;             // [N], or [n_seqs] with adv_per_seq
  bool adv_per_seq;
  const uint8_t* mask;          // nullable
  const int64_t* starts;        // nullable: n_seqs rows of row_len tokens
  int64_t n_seqs, row_len, N;
  float2 log_hi, log_lo;        // log(1 + clip_high), log(1 - clip_low), each as the sum of two fp32 numbers
  float hi, lo;                 // 1 + clip_high, 1 - clip_low
  float kl_coef;
  int mean;
  float* stats;
  float* grad;
  float* counts;                // [n_seqs] workspace: tokens that take part, as the weights take them
  TrainScratch* scratch;
};
cudaError_t launch_policy_loss(const PolicyProblem& p, cudaStream_t stream);

cudaError_t launch_clip_grad_norm(const void* const* grads, void* const* outs, const int64_t* sizes, const int* types,
                                  int n_tensors, double max_norm, int norm_type, float* norm, TrainScratch* scratch,
                                  cudaStream_t stream);

}  // namespace fs
