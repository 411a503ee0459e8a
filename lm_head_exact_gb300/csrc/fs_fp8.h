// Internals of the 8-bit path and of the norm ahead of it: quantising in blocks
// of 128, the matrix product of what was quantised, the sampler over an 8-bit
// head, layer norm and its backward pass.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "fs_internal.h"

namespace fs {

constexpr int kQuantBlock = 128;          // elements of a row that share a scale

inline int64_t quant_blocks(int64_t n) { return (n + kQuantBlock - 1) / kQuantBlock; }

// An 8-bit matrix [rows, k]: value (r, j) is q[r * stride + j] *
// scale[(r / block_rows) * s_row + (j / 128) * s_col].
struct Fp8Matrix {
  const void* q;
  int type;                 // FS_TYPE_E4M3 or FS_TYPE_E5M2
  int64_t stride;           // bytes, a multiple of 16
  const float* scale;
  int64_t s_row, s_col;
  int block_rows;           // 1 or 128
};

// x [rows, cols] of a 16- or 32-bit type, rows x_stride elements apart.
struct QuantProblem {
  const void* x;
  int x_type;
  int64_t rows, cols, x_stride;
  bool transpose;           // q holds the transposed matrix
  int block_rows;           // of q
  int q_type;
  void* q;
  int64_t q_stride;
  float* scale;
  int64_t s_row, s_col;
};
cudaError_t launch_quantize(const QuantProblem& p, cudaStream_t stream);

struct Fp8Product {
  Fp8Matrix a, b;           // a [m, k], b [n, k]
  int64_t m, n, k;
  void* out;                // [m, n] of out_type, rows out_stride elements apart
  int out_type;
  int64_t out_stride;
};
cudaError_t launch_fp8_matmul(const Fp8Product& p, int* err, cudaStream_t stream);
// The same where there is little to read (fs_fp8_rows.cu).
bool fp8_rows_takes(const Fp8Product& p);
cudaError_t launch_fp8_rows(const Fp8Product& p, cudaStream_t stream);

// The sampler: rows of a are the batch, rows of b the vocabulary (p.h, p.W and
// p.d of the Problem are not looked at).
cudaError_t launch_fp8_sample(const Problem& p, const Fp8Matrix& h, const Fp8Matrix& W, int64_t k, const Finish& f,
                              int* err, cudaStream_t stream);

// Layer norm of the rows of x [n, d]; rms: without the mean.
struct NormProblem {
  const void* x;
  int x_type;
  int64_t n, d, x_stride;
  const void* weight;       // nullable [d] of w_type
  const void* bias;         // nullable [d] of w_type
  int w_type;               // FS_TYPE_F32 or x_type
  bool rms;
  float eps;
  void* y;                  // [n, d] of x_type, rows y_stride elements apart; nullable with q
  int64_t y_stride;
  float* mean;              // nullable [n] (none with rms)
  float* rstd;              // nullable [n]
  void* q;                  // nullable: y quantised, rows q_stride bytes apart
  int q_type;
  int64_t q_stride;
  float* scale;
  int64_t s_row, s_col;
};
cudaError_t launch_norm(const NormProblem& p, cudaStream_t stream);

struct NormGradProblem {
  const void* g;            // [n, d] of x_type
  int64_t g_stride;
  const void* x;
  int x_type;
  int64_t n, d, x_stride;
  const void* weight;       // nullable
  int w_type;
  bool rms;
  const float* mean;        // none with rms
  const float* rstd;
  void* gx;                 // nullable [n, d] of x_type, gx_stride elements apart
  int64_t gx_stride;
  void* gw;                 // nullable [d] of w_type
  void* gb;                 // nullable [d] of w_type
  float* partials;          // norm_grad_blocks(n) x 2 x d
  int* err;
};
// Blocks, at most, that each leave one partial sum of the weight's and bias's gradients.
int64_t norm_grad_blocks(int64_t n);
cudaError_t launch_norm_grad(const NormGradProblem& p, cudaStream_t stream);

constexpr int64_t kNormMaxWidth = 32768;

}  // namespace fs
