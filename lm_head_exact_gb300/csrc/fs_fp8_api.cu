// C entry points of the 8-bit path and of the norm ahead of it: argument checks
// and launches.  Contracts: include/flashsample.h.
#include <algorithm>
#include <cmath>

#include "flashsample.h"
#include "fs_api_util.h"
#include "fs_fp8.h"

namespace fs {
namespace {

constexpr int64_t kMaxSize = (int64_t(1) << 31) - 1024;
constexpr int64_t kMaxDepth = int64_t(1) << 24;      // of k: a tile then takes a tenth of what a wait allows
constexpr int64_t kMaxStride = int64_t(1) << 40;

bool is_wide(int type) { return type >= FS_TYPE_F32 && type <= FS_TYPE_F16; }
bool is_fp8(int type) { return type == FS_TYPE_E4M3 || type == FS_TYPE_E5M2; }
size_t width_of(int type) { return type == FS_TYPE_F32 ? 4 : is_fp8(type) ? 1 : 2; }

// Rows of `cols` elements, `stride` apart: the stride of a single row is not
// looked at but for its size.
fs_status check_rows(int64_t rows, int64_t cols, int64_t stride, const char* name) {
  if (stride < 0 || stride >= kMaxStride || (rows > 1 && stride < cols))
    return api_fail(FS_ERR_INVALID_ARG, "%s: a row stride of %lld for rows of %lld", name, (long long)stride, (long long)cols);
  return FS_OK;
}

fs_status check_fp8(const void* q, int type, int64_t rows, int64_t cols, int64_t stride, const float* scale,
                    int64_t s_row, int64_t s_col, int block_rows, const char* name) {
  if (!is_fp8(type)) return api_fail(FS_ERR_INVALID_ARG, "%s: type %d is not an 8-bit one", name, type);
  if (block_rows != 1 && block_rows != kQuantBlock)
    return api_fail(FS_ERR_INVALID_ARG, "%s: blocks of %d rows; 1 or 128", name, block_rows);
  if (rows == 0 || cols == 0) return FS_OK;
  FS_API_TRY(check_rows(2, cols, stride, name));
  if (stride % 16 != 0) return api_fail(FS_ERR_UNSUPPORTED, "%s: a row stride of %lld bytes, not a multiple of 16", name, (long long)stride);
  if (s_row < 0 || s_col < 0 || s_row >= kMaxStride || s_col >= kMaxStride)
    return api_fail(FS_ERR_INVALID_ARG, "%s: strides of the scales must be >= 0", name);
  FS_API_TRY(api_check_array(q, 16, name));
  return api_check_array(scale, 4, name);
}

// Bytes from the first element of [rows, cols] to behind the last.
size_t span_of(int64_t rows, int64_t cols, int64_t stride, size_t width) {
  return rows == 0 || cols == 0 ? 0 : (static_cast<size_t>(rows - 1) * stride + cols) * width;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const char* x = static_cast<const char*>(a);
  const char* y = static_cast<const char*>(b);
  return x != nullptr && y != nullptr && na > 0 && nb > 0 && x < y + nb && y < x + na;
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

}  // namespace
}  // namespace fs

using namespace fs;

extern "C" {

fs_status fs_quantize_fp8(const void* x, int x_type, int64_t rows, int64_t cols, int64_t x_row_stride, int transpose,
                          int block_rows, int q_type, void* q, int64_t q_row_stride, float* scale,
                          int64_t scale_row_stride, int64_t scale_col_stride, void* stream) {
  api_begin();
  return guarded([&]() -> fs_status {
  if (rows < 0 || cols < 0) return api_fail(FS_ERR_INVALID_ARG, "need rows >= 0 and cols >= 0");
  if (rows >= (int64_t(1) << 31) || cols >= (int64_t(1) << 31))
    return api_fail(FS_ERR_UNSUPPORTED, "rows and cols must be < 2^31");
  if (!is_wide(x_type)) return api_fail(FS_ERR_INVALID_ARG, "x: unknown type %d", x_type);
  if (transpose != 0 && transpose != 1) return api_fail(FS_ERR_INVALID_ARG, "transpose must be 0 or 1");
  FS_API_TRY(check_rows(rows, cols, x_row_stride, "x"));
  const int64_t R = transpose ? cols : rows, C = transpose ? rows : cols;
  FS_API_TRY(check_fp8(q, q_type, R, C, q_row_stride, scale, scale_row_stride, scale_col_stride, block_rows, "q"));
  if (rows == 0 || cols == 0) return FS_OK;
  FS_API_TRY(api_check_array(x, width_of(x_type), "x"));
  if (overlap(q, span_of(R, C, q_row_stride, 1), x, span_of(rows, cols, x_row_stride, width_of(x_type))))
    return api_fail(FS_ERR_INVALID_ARG, "q overlaps x");
  FS_API_TRY(api_check_launch());
  const QuantProblem p{x, x_type, rows, cols, x_row_stride, transpose == 1, block_rows, q_type, q, q_row_stride, scale,
                       scale_row_stride, scale_col_stride};
  return api_launched(launch_quantize(p, static_cast<cudaStream_t>(stream)), "quantising launch");
  });
}

fs_status fs_fp8_matmul(const void* a, int a_type, int64_t a_row_stride, const float* a_scale, int64_t a_scale_row_stride,
                        int64_t a_scale_col_stride, const void* b, int b_type, int64_t b_row_stride, const float* b_scale,
                        int64_t b_scale_row_stride, int64_t b_scale_col_stride, int b_block_rows, int64_t m, int64_t n,
                        int64_t k, void* out, int out_type, int64_t out_row_stride, void* stream_) {
  api_begin();
  return guarded([&]() -> fs_status {
  if (m < 0 || n < 0 || k < 0) return api_fail(FS_ERR_INVALID_ARG, "need m, n, k >= 0");
  if (m > kMaxSize || n > kMaxSize || k > kMaxDepth)
    return api_fail(FS_ERR_UNSUPPORTED, "m and n must be <= %lld, k <= %lld", (long long)kMaxSize, (long long)kMaxDepth);
  if (!is_wide(out_type)) return api_fail(FS_ERR_INVALID_ARG, "out: unknown type %d", out_type);
  FS_API_TRY(check_rows(m, n, out_row_stride, "out"));
  FS_API_TRY(check_fp8(a, a_type, m, k, a_row_stride, a_scale, a_scale_row_stride, a_scale_col_stride, 1, "a"));
  FS_API_TRY(check_fp8(b, b_type, n, k, b_row_stride, b_scale, b_scale_row_stride, b_scale_col_stride, b_block_rows, "b"));
  if (m == 0 || n == 0) return FS_OK;
  const size_t width = width_of(out_type);
  FS_API_TRY(api_check_array(out, width, "out"));
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (k == 0)
    return api_launched(m == 1 ? cudaMemsetAsync(out, 0, n * width, stream)
                               : cudaMemset2DAsync(out, out_row_stride * width, 0, n * width, m, stream), "zeroing out");
  const size_t so = span_of(m, n, out_row_stride, width);
  if (overlap(out, so, a, span_of(m, k, a_row_stride, 1)) || overlap(out, so, b, span_of(n, k, b_row_stride, 1)))
    return api_fail(FS_ERR_INVALID_ARG, "out overlaps a or b");
  int* err = nullptr;
  FS_API_TRY(api_error_word(&err, stream));
  FS_API_TRY(api_check_launch());
  const Fp8Product p{{a, a_type, a_row_stride, a_scale, a_scale_row_stride, a_scale_col_stride, 1},
                     {b, b_type, b_row_stride, b_scale, b_scale_row_stride, b_scale_col_stride, b_block_rows},
                     m, n, k, out, out_type, out_row_stride};
  return api_launched(launch_fp8_matmul(p, err, stream), "8-bit product launch");
  });
}

fs_status fs_sample_fp8(const void* h, int64_t h_row_stride, const float* h_scale, int64_t h_scale_row_stride,
                        int64_t h_scale_col_stride, const void* W, int64_t W_row_stride, const float* W_scale,
                        int64_t W_scale_row_stride, int64_t W_scale_col_stride, int W_block_rows, int64_t B, int64_t d,
                        int64_t V, const float* temp, const float* bias, int64_t bias_row_stride, uint64_t seed,
                        uint64_t step, int64_t* out_ids, float* out_max, void* stream_) {
  api_begin();
  return guarded([&]() -> fs_status {
  if (B < 0 || d <= 0 || V < 0) return api_fail(FS_ERR_INVALID_ARG, "need B >= 0, d > 0, V >= 0 (got %lld, %lld, %lld)",
                                                (long long)B, (long long)d, (long long)V);
  if (B > kMaxSize || d > kMaxDepth || V > kMaxSize)
    return api_fail(FS_ERR_UNSUPPORTED, "B and V must be <= %lld, d <= %lld", (long long)kMaxSize, (long long)kMaxDepth);
  FS_API_TRY(check_fp8(h, FS_TYPE_E4M3, B, d, h_row_stride, h_scale, h_scale_row_stride, h_scale_col_stride, 1, "h"));
  if (B == 0) return FS_OK;
  FS_API_TRY(check_fp8(W, FS_TYPE_E4M3, V, d, W_row_stride, W_scale, W_scale_row_stride, W_scale_col_stride, W_block_rows, "W"));
  FS_API_TRY(api_check_array(temp, 4, "temp"));
  if (bias != nullptr) {
    if (bias_row_stride != 0 && bias_row_stride < V)
      return api_fail(FS_ERR_INVALID_ARG, "bias_row_stride must be 0 or >= V");
    FS_API_TRY(api_check_array(bias, 4, "bias"));
  }
  FS_API_TRY(api_check_array(out_ids, 8, "out_ids"));
  FS_API_TRY(api_check_array(out_max, 4, "out_max"));
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  Problem p{nullptr, nullptr, B, d, V, 0, temp, bias, bias_row_stride, seed, step};
  Finish f{};
  f.write_out = true;
  f.out_ids = out_ids;
  f.out_max = out_max;
  if (V == 0) return api_launched(launch_reduce(f, B, stream), "reduction kernel launch");
  const CallLock lock(stream);
  FS_API_TRY(api_finish(stream, B, &f));
  int* err = nullptr;
  FS_API_TRY(api_error_word(&err, stream));
  FS_API_TRY(api_check_launch());
  const Fp8Matrix mh{h, FS_TYPE_E4M3, h_row_stride, h_scale, h_scale_row_stride, h_scale_col_stride, 1};
  const Fp8Matrix mw{W, FS_TYPE_E4M3, W_row_stride, W_scale, W_scale_row_stride, W_scale_col_stride, W_block_rows};
  return api_launched(launch_fp8_sample(p, mh, mw, d, f, err, stream), "fused sampling kernel launch");
  });
}

namespace {

fs_status check_norm(int64_t n, int64_t d, int x_type, const void* weight, const void* bias, int w_type, int rms) {
  if (n < 0 || d <= 0) return api_fail(FS_ERR_INVALID_ARG, "need n >= 0 and d > 0 (got %lld, %lld)", (long long)n, (long long)d);
  if (n >= (int64_t(1) << 31) || d > kNormMaxWidth)
    return api_fail(FS_ERR_UNSUPPORTED, "n must be < 2^31 and d <= %lld", (long long)kNormMaxWidth);
  if (!is_wide(x_type)) return api_fail(FS_ERR_INVALID_ARG, "x: unknown type %d", x_type);
  if (w_type != FS_TYPE_F32 && w_type != x_type)
    return api_fail(FS_ERR_INVALID_ARG, "w_type %d: weights are fp32 or of x's type", w_type);
  if (rms != 0 && rms != 1) return api_fail(FS_ERR_INVALID_ARG, "rms must be 0 or 1");
  if (weight != nullptr) FS_API_TRY(api_check_array(weight, width_of(w_type), "weight"));
  if (bias != nullptr) FS_API_TRY(api_check_array(bias, width_of(w_type), "bias"));
  return FS_OK;
}

}  // namespace

fs_status fs_layer_norm(const void* x, int x_type, int64_t n, int64_t d, int64_t x_row_stride, const void* weight,
                        const void* bias, int w_type, int rms, double eps, void* y, int64_t y_row_stride, float* mean,
                        float* rstd, void* q, int q_type, int64_t q_row_stride, float* scale, int64_t scale_row_stride,
                        int64_t scale_col_stride, void* stream) {
  api_begin();
  return guarded([&]() -> fs_status {
  FS_API_TRY(check_norm(n, d, x_type, nullptr, nullptr, w_type, rms));
  if (!(eps >= 0.0) || std::isinf(eps)) return api_fail(FS_ERR_INVALID_ARG, "eps must be finite and >= 0");
  FS_API_TRY(check_rows(n, d, x_row_stride, "x"));
  if (n == 0) return FS_OK;
  if ((y == nullptr) == (q == nullptr)) return api_fail(FS_ERR_INVALID_ARG, "one of y and q");
  FS_API_TRY(check_norm(n, d, x_type, weight, bias, w_type, rms));
  const size_t width = width_of(x_type);
  FS_API_TRY(api_check_array(x, width, "x"));
  if (mean != nullptr) FS_API_TRY(api_check_array(mean, 4, "mean"));
  if (rstd != nullptr) FS_API_TRY(api_check_array(rstd, 4, "rstd"));
  const size_t sx = span_of(n, d, x_row_stride, width);
  if (y != nullptr) {
    FS_API_TRY(check_rows(n, d, y_row_stride, "y"));
    FS_API_TRY(api_check_array(y, width, "y"));
    if (!(y == x && y_row_stride == x_row_stride) && overlap(y, span_of(n, d, y_row_stride, width), x, sx))
      return api_fail(FS_ERR_INVALID_ARG, "y overlaps x without being it");
  } else {
    FS_API_TRY(check_fp8(q, q_type, n, d, q_row_stride, scale, scale_row_stride, scale_col_stride, 1, "q"));
    if (overlap(q, span_of(n, d, q_row_stride, 1), x, sx)) return api_fail(FS_ERR_INVALID_ARG, "q overlaps x");
  }
  FS_API_TRY(api_check_launch());
  const NormProblem p{x, x_type, n, d, x_row_stride, weight, bias, w_type, rms == 1, static_cast<float>(eps), y, y_row_stride,
                      rms == 1 ? nullptr : mean, rstd, q, q_type, q_row_stride, scale, scale_row_stride, scale_col_stride};
  return api_launched(launch_norm(p, static_cast<cudaStream_t>(stream)), "layer norm launch");
  });
}

size_t fs_layer_norm_backward_workspace_bytes(int64_t n, int64_t d) {
  return n <= 0 || d <= 0 || d > kNormMaxWidth ? 0 : static_cast<size_t>(norm_grad_blocks(n)) * 2 * d * sizeof(float);
}

fs_status fs_layer_norm_backward(const void* g, int64_t g_row_stride, const void* x, int x_type, int64_t n, int64_t d,
                                 int64_t x_row_stride, const void* weight, int w_type, int rms, const float* mean,
                                 const float* rstd, void* grad_x, int64_t grad_x_row_stride, void* grad_weight,
                                 void* grad_bias, void* workspace, size_t workspace_bytes, void* stream_) {
  api_begin();
  return guarded([&]() -> fs_status {
  FS_API_TRY(check_norm(n, d, x_type, nullptr, nullptr, w_type, rms));
  FS_API_TRY(check_rows(n, d, g_row_stride, "g"));
  FS_API_TRY(check_rows(n, d, x_row_stride, "x"));
  const size_t width = width_of(x_type), w_width = width_of(w_type);
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (grad_weight != nullptr) FS_API_TRY(api_check_array(grad_weight, w_width, "grad_weight"));
  if (grad_bias != nullptr) FS_API_TRY(api_check_array(grad_bias, w_width, "grad_bias"));
  if (overlap(grad_weight, d * w_width, grad_bias, d * w_width))
    return api_fail(FS_ERR_INVALID_ARG, "grad_weight and grad_bias overlap");
  if (n == 0) {                             // sums over no rows
    if (grad_weight != nullptr)
      FS_API_TRY(api_launched(cudaMemsetAsync(grad_weight, 0, d * w_width, stream), "zeroing grad_weight"));
    if (grad_bias != nullptr)
      FS_API_TRY(api_launched(cudaMemsetAsync(grad_bias, 0, d * w_width, stream), "zeroing grad_bias"));
    return FS_OK;
  }
  FS_API_TRY(check_norm(n, d, x_type, weight, nullptr, w_type, rms));
  FS_API_TRY(api_check_array(g, width, "g"));
  FS_API_TRY(api_check_array(x, width, "x"));
  FS_API_TRY(api_check_array(rstd, 4, "rstd"));
  if (rms == 0) FS_API_TRY(api_check_array(mean, 4, "mean"));
  const size_t sg = span_of(n, d, g_row_stride, width), sx = span_of(n, d, x_row_stride, width);
  if (grad_x != nullptr) {
    FS_API_TRY(check_rows(n, d, grad_x_row_stride, "grad_x"));
    FS_API_TRY(api_check_array(grad_x, width, "grad_x"));
    const size_t so = span_of(n, d, grad_x_row_stride, width);
    const bool is_g = grad_x == g && grad_x_row_stride == g_row_stride, is_x = grad_x == x && grad_x_row_stride == x_row_stride;
    if ((!is_g && overlap(grad_x, so, g, sg)) || (!is_x && overlap(grad_x, so, x, sx)) ||
        overlap(grad_x, so, weight, d * w_width) || overlap(grad_x, so, grad_weight, d * w_width) ||
        overlap(grad_x, so, grad_bias, d * w_width))
      return api_fail(FS_ERR_INVALID_ARG, "grad_x overlaps another tensor without being g or x");
  }
  for (void* sum : {grad_weight, grad_bias})
    if (overlap(sum, d * w_width, g, sg) || overlap(sum, d * w_width, x, sx) || overlap(sum, d * w_width, weight, d * w_width))
      return api_fail(FS_ERR_INVALID_ARG, "grad_weight and grad_bias must not overlap g, x or weight");
  const bool sums = grad_weight != nullptr || grad_bias != nullptr;
  if (!sums && grad_x == nullptr) return FS_OK;
  const CallLock lock(stream);
  if (sums) {
    const size_t need = fs_layer_norm_backward_workspace_bytes(n, d);
    if (workspace == nullptr && need <= FS_SMALL_WORKSPACE) {
      TrainScratch* scratch = nullptr;
      FS_API_TRY(api_train_scratch(stream, &scratch));
      workspace = scratch->small;
    } else {
      if (workspace_bytes < need)
        return api_fail(FS_ERR_INVALID_ARG, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
      FS_API_TRY(api_check_array(workspace, 16, "workspace"));
    }
  }
  int* err = nullptr;
  FS_API_TRY(api_error_word(&err, stream));
  FS_API_TRY(api_check_launch());
  const NormGradProblem p{g, g_row_stride, x, x_type, n, d, x_row_stride, weight, w_type, rms == 1, mean, rstd, grad_x,
                          grad_x_row_stride, grad_weight, grad_bias, static_cast<float*>(workspace), err};
  return api_launched(launch_norm_grad(p, stream), "layer norm gradient launch");
  });
}

}  // extern "C"
