// C entry points of the 8-bit path and of the norm ahead of it: argument checks
// and launches.  Contracts: include/flashsample.h.
#include <algorithm>
#include <cmath>
#include <initializer_list>

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

// An 8-bit matrix but for its addresses, and those.
fs_status check_fp8_form(int type, int64_t rows, int64_t cols, int64_t stride, int64_t s_row, int64_t s_col, int block_rows,
                         const char* name) {
  if (!is_fp8(type)) return api_fail(FS_ERR_INVALID_ARG, "%s: type %d is not an 8-bit one", name, type);
  if (block_rows != 1 && block_rows != kQuantBlock)
    return api_fail(FS_ERR_INVALID_ARG, "%s: blocks of %d rows; 1 or 128", name, block_rows);
  if (rows == 0 || cols == 0) return FS_OK;
  FS_API_TRY(check_rows(2, cols, stride, name));
  if (stride % 16 != 0) return api_fail(FS_ERR_UNSUPPORTED, "%s: a row stride of %lld bytes, not a multiple of 16", name, (long long)stride);
  if (s_row < 0 || s_col < 0 || s_row >= kMaxStride || s_col >= kMaxStride)
    return api_fail(FS_ERR_INVALID_ARG, "%s: strides of the scales must be >= 0", name);
  return FS_OK;
}

fs_status check_fp8_arrays(const void* q, const float* scale, int64_t rows, int64_t cols, const char* name) {
  if (rows == 0 || cols == 0) return FS_OK;
  FS_API_TRY(api_check_array(q, 16, name));
  return api_check_array(scale, 4, name);
}

fs_status check_fp8(const void* q, int type, int64_t rows, int64_t cols, int64_t stride, const float* scale,
                    int64_t s_row, int64_t s_col, int block_rows, const char* name) {
  FS_API_TRY(check_fp8_form(type, rows, cols, stride, s_row, s_col, block_rows, name));
  return check_fp8_arrays(q, scale, rows, cols, name);
}

// Memory of a matrix: rows of `width` bytes, `pitch` bytes apart (at NULL: none).
// Sums of strides pass 64 bits before they are known to be memory.
using Wide = __int128;
struct Region {
  const void* at;
  int64_t rows;
  Wide width, pitch;
  const char* name;
  bool in_place = false;      // of an output and an input: they may be the same memory
};

Region matrix(const void* at, int64_t rows, int64_t cols, int64_t stride, size_t width, const char* name, bool in_place = false) {
  return Region{at, rows, Wide(cols) * width, Wide(stride) * width, name, in_place};
}
Region vector(const void* at, int64_t n, size_t width, const char* name) { return matrix(at, 1, n, n, width, name); }
// The scales of an 8-bit [rows, cols], by rows or by columns, whichever lie further apart.
Region scales(const float* at, int64_t rows, int64_t cols, int64_t s_row, int64_t s_col, int block_rows, const char* name) {
  const int64_t r = (rows + block_rows - 1) / block_rows, c = quant_blocks(cols);
  if (r == 0 || c == 0) return Region{nullptr, 0, 0, 0, name};
  return s_row >= s_col ? Region{at, r, (Wide(c - 1) * s_col + 1) * 4, Wide(s_row) * 4, name}
                        : Region{at, c, (Wide(r - 1) * s_row + 1) * 4, Wide(s_col) * 4, name};
}

Wide floor_div(Wide a, Wide b) { return a / b - (a % b < 0 ? 1 : 0); }      // b > 0

// Whether two matrices share a byte.  Rows of one pitch may lie side by side;
// where pitches differ, matrices between each other's ends count as sharing.
bool overlap(const Region& a, const Region& b) {
  if (a.at == nullptr || b.at == nullptr || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
  const Wide apart = Wide(reinterpret_cast<uintptr_t>(b.at)) - Wide(reinterpret_cast<uintptr_t>(a.at));
  if (apart >= (a.rows - 1) * a.pitch + a.width || -apart >= (b.rows - 1) * b.pitch + b.width) return false;
  if (a.rows == 1 && b.rows == 1) return true;
  const Wide pitch = a.rows == 1 ? b.pitch : a.pitch;
  if (pitch <= 0 || (b.rows > 1 && b.pitch != pitch)) return true;
  // row i of a and row j of b meet where (i - j) pitch lies in (apart - a.width, apart + b.width)
  const Wide least = std::max<Wide>(floor_div(apart - a.width, pitch) + 1, 1 - b.rows);
  const Wide most = std::min<Wide>(floor_div(apart + b.width - 1, pitch), a.rows - 1);
  return least <= most;
}

// Outputs share no memory with one another, and none with inputs but where both
// may be the same matrix and are.
fs_status check_apart(std::initializer_list<Region> outputs, std::initializer_list<Region> inputs) {
  for (const Region* o = outputs.begin(); o != outputs.end(); ++o) {
    for (const Region* other = outputs.begin(); other != o; ++other)
      if (overlap(*o, *other)) return api_fail(FS_ERR_INVALID_ARG, "%s overlaps %s", o->name, other->name);
    for (const Region& i : inputs) {
      const bool same = o->in_place && i.in_place && o->at == i.at && (o->rows == 1 || o->pitch == i.pitch);
      if (!same && overlap(*o, i))
        return api_fail(FS_ERR_INVALID_ARG, "%s overlaps %s%s", o->name, i.name, o->in_place && i.in_place ? " without being it" : "");
    }
  }
  return FS_OK;
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
  FS_API_TRY(check_fp8_form(q_type, R, C, q_row_stride, scale_row_stride, scale_col_stride, block_rows, "q"));
  if (rows == 0 || cols == 0) return FS_OK;
  FS_API_TRY(check_apart({matrix(q, R, C, q_row_stride, 1, "q"),
                          scales(scale, R, C, scale_row_stride, scale_col_stride, block_rows, "scale")},
                         {matrix(x, rows, cols, x_row_stride, width_of(x_type), "x")}));
  FS_API_TRY(check_fp8_arrays(q, scale, R, C, "q"));
  FS_API_TRY(api_check_array(x, width_of(x_type), "x"));
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
  FS_API_TRY(check_fp8_form(a_type, m, k, a_row_stride, a_scale_row_stride, a_scale_col_stride, 1, "a"));
  FS_API_TRY(check_fp8_form(b_type, n, k, b_row_stride, b_scale_row_stride, b_scale_col_stride, b_block_rows, "b"));
  const size_t width = width_of(out_type);
  FS_API_TRY(check_apart({matrix(out, m, n, out_row_stride, width, "out")},
                         {matrix(a, m, k, a_row_stride, 1, "a"), matrix(b, n, k, b_row_stride, 1, "b"),
                          scales(a_scale, m, k, a_scale_row_stride, a_scale_col_stride, 1, "a_scale"),
                          scales(b_scale, n, k, b_scale_row_stride, b_scale_col_stride, b_block_rows, "b_scale")}));
  FS_API_TRY(check_fp8_arrays(a, a_scale, m, k, "a"));
  FS_API_TRY(check_fp8_arrays(b, b_scale, n, k, "b"));
  if (m == 0 || n == 0) return FS_OK;
  FS_API_TRY(api_check_array(out, width, "out"));
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (k == 0)
    return api_launched(m == 1 ? cudaMemsetAsync(out, 0, n * width, stream)
                               : cudaMemset2DAsync(out, out_row_stride * width, 0, n * width, m, stream), "zeroing out");
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
  if (y != nullptr)
    FS_API_TRY(check_rows(n, d, y_row_stride, "y"));
  else
    FS_API_TRY(check_fp8_form(q_type, n, d, q_row_stride, scale_row_stride, scale_col_stride, 1, "q"));
  const size_t width = width_of(x_type), w_width = width_of(w_type);
  if (rms == 1) mean = nullptr;             // not written
  FS_API_TRY(check_apart({y != nullptr ? matrix(y, n, d, y_row_stride, width, "y", true) : matrix(q, n, d, q_row_stride, 1, "q"),
                          y != nullptr ? Region{} : scales(scale, n, d, scale_row_stride, scale_col_stride, 1, "scale"),
                          vector(mean, n, 4, "mean"), vector(rstd, n, 4, "rstd")},
                         {matrix(x, n, d, x_row_stride, width, "x", true), vector(weight, d, w_width, "weight"),
                          vector(bias, d, w_width, "bias")}));
  FS_API_TRY(check_norm(n, d, x_type, weight, bias, w_type, rms));
  FS_API_TRY(api_check_array(x, width, "x"));
  if (mean != nullptr) FS_API_TRY(api_check_array(mean, 4, "mean"));
  if (rstd != nullptr) FS_API_TRY(api_check_array(rstd, 4, "rstd"));
  if (y != nullptr)
    FS_API_TRY(api_check_array(y, width, "y"));
  else
    FS_API_TRY(check_fp8_arrays(q, scale, n, d, "q"));
  FS_API_TRY(api_check_launch());
  const NormProblem p{x, x_type, n, d, x_row_stride, weight, bias, w_type, rms == 1, static_cast<float>(eps), y, y_row_stride,
                      mean, rstd, q, q_type, q_row_stride, scale, scale_row_stride, scale_col_stride};
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
  if (grad_x != nullptr && n > 0) FS_API_TRY(check_rows(n, d, grad_x_row_stride, "grad_x"));
  const bool sums = grad_weight != nullptr || grad_bias != nullptr;
  const size_t need = sums ? fs_layer_norm_backward_workspace_bytes(n, d) : 0;
  const bool own_block = workspace == nullptr && need <= FS_SMALL_WORKSPACE;
  if (sums && !own_block && workspace_bytes < need)
    return api_fail(FS_ERR_INVALID_ARG, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
  FS_API_TRY(check_apart({matrix(n > 0 ? grad_x : nullptr, n, d, grad_x_row_stride, width, "grad_x", true),
                          vector(grad_weight, d, w_width, "grad_weight"), vector(grad_bias, d, w_width, "grad_bias"),
                          vector(sums ? workspace : nullptr, static_cast<int64_t>(need), 1, "workspace")},
                         {matrix(g, n, d, g_row_stride, width, "g", true), matrix(x, n, d, x_row_stride, width, "x", true),
                          vector(n > 0 ? weight : nullptr, d, w_width, "weight"),
                          vector(rms == 0 ? mean : nullptr, n, 4, "mean"), vector(rstd, n, 4, "rstd")}));
  if (grad_weight != nullptr) FS_API_TRY(api_check_array(grad_weight, w_width, "grad_weight"));
  if (grad_bias != nullptr) FS_API_TRY(api_check_array(grad_bias, w_width, "grad_bias"));
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
  if (grad_x != nullptr) FS_API_TRY(api_check_array(grad_x, width, "grad_x"));
  if (!sums && grad_x == nullptr) return FS_OK;
  const CallLock lock(stream);
  if (own_block && sums) {
    TrainScratch* scratch = nullptr;
    FS_API_TRY(api_train_scratch(stream, &scratch));
    workspace = scratch->small;
  } else if (sums) {
    FS_API_TRY(api_check_array(workspace, 16, "workspace"));
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
