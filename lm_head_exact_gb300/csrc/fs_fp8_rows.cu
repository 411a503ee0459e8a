// The 8-bit matrix product of few rows of a (tokens of a decode step) and a b that
// is read in some microseconds:
//
//   out[i, j] = sum_b sa[i, b] sb[j, b] (sum_{k in block b} a[i, k] b[j, k])
//
// Such a product is bound by what a kernel does before its first load and after its
// last.  So nothing is staged: warps load b's rows into registers in the order in
// which mma.sync wants them, multiply, scale each block's sum and add it up.  A
// block of threads takes 16 rows of b and 8 of a; its 8 warps take its blocks of k in
// turn, and are joined through shared memory at the end, in their order.  The form
// with barriers, TMEM and a cluster around the same bytes (fs_fp8_gemm.cuh), which
// reads b once whatever the tokens, is faster where there is more to read
// (launch_fp8_rows says from where).  us, this kernel and that form:
//
//    1 x  1024 x  1024    1.8   4.5        16 x  1024 x 1024    1.9   5.0
//    1 x  4096 x  4096    5.1   8.6        16 x  4096 x 4096    7.9   8.9
//    1 x  6144 x  4096    7.6  10.8        16 x  6144 x 4096   10.9  11.6
//    1 x  4096 x 14336   12.8  15.8        16 x  8192 x 4096   13.6  12.3
//    1 x 28672 x  4096   23.3  24.0        32 x  4096 x 4096   13.2   9.8
//    4 x 128256 x 4096   92.8  82.9        64 x  1024 x 1024    3.7   6.9
//
// (32 rows of b a block of threads, or one block of k at a time instead of two: the
// same within a tenth, either way.)
#include "fs_fp8.cuh"
#include "fs_fp8.h"
#include "fs_internal.h"

namespace fs {
namespace {

constexpr int kWarps = 8;
constexpr int kTokens = 8, kRows = 16;     // of a and b a block of threads takes
constexpr int kDeep = 2;                   // blocks of k a warp loads at a time

struct Rows {
  const uint8_t* q;
  int64_t stride;
  const float* scale;
  int64_t s_row, s_col;
  int shift;                   // of a row's number to its scale's: 0 or 7
  int64_t rows;
};

struct RowsArgs {
  Rows a, b;
  int64_t k;
  unsigned groups;             // of kTokens rows of a
  void* out;
  int out_type;
  int64_t out_stride;
};

// d += w x^T over 32 elements of k: 16 rows of b by 8 of a.
template <bool kE5B, bool kE5A>
__device__ __forceinline__ void mma_rows(float (&d)[4], uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, uint32_t x0,
                                         uint32_t x1) {
#define FS_MMA_ROWS(B, A)                                                                                             \
  asm volatile("mma.sync.aligned.m16n8k32.row.col.f32." B "." A ".f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, " \
               "{%0, %1, %2, %3};"                                                                                    \
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])                                                       \
               : "r"(w0), "r"(w1), "r"(w2), "r"(w3), "r"(x0), "r"(x1))
  if constexpr (kE5B && kE5A) FS_MMA_ROWS("e5m2", "e5m2");
  else if constexpr (kE5B) FS_MMA_ROWS("e5m2", "e4m3");
  else if constexpr (kE5A) FS_MMA_ROWS("e4m3", "e5m2");
  else FS_MMA_ROWS("e4m3", "e4m3");
#undef FS_MMA_ROWS
}

// b: what further groups of tokens read again comes from L2.
__device__ __forceinline__ uint4 load_once(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// 16 bytes of a row, of which `left` exist.
__device__ __forceinline__ uint4 load_ends(const uint8_t* p, int left) {
  if (left >= 16) return *reinterpret_cast<const uint4*>(p);
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  for (int i = 0; i < left; ++i) reinterpret_cast<uint8_t*>(&v)[i] = p[i];
  return v;
}

// A lane (g = lane / 4, t = lane % 4) holds, of a block's 128 elements, 16 t .. and
// 64 + 16 t .. of rows g and g + 8: mma.sync sums over k in any order that
// both operands share, so that a load takes 16 bytes and four lanes 64 in a row.
template <bool kE5B, bool kE5A>
__global__ void __launch_bounds__(kWarps * 32, 2) rows_kernel(const RowsArgs p) {
  constexpr int kPitch = kRows + 1;
  __shared__ float parts[kWarps][kTokens * kPitch];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / p.groups) * kRows;
  const int64_t token0 = static_cast<int64_t>(blockIdx.x % p.groups) * kTokens;
  const int whole = static_cast<int>(p.k / kQuantBlock);
  // rows of b and a beyond the last one stand for it, and are dropped
  const uint8_t *w_at[2], *x_at = p.a.q + min(token0 + g, p.a.rows - 1) * p.a.stride + 16 * t;
  const float *ws_at[2], *xs_at[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t r = min(row0 + 8 * h + g, p.b.rows - 1);
    w_at[h] = p.b.q + r * p.b.stride + 16 * t;
    ws_at[h] = p.b.scale + (r >> p.b.shift) * p.b.s_row;
    xs_at[h] = p.a.scale + min(token0 + 2 * t + h, p.a.rows - 1) * p.a.s_row;
  }
  const auto skip = [&](int blocks) {                      // moves every pointer on
    x_at += blocks * kQuantBlock;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      w_at[h] += blocks * kQuantBlock;
      ws_at[h] += blocks * p.b.s_col;
      xs_at[h] += blocks * p.a.s_col;
    }
  };
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};                 // rows g, g + 8 by tokens 2 t, 2 t + 1
  const auto add = [&](const uint4 (&w)[2][2], const uint4 (&x)[2], const float (&ws)[2], const float (&xs)[2]) {
    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      mma_rows<kE5B, kE5A>(d, w[0][c].x, w[1][c].x, w[0][c].y, w[1][c].y, x[c].x, x[c].y);
      mma_rows<kE5B, kE5A>(d, w[0][c].z, w[1][c].z, w[0][c].w, w[1][c].w, x[c].z, x[c].w);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] = fmaf(d[e], xs[e & 1] * ws[e >> 1], sum[e]);
  };
  skip(warp);
  pdl_wait();
  int kb = warp;
#pragma unroll 1
  for (; kb < whole; kb += kWarps * kDeep) {
    uint4 w[kDeep][2][2], x[kDeep][2];
    float ws[kDeep][2], xs[kDeep][2];
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      if (kb + kWarps * d >= whole) break;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int c = 0; c < 2; ++c) w[d][h][c] = load_once(w_at[h] + d * (kWarps * kQuantBlock) + 64 * c);
        ws[d][h] = ws_at[h][d * kWarps * p.b.s_col];
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        x[d][h] = *reinterpret_cast<const uint4*>(x_at + d * (kWarps * kQuantBlock) + 64 * h);
        xs[d][h] = xs_at[h][d * kWarps * p.a.s_col];
      }
    }
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      if (kb + kWarps * d >= whole) break;
      add(w[d], x[d], ws[d], xs[d]);
    }
    skip(kWarps * kDeep);
  }
  const int rest = static_cast<int>(p.k - static_cast<int64_t>(whole) * kQuantBlock);
  if (rest > 0 && whole % kWarps == warp) {                // the last block's elements that exist
    skip(whole - kb);
    uint4 w[2][2], x[2];
    float ws[2], xs[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int c = 0; c < 2; ++c) w[h][c] = load_ends(w_at[h] + 64 * c, rest - 64 * c - 16 * t);
      x[h] = load_ends(x_at + 64 * h, rest - 64 * h - 16 * t);
      ws[h] = *ws_at[h];
      xs[h] = *xs_at[h];
    }
    add(w, x, ws, xs);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) parts[warp][(2 * t + (e & 1)) * kPitch + 8 * (e >> 1) + g] = sum[e];
  __syncthreads();
  const int token = threadIdx.x / kRows, row = threadIdx.x % kRows;
  if (token >= kTokens || token0 + token >= p.a.rows || row0 + row >= p.b.rows) return;
  float s = parts[0][token * kPitch + row];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) s += parts[w][token * kPitch + row];
  const int64_t to = (token0 + token) * p.out_stride + row0 + row;
  if (p.out_type == FS_TYPE_F32)
    static_cast<float*>(p.out)[to] = s;
  else if (p.out_type == FS_TYPE_BF16)
    static_cast<__nv_bfloat16*>(p.out)[to] = __float2bfloat16_rn(s);
  else
    static_cast<__half*>(p.out)[to] = __float2half_rn(s);
}

Rows rows_of(const Fp8Matrix& m, int64_t rows) {
  return Rows{static_cast<const uint8_t*>(m.q), m.stride, m.scale, m.s_row, m.s_col, m.block_rows == 1 ? 0 : 7, rows};
}

int64_t groups_of(int64_t m) { return (m + kTokens - 1) / kTokens; }

}  // namespace

// One group of tokens reads b once, as the other form does: up to 2^27 bytes of it.
// Further groups read it from L2: up to 3 * 2^24 in all, and 64 tokens.  (Times above.)
bool fp8_rows_takes(const Fp8Product& p) {
  const int64_t groups = groups_of(p.m), most = groups == 1 ? int64_t(1) << 27 : int64_t(3) << 24;
  return p.m <= 64 && p.n <= most && p.k <= most && groups * p.n * p.k <= most;
}

cudaError_t launch_fp8_rows(const Fp8Product& p, cudaStream_t stream) {
  const unsigned groups = static_cast<unsigned>(groups_of(p.m));
  const RowsArgs a{rows_of(p.a, p.m), rows_of(p.b, p.n), p.k, groups, p.out, p.out_type, p.out_stride};
  const bool e5_b = p.b.type == FS_TYPE_E5M2, e5_a = p.a.type == FS_TYPE_E5M2;
  const auto kernel = e5_b ? (e5_a ? rows_kernel<true, true> : rows_kernel<true, false>)
                           : (e5_a ? rows_kernel<false, true> : rows_kernel<false, false>);
  return launch_kernel(kernel, dim3(static_cast<unsigned>((p.n + kRows - 1) / kRows) * groups), dim3(kWarps * 32), 0, stream,
                       true, a);
}

}  // namespace fs
