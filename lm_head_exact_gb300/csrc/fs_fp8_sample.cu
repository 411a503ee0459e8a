// The sampler over an 8-bit head: the product's kernel (fs_fp8_gemm.cuh) with the
// sampling kernels' scan and finish in place of the output.
#include "fs_fp8_gemm.cuh"

namespace fs {
namespace {

using namespace fp8;

template <Form kForm, int kBN>
cudaError_t sample(const Args& a, const Fp8Matrix& h, const Fp8Matrix& W, const Problem& p, int64_t k, int ctas,
                   cudaStream_t stream) {
  constexpr bool kSwap = kForm == kThin;
  return W.block_rows == 1 ? launch<kForm, kBN, true, true, true, false>(a, h, W, p.B, p.V_local, k, ctas, stream)
                           : launch<kForm, kBN, true, !kSwap, kSwap, false>(a, h, W, p.B, p.V_local, k, ctas, stream);
}

// As few CTAs as give each the same number of tiles.
int even_share(int tiles, int most) {
  const int per = (tiles + most - 1) / most;
  return (tiles + per - 1) / per;
}

}  // namespace

cudaError_t launch_fp8_sample(const Problem& p, const Fp8Matrix& h, const Fp8Matrix& W, int64_t k, const Finish& f,
                              int* err, cudaStream_t stream) {
  Args a{};
  a.n_kb = static_cast<int>(quant_blocks(k));
  a.splits = 1;
  a.p = p;
  a.f = f;
  a.err = err;
  const int sms = sm_count();
  const int64_t m = p.B, n = p.V_local;
  if (m <= kThinMaxRows) {
    const int bn = thin_columns(m);
    if (!set_tiles(&a, n, m, kLanes, bn, 1)) return cudaErrorInvalidValue;
    const int ctas = even_share(a.n_tiles, sms);
    return bn == 16   ? sample<kThin, 16>(a, h, W, p, k, ctas, stream)
           : bn == 32 ? sample<kThin, 32>(a, h, W, p, k, ctas, stream)
                      : sample<kThin, 64>(a, h, W, p, k, ctas, stream);
  }
  const bool pair = m > kLanes;
  const int most = pair ? sms / 2 : sms;
  if (!set_tiles(&a, m, n, pair ? 2 * kLanes : kLanes, 192, 0)) return cudaErrorInvalidValue;
  int ctas = std::min(a.n_tiles, most);
  if (a.n_lt <= most) ctas = even_share(a.n_ct, most / a.n_lt) * a.n_lt;   // a multiple of the row tiles: a CTA keeps its rows
  return pair ? sample<kPair, 192>(a, h, W, p, k, ctas, stream) : sample<kWide, 192>(a, h, W, p, k, ctas, stream);
}

}  // namespace fs
