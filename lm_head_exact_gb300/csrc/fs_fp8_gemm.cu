// The 8-bit matrix product: how it is cut, and its launches (the kernel:
// fs_fp8_gemm.cuh).
#include "fs_fp8_gemm.cuh"

namespace fs {
namespace fp8 {

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 152;
  }
  return sms > 0 ? sms : 152;
}

namespace {

constexpr int kBand = 12;                      // column tiles that a wave of CTAs works on, by as many lane tiles

// How a product is cut: form, columns of a tile, splits of k.
struct Plan {
  Form form;
  int bn, splits;
};

Plan plan(int64_t m, int64_t n, int n_kb, int sms) {
  const auto split_of = [&](int64_t tiles, int ctas) {
    return tiles * ctas >= sms ? 1 : static_cast<int>(std::min<int64_t>({kMaxSplits / ctas, n_kb, sms / (tiles * ctas)}));
  };
  if (m <= kThinMaxRows) return Plan{kThin, thin_columns(m), split_of((n + kLanes - 1) / kLanes, 1)};
  Plan best{kWide, 192, 1};
  double best_time = 1e300;
  const struct { Form form; int bn, ctas; double clocks; } forms[] = {{kPair, 192, 2, 1000}, {kWide, 192, 1, 1000}};
  for (const auto& f : forms) {
    const int64_t tile_m = kLanes * f.ctas;
    const int64_t tiles = (m + tile_m - 1) / tile_m * ((n + f.bn - 1) / f.bn);
    const int splits = split_of(tiles, f.ctas);
    const double rounds = static_cast<double>((tiles * f.ctas + sms - 1) / sms);
    const double time = rounds * ((n_kb + splits - 1) / splits) * f.clocks + (splits > 1 ? 3000.0 : 0.0);
    if (time < best_time) {
      best_time = time;
      best = Plan{f.form, f.bn, splits};
    }
  }
  return best;
}

template <Form kForm, int kBN, bool kLaneScales, bool kColScales>
cudaError_t store(const Args& a, const Fp8Product& p, cudaStream_t stream) {
  if (a.splits > 1) return launch<kForm, kBN, false, kLaneScales, kColScales, true>(a, p.a, p.b, p.m, p.n, p.k, a.n_tiles, stream);
  const int most = sm_count() / (kForm == kPair ? 2 : 1);
  return launch<kForm, kBN, false, kLaneScales, kColScales, false>(a, p.a, p.b, p.m, p.n, p.k, std::min(a.n_tiles, most), stream);
}

template <int kBN>
cudaError_t thin(const Args& a, const Fp8Product& p, cudaStream_t stream) {
  return p.b.block_rows == 1 ? store<kThin, kBN, true, true>(a, p, stream) : store<kThin, kBN, false, true>(a, p, stream);
}

template <Form kForm, int kBN>
cudaError_t wide(const Args& a, const Fp8Product& p, cudaStream_t stream) {
  return p.b.block_rows == 1 ? store<kForm, kBN, true, true>(a, p, stream) : store<kForm, kBN, true, false>(a, p, stream);
}

}  // namespace
}  // namespace fp8

cudaError_t launch_fp8_matmul(const Fp8Product& p, int* err, cudaStream_t stream) {
  using namespace fp8;
  Args a{};
  a.n_kb = static_cast<int>(quant_blocks(p.k));
  const Plan s = plan(p.m, p.n, a.n_kb, sm_count());
  if (!(s.form == kThin ? set_tiles(&a, p.n, p.m, kLanes, s.bn, 1)
                        : set_tiles(&a, p.m, p.n, s.form == kPair ? 2 * kLanes : kLanes, s.bn, kBand)))
    return cudaErrorInvalidValue;
  a.splits = s.splits;
  a.out = p.out;
  a.out_type = p.out_type;
  a.out_stride = p.out_stride;
  a.err = err;
  if (s.form == kThin) return s.bn == 16 ? thin<16>(a, p, stream) : s.bn == 32 ? thin<32>(a, p, stream) : thin<64>(a, p, stream);
  return s.form == kPair ? wide<kPair, 192>(a, p, stream) : wide<kWide, 192>(a, p, stream);
}

}  // namespace fs
