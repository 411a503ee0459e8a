// The 8-bit matrix product: how it is cut, and its launches (the kernel:
// fs_fp8_gemm.cuh).
#include <atomic>

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

// Clusters of `size` CTAs of one to an SM that this GPU holds at a time: fewer
// than its SMs give, as clusters do not cross its groups of SMs (152 SMs: 76 of 2,
// 46 of 3, 36 of 4, 28 of 5, 23 of 6, 15 of 7 or 8).
int clusters_at_once(int size, int sms) {
  if (size == 1) return sms;
  static std::atomic<int> known[64][kMaxSplits + 1];       // (0: not asked yet)
  int dev = 0;
  const bool cached = cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64;
  if (cached) {
    const int n = known[dev][size].load(std::memory_order_relaxed);
    if (n > 0) return n;
  }
  using S = Shape<kThin, 16, false, true>;
  constexpr auto fn = kernel<kThin, 16, false, false, true, true>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(size));
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (raise_smem_limit<fn>(dev, S::kSmem) != cudaSuccess || cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess ||
      n <= 0) {
    cudaGetLastError();
    return std::max(1, sms / (size + 1));
  }
  if (cached) known[dev][size].store(n, std::memory_order_relaxed);
  return n;
}

// The cut of the least time, in clocks: a block of k takes a tile's 1000 (of
// kThin some 400 where bytes are not what counts), a CTA's start and end 14000,
// a joined tile 2000 more.  (16 x 6144 x 4096, 48 tiles: 18.3 us with 3 splits, whose
// 48 clusters do not run at once, 11.5 with 1 or 2.)
Plan plan(int64_t m, int64_t n, int n_kb, int sms) {
  constexpr double kEnds = 14000, kJoin = 2000;
  struct Choice {
    Form form;
    int bn, ctas;
    double clocks;
  };
  const bool few = m <= kThinMaxRows;
  const Choice thin[] = {{kThin, few ? thin_columns(m) : 0, 1, 400}}, wide[] = {{kPair, 192, 2, 1000}, {kWide, 192, 1, 1000}};
  Plan best{};
  double best_time = 1e300;
  for (const Choice* f = few ? thin : wide; f != (few ? thin + 1 : wide + 2); ++f) {
    const int64_t tile_m = f->form == kPair ? 2 * kLanes : kLanes;
    const int64_t tiles = few ? (n + kLanes - 1) / kLanes : (m + tile_m - 1) / tile_m * ((n + f->bn - 1) / f->bn);
    for (int splits = 1; splits <= std::min(kMaxSplits / f->ctas, n_kb); ++splits) {
      if (splits > 1 && tiles * f->ctas * (splits - 1) >= sms) break;   // (the SMs were busy with fewer)
      const int at_once = splits > 1 ? clusters_at_once(f->ctas * splits, sms) : sms / f->ctas;
      const double rounds = static_cast<double>((tiles + at_once - 1) / at_once);
      const double work = (n_kb + splits - 1) / splits * f->clocks;
      const double time = splits > 1 ? rounds * (work + kEnds + kJoin) : rounds * work + kEnds;
      if (time < best_time) {
        best_time = time;
        best = Plan{f->form, f->bn, splits};
      }
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
  if (fp8_rows_takes(p)) return launch_fp8_rows(p, stream);
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
