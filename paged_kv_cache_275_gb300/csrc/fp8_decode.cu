// Decode and chunks of a few tokens over the 8-bit cache (fp8_decode.cuh): instances and launches.
#include "fp8_decode.cuh"

namespace pkv {
namespace {

// Which form a call takes: clusters if those of all its pairs run at once and are expected to be done before the stream form.
// Microseconds a call, measured (32 q and 8 kv heads of 128 dims, sequences of half a length to all of it; stream, clusters):
//   1 x 128 8.4, 5.2; 1 x 8192 14.1, 10.1; 1 x 32768 22.7, 23.0; 8 x 2048 15.4, 9.7; 8 x 8192 29, 24; 32 x 2048 30, 24;
//   32 x 8192 77, 77; of one kv head 16 x 8192 15.6, 13.4 and 16 x 32768 29, 35.
// As large as the pairs leave room for, up to 16 CTAs (1 x 8192: 12.6 with 8).
// The lengths are not known here, only the table's width.  In a table that is much wider than its sequences a call that clusters
// would do in 5.1, 7.6 or 9.5 us (one of 512, one of 4097, eight of 2048 tokens; 8192 blocks wide) takes the stream form, 8.0,
// 12.6 and 13.3; clusters over a context that does fill it would take, by the estimate, up to twice the stream form's time.
// A cluster's units come one after the other; the stream form has a second launch and a pass over the lengths; and either takes
// the bytes' time, of a batch whose tables are filled to three quarters.
constexpr float kClusterUs = 4.6f, kStreamUs = 10.5f;
constexpr float kBytesPerUs = 7.0e6f, kFilled = 0.75f;
template <int D, int NC>
constexpr float kClusterUnitUs = (D == 128 ? 1.05f : 1.4f) + 0.4f * (NC - 1);

template <int D, int NC>
struct Instance {
  using Stream = Few<D, NC, false>;
  using Cluster = Few<D, NC, true>;
  static constexpr int kMost = Stream::smem(kFp8LaunchSeqs);
  static constexpr int kClusterSmem = Cluster::smem(0);
  static_assert(Stream::kCtas * (kMost + 1024 + 256) <= 228 * 1024, "shared memory of an SM's CTAs");
  static_assert(Cluster::kCols * (D * 4 + 8) <= Cluster::kOffScales, "a cluster CTA's state lies in the rings");
  static constexpr int kSizes = 5;  // of clusters
  static_assert(1 << (kSizes - 1) == kMostCluster, "the largest cluster");
  static constexpr auto kStream = &few_rows_fp8_kernel<D, NC, false>;
  static constexpr auto kCluster = &few_rows_fp8_kernel<D, NC, true>;

  static cudaLaunchConfig_t cluster_config(unsigned pairs, int ctas, cudaStream_t stream, cudaLaunchAttribute (&attr)[2]) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(pairs * static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kClusterSmem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cfg;
  }

  // Clusters of 1, 2, 4, 8 and 16 CTAs that the current device holds at once; both kernels' attributes are set on the way.
  static cudaError_t prepare(const int** counts) {
    static std::mutex mu;
    static int known[64][kSizes];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (known[dev][0] == 0) {
      if ((e = cudaFuncSetAttribute(kStream, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost)) != cudaSuccess) return e;
      if ((e = cudaFuncSetAttribute(kStream, cudaFuncAttributePreferredSharedMemoryCarveout, 100)) != cudaSuccess) return e;
      if ((e = cudaFuncSetAttribute(kCluster, cudaFuncAttributeMaxDynamicSharedMemorySize, kClusterSmem)) != cudaSuccess) return e;
      if ((e = cudaFuncSetAttribute(kCluster, cudaFuncAttributePreferredSharedMemoryCarveout, 100)) != cudaSuccess) return e;
      if ((e = cudaFuncSetAttribute(kCluster, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) return e;
      for (int k = kSizes - 1; k >= 0; --k) {
        cudaLaunchAttribute attr[2];
        cudaLaunchConfig_t cfg = cluster_config(1, 1 << k, nullptr, attr);
        cfg.numAttrs = 1;
        if ((e = cudaOccupancyMaxActiveClusters(&known[dev][k], kCluster, &cfg)) != cudaSuccess) {
          known[dev][0] = 0;
          return e;
        }
      }
    }
    *counts = known[dev];
    return cudaSuccess;
  }

  static int choose(const int* counts, int64_t pairs, int max_blocks_per_seq) {
    const int units = (max_blocks_per_seq + Cluster::kUnitTiles - 1) / Cluster::kUnitTiles;
    int k = 0;
    while (k < kSizes - 1 && (1 << k) < units && pairs <= counts[k + 1]) ++k;
    if (pairs > counts[k]) return 0;
    const float bytes_us =
        kFilled / kBytesPerUs * static_cast<float>(pairs) * units * (2.f * Cluster::kUnitTiles * Cluster::kTile);
    const float units_us = kClusterUnitUs<D, NC> * static_cast<float>(units) / (1 << k);
    return kClusterUs + (units_us > bytes_us ? units_us : bytes_us) <= kStreamUs + bytes_us ? 1 << k : 0;
  }

  // CTAs a pair of a call; *fewer: whether every smaller batch, and narrower table, takes clusters too.  With as many CTAs a
  // pair the smallest batch is the first not to (the stream form has fewest bytes then), so one batch for each number of CTAs
  // is looked at; a table that is not too wide for a batch leaves none narrower that is, for a cluster's time over the stream
  // form's is linear in the units.
  static cudaError_t cluster_ctas(int num_seqs, int num_kv_heads, int max_blocks_per_seq, int* ctas, bool* fewer) {
    const int* counts = nullptr;
    const cudaError_t e = prepare(&counts);
    if (e != cudaSuccess) return e;
    auto takes = [&](int64_t seqs) { return choose(counts, seqs * num_kv_heads, max_blocks_per_seq); };
    *ctas = takes(num_seqs);
    *fewer = *ctas != 0 && takes(1) != 0;
    for (int k = 1; k < kSizes; ++k) {
      const int64_t first = counts[k] / num_kv_heads + 1;  // the smallest batch whose pairs get no more than 2^(k - 1)
      if (first < num_seqs) *fewer = *fewer && takes(first) != 0;
    }
    return cudaSuccess;
  }

  static cudaError_t launch(const Fp8AttentionParams& p, cudaStream_t stream) {
    const int* counts = nullptr;
    cudaError_t e = prepare(&counts);
    if (e != cudaSuccess) return e;
    const unsigned pairs = static_cast<unsigned>(p.num_seqs) * p.num_kv_heads;
    if (p.cluster_ctas) {
      cudaLaunchAttribute attr[2];
      const cudaLaunchConfig_t cfg = cluster_config(pairs, p.cluster_ctas, stream, attr);
      return cudaLaunchKernelEx(&cfg, kCluster, p);
    }
    e = launch_pdl(kStream, dim3(p.num_pieces), dim3(kThreads), Stream::smem(p.num_seqs), stream, p);
    if (e != cudaSuccess) return e;
    const unsigned cols = p.state_rows;
    // A pair has about as many states as pieces come to it.  Up to twice the eight that a warp fetches at once it takes them
    // alone.
    if (p.num_pieces > 16 * p.num_seqs * (p.num_kv_heads / p.unit_heads))
      return launch_pdl(join_fp8_kernel<D, 16>, dim3(pairs, cols), dim3(512), 0, stream, p);
    return launch_pdl(join_fp8_kernel<D, 1>, dim3(pairs, (cols + 3) / 4), dim3(128), 0, stream, p);
  }
};

template <typename F>
cudaError_t dispatch(int head_dim, int rows, F&& f) {
  switch (head_dim * 8 + fp8_columns(rows)) {
    case 64 * 8 + 1: return f(Instance<64, 1>{});
    case 64 * 8 + 2: return f(Instance<64, 2>{});
    case 64 * 8 + 3: return f(Instance<64, 3>{});
    case 128 * 8 + 1: return f(Instance<128, 1>{});
    case 128 * 8 + 2: return f(Instance<128, 2>{});
    case 128 * 8 + 3: return f(Instance<128, 3>{});
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_few_rows_fp8(const Fp8AttentionParams& p, int head_dim, cudaStream_t stream) {
  return dispatch(head_dim, p.state_rows, [&](auto instance) { return instance.launch(p, stream); });
}

cudaError_t fp8_cluster_ctas(int head_dim, int rows, int num_seqs, int num_kv_heads, int max_blocks_per_seq, int* ctas,
                             bool* fewer) {
  return dispatch(head_dim, rows, [&](auto instance) {
    return instance.cluster_ctas(num_seqs, num_kv_heads, max_blocks_per_seq, ctas, fewer);
  });
}

}  // namespace pkv
