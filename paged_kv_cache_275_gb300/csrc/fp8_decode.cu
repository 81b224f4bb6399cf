// Decode and chunks of a few tokens over the 8-bit cache (fp8_decode.cuh): instances and launches.
#include "fp8_decode.cuh"

namespace pkv {
namespace {

// The cache's codes as rows of 128 bytes (a token of 128 dims, or two of 64), a box the rows of a unit's heads of one block,
// swizzled.  (With boxes of 64-byte rows, 64 dims are copied at 5.0 TB/s, so XXX.)
cudaError_t code_map(CUtensorMap* map, const void* cache, int64_t bytes, int box_bytes) {
  const cuuint64_t dims[2] = {128, static_cast<cuuint64_t>(bytes / 128)};
  const cuuint64_t strides[1] = {128};
  const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_bytes / 128)};
  return encode_code_map(map, cache, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int D, int NC>
cudaError_t launch(const Fp8AttentionParams& p, cudaStream_t stream) {
  constexpr int kMost = Few<D, NC>::smem(kFp8LaunchSeqs);
  static_assert(Few<D, NC>::kCtas * (kMost + 1024 + 256) <= 228 * 1024, "shared memory of an SM's CTAs");
  static std::mutex mu;
  static uint64_t ready = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!(dev < 64 && ((ready >> dev) & 1u))) {
      e = cudaFuncSetAttribute(&few_rows_fp8_kernel<D, NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
      if (e != cudaSuccess) return e;
      e = cudaFuncSetAttribute(&few_rows_fp8_kernel<D, NC>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
      if (e != cudaSuccess) return e;
      if (dev < 64) ready |= uint64_t{1} << dev;
    }
  }
  CUtensorMap mk, mv;
  const int64_t bytes = p.num_blocks * p.num_kv_heads * Few<D, NC>::kTile;
  if ((e = code_map(&mk, p.k_cache, bytes, p.unit_heads * Few<D, NC>::kTile)) != cudaSuccess) return e;
  if ((e = code_map(&mv, p.v_cache, bytes, p.unit_heads * Few<D, NC>::kTile)) != cudaSuccess) return e;
  e = launch_pdl(few_rows_fp8_kernel<D, NC>, dim3(p.num_pieces), dim3(kThreads), Few<D, NC>::smem(p.num_seqs), stream, p, mk, mv);
  if (e != cudaSuccess) return e;
  const unsigned pairs = static_cast<unsigned>(p.num_seqs) * p.num_kv_heads;
  const unsigned cols = p.state_rows;
  // Few pairs have many states each.
  if (pairs * cols <= 1216) return launch_pdl(join_fp8_kernel<D, 8>, dim3(pairs, cols), dim3(256), 0, stream, p);
  return launch_pdl(join_fp8_kernel<D, 1>, dim3(pairs, (cols + 3) / 4), dim3(128), 0, stream, p);
}

}  // namespace

cudaError_t launch_few_rows_fp8(const Fp8AttentionParams& p, int head_dim, cudaStream_t stream) {
  const int nc = fp8_columns(p.state_rows);
  switch (head_dim * 8 + nc) {
    case 64 * 8 + 1: return launch<64, 1>(p, stream);
    case 64 * 8 + 2: return launch<64, 2>(p, stream);
    case 64 * 8 + 3: return launch<64, 3>(p, stream);
    case 64 * 8 + 4: return launch<64, 4>(p, stream);
    case 128 * 8 + 1: return launch<128, 1>(p, stream);
    case 128 * 8 + 2: return launch<128, 2>(p, stream);
    case 128 * 8 + 3: return launch<128, 3>(p, stream);
    case 128 * 8 + 4: return launch<128, 4>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pkv
