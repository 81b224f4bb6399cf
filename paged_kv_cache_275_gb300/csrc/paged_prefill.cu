// Chunked causal prefill: the kCausal instances of the prefill kernel (paged_prefill_kernel.cuh), and the
// cache's tensor map for the decode kernels.
#include "paged_prefill_kernel.cuh"

namespace pkv {

cudaError_t encode_cache_map(CUtensorMap_st* map, const void* cache, int64_t rows, int head_dim) {
  return cache_map(map, cache, rows, head_dim);
}

cudaError_t launch_paged_prefill(const PrefillParams& p, int head_dim, int group, int max_query_len,
                                 cudaStream_t stream) {
  return p.num_splits > 1 ? dispatch_prefill<true, Mask::kCausal>(p, head_dim, group, max_query_len, stream)
                          : dispatch_prefill<false, Mask::kCausal>(p, head_dim, group, max_query_len, stream);
}

}  // namespace pkv
