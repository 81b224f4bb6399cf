// Attention of groups of single query tokens over the blocks that each group shares, as partial states: the
// kShared instances of the prefill kernel (paged_prefill_kernel.cuh).  prefix_decode.cu merges them with the
// states of what follows.
#include "paged_prefill_kernel.cuh"

namespace pkv {

cudaError_t launch_shared_prefix(const PrefillParams& p, int head_dim, int group, cudaStream_t stream) {
  return dispatch_prefill<true, Mask::kShared>(p, head_dim, group, 1, stream);
}

}  // namespace pkv
