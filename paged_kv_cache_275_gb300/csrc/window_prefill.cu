// Chunked prefill with a sliding window and sinks: a chunk row at position P sees the cached tokens j <= P
// with j > P - window or j < sinks.  The kWindow instances of the prefill kernel (paged_prefill_kernel.cuh).
//
// A CTA's 256 / G tokens see the pages from the oldest key of its first row on, and the sink pages.  Those
// pages are one stream, sinks first, cut into steps of 128 keys like any other: a sink page shares its step
// with the first pages of the window, and no page that no row sees is read (its table entry may be anything).
#include "paged_prefill_kernel.cuh"

namespace pkv {

cudaError_t launch_window_prefill(const PrefillParams& p, int head_dim, int group, int max_query_len,
                                  cudaStream_t stream) {
  return p.num_splits > 1 ? dispatch_prefill<true, Mask::kWindow>(p, head_dim, group, max_query_len, stream)
                          : dispatch_prefill<false, Mask::kWindow>(p, head_dim, group, max_query_len, stream);
}

}  // namespace pkv
