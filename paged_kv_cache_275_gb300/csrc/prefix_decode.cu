// Paged decode attention for groups of sequences that share a prefix: the tail's partition kernel and the
// join of prefix and tail, the kTail instances of paged_decode_kernel.cuh.
//
// The prefix's states come from the prefill kernel (paged_prefill_kernel.cuh, Mask::kShared, shared_prefix.cu):
// a group's query rows are the rows of a tensor-core product with the prefix's keys, which are read once for
// the group (once per 256 rows) instead of once per sequence.  What follows the shared blocks is each
// sequence's own and streams through the partition kernel (View::kTail).
#include "paged_decode_kernel.cuh"

namespace pkv {
cudaError_t resident_tail_pieces(int head_dim, int group, int num_seqs, int* pieces) {
  return dispatch<View::kTail>(head_dim, group,
                               [&](auto inst) { return decltype(inst)::resident_pieces(num_seqs, pieces); });
}

cudaError_t launch_tail_partition(const DecodeViewParams& p, int head_dim, int group, cudaStream_t stream) {
  return dispatch<View::kTail>(head_dim, group, [&](auto inst) { return decltype(inst)::partition(p, stream); });
}

cudaError_t launch_prefix_join(const DecodeViewParams& p, int head_dim, int group, cudaStream_t stream) {
  return dispatch<View::kTail>(head_dim, group, [&](auto inst) { return decltype(inst)::merge(p, stream); });
}

}  // namespace pkv
