// Paged decode attention for groups of sequences that share a prefix: the tail's partition kernel and the
// join of prefix and tail, the kTail instances of paged_decode_kernel.cuh.
//
// The prefix's states come from the prefill kernel (paged_prefill_kernel.cuh, Mask::kShared, shared_prefix.cu):
// a group's query rows are the rows of a tensor-core product with the prefix's keys, which are read once for
// the group (once per 256 rows) instead of once per sequence.  What follows the shared blocks is each
// sequence's own and streams through the partition kernel (View::kTail).
#include "cluster_decode.cuh"

namespace pkv {
cudaError_t prefix_cluster_ctas(int head_dim, int group, int num_seqs, int num_kv_heads, int visible_blocks, int* ctas) {
  // What the three kernels take depends on lengths that only the device knows: 10 us at least, 13 to 14 where a warp here
  // has 8 blocks (which takes 12), and less than here where it has 16 (16 sequences of 8 kv heads behind 2048 tokens: 14.3
  // and 18.7 us).
  return dispatch_cluster<View::kTail>(head_dim, group, [&](auto form) {
    return decltype(form)::ctas(num_seqs, num_kv_heads, visible_blocks, 13.2f, false, ctas);
  });
}

cudaError_t launch_prefix_cluster(const DecodeViewParams& p, int head_dim, int group, int ctas, cudaStream_t stream) {
  return dispatch_cluster<View::kTail>(
      head_dim, group, [&](auto form) { return decltype(form)::launch(p, ctas, stream); });
}

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
