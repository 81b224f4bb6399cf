// Paged decode attention with a sliding window and sinks: the query token, at position P = L - 1, sees the
// cached tokens j with j > P - window or j < sinks.
//
// Two forms.  Large calls are the kWindow instances of the partition and join kernels (paged_decode_kernel.cuh): the block
// stream holds the sink blocks and the window's blocks of each sequence, and nothing else of it is read (table entries
// in between may be anything, so their blocks can be freed).  Calls with few (sequence, kv head) pairs and short windows
// are bound by latency, not by bytes, and take the cluster form (cluster_decode.cuh).
#include "cluster_decode.cuh"

namespace pkv {

// The partition and join kernels take 8.7 us besides streaming if the pairs are many; of few pairs the join has so many
// states that they lose up to 16 blocks a warp.
constexpr float kOtherFormUs = 18.4f;

cudaError_t window_cluster_ctas(int head_dim, int group, int num_seqs, int num_kv_heads, int visible_blocks, int* ctas) {
  return dispatch_cluster<View::kWindow>(head_dim, group, [&](auto form) {
    return decltype(form)::ctas(num_seqs, num_kv_heads, visible_blocks, kOtherFormUs, true, ctas);
  });
}

cudaError_t window_cluster_takes_all(int head_dim, int group, int num_seqs, int num_kv_heads, int visible_blocks, bool* all) {
  return dispatch_cluster<View::kWindow>(head_dim, group, [&](auto form) {
    return decltype(form)::takes_all(num_seqs, num_kv_heads, visible_blocks, kOtherFormUs, true, all);
  });
}

cudaError_t launch_window_cluster(const DecodeViewParams& p, int head_dim, int group, int ctas, cudaStream_t stream) {
  return dispatch_cluster<View::kWindow>(
      head_dim, group, [&](auto form) { return decltype(form)::launch(p, ctas, stream); });
}

cudaError_t resident_window_pieces(int head_dim, int group, int num_seqs, int* pieces) {
  return dispatch<View::kWindow>(head_dim, group,
                                 [&](auto inst) { return decltype(inst)::resident_pieces(num_seqs, pieces); });
}

cudaError_t launch_window_decode(const DecodeViewParams& p, int head_dim, int group, cudaStream_t stream) {
  return dispatch<View::kWindow>(head_dim, group, [&](auto inst) {
    const cudaError_t e = decltype(inst)::partition(p, stream);
    return e != cudaSuccess ? e : decltype(inst)::merge(p, stream);
  });
}

}  // namespace pkv
