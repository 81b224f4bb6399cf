// Paged decode attention with a sliding window and sinks: the query token, at position P = L - 1, sees the
// cached tokens j with j > P - window or j < sinks.  The kWindow instances of the partition and merge kernels
// (paged_decode_kernel.cuh): the block stream holds the sink blocks and the window's blocks of each sequence,
// and nothing else of it is read (table entries in between may be anything, so their blocks can be freed).
#include "paged_decode_kernel.cuh"

namespace pkv {

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
