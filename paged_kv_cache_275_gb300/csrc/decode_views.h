// Internal interface of the windowed and the shared-prefix decode kernels (window_decode.cu, prefix_decode.cu), used by
// capi.cu: views of a sequence other than the whole of it.
#pragma once

#include "pkv_internal.h"

namespace pkv {

// What the views of a sequence other than the whole of it need besides.
struct DecodeViewParams : DecodeParams {
  int min_piece_blocks;  // window and tail views: the least blocks a piece is cut to
  // Window view: a sequence's last `window` tokens and its first `sinks` (both at most 16 * max_blocks_per_seq).
  int window;
  int sinks;
  // Tail view: groups of consecutive sequences whose first prefix_lens[g] / 16 blocks are shared.
  const int32_t* group_start;  // [num_groups + 1]
  const int32_t* prefix_lens;  // [num_groups]
  int num_groups;
  int32_t* ws_shared;          // workspace: int32 [num_seqs], each sequence's shared blocks
  float* ws_whole;             // workspace: fp32 states of pairs that lie whole in a piece, [num_seqs * num_kv_heads]
  const int32_t* ws_plan_ok;   // workspace: whether the groups are in order (0: the records are not to be used)
  const int2* ws_records;      // workspace: [num_seqs * num_kv_heads]: (first row, splits) of a pair's prefix states
  const float* ws_prefix_o;    // workspace: prefix states, rows of D floats (a pair's splits 256 rows apart)
  const float2* ws_prefix_ml;  // workspace: their (m, l)
};

// Blocks of a shared prefix of len tokens: whole blocks only, within the table.
__host__ __device__ __forceinline__ int shared_prefix_blocks(int len, int max_blocks_per_seq) {
  const int blocks = len > 0 ? len / kBlockTokens : 0;
  return blocks < max_blocks_per_seq ? blocks : max_blocks_per_seq;
}

// Pieces the partition kernel keeps in flight on the current device, as resident_partition_pieces.
cudaError_t resident_window_pieces(int head_dim, int group, int num_seqs, int* pieces);
cudaError_t resident_tail_pieces(int head_dim, int group, int num_seqs, int* pieces);
// Windowed decode, a cluster of `ctas` CTAs a (sequence, kv head): how many suit a call (0: it is too large for this
// form), and the launch (no workspace).
cudaError_t window_cluster_ctas(int head_dim, int group, int num_seqs, int num_kv_heads, int visible_blocks, int* ctas);
// Whether a windowed call of every number of sequences up to num_seqs takes that form.
cudaError_t window_cluster_takes_all(int head_dim, int group, int num_seqs, int num_kv_heads, int visible_blocks, bool* all);
cudaError_t launch_window_cluster(const DecodeViewParams& p, int head_dim, int group, int ctas, cudaStream_t stream);
// The same for sequences that share prefixes (each pair reads its group's blocks for itself).
cudaError_t prefix_cluster_ctas(int head_dim, int group, int num_seqs, int num_kv_heads, int visible_blocks, int* ctas);
cudaError_t launch_prefix_cluster(const DecodeViewParams& p, int head_dim, int group, int ctas, cudaStream_t stream);
// Windowed decode (partition, then join).
cudaError_t launch_window_decode(const DecodeViewParams& p, int head_dim, int group, cudaStream_t stream);
// What follows shared prefixes: the partition (behind launch_shared_prefix), and the join of both.
cudaError_t launch_tail_partition(const DecodeViewParams& p, int head_dim, int group, cudaStream_t stream);
cudaError_t launch_prefix_join(const DecodeViewParams& p, int head_dim, int group, cudaStream_t stream);

}  // namespace pkv
