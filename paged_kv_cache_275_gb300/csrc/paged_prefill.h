// Internal interface of the chunked prefill kernel (paged_prefill.cu), used by capi.cu.
#pragma once

#include "pkv_internal.h"

namespace pkv {

struct PrefillParams {
  const void* q;               // bf16 [T][num_q_heads][head_dim]
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;  // prefix + chunk
  const int32_t* query_start;   // [num_seqs + 1]
  void* out;                    // bf16 [T][num_q_heads][head_dim]
  unsigned* err;
  int64_t num_blocks;
  int num_seqs;
  int num_q_heads;
  int num_kv_heads;
  int max_blocks_per_seq;
  int max_query_len;  // host's bound on the chunk lengths (sizes the grid)
  float scale;
  // Split-K over the key steps: each (tile pair, kv head, sequence) runs as num_splits CTAs, each over
  // a contiguous share of the key steps.  With num_splits > 1 the CTAs write fp32 partial states
  // (O unnormalised, m in base 2, l) to ws and a merge kernel forms out.
  int num_splits = 1;
  int ws_rows = 0;     // chunk rows per sequence in ws (the grid's tiles x chunk tokens per CTA)
  float* ws = nullptr;  // [split][seq][ws_rows][num_q_heads]: D floats of O; then the same index: (m, l)
  // Window: a row sees its last `window` tokens and the first `sinks` (both at most 16 * max_blocks_per_seq).
  int window = 0;
  int sinks = 0;
  int64_t query_rows = 0;  // rows of q and out: no chunk may reach past them
  // Windowed calls, of up to kPrefillRankedSeqs sequences a launch: with num_splits > 1 a unit (a tile pair of a chunk and a
  // kv head) runs as up to num_splits CTAs.  ws: [CTA][256 rows]: D floats of O; then the same index: (m, l).
  int4* ws_units = nullptr;     // [unit]: first row of out, chunk tokens, kv head, splits
  int32_t* ws_count = nullptr;  // units
  // Shared prefixes (one query token a sequence; q and out rows are sequences): groups of consecutive
  // sequences and the tokens they share.  ws: [CTA][256 rows]: D floats of O; then the same index: (m, l).
  const int32_t* group_start = nullptr;  // [num_groups + 1]
  const int32_t* prefix_lens = nullptr;  // [num_groups]
  int num_groups = 0;
  int shared_ctas = 0;               // grid: whole waves of num_sms
  int num_sms = 0;                   // CTAs of a wave (also windowed calls)
  int2* ws_records = nullptr;        // [num_seqs][num_kv_heads]: (first row in ws, splits 256 rows apart)
  int32_t* ws_plan_ok = nullptr;     // whether group_start is in order (records are valid)
};

// Chunked prefill attention (tensor cores); grid covers max_query_len rows per sequence.
cudaError_t launch_paged_prefill(const PrefillParams& p, int head_dim, int group, int max_query_len,
                                 cudaStream_t stream);
// The same for rows with a window and sinks, and for shared prefixes (partial states).
cudaError_t launch_window_prefill(const PrefillParams& p, int head_dim, int group, int max_query_len,
                                  cudaStream_t stream);
cudaError_t launch_shared_prefix(const PrefillParams& p, int head_dim, int group, cudaStream_t stream);
// Chunk tokens one CTA covers (two 128-row tiles of 128 / group tokens).
inline int prefill_cta_tokens(int group) { return 256 / group; }
// Workspace bytes of a split call: partial states of every split.
inline size_t prefill_workspace_bytes(int num_seqs, int max_query_len, int num_q_heads, int num_kv_heads,
                                      int head_dim, int num_splits) {
  if (num_splits <= 1) return 0;
  const int cta = prefill_cta_tokens(num_q_heads / num_kv_heads);
  const size_t rows = static_cast<size_t>((max_query_len + cta - 1) / cta) * cta;
  return static_cast<size_t>(num_splits) * num_seqs * rows * num_q_heads * (head_dim + 2) * sizeof(float);
}
// Most sequences whose units a CTA ranks, a thread each; and CTAs of a split windowed call at most.
constexpr int kPrefillRankedSeqs = 320;
constexpr int kWindowSplitCtas = 160;
// No more units than these in a windowed call.
inline int64_t window_units(const PrefillParams& p, int group, int max_query_len) {
  const int64_t cta = prefill_cta_tokens(group);
  const int64_t grid = p.num_seqs * ((max_query_len + cta - 1) / cta), rows = p.query_rows / cta + p.num_seqs;
  return (grid < rows ? grid : rows) * p.num_kv_heads;
}
// Whether its units are split: if two CTAs each are no more than SMs.
inline bool window_splits(const PrefillParams& p, int group, int max_query_len) {
  return p.num_splits > 1 && 2 * window_units(p, group, max_query_len) <= p.num_sms;
}
// Workspace of a windowed call that splits: states, then the units and their count.
struct WindowSplitLayout {
  size_t units, count, bytes;
  WindowSplitLayout(int head_dim, int num_splits) {
    units = static_cast<size_t>(kWindowSplitCtas) * 256 * (head_dim + 2) * sizeof(float);
    count = units + kWindowSplitCtas / 2 * sizeof(int4);
    bytes = num_splits > 1 ? count + 16 : 0;
  }
};

}  // namespace pkv
