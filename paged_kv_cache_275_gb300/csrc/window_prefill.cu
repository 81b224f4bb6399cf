// Chunked prefill with a sliding window and sinks: a chunk row at position P sees the cached tokens j <= P
// with j > P - window or j < sinks.  The kWindow instances of the prefill kernel (paged_prefill_kernel.cuh).
//
// A CTA's 256 / G tokens see the pages from the oldest key of its first row on, and the sink pages.  Those
// pages are one stream, sinks first, cut into steps of 128 keys like any other: a sink page shares its step
// with the first pages of the window, and no page that no row sees is read (its table entry may be anything).
//
// A window bounds a unit's work (a unit: a tile pair and a kv head), so the parts around the steps count.  One chunk of 512
// tokens, 16 q / 8 kv heads, window 1024 (32 units of 10 steps) takes 18.5 us in four splits with their own merge (25.6
// unsplit).  Splits as a cluster that joins through its shared memory take 19.1: a quarter of four CTAs' 128 KB of states
// takes 5.7 us to read from there, longer than the merge kernel with its launch.
//
// Calls that fill the GPU keep their CTAs: a unit is 4 us of Q, first S and epilogue besides its steps of 1.7 us, of which a
// CTA a unit would add 2 more for launch and set-up, and the copies of a unit's first keys overlap the end of the unit before.
// Two whole prompts of 8192 tokens, 32 q / 8 kv heads, window 4096, take 632 us a call in a long run at the power cap, 1300
// TFLOP/s, 0.68 of the measured bf16 burst rate; in a burst of 30 calls 610 to 620 us, 0.70 (and there 652 with a CTA a unit and
// lane 0 alone in the MMA loop).  The softmax of a step bounds them, as it does the causal kernel.
// Eight ragged chunks of 33 to 1001 tokens, window 1024, take 68 us (610 TFLOP/s): 344 units of at most 9 steps, three rounds
// of 152 CTAs, of which the third fills a quarter.  Its 40 units as 80 of a query tile each, 71 otherwise; keys split over
// three CTAs each by a kernel beside, with a merge behind, 69 to 70.  What every CTA's registers hold counts: while lane 0
// alone went through the MMA loop, the two prompts took 756 us with the job kept in registers through the steps and 735 with
// it in shared memory.
// Computing a share of the weights' exponentials on the FMA pipe instead of the special function unit only adds instructions
// (an eighth of them 5 %, half 19 %).
#include <algorithm>

#include "paged_prefill_kernel.cuh"

namespace pkv {

cudaError_t launch_window_prefill(const PrefillParams& p, int head_dim, int group, int max_query_len,
                                  cudaStream_t stream) {
  for (int first = 0; first < p.num_seqs; first += kPrefillRankedSeqs) {  // (a call of more than that is not split)
    PrefillParams q = p;
    q.num_seqs = std::min(p.num_seqs - first, kPrefillRankedSeqs);
    q.query_start = p.query_start + first;
    q.context_lens = p.context_lens + first;
    q.block_tables = p.block_tables + static_cast<size_t>(first) * p.max_blocks_per_seq;
    const cudaError_t e = window_splits(p, group, max_query_len)
                              ? dispatch_prefill<true, Mask::kWindow>(q, head_dim, group, max_query_len, stream)
                              : dispatch_prefill<false, Mask::kWindow>(q, head_dim, group, max_query_len, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace pkv
