// Chunked prefill with a sliding window and sinks: a chunk row at position P sees the cached tokens j <= P
// with j > P - window or j < sinks.  The kWindow instances of the prefill kernel (paged_prefill_kernel.cuh).
//
// A CTA's 256 / G tokens see the pages from the oldest key of its first row on, and the sink pages.  Those
// pages are one stream, sinks first, cut into steps of 128 keys like any other: a sink page shares its step
// with the first pages of the window, and no page that no row sees is read (its table entry may be anything).
//
// A window bounds a CTA's work, so calls with few tiles are short and the parts around the steps count.  One chunk of 512
// tokens, 16 q / 8 kv heads, window 1024 (32 tile pairs of 9 steps) takes 18.3 us in four splits with their own merge
// (25.7 unsplit).  Splits as a cluster that joins through its shared memory take 19.1: a quarter of four CTAs' 128 KB of
// states takes 5.7 us to read from there, longer than the merge kernel with its launch.
//
// Eight ragged chunks of 33 to 1001 tokens, 32 q / 8 kv heads, window 1024, take 71 us (590 TFLOP/s): 344 CTAs of 9 or 10 steps,
// 22 us each, on 152 SMs, of which the third wave fills a quarter.  Two whole prompts of 8192 tokens with a window of 4096 take
// 651 us, 1267 TFLOP/s, 0.66 of the measured bf16 burst rate, bound as the causal kernel is (3300 cycles a step, 2048 of them
// math).  Computing a share of the weights' exponentials on the FMA pipe instead of the special function unit only adds
// instructions (an eighth of them: 686 us, half: 776).
#include "paged_prefill_kernel.cuh"

namespace pkv {

cudaError_t launch_window_prefill(const PrefillParams& p, int head_dim, int group, int max_query_len,
                                  cudaStream_t stream) {
  return p.num_splits > 1 ? dispatch_prefill<true, Mask::kWindow>(p, head_dim, group, max_query_len, stream)
                          : dispatch_prefill<false, Mask::kWindow>(p, head_dim, group, max_query_len, stream);
}

}  // namespace pkv
