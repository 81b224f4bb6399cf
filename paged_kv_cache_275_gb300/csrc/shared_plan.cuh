// How the prefixes of a shared-prefix decode call are cut into splits over the CTAs of the prefix kernel
// (paged_prefill_kernel.cuh, Mask::kShared).  Every CTA works the plan out for itself from the call's lengths, a warp
// a CTA, so that nothing waits for another launch or for the host.
#pragma once

#include "decode_views.h"

namespace pkv {
namespace {

constexpr int kPlanKeys = 128;  // keys of a step
constexpr int kPlanRows = 256;  // query rows of a unit (a tile pair)

// The plan's estimate: microseconds of a prefix CTA besides its steps and of a step, with two query tiles and with one;
// bytes a microsecond that an SM streams of a tail, beside the prefix and when all SMs stream; and microseconds that a
// tail which outlasts the prefix takes to get going.  Chosen so that the splits they lead to are near the best of all
// splits, measured over 24 calls (16 to 128 sequences, one to six groups, prefixes of 200 to 16384 tokens, 1 to 8 kv heads):
// 46.2 us in the geometric mean (44.4 since the join fetches eight states ahead), against 47.0 with (4, 1.85, 1, 3.8e4,
// 3.6e4, 2), the choice for steps with weights in one part, 46.4 with (4, 2.6, 1.4, 4.1e4, 3.9e4, 2), 46.3 with (5, 2.6,
// 1.4, 4.4e4, 4.2e4, 2) and 47.3, with one call half as slow again, with (4, 2.45, 1.4, 3.8e4, 3.6e4, 2).
constexpr float kSharedCtaUs = 4.f, kSharedStepUs = 2.45f, kSharedOneTileStepUs = 1.4f;
constexpr float kTailEarlyRate = 4.4e4f, kTailLateRate = 4.2e4f, kTailLateUs = 2.f;

struct SharedGroup {
  int first, rows, keys;  // its sequences, and the tokens of its shared blocks
  bool fine;              // its bounds are in order
};

struct SharedPlan {
  bool fine;        // every group's bounds are in order: group_start starts at 0 or above, does not fall, and ends at
                    // num_seqs or below
  int split_steps;  // most key steps of a split; 0: nothing is shared
};

// One instance a head dim and group size: the plan of a call, worked out by a whole warp.
template <int D, int G>
struct SharedPlanner {
  static constexpr int kUnitRows = kPlanRows / G;  // sequences of a unit
  const int32_t* group_start;
  const int32_t* prefix_lens;
  const int32_t* context_lens;
  int num_groups, num_seqs, num_kv_heads, max_blocks_per_seq, num_sms, grid;

  __device__ __forceinline__ SharedGroup group(int g) const {
    SharedGroup x{0, 0, 0, true};
    if (g < num_groups) {
      const int a = __ldg(group_start + g), e = __ldg(group_start + g + 1), len = __ldg(prefix_lens + g);
      x.fine = a >= 0 && a <= e && e <= num_seqs;
      if (x.fine && a < e) {  // an empty group's length says nothing
        x.first = a;
        x.rows = e - a;
        x.keys = shared_prefix_blocks(len, max_blocks_per_seq) * kBlockTokens;
      }
    }
    return x;
  }
  __device__ __forceinline__ int units(const SharedGroup& x) const {
    return x.keys > 0 ? (x.rows + kUnitRows - 1) / kUnitRows * num_kv_heads : 0;
  }
  static __device__ __forceinline__ int steps(const SharedGroup& x) { return (x.keys + kPlanKeys - 1) / kPlanKeys; }

  // All groups' units are cut into splits of at most s steps, so that the CTAs finish about together whatever the
  // groups' sizes and lengths (the grid holds no less than one CTA a unit, so some s always fits).  The tail takes the
  // SMs that are left and, behind the prefix, all of them, so s is not the least that fits but the one with the least
  // estimated time for both: few long splits give the tail more SMs, and the join fewer states.
  __device__ __forceinline__ SharedPlan plan(int lane, const SharedGroup& mine) const {
    constexpr unsigned kAll = 0xffffffffu;
    SharedPlan r{};
    // The sequences' lengths, of at most 256 of them, requested together.
    const int every = (num_seqs + 255) / 256;
    int lens[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int b = (lane + 32 * i) * every;
      lens[i] = b < num_seqs ? __ldg(context_lens + b) : 0;
    }
    bool fine = true, two_tiles = false;
    int most = 1;      // the longest unit's steps
    float work = 0.f;  // steps of all units
    float tokens = 0.f;
    for (int g0 = 0; g0 < num_groups; g0 += 32) {
      const SharedGroup x = g0 == 0 ? mine : group(g0 + lane);
      fine = fine && x.fine;
      most = max(most, steps(x));
      work += static_cast<float>(units(x)) * static_cast<float>(steps(x));
      two_tiles = two_tiles || x.rows * G > kPlanRows / 2;
      tokens -= static_cast<float>(x.rows) * static_cast<float>(x.keys);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) tokens += static_cast<float>(max(0, lens[i]) * every);
    r.fine = __all_sync(kAll, fine);
    two_tiles = __any_sync(kAll, two_tiles);
    most = __reduce_max_sync(kAll, most);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      work += __shfl_xor_sync(kAll, work, off);
      tokens += __shfl_xor_sync(kAll, tokens, off);
    }
    const float tail = fmaxf(tokens, 0.f) * (4.f * D) * num_kv_heads;  // about how many bytes follow the shared blocks
    if (!r.fine || work == 0.f) return r;
    const int least_s = min(most, max(1, static_cast<int>(work / grid)));
    if (num_groups > 32) {  // many groups: the least s that fits, with a group a lane at a time (the longest unit's does)
      int lo = least_s, hi = most;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        int n = 0;
        for (int g0 = 0; g0 < num_groups; g0 += 32) {
          const SharedGroup x = group(g0 + lane);
          n += units(x) * ((steps(x) + mid - 1) / mid);
        }
        if (__reduce_add_sync(kAll, n) <= grid) hi = mid;
        else lo = mid + 1;
      }
      r.split_steps = lo;
      return r;
    }
    // The lane's candidate s: from the least that could fit on, an eighth of it apart; the last is the longest unit.
    const int s = lane == 31 ? most : min(most, least_s + lane * ((least_s + 7) / 8));
    const int u = units(mine), t = steps(mine);
    int n = 0;  // its CTAs
    for (int k = 0; k < num_groups; ++k)
      n += __shfl_sync(kAll, u, k) * ((__shfl_sync(kAll, t, k) + s - 1) / s);
    const int waves = (n + num_sms - 1) / num_sms;
    const float us = waves * (kSharedCtaUs + s * (two_tiles ? kSharedStepUs : kSharedOneTileStepUs));
    const float behind = tail - max(num_sms - n, 0) * kTailEarlyRate * us;
    float cost = us + (behind > 0.f ? kTailLateUs + behind / (num_sms * kTailLateRate) : 0.f);
    if (n > grid) cost = INFINITY;  // does not fit
    float best = cost;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) best = fminf(best, __shfl_xor_sync(kAll, best, off));
    r.split_steps = __shfl_sync(kAll, s, __ffs(__ballot_sync(kAll, cost == best)) - 1);
    return r;
  }
};

}  // namespace
}  // namespace pkv
