// Paged decode attention for groups of sequences that share a prefix: the tail's partition kernel and the
// merge of prefix and tail.
//
//   out[b][h] = sum over the prefix and the tail of softmax weights times V, as one softmax:
//   with states (m, l, O) of disjoint parts of the keys, M = max m, out = sum 2^(m - M) O / sum 2^(m - M) l.
//
// The prefix's states come from the prefill kernel (paged_prefill_kernel.cuh, Mask::kShared, shared_prefix.cu):
// a group's query rows are the rows of a tensor-core product with the prefix's keys, which are read once for
// the group (once per 256 rows) instead of once per sequence.  What follows the shared blocks is each
// sequence's own and streams through the partition kernel (View::kTail).
#include "paged_decode_kernel.cuh"

namespace pkv {
namespace {

// One CTA per (sequence, kv head), one warp per q head, a lane D / 32 dims.  States are fetched kAhead at a
// time before any is combined.
template <int D, int G>
__global__ void __launch_bounds__(G * 32) prefix_merge_kernel(const DecodeParams p) {
  constexpr int kPieceFloats = Geo<D, G>::kPieceFloats;
  constexpr int kPer = D / 32;
  constexpr int kAhead = 8;
  const int hkv = p.num_kv_heads;
  const int b = blockIdx.x / hkv;
  const int kvh = blockIdx.x - b * hkv;
  const int g = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  pdl_trigger();
  pdl_wait();
  const int len = min(p.context_lens[b], p.max_blocks_per_seq * kBlockTokens);
  const int shared = *p.ws_plan_ok ? p.ws_shared[b] : 0;
  const size_t pair = blockIdx.x;

  float M = -INFINITY, l = 0.f;
  float acc[kPer];
#pragma unroll
  for (int x = 0; x < kPer; ++x) acc[x] = 0.f;
  // Adds up to kAhead states; row(u) and ml(u) are state u's D floats of O for this head and its (m, l).
  auto add = [&](int count, auto row, auto ml) {
    float2 s[kAhead];
    float a[kAhead][kPer];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      s[u] = make_float2(-INFINITY, 0.f);
      if (u < count) {
        s[u] = ml(u);
        const float* src = row(u) + lane * kPer;
        if constexpr (kPer == 4) {
          const float4 v = *reinterpret_cast<const float4*>(src);
          a[u][0] = v.x; a[u][1] = v.y; a[u][2] = v.z; a[u][3] = v.w;
        } else {
          const float2 v = *reinterpret_cast<const float2*>(src);
          a[u][0] = v.x; a[u][1] = v.y;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (u >= count || s[u].x == -INFINITY) continue;  // a state that saw no key
      const float mn = fmaxf(M, s[u].x);
      const float alpha = exp2f(M - mn), beta = exp2f(s[u].x - mn);
      l = l * alpha + s[u].y * beta;
#pragma unroll
      for (int x = 0; x < kPer; ++x) acc[x] = acc[x] * alpha + a[u][x] * beta;
      M = mn;
    }
  };

  if (shared > 0 && len > 0) {
    const int2 rec = p.ws_records[pair];
    for (int s0 = 0; s0 < rec.y; s0 += kAhead) {
      const size_t r0 = static_cast<size_t>(rec.x) + g + static_cast<size_t>(s0) * 256;
      add(min(kAhead, rec.y - s0), [&](int u) { return p.ws_prefix_o + (r0 + u * 256) * D; },
          [&](int u) { return p.ws_prefix_ml[r0 + u * 256]; });
    }
  }
  const int tail_shared = p.ws_shared[b];  // what the partition kernel skipped
  if (len > tail_shared * kBlockTokens) {
    const int rec_a = p.ws_pairs[2 * pair], wb = p.ws_pairs[2 * pair + 1], wa = rec_a >> 1;
    if (wa < 0 || wa > wb || wb >= p.num_partitions) {
      // The partition gave up on the pair's piece and recorded nothing (its timeout is flagged).
    } else if (wa == wb) {
      const float* state = p.ws_whole + pair * kPieceFloats;
      add(1, [&](int) { return state + g * D; }, [&](int) { return make_float2(state[G * D + g], state[G * D + G + g]); });
    } else {
      // With more pieces than items some pieces are empty and hold no state (piece w covers items
      // [w N / P, (w + 1) N / P)).
      const long long total = static_cast<long long>(hkv) * p.ws_prefix[p.num_seqs];
      const long long W = p.num_partitions;
      auto piece = [&](int w) { return p.ws_pieces + (static_cast<size_t>(w) * 2 + (w == wa ? (rec_a & 1) : 0)) * kPieceFloats; };
      for (int w0 = wa; w0 <= wb; w0 += kAhead)
        add(min(kAhead, wb - w0 + 1), [&](int u) { return piece(w0 + u) + g * D; },
            [&](int u) {
              const int w = w0 + u;
              if (W > total && w * total / W == (w + 1) * total / W) return make_float2(-INFINITY, 0.f);
              return make_float2(piece(w)[G * D + g], piece(w)[G * D + G + g]);
            });
    }
  }
  const float inv = l > 0.f ? 1.0f / l : 0.f;  // no token: zeros
  __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(p.out) +
                        (static_cast<size_t>(b) * p.num_q_heads + kvh * G + g) * D + lane * kPer;
  if constexpr (kPer == 4) {
    uint2 o;
    o.x = float2_to_bf16x2(acc[0] * inv, acc[1] * inv);
    o.y = float2_to_bf16x2(acc[2] * inv, acc[3] * inv);
    *reinterpret_cast<uint2*>(orow) = o;
  } else {
    *reinterpret_cast<uint32_t*>(orow) = float2_to_bf16x2(acc[0] * inv, acc[1] * inv);
  }
}

template <int D, int G>
cudaError_t merge(const DecodeParams& p, cudaStream_t stream) {
  return launch_pdl(prefix_merge_kernel<D, G>, dim3(static_cast<unsigned>(p.num_seqs) * p.num_kv_heads), dim3(G * 32),
                    0, stream, p);
}

}  // namespace

cudaError_t resident_tail_pieces(int head_dim, int group, int num_seqs, int* pieces) {
  return dispatch<View::kTail>(head_dim, group,
                               [&](auto inst) { return decltype(inst)::resident_pieces(num_seqs, pieces); });
}

cudaError_t launch_tail_partition(const DecodeParams& p, int head_dim, int group, cudaStream_t stream) {
  return dispatch<View::kTail>(head_dim, group, [&](auto inst) { return decltype(inst)::partition(p, stream); });
}

cudaError_t launch_prefix_merge(const DecodeParams& p, int head_dim, int group, cudaStream_t stream) {
  switch (head_dim * 16 + group) {
    case 64 * 16 + 1: return merge<64, 1>(p, stream);
    case 64 * 16 + 2: return merge<64, 2>(p, stream);
    case 64 * 16 + 4: return merge<64, 4>(p, stream);
    case 64 * 16 + 8: return merge<64, 8>(p, stream);
    case 128 * 16 + 1: return merge<128, 1>(p, stream);
    case 128 * 16 + 2: return merge<128, 2>(p, stream);
    case 128 * 16 + 4: return merge<128, 4>(p, stream);
    case 128 * 16 + 8: return merge<128, 8>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pkv
