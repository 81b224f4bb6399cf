// Attention over the 8-bit cache, decode and chunks alike: out = softmax(scale q K^T) V over the tokens that a row sees.
//
// The simplest kernel that holds for every case: a CTA takes a query row and q head and goes through the row's tokens 128 at
// a time, a thread a token for the scores, then a thread a dim for the weighted sum, with the running maximum and sum of the
// softmax.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fp8_cache.h"
#include "fp8_format.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 128;

template <int D>
__global__ void __launch_bounds__(kThreads) attention_fp8_kernel(const Fp8AttentionParams p) {
  __shared__ float s_q[D], s_p[kThreads], s_red[kThreads / 32];
  __shared__ int64_t s_tile[kThreads];
  __shared__ float s_vs[kThreads];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, h = blockIdx.x, b = blockIdx.z;
  const int kvh = h / (p.num_q_heads / p.num_kv_heads);
  const int cap = p.max_blocks_per_seq * kBlockTokens;
  int64_t row = b;
  int len = p.context_lens[b];
  if (p.query_start) {
    const int q0 = p.query_start[b], chunk = p.query_start[b + 1] - q0, i = blockIdx.y;
    const bool bad = chunk < 0 || len < chunk || len > cap || q0 < 0 || static_cast<int64_t>(q0) + chunk > p.query_rows;
    if ((bad || chunk > p.max_query_len) && tid == 0 && h == 0 && i == 0) atomicOr(p.err, kErrLenTooLong);
    if (bad || i >= chunk) return;
    row = q0 + i;
    len = len - chunk + i + 1;
  } else {
    if (len < 0 || len > cap) {
      if (tid == 0 && h == 0) atomicOr(p.err, len < 0 ? kErrLenNegative : kErrLenTooLong);
      len = len < 0 ? 0 : cap;
    }
  }
  const int64_t at = (row * p.num_q_heads + h) * D;
  if (tid < D) s_q[tid] = __bfloat162float(static_cast<const __nv_bfloat16*>(p.q)[at + tid]);
  float m = -INFINITY, l = 0.f, acc = 0.f;
  const float scale = p.scale * 1.4426950408889634f;
  for (int t0 = 0; t0 < len; t0 += kThreads) {
    __syncthreads();
    const int t = t0 + tid;
    float s = -INFINITY;
    if (t < len) {
      int id = p.block_tables[static_cast<int64_t>(b) * p.max_blocks_per_seq + t / kBlockTokens];
      if (id < 0 || id >= p.num_blocks) {
        atomicOr(p.err, kErrBlockId);
        id = 0;
      }
      const int64_t tile = static_cast<int64_t>(id) * p.num_kv_heads + kvh;
      const uint8_t* k = p.k_cache + (tile * kBlockTokens + t % kBlockTokens) * D;
      float dot = 0.f;
      for (int d = 0; d < D; d += 2) {
        const float2 x = fp8_floats(*reinterpret_cast<const uint16_t*>(k + d));
        dot += x.x * s_q[d] + x.y * s_q[d + 1];
      }
      s = dot * fp8_scale(p.kv_scales[tile * 2 * kBlockTokens + t % kBlockTokens]) * scale;
      s_tile[tid] = tile * kBlockTokens + t % kBlockTokens;
      s_vs[tid] = fp8_scale(p.kv_scales[(tile * 2 + 1) * kBlockTokens + t % kBlockTokens]);
    }
    float top = s;
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    if ((tid & 31) == 0) s_red[tid >> 5] = top;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) top = fmaxf(top, s_red[w]);
    const float m_new = fmaxf(m, top), alpha = m == -INFINITY ? 0.f : exp2f(m - m_new);
    s_p[tid] = t < len ? exp2f(s - m_new) : 0.f;
    m = m_new;
    l *= alpha;
    acc *= alpha;
    __syncthreads();
    const int n = min(kThreads, len - t0);
    for (int x = 0; x < n; ++x) {
      l += s_p[x];
      if (tid < D) {
        const float2 v = fp8_floats(p.v_cache[s_tile[x] * D + tid]);
        acc += s_p[x] * (v.x * s_vs[x]);
      }
    }
  }
  if (tid < D) static_cast<__nv_bfloat16*>(p.out)[at + tid] = __float2bfloat16_rn(len > 0 ? acc / l : 0.f);
}

}  // namespace

cudaError_t launch_attention_fp8(const Fp8AttentionParams& p, int head_dim, cudaStream_t stream) {
  const dim3 grid(p.num_q_heads, p.query_start ? p.max_query_len : 1, p.num_seqs);
  return launch_pdl(head_dim == 128 ? attention_fp8_kernel<128> : attention_fp8_kernel<64>, grid, dim3(kThreads), 0, stream, p);
}

}  // namespace pkv
