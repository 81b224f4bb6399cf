// rope_append: rotate q and k at their tokens' positions and append k and v to the paged cache.
//
// For every token t with slot s >= 0, frequency i < D / 2 and pos = positions[axis(i)][t]:
//   c = cos_sin[pos][i], n = cos_sin[pos][D / 2 + i]
//   x'[i] = x[i] c - x[i + D / 2] n,  x'[i + D / 2] = x[i + D / 2] c + x[i] n
// for each q row (to q_out) and each k row (to its cache slot); v rows are copied to their slot.  Each product,
// difference and sum is one fp32 operation rounded to nearest and the result is rounded to bf16, the steps of
// the fused decode step, so that a token's cache row has the same bits whichever call appended it.
//
// A lane owns the 16-byte chunks c and c + D / 16 of a row, the rotation's two halves, so D / 16 lanes cover a
// row and a warp 4 (D = 128) or 8 rows at a time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}
__device__ __forceinline__ float2 widen(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t narrow(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Rotates eight pairs: (a, b) are the chunks of the first and the second half.
__device__ __forceinline__ void rotate(uint4& a, uint4& b, const float (&cs)[8], const float (&sn)[8]) {
  uint32_t* aw = &a.x;
  uint32_t* bw = &b.x;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float2 x = widen(aw[w]), y = widen(bw[w]);
    aw[w] = narrow(__fsub_rn(__fmul_rn(x.x, cs[2 * w]), __fmul_rn(y.x, sn[2 * w])),
                   __fsub_rn(__fmul_rn(x.y, cs[2 * w + 1]), __fmul_rn(y.y, sn[2 * w + 1])));
    bw[w] = narrow(__fadd_rn(__fmul_rn(y.x, cs[2 * w]), __fmul_rn(x.x, sn[2 * w])),
                   __fadd_rn(__fmul_rn(y.y, cs[2 * w + 1]), __fmul_rn(x.y, sn[2 * w + 1])));
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const RopeAppendParams p) {
  pdl_trigger();
  pdl_wait();
  constexpr int kLanes = D / 16;          // lanes of a row
  constexpr int kRowsAtOnce = 32 / kLanes;
  constexpr int kChunks = D / 8;          // 16-byte chunks of a row
  const int lane = threadIdx.x & 31;
  const int c = lane % kLanes, sub = lane / kLanes;
  const int rows = p.num_q_heads + 2 * p.num_kv_heads;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); t < p.num_tokens; t += warps) {
    const int64_t slot = p.slot_mapping[t];
    if (slot < 0) continue;  // padding
    const bool stored = slot < p.num_slots;
    if (!stored && lane == 0) atomicOr(p.err, kErrSlot);
    float cs[8], sn[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int f = 8 * c + e;
      int64_t pos = p.positions[p.freq_axis[f] * p.axis_stride + t];
      if (pos < 0 || pos >= p.max_position) {
        atomicOr(p.err, kErrPosition);
        pos = pos < 0 ? 0 : p.max_position - 1;
      }
      cs[e] = __ldg(p.cos_sin + pos * D + f);
      sn[e] = __ldg(p.cos_sin + pos * D + D / 2 + f);
    }
    for (int r = sub; r < rows; r += kRowsAtOnce) {
      const bool is_q = r < p.num_q_heads;
      const int head = is_q ? r : (r - p.num_q_heads) % p.num_kv_heads;
      const bool is_v = r >= p.num_q_heads + p.num_kv_heads;
      if (!is_q && !stored) continue;
      const uint4* src = is_q ? static_cast<const uint4*>(p.q) + t * p.q_stride
                              : is_v ? static_cast<const uint4*>(p.v) + t * p.v_stride
                                     : static_cast<const uint4*>(p.k) + t * p.k_stride;
      uint4* dst = is_q ? static_cast<uint4*>(p.q_out) + t * p.q_out_stride + static_cast<int64_t>(head) * kChunks
                        : static_cast<uint4*>(is_v ? p.v_cache : p.k_cache) +
                              (((slot / kBlockTokens) * p.num_kv_heads + head) * kBlockTokens + slot % kBlockTokens) *
                                  kChunks;
      uint4 a = load_once(src + head * kChunks + c);
      uint4 b = load_once(src + head * kChunks + c + kLanes);
      if (!is_v) rotate(a, b, cs, sn);
      dst[c] = a;
      dst[c + kLanes] = b;
    }
  }
}

template <int D>
cudaError_t launch(const RopeAppendParams& p, int num_sms, cudaStream_t stream) {
  int64_t blocks = (p.num_tokens + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t cap = static_cast<int64_t>(num_sms) * 8;
  if (blocks > cap) blocks = cap;
  return launch_pdl(rope_append_kernel<D>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppendParams& p, int head_dim, int num_sms, cudaStream_t stream) {
  return head_dim == 128 ? launch<128>(p, num_sms, stream) : launch<64>(p, num_sms, stream);
}

}  // namespace pkv
