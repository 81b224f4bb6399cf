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

#include "rope_append.h"

namespace pkv {
namespace {

// Bound by HBM: every row is read once and written once.  32773 tokens of 32 q / 8 kv heads, D 128 (823 MB) take 128.6 us,
// 6.40 TB/s, 0.96 of the measured copy bandwidth; 4096 tokens (103 MB) 19.8 us, where a wave of loads and stores and the
// launch's start and end are a fifth of the time.  A warp takes a token, so that the angles are fetched once for all its
// rows.  Rows of a lane in flight: with 1 131 us, with 3 145, with 4 142 (74 registers); CTAs of 256 threads instead of 128
// leave the 4096 tokens' last wave uneven (21.3 us with one row in flight).
constexpr int kThreads = 128;
constexpr int kAhead = 2;      // rows of a lane in flight
constexpr int kMostCtas = 16;  // per SM; beyond that a warp takes several tokens

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
  const int64_t items = p.num_tokens * p.parts;  // a token's rows in `parts` parts
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); item < items;
       item += warps) {
    const int64_t t = item / p.parts;
    const int part = static_cast<int>(item - t * p.parts);
    const int first = part * kRowsAtOnce + sub, step = p.parts * kRowsAtOnce;
    uint4 a[kAhead], b[kAhead];
    auto fetch = [&](int r0) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int r = r0 + k * step;
        if (r >= rows) continue;
        const int kr = r - p.num_q_heads, vr = kr - p.num_kv_heads;
        const uint4* src = kr < 0 ? static_cast<const uint4*>(p.q) + t * p.q_stride + r * kChunks
                           : vr < 0 ? static_cast<const uint4*>(p.k) + t * p.k_stride + kr * kChunks
                                    : static_cast<const uint4*>(p.v) + t * p.v_stride + vr * kChunks;
        a[k] = load_once(src + c);
        b[k] = load_once(src + c + kLanes);
      }
    };
    // The first rows are on their way while the position and then its table row are looked up.
    fetch(first);
    const int64_t slot = p.slot_mapping[t];
    if (slot < 0) continue;  // padding
    const bool stored = slot < p.num_slots;
    if (!stored && lane == 0 && part == 0) atomicOr(p.err, kErrSlot);
    auto row_of = [&](int axis) -> const float* {
      int64_t pos = p.positions[axis * p.axis_stride + t];
      if (pos < 0 || pos >= p.max_position) {
        atomicOr(p.err, kErrPosition);
        pos = pos < 0 ? 0 : p.max_position - 1;
      }
      return p.cos_sin + pos * D;
    };
    float cs[8], sn[8];
    if (p.num_axes == 1) {
      const float4* row = reinterpret_cast<const float4*>(row_of(0)) + 2 * c;
      const float4 c0 = __ldg(row), c1 = __ldg(row + 1), s0 = __ldg(row + D / 8), s1 = __ldg(row + D / 8 + 1);
      cs[0] = c0.x; cs[1] = c0.y; cs[2] = c0.z; cs[3] = c0.w; cs[4] = c1.x; cs[5] = c1.y; cs[6] = c1.z; cs[7] = c1.w;
      sn[0] = s0.x; sn[1] = s0.y; sn[2] = s0.z; sn[3] = s0.w; sn[4] = s1.x; sn[5] = s1.y; sn[6] = s1.z; sn[7] = s1.w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int f = 8 * c + e;
        const float* row = row_of(p.freq_axis[f]);
        cs[e] = __ldg(row + f);
        sn[e] = __ldg(row + D / 2 + f);
      }
    }
    const int64_t cache_row = (slot / kBlockTokens) * p.num_kv_heads * kBlockTokens + slot % kBlockTokens;
    for (int r0 = first; r0 < rows; r0 += kAhead * step) {
      if (r0 != first) fetch(r0);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int r = r0 + k * step;
        if (r >= rows) continue;
        const int kr = r - p.num_q_heads, vr = kr - p.num_kv_heads;
        if (vr < 0) rotate(a[k], b[k], cs, sn);
        if (kr >= 0 && !stored) continue;
        uint4* dst = kr < 0 ? static_cast<uint4*>(p.q_out) + t * p.q_out_stride + static_cast<int64_t>(r) * kChunks
                            : static_cast<uint4*>(vr < 0 ? p.k_cache : p.v_cache) +
                                  (cache_row + static_cast<int64_t>(vr < 0 ? kr : vr) * kBlockTokens) * kChunks;
        dst[c] = a[k];
        dst[c + kLanes] = b[k];
      }
    }
  }
}

template <int D>
cudaError_t launch(const RopeAppendParams& p, int num_sms, cudaStream_t stream) {
  constexpr int kRowsAtOnce = 512 / D;
  const int rounds = (p.num_q_heads + 2 * p.num_kv_heads + kRowsAtOnce - 1) / kRowsAtOnce;
  const int64_t cap = static_cast<int64_t>(num_sms) * kMostCtas;
  // Few tokens: a token's rows over several warps, as long as that leaves one CTA per SM at most (eight tokens 1.9 us
  // instead of 5.2).
  RopeAppendParams q = p;
  const int64_t parts = num_sms * static_cast<int64_t>(kThreads / 32) / p.num_tokens;
  q.parts = static_cast<int>(parts < 1 ? 1 : parts > rounds ? rounds : parts);
  int64_t blocks = (p.num_tokens * q.parts + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > cap) blocks = cap;
  return launch_pdl(rope_append_kernel<D>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream, q);
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppendParams& p, int head_dim, int num_sms, cudaStream_t stream) {
  return head_dim == 128 ? launch<128>(p, num_sms, stream) : launch<64>(p, num_sms, stream);
}

}  // namespace pkv
