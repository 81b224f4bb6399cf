// The 8-bit cache's writes, reads and copies: quantising append (with or without the rotation of q and k), rows read back
// as bf16, and whole-block copies.  All are bound by HBM: each row is read once and written once.  Measured: 32773 tokens of 8
// kv heads of 128 dims appended in 34.4 us (0.88 of the copy bandwidth), with the rotation of 32 q heads in 123 us (0.92);
// 65536 of 64 dims read back in 35.3 us (0.86); 2048 blocks copied in 17.2 us (part of them from L2); the smallest calls 3 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fp8_cache.h"
#include "fp8_format.cuh"

namespace pkv {
namespace {

constexpr unsigned kFull = 0xffffffffu;

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

// Largest magnitude of a lane's 16 values as bf16 bits (infinities and NaN count by their bits), or of the finite ones.
__device__ __forceinline__ uint32_t top_bits(const uint4& a, const uint4& b) {
  const uint32_t* w[2] = {&a.x, &b.x};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = __vmaxu2(top, w[i / 4][i % 4] & 0x7fff7fffu);
  return max(top & 0xffffu, top >> 16);
}
__device__ __forceinline__ uint32_t top_finite_bits(const uint4& a, const uint4& b) {
  const uint32_t* w[2] = {&a.x, &b.x};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t x = (w[i / 8][i / 2 % 4] >> 16 * (i & 1)) & 0x7fffu;
    if (x < 0x7f80u) top = max(top, x);
  }
  return top;
}
// Eight codes of a chunk; infinities become NaN, as the type has none.
__device__ __forceinline__ uint2 quantise(const uint4& a, float inverse, bool odd) {
  const uint32_t* w = &a.x;
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 x = widen(w[i]);
    if (odd) {
      if (!(fabsf(x.x) < INFINITY)) x.x = __int_as_float(0x7fffffff);
      if (!(fabsf(x.y) < INFINITY)) x.y = __int_as_float(0x7fffffff);
    }
    r[i] = fp8_codes(x.x * inverse, x.y * inverse);
  }
  return make_uint2(r[0] | r[1] << 16, r[2] | r[3] << 16);
}

constexpr int kAppendThreads = 128;
constexpr int kAppendCtas = 64;  // per SM at most; beyond that a warp takes several tokens

// A lane owns two 16-byte chunks of a row, so that D / 16 lanes cover it and a warp takes 4 (D = 128) or 8 rows at a time:
// the chunks c and c + D / 16, the rotation's two halves, or without rotation 2 c and 2 c + 1, whose codes are 16 bytes.
// A warp takes a token, or a part of its rows, and has kAhead rows a lane in flight, the first while it looks up the slot (up
// to 37.8 us with other numbers of rows and CTAs where this takes 34.4).  Rows that hold an infinity or NaN look for their
// largest finite value a second time.
template <int D, bool kRotary>
__global__ void __launch_bounds__(kAppendThreads) append_fp8_kernel(const Fp8AppendParams p) {
  pdl_trigger();
  pdl_wait();
  constexpr int kAhead = 2;
  constexpr int kLanes = D / 16;  // lanes of a row
  constexpr int kRowsAtOnce = 32 / kLanes;
  constexpr int kChunks = D / 8;  // 16-byte chunks of a bf16 row
  const int lane = threadIdx.x & 31;
  const int c = lane % kLanes, sub = lane / kLanes;
  const int chunk_a = kRotary ? c : 2 * c, chunk_b = kRotary ? c + kLanes : 2 * c + 1;
  const int rows = p.num_q_heads + 2 * p.num_kv_heads;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kAppendThreads / 32);
  const int64_t items = p.num_tokens * p.parts;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * (kAppendThreads / 32) + (threadIdx.x >> 5); item < items;
       item += warps) {
    const int64_t t = item / p.parts;
    const int part = static_cast<int>(item - t * p.parts);
    const int step = p.parts * kRowsAtOnce;
    uint4 a[kAhead], b[kAhead];
    auto fetch = [&](int r0) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int r = r0 + k * step + sub;
        a[k] = b[k] = make_uint4(0u, 0u, 0u, 0u);
        if (r >= rows) continue;
        const int kr = r - p.num_q_heads, vr = kr - p.num_kv_heads;
        const uint4* src = kr < 0 ? static_cast<const uint4*>(p.q) + t * p.q_stride + r * kChunks
                           : vr < 0 ? static_cast<const uint4*>(p.k) + t * p.k_stride + kr * kChunks
                                    : static_cast<const uint4*>(p.v) + t * p.v_stride + vr * kChunks;
        a[k] = load_once(src + chunk_a);
        b[k] = load_once(src + chunk_b);
      }
    };
    fetch(part * kRowsAtOnce);
    const int64_t slot = p.slot_mapping[t];
    if (slot < 0) continue;  // padding
    const bool stored = slot < p.num_slots;
    if (!stored && lane == 0 && part == 0) atomicOr(p.err, kErrSlot);
    float cs[8], sn[8];
    if constexpr (kRotary) {
      auto row_of = [&](int axis) -> const float* {
        int64_t pos = p.positions[axis * p.axis_stride + t];
        if (pos < 0 || pos >= p.max_position) {
          atomicOr(p.err, kErrPosition);
          pos = pos < 0 ? 0 : p.max_position - 1;
        }
        return p.cos_sin + pos * D;
      };
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
    }
    const int64_t block_head = (slot / kBlockTokens) * p.num_kv_heads;
    const int offset = static_cast<int>(slot % kBlockTokens);
    // The whole warp goes through the rows together (the row's lanes exchange their maxima).
    for (int r0 = part * kRowsAtOnce; r0 < rows; r0 += kAhead * step) {
      if (r0 != part * kRowsAtOnce) fetch(r0);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int r = r0 + k * step + sub;
        const int kr = r - p.num_q_heads, vr = kr - p.num_kv_heads;
        if (kRotary && vr < 0) rotate(a[k], b[k], cs, sn);
        uint32_t top = top_bits(a[k], b[k]);
        const bool odd = __any_sync(kFull, top >= 0x7f80u);  // some value of the warp's rows is not finite
        if (odd) top = top_finite_bits(a[k], b[k]);
#pragma unroll
        for (int off = 1; off < kLanes; off <<= 1) top = max(top, __shfl_xor_sync(kFull, top, off));
        if (r >= rows) continue;
        if (kRotary && kr < 0) {
          uint4* dst = static_cast<uint4*>(p.q_out) + t * p.q_out_stride + static_cast<int64_t>(r) * kChunks;
          dst[chunk_a] = a[k];
          dst[chunk_b] = b[k];
        }
        if (kr < 0 || !stored) continue;
        const uint32_t e = fp8_exponent(top);
        const float inverse = fp8_inverse(e);
        const int64_t tile = block_head + (vr < 0 ? kr : vr);
        uint8_t* dst = (vr < 0 ? p.k_cache : p.v_cache) + (tile * kBlockTokens + offset) * D;
        const uint2 x = quantise(a[k], inverse, odd), y = quantise(b[k], inverse, odd);
        if constexpr (kRotary) {
          *reinterpret_cast<uint2*>(dst + 8 * chunk_a) = x;
          *reinterpret_cast<uint2*>(dst + 8 * chunk_b) = y;
        } else {
          *reinterpret_cast<uint4*>(dst + 8 * chunk_a) = make_uint4(x.x, x.y, y.x, y.y);
        }
        if (c == 0) p.kv_scales[(tile * 2 + (vr < 0 ? 0 : 1)) * kBlockTokens + offset] = static_cast<uint8_t>(e);
      }
    }
  }
}

// A thread reads 8 codes of a row of K and of V, of kGatherTokens tokens at once, and writes 8 bf16 values of each: so the
// loads and the stores of a warp are whole rows.  A CTA's tokens are neighbours (39.4 us where this takes 35.3 without).
constexpr int kGatherThreads = 256;
constexpr int kGatherTokens = 2;
constexpr int kGatherCtas = 64;  // per SM at most
template <int D>
__global__ void __launch_bounds__(kGatherThreads) gather_fp8_kernel(const Fp8GatherParams p) {
  pdl_trigger();
  pdl_wait();
  constexpr int kChunks = D / 8;
  const int per_token = p.num_kv_heads * kChunks;
  const int64_t total = p.num_tokens * per_token;
  // A CTA's are neighbours, so that blocks are read whole.
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kGatherThreads * kGatherTokens;
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * kGatherThreads * kGatherTokens + threadIdx.x; first < total; first += stride) {
    int64_t token[kGatherTokens], slot[kGatherTokens];
    int rem[kGatherTokens];
#pragma unroll
    for (int k = 0; k < kGatherTokens; ++k) {
      const int64_t idx = first + k * kGatherThreads;
      token[k] = idx / per_token;
      rem[k] = static_cast<int>(idx - token[k] * per_token);
      slot[k] = idx < total ? __ldg(p.slot_mapping + token[k]) : -1;
    }
    uint2 codes[kGatherTokens][2];
    uint8_t e[kGatherTokens][2];
#pragma unroll
    for (int k = 0; k < kGatherTokens; ++k) {
      if (slot[k] >= p.num_slots) {
        atomicOr(p.err, kErrSlot);
        slot[k] = -1;
      }
      if (slot[k] < 0) continue;  // padding
      const int64_t tile = (slot[k] / kBlockTokens) * p.num_kv_heads + rem[k] / kChunks;
      const int offset = static_cast<int>(slot[k] % kBlockTokens);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint8_t* src = (i ? p.v_cache : p.k_cache) + (tile * kBlockTokens + offset) * D + rem[k] % kChunks * 8;
        asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(codes[k][i].x), "=r"(codes[k][i].y) : "l"(src) : "memory");
        e[k][i] = p.kv_scales[(tile * 2 + i) * kBlockTokens + offset];
      }
    }
#pragma unroll
    for (int k = 0; k < kGatherTokens; ++k) {
      if (slot[k] < 0) continue;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float s = fp8_scale(e[k][i]);
        const uint32_t w[2] = {codes[k][i].x, codes[k][i].y};
        uint32_t r[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float2 f = fp8_floats(static_cast<uint16_t>(w[x / 2] >> 16 * (x & 1)));
          r[x] = narrow(f.x * s, f.y * s);
        }
        static_cast<uint4*>(i ? p.v : p.k)[token[k] * (i ? p.v_stride : p.k_stride) + rem[k]] = make_uint4(r[0], r[1], r[2], r[3]);
      }
    }
  }
}

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;

// One CTA per pair and K or V: the block's codes are one contiguous run; V's CTA copies the exponents too.
__global__ void __launch_bounds__(kCopyThreads) copy_blocks_fp8_kernel(const Fp8CopyParams p) {
  pdl_trigger();
  pdl_wait();
  const int pair = blockIdx.x >> 1;
  const bool v = blockIdx.x & 1;
  const int64_t src = p.src_dst[2 * pair];
  const int64_t dst = p.src_dst[2 * pair + 1];
  if (src < 0 || src >= p.num_blocks || dst < 0 || dst >= p.num_blocks) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrCopyRange);
    return;
  }
  auto run = [&](void* area, int64_t n) {
    const uint4* from = static_cast<const uint4*>(area) + src * n;
    uint4* to = static_cast<uint4*>(area) + dst * n;
    for (int64_t i = threadIdx.x; i < n; i += kCopyThreads * kCopyUnroll) {
      uint4 r[kCopyUnroll];
#pragma unroll
      for (int u = 0; u < kCopyUnroll; ++u)
        if (i + u * kCopyThreads < n) r[u] = from[i + u * kCopyThreads];
#pragma unroll
      for (int u = 0; u < kCopyUnroll; ++u)
        if (i + u * kCopyThreads < n) to[i + u * kCopyThreads] = r[u];
    }
  };
  run(v ? p.v_cache : p.k_cache, p.cache_chunks);
  if (v) run(p.kv_scales, p.scale_chunks);
}

template <int D>
cudaError_t append(const Fp8AppendParams& p, int num_sms, cudaStream_t stream) {
  constexpr int kRowsAtOnce = 512 / D;
  const int rounds = (p.num_q_heads + 2 * p.num_kv_heads + kRowsAtOnce - 1) / kRowsAtOnce;
  const int64_t cap = static_cast<int64_t>(num_sms) * kAppendCtas;
  // Few tokens: a token's rows over several warps, as long as that leaves one CTA per SM at most.
  Fp8AppendParams q = p;
  const int64_t parts = num_sms * static_cast<int64_t>(kAppendThreads / 32) / p.num_tokens;
  q.parts = static_cast<int>(parts < 1 ? 1 : parts > rounds ? rounds : parts);
  int64_t blocks = (p.num_tokens * q.parts + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
  if (blocks > cap) blocks = cap;
  return launch_pdl(p.cos_sin ? append_fp8_kernel<D, true> : append_fp8_kernel<D, false>, dim3(static_cast<unsigned>(blocks)),
                    dim3(kAppendThreads), 0, stream, q);
}

}  // namespace

cudaError_t launch_append_fp8(const Fp8AppendParams& p, int head_dim, int num_sms, cudaStream_t stream) {
  return head_dim == 128 ? append<128>(p, num_sms, stream) : append<64>(p, num_sms, stream);
}

cudaError_t launch_gather_fp8(const Fp8GatherParams& p, int head_dim, int num_sms, cudaStream_t stream) {
  const int64_t total = p.num_tokens * p.num_kv_heads * (head_dim / 8);
  constexpr int kPerCta = kGatherThreads * kGatherTokens;
  int64_t blocks = (total + kPerCta - 1) / kPerCta;
  const int64_t cap = static_cast<int64_t>(num_sms) * kGatherCtas;
  if (blocks > cap) blocks = cap;
  return launch_pdl(head_dim == 128 ? gather_fp8_kernel<128> : gather_fp8_kernel<64>, dim3(static_cast<unsigned>(blocks)),
                    dim3(kGatherThreads), 0, stream, p);
}

cudaError_t launch_copy_blocks_fp8(const Fp8CopyParams& p, int num_pairs, cudaStream_t stream) {
  return launch_pdl(copy_blocks_fp8_kernel, dim3(static_cast<unsigned>(num_pairs) * 2u), dim3(kCopyThreads), 0, stream, p);
}

}  // namespace pkv
