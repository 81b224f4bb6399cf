// Decode attention of few (sequence, kv head) pairs, for calls that are bound by latency and not by bytes: a thread-block
// cluster takes a pair, its warps a few of the pair's blocks each, and the warps' states are joined first in a CTA and
// then through the cluster's shared memory.  One launch, no workspace, and no pass over the batch's lengths before the
// first copy.  Used with a window (window_decode.cu), and for whole sequences whose leading blocks are their group's
// (View::kTail, prefix_decode.cu: the pair reads shared blocks for itself, through the group's first table).
#pragma once

#include "paged_decode_kernel.cuh"

namespace pkv {
namespace {

constexpr int kClusterWarps = 8;   // of a CTA
constexpr int kClusterStages = 2;
constexpr int kMostClusterCtas = 8;

// Estimates that choose between this form and the others, microseconds and bytes a microsecond, as measured on one GB300
// with tables full of visible blocks: a call takes about 4.5 us and 0.87 (D 128) or 0.6 (D 64) a block of a warp.  Windows
// of 1024, 4096 and 8192 tokens, D 128, us a call here and in the partition and join kernels: one sequence of 8 kv heads
// 5.1, 7.6, 10.9 and 8.9, 11.5, 14.5; of one kv head with eight q heads 6.4, 9.1, 12.2 and 10.3, 18.5, 28.4; 16 sequences of 8 kv
// heads 15.3, 43.6, 81.0 and 18.9, 48.4, 87.3; two of 8 kv heads, half the SMs and 16 blocks a warp, 18.3 and 19.0 at 8192,
// where the forms meet.  (16 pairs take 5.8 us in clusters of four but 9.7 in clusters of eight, of which fewer than 16 run
// at once.)
constexpr float kClusterUs = 4.5f, kStreamRate = 6.4e6f, kUneven = 0.5f;
template <int D>
constexpr float kBlockUs = D == 128 ? 0.87f : 0.6f;

// Shared memory of a CTA: the warps' rings, their P tiles, the CTA's joined state, the warps' (m, l), the barriers.
template <int D, int G, View kView>
struct ClusterSmem {
  static constexpr int kStage = stage_bytes<D, G, kView>();
  static constexpr int kPTile = ptile_bytes<D, G, kView>();
  static constexpr int kOffPTile = kClusterWarps * kClusterStages * kStage;
  static constexpr int kOffState = kOffPTile + kClusterWarps * kPTile;     // fp32 [G][D], then (m, l) [G]
  static constexpr int kOffMl = kOffState + G * D * 4 + G * 8;             // (m, l) [warp][G]
  static constexpr int kOffBar = kOffMl + kClusterWarps * G * 8;
  static constexpr int kBytes = 1024 + kOffBar + kClusterWarps * kClusterStages * 8;  // 1024: to align the first stage
  static_assert(kOffState % 16 == 0 && kOffMl % 8 == 0 && kOffBar % 8 == 0, "alignment");
  static_assert(G * D * 4 <= kStage, "a warp's O fits its first stage");
};

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of the same shared-memory location in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 peer_load4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 peer_load2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

template <int D, int G, View kView>
__global__ void __launch_bounds__(kClusterWarps * 32)
    cluster_decode_kernel(const DecodeViewParams p, const __grid_constant__ CUtensorMap map_k,
                          const __grid_constant__ CUtensorMap map_v, int ctas) {
  using M = ClusterSmem<D, G, kView>;
  constexpr int kTileBytes = Geo<D, G>::kTileBytes, kQBytes = Geo<D, G>::kQBytes;
  extern __shared__ __align__(128) unsigned char smem[];
  unsigned char* base = smem + ((1024u - (smem_addr(smem) & 1023u)) & 1023u);  // (the same offset in every CTA)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int pair = blockIdx.x / ctas, rank = blockIdx.x % ctas;
  const int hkv = p.num_kv_heads;
  const int b = pair / hkv, kvh = pair - b * hkv;
  unsigned char* ring_ptr = base + warp * kClusterStages * M::kStage;
  const uint32_t ring = smem_addr(ring_ptr);
  const uint32_t sP = smem_addr(base + M::kOffPTile + warp * M::kPTile);
  const uint32_t bar0 = smem_addr(base + M::kOffBar) + warp * kClusterStages * 8;
  float* s_state = reinterpret_cast<float*>(base + M::kOffState);
  float2* s_state_ml = reinterpret_cast<float2*>(s_state + G * D);
  float2* s_ml = reinterpret_cast<float2*>(base + M::kOffMl);
  if (lane == 0) {
    for (int s = 0; s < kClusterStages; ++s) mbar_init(bar0 + 8 * s, 1);
    fence_mbar_init();
  }
  __syncwarp();
  pdl_trigger();
  pdl_wait();

  int len = __ldg(p.context_lens + b);
  const int cap = p.max_blocks_per_seq * kBlockTokens;
  if (len < 0 || len > cap) {
    if (kvh == 0 && rank == 0 && tid == 0) atomicOr(p.err, len < 0 ? kErrLenNegative : kErrLenTooLong);
    len = len < 0 ? 0 : cap;
  }
  int blocks = (len + kBlockTokens - 1) / kBlockTokens;
  const int32_t* table = p.block_tables + static_cast<size_t>(b) * p.max_blocks_per_seq;
  const WindowBlocks window(len, p.window, p.sinks);  // (not used without a window)
  SharedRow shared{0, 0};
  if constexpr (kView == View::kWindow) {
    blocks -= window.skip;
  } else {
    shared = shared_blocks_of_row(p, b);
    if (blockIdx.x == 0) report_groups(p);
  }
  auto column = [&](int n) -> int {  // of block n of the pair's stream
    if constexpr (kView == View::kWindow) return window.column(n);
    return n;
  };
  // This warp's blocks [first, first + n) of the pair's stream.
  const int warps = ctas * kClusterWarps, w = rank * kClusterWarps + warp;
  const int first = static_cast<int>(static_cast<int64_t>(w) * blocks / warps);
  const int n = static_cast<int>(static_cast<int64_t>(w + 1) * blocks / warps) - first;
  auto fetch_id = [&](int i) -> int {  // table entry of block first + i
    if (i >= n) return 0;
    const int col = column(first + i);
    const int32_t* row = table;
    if (kView == View::kTail && col < shared.blocks)
      row = p.block_tables + static_cast<size_t>(shared.first_row) * p.max_blocks_per_seq;
    int id = __ldg(row + col);
    if (id < 0 || id >= p.num_blocks) {
      atomicOr(p.err, kErrBlockId);
      id = 0;
    }
    return id;
  };
  int ids = fetch_id(lane);  // 32 at a time, one a lane
  auto issue = [&](int i, int id) {  // lane 0
    const int stage = i % kClusterStages;
    const uint32_t dst = ring + stage * M::kStage, bar = bar0 + 8 * stage;
    mbar_arrive_expect_tx(bar, 2 * kTileBytes + (i == 0 ? kQBytes : 0));
    const int row = (id * hkv + kvh) * kBlockTokens;  // < 2^31: checked on the host
#pragma unroll
    for (int h = 0; h < D / 64; ++h) {
      tensor_load(dst + h * 2048, &map_k, 64 * h, row, bar);
      tensor_load(dst + kTileBytes + h * 2048, &map_v, 64 * h, row, bar);
    }
    if (i == 0)
      bulk_load(dst + 2 * kTileBytes,
                static_cast<const __nv_bfloat16*>(p.q) + (static_cast<size_t>(b) * p.num_q_heads + kvh * G) * D, kQBytes, bar);
  };
  for (int i = 0; i < kClusterStages; ++i) {
    const int id = __shfl_sync(kFull, ids, i);
    if (lane == 0 && i < n) issue(i, id);
  }

  uint32_t qf[D / 16][2];
  float o[D / 16][4];
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int mt = 0; mt < D / 16; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
  bool failed = false;
  for (int i = 0; i < n; ++i) {
    const int stage = i % kClusterStages;
    if (!__all_sync(kFull, mbar_wait(bar0 + 8 * stage, (i / kClusterStages) & 1, kWaitTimeoutNs))) {
      // Give up on this warp's blocks: flag it, let the copies in flight land, and go on to the join.
      if (lane == 0) atomicOr(p.err, kErrTimeout);
      for (int x = i; x < n && x < i + kClusterStages; ++x)
        mbar_wait(bar0 + 8 * (x % kClusterStages), (x / kClusterStages) & 1, kDrainTimeoutNs);
      failed = true;
      break;
    }
    unsigned char* st = ring_ptr + stage * M::kStage;
    if (i == 0) {  // q^T fragments: head lane / 4 (a zero column past the group)
      const int g = lane >> 2, t = lane & 3;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const unsigned char* qrow = st + 2 * kTileBytes + g * (D * 2) + (16 * kk + 2 * t) * 2;
        qf[kk][0] = g < G ? *reinterpret_cast<const uint32_t*>(qrow) : 0u;
        qf[kk][1] = g < G ? *reinterpret_cast<const uint32_t*>(qrow + 16) : 0u;
      }
    }
    const int col = column(first + i);
    typename SeesOf<kView>::type sees;
    sees.end = len - col * kBlockTokens;
    bool whole = sees.end >= kBlockTokens;
    if constexpr (kView == View::kWindow) {
      sees.first = sees.end - p.window;
      sees.sinks = p.sinks - col * kBlockTokens;
      whole = whole && (sees.first <= 0 || sees.sinks >= kBlockTokens);
    }
    const uint32_t sk = ring + stage * M::kStage;
    if (whole)
      process_block_mma<D, false>(sk, st + kTileBytes, sk + kTileBytes, sP, qf, o, m, l, p.qscale, lane, sees);
    else
      process_block_mma<D, true>(sk, st + kTileBytes, sk + kTileBytes, sP, qf, o, m, l, p.qscale, lane, sees);
    __syncwarp();
    const int next = i + kClusterStages;
    if (next < n) {  // uniform for the warp
      if (next % 32 == 0) ids = fetch_id(next + lane);
      const int id = __shfl_sync(kFull, ids, next % 32);
      if (lane == 0) {
        fence_proxy_async_smem();
        issue(next, id);
      }
    }
  }

  // The warp's state: O in the ring's first stage (every copy has landed and been read), m and l beside.
  float la = l[0], lb = l[1];
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
    la += __shfl_xor_sync(kFull, la, off);
    lb += __shfl_xor_sync(kFull, lb, off);
  }
  const int go = lane >> 2, ha = 2 * (lane & 3), hb = ha + 1;
  float* mine = reinterpret_cast<float*>(ring_ptr);
#pragma unroll
  for (int mt = 0; mt < D / 16; ++mt) {
    const int d0 = 16 * mt + go, d1 = d0 + 8;
    if (ha < G) {
      mine[ha * D + d0] = o[mt][0];
      mine[ha * D + d1] = o[mt][2];
    }
    if (hb < G) {
      mine[hb * D + d0] = o[mt][1];
      mine[hb * D + d1] = o[mt][3];
    }
  }
  const bool empty = n == 0 || failed;
  if (go == 0) {
    if (ha < G) s_ml[warp * G + ha] = empty ? make_float2(-INFINITY, 0.f) : make_float2(m[0], la);
    if (hb < G) s_ml[warp * G + hb] = empty ? make_float2(-INFINITY, 0.f) : make_float2(m[1], lb);
  }
  __syncthreads();

  // The CTA's state: sum_w 2^(m_w - M) O_w, four dims a thread at a time.  (A state without a key is skipped: its m is
  // -infinity and its l is 0.  One whose scores were not numbers has l so, and spoils the sum.)
  for (int x = tid; x < G * D / 4; x += kClusterWarps * 32) {
    const int g = x / (D / 4);
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < kClusterWarps; ++k) top = fmaxf(top, s_ml[k * G + g].x);
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum_l = 0.f;
#pragma unroll
    for (int k = 0; k < kClusterWarps; ++k) {
      const float2 s = s_ml[k * G + g];
      if (s.x == -INFINITY && s.y == 0.f) continue;
      const float f = exp2f(s.x - top);
      const float4 v = *reinterpret_cast<const float4*>(base + k * kClusterStages * M::kStage + x * 16);
      sum.x += f * v.x;
      sum.y += f * v.y;
      sum.z += f * v.z;
      sum.w += f * v.w;
      sum_l += f * s.y;
    }
    *reinterpret_cast<float4*>(s_state + 4 * x) = sum;
    if (x % (D / 4) == 0) s_state_ml[g] = make_float2(top, sum_l);
  }
  cluster_sync();

  // Every CTA joins its share of the pair's outputs over the cluster's states.
  const uint32_t state = smem_addr(s_state), state_ml = smem_addr(s_state_ml);
  for (int x = rank * kClusterWarps * 32 + tid; x < G * D / 4; x += ctas * kClusterWarps * 32) {
    const int g = x / (D / 4);
    float2 s[kMostClusterCtas];
    float4 v[kMostClusterCtas];
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < kMostClusterCtas; ++k) {
      s[k] = make_float2(-INFINITY, 0.f);
      if (k < ctas) {
        s[k] = peer_load2(peer(state_ml + g * 8, k));
        v[k] = peer_load4(peer(state + x * 16, k));
      }
      top = fmaxf(top, s[k].x);
    }
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum_l = 0.f;
#pragma unroll
    for (int k = 0; k < kMostClusterCtas; ++k) {
      if (s[k].x == -INFINITY && s[k].y == 0.f) continue;
      const float f = exp2f(s[k].x - top);
      sum.x += f * v[k].x;
      sum.y += f * v[k].y;
      sum.z += f * v[k].z;
      sum.w += f * v[k].w;
      sum_l += f * s[k].y;
    }
    const float inv = sum_l != 0.f ? 1.f / sum_l : 0.f;  // no token: zeros
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + (static_cast<size_t>(b) * p.num_q_heads + kvh * G) * D + 4 * x;
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(float2_to_bf16x2(sum.x * inv, sum.y * inv), float2_to_bf16x2(sum.z * inv, sum.w * inv));
  }
  cluster_sync();  // no CTA leaves while another reads its state
}

template <int D, int G, View kView>
struct ClusterForm {
  using M = ClusterSmem<D, G, kView>;
  static constexpr auto kKernel = &cluster_decode_kernel<D, G, kView>;

  static cudaLaunchConfig_t config(unsigned pairs, int ctas, cudaStream_t stream, cudaLaunchAttribute (&attr)[2]) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(pairs * ctas);
    cfg.blockDim = dim3(kClusterWarps * 32);
    cfg.dynamicSmemBytes = M::kBytes;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cfg;
  }

  // Clusters of 1, 2, 4 and 8 CTAs that the current device holds at once (a cluster stays within a GPC, so of the larger
  // ones fewer fit than the SMs suggest).  Looked up once per device, with the kernel's shared-memory limit raised.
  static cudaError_t resident(const int** counts) {
    static std::mutex mu;
    static int known[64][4];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (known[dev][0] == 0) {
      if ((e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, M::kBytes)) != cudaSuccess) return e;
      for (int k = 3; k >= 0; --k) {
        cudaLaunchAttribute attr[2];
        cudaLaunchConfig_t cfg = config(1, 1 << k, nullptr, attr);
        cfg.numAttrs = 1;
        if ((e = cudaOccupancyMaxActiveClusters(&known[dev][k], kKernel, &cfg)) != cudaSuccess) {
          known[dev][0] = 0;
          return e;
        }
      }
    }
    *counts = known[dev];
    return cudaSuccess;
  }

  // CTAs a pair: as many as give every warp two blocks, if that many clusters run at once.  0: this form is not for the
  // call, because the pairs are too many or it would take longer than the other form, which takes `other_us` or, if
  // `streamed`, that and the time of streaming the call's blocks over the whole GPU (of which kUneven are taken to exist, as
  // sequences may be shorter than their tables).
  static int choose(const int* counts, int64_t pairs, int visible_blocks, float other_us, bool streamed) {
    int k = 0;
    while (k < 3 && (kClusterWarps * 2 << k) < visible_blocks && pairs <= counts[k + 1]) ++k;
    const float bytes = static_cast<float>(pairs) * visible_blocks * (2.f * Geo<D, G>::kTileBytes);
    const float mine = kClusterUs + kBlockUs<D> * visible_blocks / (kClusterWarps << k);
    const float other = other_us + (streamed ? kUneven * bytes / kStreamRate : 0.f);
    return pairs <= counts[k] && mine <= other ? 1 << k : 0;
  }
  static cudaError_t ctas(int num_seqs, int num_kv_heads, int visible_blocks, float other_us, bool streamed, int* out) {
    const int* counts = nullptr;
    const cudaError_t e = resident(&counts);
    if (e != cudaSuccess) return e;
    *out = choose(counts, static_cast<int64_t>(num_seqs) * num_kv_heads, visible_blocks, other_us, streamed);
    return cudaSuccess;
  }
  // Whether a call of every number of sequences up to num_seqs takes this form.  With as many CTAs a pair the smallest batch
  // is the first not to (its other form streams least), so one batch for each number of CTAs is looked at.
  static cudaError_t takes_all(int num_seqs, int num_kv_heads, int visible_blocks, float other_us, bool streamed, bool* out) {
    const int* counts = nullptr;
    const cudaError_t e = resident(&counts);
    if (e != cudaSuccess) return e;
    auto takes = [&](int64_t seqs) { return choose(counts, seqs * num_kv_heads, visible_blocks, other_us, streamed) != 0; };
    *out = takes(num_seqs) && takes(1);
    for (int k = 1; k <= 3; ++k) {
      const int64_t fewer_ctas = counts[k] / num_kv_heads + 1;  // the first batch with so many pairs that they get fewer
      if (fewer_ctas < num_seqs) *out = *out && takes(fewer_ctas);
    }
    return cudaSuccess;
  }

  static cudaError_t launch(const DecodeViewParams& p, int ctas, cudaStream_t stream) {
    const int* counts = nullptr;  // (the kernel's attributes are set)
    cudaError_t e = resident(&counts);
    if (e != cudaSuccess) return e;
    CUtensorMap mk, mv;
    const int64_t rows = p.num_blocks * p.num_kv_heads * kBlockTokens;
    if (rows > INT32_MAX) return cudaErrorInvalidValue;  // tensor-copy row coordinates are 32-bit
    if ((e = encode_cache_map(&mk, p.k_cache, rows, D)) != cudaSuccess) return e;
    if ((e = encode_cache_map(&mv, p.v_cache, rows, D)) != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = config(static_cast<unsigned>(p.num_seqs) * p.num_kv_heads, ctas, stream, attr);
    return cudaLaunchKernelEx(&cfg, kKernel, p, mk, mv, ctas);
  }
};

template <View kView, typename F>
cudaError_t dispatch_cluster(int head_dim, int group, F&& f) {
  switch (head_dim * 16 + group) {
    case 64 * 16 + 1: return f(ClusterForm<64, 1, kView>{});
    case 64 * 16 + 2: return f(ClusterForm<64, 2, kView>{});
    case 64 * 16 + 4: return f(ClusterForm<64, 4, kView>{});
    case 64 * 16 + 8: return f(ClusterForm<64, 8, kView>{});
    case 128 * 16 + 1: return f(ClusterForm<128, 1, kView>{});
    case 128 * 16 + 2: return f(ClusterForm<128, 2, kView>{});
    case 128 * 16 + 4: return f(ClusterForm<128, 4, kView>{});
    case 128 * 16 + 8: return f(ClusterForm<128, 8, kView>{});
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace
}  // namespace pkv
