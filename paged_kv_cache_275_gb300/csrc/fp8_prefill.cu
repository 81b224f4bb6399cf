// Chunk attention over the 8-bit cache on the 5th-generation tensor cores: causal rows, as paged_prefill_kernel.cuh does it
// over a bf16 cache, whose tiles, tensor-memory layout and products this kernel shares.  Long chunks, whose blocks many CTAs see,
// have them turned into bf16 once (unpack_fp8_kernel) and take the bf16 kernel itself.
//
// Bound by the products (bf16, 4 D flop a row and key it sees).  They stay bf16: q has eight significant bits and the softmax
// weights need as many, so 8-bit products would take two parts of each and save nothing; and a code times its row's power of
// two is a bf16 value exactly.  So the cache's rows become bf16 on their way into shared memory, and everything behind that,
// and every result's bits, are those of the bf16 kernel over the values that the cache stands for.
//
// Roles (16 warps, one CTA an SM, two 128-row query tiles):
//   * warps 9-15: convert.  A tile of the K/V ring is four units of 32 rows, and the units go to the warps in turns.  A lane
//     takes 16 codes at a time (to fp16, to fp32, times the row's scale, to bf16, all exact), stores them where the products
//     read them (128-byte swizzle) and requests those of the same place of its next unit.  Rows past the last key become
//     zeros.
//   * warp 8: issues the products, as there; it owns the tensor memory.
//   * warps 0-7: softmax and epilogue, a row a thread, as there.
// A chunk call that does not fill the GPU has each tile pair's key steps split over CTAs, as there, with a merge.
// Measured (8 kv heads of 128 dims): eight chunks of 256 behind 3840 tokens, 32 q heads, 147 us; 512 tokens behind 8192, 16 q
// heads, 50 us: four splits of 17 steps on 128 of 152 SMs, and the merge.  Seven converters and eight softmax warps share the
// issue slots, 1.26 times the bf16 kernel's time over a bf16 cache (two prompts of 8192 925 us, 734 there, 746 unpacked, in one
// loop over one input; 946 and 789 over several in turn).  A single query
// tile dealt to both tiles' places by steps gained nothing (64 sequences of 8 tokens 165 to 172 us).
// The softmax warps take 168 registers a thread and leave the others 88: 256 (168 + 88) is the block's 512 * 128.  (The compiler
// plans with 128 for all and spills 16 to 24 bytes a thread.)
#include "paged_prefill_kernel.cuh"

#include "fp8_cache.h"
#include "fp8_format.cuh"

namespace pkv {
namespace {

constexpr int kIssuer = 4 * kTiles;
constexpr int kConverters = 7;
constexpr int kFp8Threads = 32 * (kIssuer + 1 + kConverters);
constexpr int kUnitRows = 32, kUnits = kKeys / kUnitRows;  // a converter's unit, and units of a tile
static_assert(kRing * kUnits >= kConverters, "a converter's next unit may not wait for a tile that it has yet to fill");
constexpr int kSoftmaxRegs = 168, kOtherRegs = 88;
static_assert(kFp8Threads == 512 && 256 * (kSoftmaxRegs + kOtherRegs) == 512 * 128, "the block's registers");

struct Fp8PrefillParams : PrefillParams {
  const uint8_t* kv_scales;
};

__device__ __forceinline__ uint4 load_codes(const uint8_t* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

template <int D, int G, bool kSplit>
__global__ void __launch_bounds__(kFp8Threads, 1)
    prefill_fp8_kernel(const Fp8PrefillParams p, const __grid_constant__ CUtensorMap map_out) {
  using T = Pf<D>;
  constexpr int kTokens = kRows / G;
  constexpr int kCtaTokens = kTiles * kTokens;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t s_base = saddr(smem);
  pdl_trigger();
  pdl_wait();

  // Longest first, as in the bf16 kernel: x the kv head, y a sequence's tile pairs from the last on, z the sequences by
  // decreasing context length (and a sequence's splits).
  const int tile = static_cast<int>(gridDim.y) - 1 - static_cast<int>(blockIdx.y), kvh = blockIdx.x;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = kSplit ? static_cast<int>(blockIdx.z) % p.num_splits : 0;
  const int zrank = kSplit ? static_cast<int>(blockIdx.z) / p.num_splits : static_cast<int>(blockIdx.z);
  int b = zrank;
  if (p.num_seqs <= kFp8Threads && p.num_seqs > 1) {
    int* s_lens = reinterpret_cast<int*>(smem + T::kOffKV);  // (the ring is not in use yet)
    int& s_pick = *reinterpret_cast<int*>(smem + T::kOffBar + kTmemSlotOffset + 4);
    const int mine = tid < p.num_seqs ? __ldg(p.context_lens + tid) : 0;
    if (tid < p.num_seqs) s_lens[tid] = mine;
    __syncthreads();
    if (tid < p.num_seqs) {
      int rank = 0;
      for (int u = 0; u < p.num_seqs; ++u) {
        const int other = s_lens[u];
        rank += (other > mine) || (other == mine && u < tid);
      }
      if (rank == zrank) s_pick = tid;
    }
    __syncthreads();
    b = s_pick;
  }
  const int q0 = __ldg(p.query_start + b), q1 = __ldg(p.query_start + b + 1), len = __ldg(p.context_lens + b);
  const int64_t chunk = static_cast<int64_t>(q1) - q0;
  const bool bad = chunk < 0 || len < chunk || len > p.max_blocks_per_seq * kBlockTokens || q0 < 0 || q1 > p.query_rows;
  if ((bad || chunk > p.max_query_len) && tile == 0 && tid == 0) atomicOr(p.err, kErrLenTooLong);
  if (bad) return;
  const int C = min(static_cast<int>(chunk), p.max_query_len);  // rows past max_query_len are not computed
  const int prefix = len - static_cast<int>(chunk);
  const int i0 = tile * kCtaTokens;
  if (i0 >= C) return;    // uniform for the CTA: nothing allocated yet
  if (s_base & 1023u) {   // the swizzled operands need 1024-byte alignment
    if (tid == 0) atomicOr(p.err, kErrSmemAlign);
    return;
  }
  const int i_last = min(C, i0 + kCtaTokens) - 1;
  const int n_tiles = i0 + kTokens < C ? 2 : 1;
  const int kv_end = prefix + i_last + 1;  // keys that the last row sees
  const int steps_all = (kv_end + kKeys - 1) / kKeys;
  const int j0 = kSplit ? split * steps_all / p.num_splits : 0;
  const int nsteps = kSplit ? (split + 1) * steps_all / p.num_splits - j0 : steps_all;
  float2* const ws_ml = !kSplit ? nullptr
                                : reinterpret_cast<float2*>(p.ws + static_cast<size_t>(p.num_splits) * p.num_seqs * p.ws_rows *
                                                                       p.num_q_heads * D);
  auto ws_row = [&](int token, int head) -> size_t {  // token: of the chunk; head: of the group
    return ((static_cast<size_t>(split) * p.num_seqs + b) * p.ws_rows + token) * p.num_q_heads + kvh * G + head;
  };
  if (kSplit && nsteps == 0) {  // uniform for the CTA
    for (int x = tid; x < kCtaTokens * G; x += kFp8Threads)
      if (i0 + x / G < C) ws_ml[ws_row(i0 + x / G, x % G)] = make_float2(-INFINITY, 0.f);
    return;
  }

  // Barriers as in the bf16 kernel, but that a ring slot is full when its converter says so.
  const uint32_t bar = s_base + T::kOffBar;
  const uint32_t r_full = bar, r_empty = r_full + 8 * kRing, s_full = r_empty + 8 * kRing, p_full = s_full + 8 * kTiles,
                 o_full = p_full + 8 * kTiles, q_ready = o_full + 8 * kTiles, mma_drained = q_ready + 8 * kTiles,
                 o_staged = mma_drained + 8;
  static_assert(8 * (2 * kRing + 5 * kTiles + 1) <= kTmemSlotOffset, "the barriers must end below the TMEM slot");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + T::kOffBar + kTmemSlotOffset);

  // Stage Q (zero rows past the chunk) in the swizzled K-major layout, ahead of the set-up.
  if ((warp >> 2) < n_tiles && warp < kIssuer) {
    constexpr int kChunks = D / 8;
    const int t = warp >> 2, r = tid & (kRows - 1);
    const __nv_bfloat16* qg = static_cast<const __nv_bfloat16*>(p.q);
    const uint32_t qt = s_base + T::kOffQ + t * T::kQTile;
#pragma unroll
    for (int c = r; c < kRows * kChunks; c += kRows) {
      const int rr = c / kChunks, ch = c % kChunks, ii = i0 + t * kTokens + rr / G;
      const bool in_chunk = ii < C;
      const __nv_bfloat16* src =
          in_chunk ? qg + (static_cast<size_t>(q0 + ii) * p.num_q_heads + kvh * G + rr % G) * D + ch * 8 : qg;
      cp_async_16(qt + (ch / 8) * T::kQHalf + swz(rr, ch % 8), src, in_chunk ? 16u : 0u);
    }
  }
  if (tid == 0) {
    for (int s = 0; s < kRing; ++s) {
      bar_init(r_full + 8 * s, kUnits);
      bar_init(r_empty + 8 * s, 1);
    }
    for (int t = 0; t < kTiles; ++t) {
      bar_init(s_full + 8 * t, 1);
      bar_init(p_full + 8 * t, 128);
      bar_init(o_full + 8 * t, 1);
      bar_init(q_ready + 8 * t, 128);
      bar_init(o_staged + 8 * t, kRows);
    }
    bar_init(mma_drained, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kIssuer) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  const uint32_t tmem = *tmem_slot;
  bool failed = false;

  if (warp > kIssuer) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    // ---------------- converters (tile n = 2 j is K of step j, n = 2 j + 1 its V; unit u is rows of tile u / 4) ------------
    constexpr int kChunks = D / 16;                   // 16-code chunks of a row
    constexpr int kLoads = kUnitRows * kChunks / 32;  // of a unit a lane
    constexpr int kPages = kKeys / kBlockTokens;
    constexpr int kLoadRows = 32 / kChunks;           // rows of a load instruction
    // Eight consecutive lanes hold four chunks of two rows, whose swizzled bf16 places are in different banks.
    const int my_row = D == 128 ? (lane >> 2) & 3 : lane >> 2, my_chunk = D == 128 ? (lane & 3) + ((lane >> 4) << 2) : lane & 3;
    const int npages = (kv_end + kBlockTokens - 1) / kBlockTokens;
    const int32_t* table = p.block_tables + static_cast<size_t>(b) * p.max_blocks_per_seq;
    const int units = 2 * nsteps * kUnits;
    // A unit is two blocks.  What a lane knows of one: the id of block lane / 4 % 2 (-1: none), and the exponents of rows
    // 4 (lane % 8) .. + 3.
    auto block_of = [&](int u) -> int {
      const int page = (j0 + u / (2 * kUnits)) * kPages + (u % kUnits) * 2 + ((lane >> 2) & 1);
      if (u >= units || page >= npages) return -1;
      int id = __ldg(table + page);
      if (id < 0 || id >= p.num_blocks) {
        atomicOr(p.err, kErrBlockId);
        id = 0;
      }
      return id;
    };
    auto exponents_of = [&](int u, int id) -> uint32_t {
      if (id < 0) return 0x7f7f7f7fu;
      return __ldg(reinterpret_cast<const uint32_t*>(p.kv_scales + (static_cast<int64_t>(id) * p.num_kv_heads + kvh) * 2 * kBlockTokens +
                                                     (u / kUnits & 1) * kBlockTokens + 4 * (lane & 3)));
    };
    // Where a lane's codes of each of the unit's blocks are; null: there is none.
    auto codes_of = [&](int u, int id, int block) -> const uint8_t* {
      const int of = __shfl_sync(0xffffffffu, id, 4 * block);
      if (of < 0) return nullptr;
      return static_cast<const uint8_t*>((u / kUnits & 1) ? p.v_cache : p.k_cache) +
             ((static_cast<int64_t>(of) * p.num_kv_heads + kvh) * kBlockTokens + my_row) * D + my_chunk * 16;
    };
    constexpr int kHalf = kLoads / 2;  // loads of a block
    auto load = [&](const uint8_t* from, int i) -> uint4 {
      return from ? load_codes(from + (i % kHalf) * kLoadRows * D) : make_uint4(0u, 0u, 0u, 0u);
    };
    // Chunk i's bf16 places: row 16 (i / kHalf) + (i % kHalf) kLoadRows + my_row, so that of its place in the swizzle only
    // bit 2 of the row goes by i, and only with 128 dims.
    const uint32_t even = kv_off<D>(my_row, 2 * my_chunk / 8, 2 * my_chunk % 8);
    const uint32_t odd = D == 128 ? kv_off<D>(my_row + 4, 2 * my_chunk / 8, 2 * my_chunk % 8) : 0u;
    auto place = [&](int i) -> uint32_t {
      const uint32_t at = (i / kHalf) * T::kPageBytes;
      if (D == 128) return at + ((i >> 1) & 1) * T::kGroupBytes + (i & 1 ? odd : even);
      return at + (i & 1) * T::kGroupBytes + even;
    };
    const uint32_t pick = 0x0444u | (lane >> 2 & 3) << 12;  // a row's exponent, byte my_row % 4, to the top byte

    int u = warp - kIssuer - 1;
    int id = block_of(u), next_id = block_of(u + kConverters), second_id = block_of(u + 2 * kConverters);
    uint32_t exponents = exponents_of(u, id);
    uint4 x[kLoads];
    {
      const uint8_t *first = codes_of(u, id, 0), *second = codes_of(u, id, 1);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) x[i] = load(i < kHalf ? first : second, i);
    }
    for (; u < units; u += kConverters) {
      const int n = u / kUnits, slot = n % kRing;
      const int third_id = block_of(u + 3 * kConverters);
      // The unit behind the next is on its way to L2 (28 KB in registers on their way from HBM would be too few).
      if ((lane & ~4) == 0 && second_id >= 0)
        l2_prefetch(static_cast<const uint8_t*>((u + 2 * kConverters) / kUnits & 1 ? p.v_cache : p.k_cache) +
                        (static_cast<int64_t>(second_id) * p.num_kv_heads + kvh) * kBlockTokens * D,
                    kBlockTokens * D);
      const uint32_t next_exponents = exponents_of(u + kConverters, next_id);
      const uint8_t *first = codes_of(u + kConverters, next_id, 0), *second = codes_of(u + kConverters, next_id, 1);
      if (n >= kRing && !__all_sync(0xffffffffu, bar_wait(r_empty + 8 * slot, (n / kRing + 1) & 1))) {
        failed = true;
        break;
      }
      unsigned char* unit_at = smem + T::kOffKV + slot * T::kTile + (u % kUnits) * 2 * T::kPageBytes;
      const int left = kv_end - (j0 + (n >> 1)) * kKeys - (u % kUnits) * kUnitRows;  // the unit's rows that hold keys
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const uint32_t four = __shfl_sync(0xffffffffu, exponents, (i * kLoadRows + my_row) >> 2);
        // 2^(e - 127), as fp8_scale.
        const float f = __uint_as_float(max(__byte_perm(four, 0, pick) >> 1, 0x00400000u));
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t r[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 v = __fmul2_rn(fp8_floats(static_cast<uint16_t>(w[k / 2] >> 16 * (k & 1))), make_float2(f, f));
          r[k] = pack_bf16(v.x, v.y);
        }
        x[i] = load(i < kHalf ? first : second, i);
        if (left < kUnitRows && i * kLoadRows + my_row >= left)
#pragma unroll
          for (int k = 0; k < 8; ++k) r[k] = 0u;
        *reinterpret_cast<uint4*>(unit_at + place(i)) = make_uint4(r[0], r[1], r[2], r[3]);
        *reinterpret_cast<uint4*>(unit_at + (place(i) ^ 16)) = make_uint4(r[4], r[5], r[6], r[7]);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) bar_arrive(r_full + 8 * slot);
      id = next_id;
      next_id = second_id;
      second_id = third_id;
      exponents = next_exponents;
    }
    if (failed && lane == 0) atomicOr(p.err, kErrTimeout);
  } else if (warp == kIssuer) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    // ---------------- MMA issuer: S of both tiles for step 0, then per step and tile P V and S of the next ----------------
    constexpr uint32_t kIdS = idesc_bf16(kKeys, false);
    constexpr uint32_t kIdPV = idesc_bf16(D, true);
    const uint64_t d_q = sdesc(s_base + T::kOffQ), d_kv = sdesc(s_base + T::kOffKV, 1024, T::kGroupBytes);
    const bool issuer = elect_one();
    auto poll = [&](uint32_t at, uint32_t parity) -> bool { return __all_sync(0xffffffffu, bar_poll(at, parity)); };
    auto issue_s = [&](int t, int slot) {
      const uint64_t q = d_q + static_cast<uint32_t>((t * T::kQTile) >> 4);
      const uint64_t k = d_kv + static_cast<uint32_t>((slot * T::kTile) >> 4);
#pragma unroll
      for (int h = 0; h < T::kHalves; ++h)
        mma4_ss<kIdS, 2, 2>(tmem + col_s(t), q + static_cast<uint32_t>((h * T::kQHalf) >> 4),
                            k + static_cast<uint32_t>((h * 1024) >> 4), h != 0);
      mma_commit(s_full + 8 * t);
    };
    for (int t = 0; t < n_tiles; ++t)
      if (!poll(q_ready + 8 * t, 0)) failed = true;
    if (!failed && !poll(r_full, 0)) failed = true;
    if (!failed) {
      tc_after_sync();
      if (issuer) {
        for (int t = 0; t < n_tiles; ++t) issue_s(t, 0);
        mma_commit(r_empty);
      }
      __syncwarp();
    }
    for (int j = 0; j < nsteps && !failed; ++j) {
      const int nv = 2 * j + 1, nk = 2 * j + 2;
      const int sv = nv % kRing, sk = nk % kRing;
      const bool last = j == nsteps - 1;
      if (!poll(r_full + 8 * sv, (nv / kRing) & 1) || (!last && !poll(r_full + 8 * sk, (nk / kRing) & 1))) {
        failed = true;
        break;
      }
      const uint64_t v = d_kv + static_cast<uint32_t>((sv * T::kTile) >> 4);
      for (int t = 0; t < n_tiles; ++t) {
        if (!poll(p_full + 8 * t, j & 1)) {
          failed = true;
          break;
        }
        tc_after_sync();
        if (issuer) {
          const uint32_t d_s = tmem + col_s(t);
#pragma unroll
          for (int g = 0; g < kKeys / 64; ++g)
            mma4_ts<kIdPV, 8, T::kPageBytes / 16>(tmem + col_o(t), d_s + g * 32,
                                                  v + static_cast<uint32_t>((g * 4 * T::kPageBytes) >> 4), (j | g) != 0);
          if (last) mma_commit(o_full + 8 * t);
          if (t == n_tiles - 1) mma_commit(r_empty + 8 * sv);
          if (!last) issue_s(t, sk);
        }
        __syncwarp();
      }
      if (failed) break;
      if (!last && issuer) mma_commit(r_empty + 8 * sk);
    }
    if (issuer) {
      if (failed) atomicOr(p.err, kErrTimeout);
      mma_commit(mma_drained);  // every MMA must have completed before the tensor memory is freed
      bar_poll(mma_drained, 0);
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ---------------- softmax / epilogue (thread = row of tile warp / 4) ----------------
    const int t = warp >> 2;
    if (t < n_tiles) {
      const int r = tid & (kRows - 1);
      constexpr int kChunks = D / 8;
      const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
      const uint32_t s_cols = lane_base + col_s(t), o_cols = lane_base + col_o(t);
      const float qk = p.scale * kLog2e;
      const int i = i0 + t * kTokens + r / G;
      const bool row_ok = i < C;
      cp_async_wait_all();
      fence_async_smem();
      bar_arrive(q_ready + 8 * t);
      const int limit = row_ok ? prefix + i + 1 : 0;
      // A warp without rows of the chunk leaves its part of P as it is: a row of O takes only its own row of P.
      // (In a loop of its own: as a branch of the loop below it costs that a sixth of its speed.)
      const bool idle = i0 + t * kTokens + (warp & 3) * 32 / G >= C;
      for (int j = 0; idle && j < nsteps && !failed; ++j) {
        if (!__all_sync(0xffffffffu, bar_wait(s_full + 8 * t, j & 1))) failed = true;
        else bar_arrive(p_full + 8 * t);
      }
      const bool sees = kSplit ? limit > j0 * kKeys : row_ok;  // (a split's range may start behind the row's last key)
      float m_used = -INFINITY, l = 0.f;
      for (int j = idle ? nsteps : 0; j < nsteps && !failed; ++j) {
        if (!__all_sync(0xffffffffu, bar_wait(s_full + 8 * t, j & 1))) {
          failed = true;
          break;
        }
        tc_after_sync();
        float s[kKeys];
        tmem_ld64(s_cols, *reinterpret_cast<float(*)[64]>(&s[0]));
        tmem_ld64(s_cols + 64, *reinterpret_cast<float(*)[64]>(&s[64]));
        const int ja = j0 + j;
        if (__any_sync(0xffffffffu, (ja + 1) * kKeys > limit)) {
#pragma unroll
          for (int x = 0; x < kKeys; ++x) s[x] = (ja * kKeys + x) < limit ? s[x] : -INFINITY;
        }
        float mc[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) mc[k] = fmax3(s[k], s[k + 8], s[k + 16]);
        static_assert(kKeys == 128, "row max layout");
#pragma unroll
        for (int x = 24; x < 120; x += 16)
#pragma unroll
          for (int k = 0; k < 8; ++k) mc[k] = fmax3(mc[k], s[x + k], s[x + 8 + k]);
#pragma unroll
        for (int k = 0; k < 8; ++k) mc[k] = fmaxf(mc[k], s[120 + k]);
        const float bm = qk * fmax3(fmax3(mc[0], mc[1], mc[2]), fmax3(mc[3], mc[4], mc[5]), fmaxf(mc[6], mc[7]));
        const bool raise = sees && bm > m_used + kSlack;
        const float m_new = raise ? bm : m_used;
        const float alpha = raise ? ex2_approx(m_used - m_new) : 1.f;
        const float neg_m = sees ? -m_new : 0.f;
        float2 acc4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        uint32_t packed[kKeys / 2];
        const float2 qk2 = make_float2(qk, qk), neg_m2 = make_float2(neg_m, neg_m);
#pragma unroll
        for (int x = 0; x < kKeys; x += 2) {
          // The denominator sums the fp32 weights, within 2^-9 of the bf16 ones that P carries.
          const float2 e = __ffma2_rn(make_float2(s[x], s[x + 1]), qk2, neg_m2);
          const float p0 = ex2_approx(e.x), p1 = ex2_approx(e.y);
          packed[x / 2] = pack_bf16(p0, p1);
          acc4[(x / 2) & 3] = __fadd2_rn(acc4[(x / 2) & 3], make_float2(p0, p1));
        }
        const float2 a = __fadd2_rn(__fadd2_rn(acc4[0], acc4[1]), __fadd2_rn(acc4[2], acc4[3]));
        l = l * alpha + (a.x + a.y);
        m_used = m_new;
        if (j >= 1 && __any_sync(0xffffffffu, raise)) {
#pragma unroll
          for (int c0 = 0; c0 < D; c0 += 32) {
            float o[32];
            tmem_ld32(o_cols + c0, o);
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] *= alpha;
            tmem_st32(o_cols + c0, o);
          }
        }
        tmem_st32_raw(s_cols, *reinterpret_cast<const uint32_t(*)[32]>(&packed[0]));
        tmem_st32_raw(s_cols + 32, *reinterpret_cast<const uint32_t(*)[32]>(&packed[32]));
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_before_sync();
        bar_arrive(p_full + 8 * t);
      }
      if constexpr (kSplit) {
        // Partial states through the warp's own 4 KB of the tile's Q buffer, 32 columns at a time, so that each store writes
        // four 128-byte row segments.
        if (!failed && __all_sync(0xffffffffu, bar_wait(o_full + 8 * t, 0))) {
          tc_after_sync();
          float* scratch = reinterpret_cast<float*>(smem + T::kOffQ + t * T::kQTile) + (warp & 3) * 32 * 32;
#pragma unroll
          for (int c0 = 0; c0 < D; c0 += 32) {
            float o[32];
            tmem_ld32(o_cols + c0, o);
#pragma unroll
            for (int q4 = 0; q4 < 8; ++q4)
              *reinterpret_cast<float4*>(scratch + lane * 32 + ((q4 + lane) & 7) * 4) =
                  make_float4(o[4 * q4], o[4 * q4 + 1], o[4 * q4 + 2], o[4 * q4 + 3]);
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int rr = 4 * k + (lane >> 3), q4 = lane & 7;
              const float4 v = *reinterpret_cast<const float4*>(scratch + rr * 32 + ((q4 + rr) & 7) * 4);
              const int tr = (warp & 3) * 32 + rr, ii = i0 + t * kTokens + tr / G;
              if (ii < C) *reinterpret_cast<float4*>(p.ws + ws_row(ii, tr % G) * D + c0 + q4 * 4) = v;
            }
            __syncwarp();
          }
          if (row_ok) ws_ml[ws_row(i, r % G)] = make_float2(m_used, l);
        } else {
          failed = true;
        }
      } else {
        bool staged = false;
        unsigned char* ot = smem + T::kOffQ + t * T::kQTile;  // (every S that read Q has retired)
        if (!failed && __all_sync(0xffffffffu, bar_wait(o_full + 8 * t, 0))) {
          tc_after_sync();
          const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
          for (int c0 = 0; c0 < D; c0 += 32) {
            float o[32];
            tmem_ld32(o_cols + c0, o);
#pragma unroll
            for (int x = 0; x < 32; x += 8) {
              const int ch = (c0 + x) / 8;
              *reinterpret_cast<uint4*>(ot + (ch / 8) * T::kQHalf + swz(r, ch % 8)) =
                  make_uint4(pack_bf16(o[x] * inv, o[x + 1] * inv), pack_bf16(o[x + 2] * inv, o[x + 3] * inv),
                             pack_bf16(o[x + 4] * inv, o[x + 5] * inv), pack_bf16(o[x + 6] * inv, o[x + 7] * inv));
            }
          }
          fence_async_smem();
          staged = true;
        } else {
          failed = true;
        }
        bar_arrive(o_staged + 8 * t);  // (staged or not, so that the wait below ends)
        if (__all_sync(0xffffffffu, staged && bar_wait(o_staged + 8 * t, 0))) {
          const int tok0 = i0 + t * kTokens;
          if (tok0 + kTokens <= C) {  // a whole tile leaves by tensor stores
            if (r == 0) {
#pragma unroll
              for (int h = 0; h < T::kHalves; ++h)
                tma_store_3d(&map_out, 64 * h, kvh * G, q0 + tok0, s_base + T::kOffQ + t * T::kQTile + h * T::kQHalf);
              tma_store_commit_and_wait_read();
            }
          } else {
            __nv_bfloat16* og = static_cast<__nv_bfloat16*>(p.out);
#pragma unroll 4
            for (int c = r; c < kRows * kChunks; c += kRows) {
              const int rr = c / kChunks, ch = c % kChunks, ii = tok0 + rr / G;
              if (ii < C)
                reinterpret_cast<uint4*>(og + (static_cast<size_t>(q0 + ii) * p.num_q_heads + kvh * G + rr % G) * D)[ch] =
                    *reinterpret_cast<const uint4*>(ot + (ch / 8) * T::kQHalf + swz(rr, ch % 8));
            }
          }
        } else {
          failed = true;
        }
      }
      if (failed && lane == 0) atomicOr(p.err, kErrTimeout);
    }
  }

  tc_before_sync();
  __syncthreads();
  if (warp == kIssuer) {
    tc_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// Merge of a split call: for every row, over the splits whose m is finite, M = max m_s and out = sum_s 2^(m_s - M) O_s /
// sum_s 2^(m_s - M) l_s.  A warp takes kMergeRows (chunk token, q head) rows at a time, lane s the (m, l) of split s.  It is
// latency that counts: the first kFirst splits' O are requested before their (m, l) say which of them saw a key.
constexpr int kMergeRows = 2;
template <int D>
__global__ void __launch_bounds__(256) merge_fp8_kernel(const Fp8PrefillParams p) {
  constexpr int kCols = D / 32, kFirst = 8;
  const int b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  pdl_wait();
  const int q0 = p.query_start[b], q1 = p.query_start[b + 1], len = p.context_lens[b];
  const int64_t chunk = static_cast<int64_t>(q1) - q0;
  const size_t stride = static_cast<size_t>(p.num_seqs) * p.ws_rows * p.num_q_heads;  // rows of a split
  const float2* ml = reinterpret_cast<const float2*>(p.ws + static_cast<size_t>(p.num_splits) * stride * D);
  if (chunk < 0 || len < chunk || len > p.max_blocks_per_seq * kBlockTokens || q0 < 0 || q1 > p.query_rows) return;
  const int rows = min(static_cast<int>(chunk), p.max_query_len) * p.num_q_heads;
  auto load = [&](const float* o, float (&v)[kCols]) {
    if constexpr (kCols == 4) {
      const float4 x = *reinterpret_cast<const float4*>(o);
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else {
      const float2 x = *reinterpret_cast<const float2*>(o);
      v[0] = x.x; v[1] = x.y;
    }
  };
  for (int row0 = (blockIdx.x * 8 + warp) * kMergeRows; row0 < rows; row0 += gridDim.x * 8 * kMergeRows) {
    const size_t r0 = static_cast<size_t>(b) * p.ws_rows * p.num_q_heads + row0;
    float2 s[kMergeRows];
    float v[kMergeRows][kFirst][kCols];
#pragma unroll
    for (int k = 0; k < kMergeRows; ++k) {
      s[k] = make_float2(-INFINITY, 0.f);
      if (row0 + k < rows && lane < p.num_splits) s[k] = ml[lane * stride + r0 + k];
    }
#pragma unroll
    for (int k = 0; k < kMergeRows; ++k)
#pragma unroll
      for (int f = 0; f < kFirst; ++f)
        if (row0 + k < rows && f < p.num_splits) load(p.ws + (f * stride + r0 + k) * D + lane * kCols, v[k][f]);
#pragma unroll
    for (int k = 0; k < kMergeRows; ++k) {
      if (row0 + k >= rows) break;
      float mx = s[k].x;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      const float w = s[k].x == -INFINITY ? 0.f : exp2f(s[k].x - mx);
      float den = w * s[k].y;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) den += __shfl_xor_sync(0xffffffffu, den, off);
      const float inv = den != 0.f ? 1.f / den : 0.f;
      float acc[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c) acc[c] = 0.f;
#pragma unroll
      for (int f = 0; f < kFirst; ++f) {
        const float wf = __shfl_sync(0xffffffffu, w, f);
        if (wf == 0.f) continue;  // no such split, or one that saw no key and wrote no O
#pragma unroll
        for (int c = 0; c < kCols; ++c) acc[c] += wf * v[k][f][c];
      }
      for (int f = kFirst; f < p.num_splits; ++f) {
        const float wf = __shfl_sync(0xffffffffu, w, f);
        if (wf == 0.f) continue;
        float o[kCols];
        load(p.ws + (f * stride + r0 + k) * D + lane * kCols, o);
#pragma unroll
        for (int c = 0; c < kCols; ++c) acc[c] += wf * o[c];
      }
      uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) +
                                                  (static_cast<size_t>(q0) * p.num_q_heads + row0 + k) * D + lane * kCols);
#pragma unroll
      for (int c = 0; c < kCols; c += 2) dst[c / 2] = pack_bf16(acc[c] * inv, acc[c + 1] * inv);
    }
  }
}

// Unpacked form: the blocks that a sequence's rows see, in order, as bf16 ([sequence][block of its table], both with all heads),
// the table that numbers them so, and the context lengths, -1 for a sequence that the call skips.  Bound by HBM, two bytes
// written for each read: 16384 tokens of 8 heads of 128 dims 23 us with cold caches, 12 of the call's 746 us in a loop.
constexpr int kUnpackThreads = 256, kUnpackCtas = 8;  // CTAs an SM
template <int D>
__global__ void __launch_bounds__(kUnpackThreads) unpack_fp8_kernel(const Fp8AttentionParams p, const Fp8Unpacked to) {
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, ctas = static_cast<int>(gridDim.x);
  const int64_t thread = static_cast<int64_t>(blockIdx.x) * kUnpackThreads + tid, threads = static_cast<int64_t>(ctas) * kUnpackThreads;
  const int64_t slots = static_cast<int64_t>(p.num_seqs) * p.max_blocks_per_seq;
  for (int64_t i = thread; i < slots; i += threads) to.block_tables[i] = static_cast<int32_t>(i);
  auto blocks_of = [&](int b, bool& skipped) -> int {
    const int q0 = __ldg(p.query_start + b), q1 = __ldg(p.query_start + b + 1), len = __ldg(p.context_lens + b);
    const int64_t chunk = static_cast<int64_t>(q1) - q0;
    skipped = chunk < 0 || len < chunk || len > p.max_blocks_per_seq * kBlockTokens || q0 < 0 || q1 > p.query_rows;
    return skipped || chunk == 0 ? 0 : (len + kBlockTokens - 1) / kBlockTokens;
  };
  for (int64_t b = thread; b < p.num_seqs; b += threads) {
    bool skipped;
    blocks_of(static_cast<int>(b), skipped);
    to.context_lens[b] = skipped ? -1 : __ldg(p.context_lens + b);
  }
  const int pieces = p.num_kv_heads * D;  // of 16 codes, in a block of K (or V)
  const int parts = (pieces + kUnpackThreads - 1) / kUnpackThreads;
  auto unpack = [&](int b, int64_t item) {  // a part of a block: a piece of K and of V a thread
    const int j = static_cast<int>(item / parts), x = static_cast<int>(item % parts) * kUnpackThreads + tid;
    if (x >= pieces) return;
    const int64_t at = static_cast<int64_t>(b) * p.max_blocks_per_seq + j;
    int id = __ldg(p.block_tables + at);
    if (id < 0 || id >= p.num_blocks) {
      if (tid == 0) atomicOr(p.err, kErrBlockId);
      id = 0;
    }
    const int64_t from = static_cast<int64_t>(id) * pieces;
    const int head = x / D, row = x % D / (D / 16);
    const uint8_t* e = p.kv_scales + (static_cast<int64_t>(id) * p.num_kv_heads + head) * 2 * kBlockTokens + row;
    const uint4 codes[2] = {load_codes(p.k_cache + (from + x) * 16), load_codes(p.v_cache + (from + x) * 16)};
    const float scale[2] = {fp8_scale(__ldg(e)), fp8_scale(__ldg(e + kBlockTokens))};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w[4] = {codes[i].x, codes[i].y, codes[i].z, codes[i].w};
      uint32_t r[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 f = fp8_floats(static_cast<uint16_t>(w[k / 2] >> 16 * (k & 1)));
        r[k] = pack_bf16(f.x * scale[i], f.y * scale[i]);
      }
      uint4* dst = reinterpret_cast<uint4*>(i ? to.v : to.k) + (at * pieces + x) * 2;
      dst[0] = make_uint4(r[0], r[1], r[2], r[3]);
      dst[1] = make_uint4(r[4], r[5], r[6], r[7]);
    }
  };
  // The sequences' items are dealt to the CTAs in turns.
  __shared__ int s_blocks[kUnpackThreads];
  int64_t turn = blockIdx.x;  // items ahead until this CTA's next
  for (int b0 = 0; b0 < p.num_seqs; b0 += kUnpackThreads) {
    const int n = min(kUnpackThreads, p.num_seqs - b0);
    bool skipped;
    if (tid < n) s_blocks[tid] = blocks_of(b0 + tid, skipped);
    __syncthreads();
    for (int x = 0; x < n; ++x) {
      const int64_t items = static_cast<int64_t>(s_blocks[x]) * parts;
      for (; turn < items; turn += ctas) unpack(b0 + x, turn);
      turn -= items;
    }
    __syncthreads();
  }
}

template <int D, int G, bool kSplit>
cudaError_t launch_fp8(Fp8PrefillParams p, cudaStream_t stream) {
  constexpr int kCtaTokens = kTiles * kRows / G;
  static std::mutex mu;
  static uint64_t ready = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!(dev < 64 && ((ready >> dev) & 1u))) {
      e = cudaFuncSetAttribute(&prefill_fp8_kernel<D, G, kSplit>, cudaFuncAttributeMaxDynamicSharedMemorySize, Pf<D>::kSmem);
      if (e != cudaSuccess) return e;
      if (dev < 64) ready |= uint64_t{1} << dev;
    }
  }
  CUtensorMap mo;
  const int64_t tokens = p.query_rows < INT32_MAX ? p.query_rows : INT32_MAX;
  if ((e = out_map(&mo, p.out, tokens, p.num_q_heads, D, G, kRows / G)) != cudaSuccess) return e;
  const int tiles = (p.max_query_len + kCtaTokens - 1) / kCtaTokens;
  p.ws_rows = tiles * kCtaTokens;
  const dim3 grid(p.num_kv_heads, tiles, p.num_seqs * (kSplit ? p.num_splits : 1));
  e = launch_pdl(prefill_fp8_kernel<D, G, kSplit>, grid, dim3(kFp8Threads), Pf<D>::kSmem, stream, p, mo);
  if (!kSplit || e != cudaSuccess) return e;
  const int64_t blocks = (static_cast<int64_t>(p.max_query_len) * p.num_q_heads + 8 * kMergeRows - 1) / (8 * kMergeRows);
  return launch_pdl(merge_fp8_kernel<D>, dim3(static_cast<unsigned>(blocks < 65535 ? blocks : 65535), p.num_seqs), dim3(256), 0,
                    stream, p);
}

template <bool kSplit>
cudaError_t dispatch_fp8(const Fp8PrefillParams& p, int head_dim, int group, cudaStream_t stream) {
  switch (head_dim * 16 + group) {
    case 64 * 16 + 1: return launch_fp8<64, 1, kSplit>(p, stream);
    case 64 * 16 + 2: return launch_fp8<64, 2, kSplit>(p, stream);
    case 64 * 16 + 4: return launch_fp8<64, 4, kSplit>(p, stream);
    case 64 * 16 + 8: return launch_fp8<64, 8, kSplit>(p, stream);
    case 128 * 16 + 1: return launch_fp8<128, 1, kSplit>(p, stream);
    case 128 * 16 + 2: return launch_fp8<128, 2, kSplit>(p, stream);
    case 128 * 16 + 4: return launch_fp8<128, 4, kSplit>(p, stream);
    case 128 * 16 + 8: return launch_fp8<128, 8, kSplit>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_prefill_unpacked_fp8(const Fp8AttentionParams& a, int head_dim, int num_splits, const Fp8Unpacked& to, float* ws,
                                        int num_sms, cudaStream_t stream) {
  const int64_t blocks = static_cast<int64_t>(a.num_seqs) * a.max_blocks_per_seq, most = static_cast<int64_t>(num_sms) * kUnpackCtas;
  const int64_t items = blocks * ((a.num_kv_heads * head_dim + kUnpackThreads - 1) / kUnpackThreads);
  const cudaError_t e = launch_pdl(head_dim == 128 ? unpack_fp8_kernel<128> : unpack_fp8_kernel<64>,
                                   dim3(static_cast<unsigned>(items < most ? items : most)), dim3(kUnpackThreads), 0, stream, a, to);
  if (e != cudaSuccess) return e;
  PrefillParams p{};
  p.q = a.q;
  p.k_cache = to.k;
  p.v_cache = to.v;
  p.block_tables = to.block_tables;
  p.context_lens = to.context_lens;
  p.query_start = a.query_start;
  p.out = a.out;
  p.err = a.err;
  p.num_blocks = blocks;
  p.num_seqs = a.num_seqs;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.max_query_len = a.max_query_len;
  p.scale = a.scale;
  p.num_splits = num_splits;
  p.ws = ws;
  return launch_paged_prefill(p, head_dim, a.num_q_heads / a.num_kv_heads, a.max_query_len, stream);
}

cudaError_t launch_prefill_fp8(const Fp8AttentionParams& a, int head_dim, int num_splits, float* ws, cudaStream_t stream) {
  Fp8PrefillParams p{};
  p.q = a.q;
  p.k_cache = a.k_cache;
  p.v_cache = a.v_cache;
  p.kv_scales = a.kv_scales;
  p.block_tables = a.block_tables;
  p.context_lens = a.context_lens;
  p.query_start = a.query_start;
  p.out = a.out;
  p.err = a.err;
  p.num_blocks = a.num_blocks;
  p.num_seqs = a.num_seqs;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.max_query_len = a.max_query_len;
  p.scale = a.scale;
  p.query_rows = a.query_rows;
  p.num_splits = num_splits;
  p.ws = ws;
  const int group = a.num_q_heads / a.num_kv_heads;
  return num_splits > 1 ? dispatch_fp8<true>(p, head_dim, group, stream) : dispatch_fp8<false>(p, head_dim, group, stream);
}

}  // namespace pkv
