// Attention of few query rows a sequence over the 8-bit cache: decode (one query token), and chunks of a few tokens.
//
//   out[row][h] = softmax_j(scale <q[row][h], K_j>) V_j  over the tokens j that the row sees,
//   K_j = 2^(ke_j) kc_j,  V_j = 2^(ve_j) vc_j   (codes kc, vc in e4m3; one exponent a row and kv head)
//
// Bound by HBM: a token's K and V of a kv head are 2 D + 2 bytes, read once, and feed 4 D flop a query row.
//
// Products.  The rows of a (sequence, kv head), G heads of up to a few tokens, are the columns of two small products on the
// warp-level tensor cores, a block of 16 tokens at a time:
//   S^T [16 tokens x columns] = Kc q^T,   O^T [D x columns] += Vc^T W^T,
// in fp16 with 32-bit sums: fp16 holds every e4m3 code exactly, and q too (bf16, eight significant bits) once a row is
// brought to a largest value of 2^14 by a power of two, down to 2^-28 of it; smaller values lose bits that a score does not
// show.  The exponents stay outside of the products: a score is S 2^(ke) scale, and a weight takes V's exponent with it,
//   w_j = 2^((s_j - m) + ve_j - r),   O = 2^r sum_j w_j vc_j,   l = sum_j 2^(s_j - m),
// with running references (base 2) m of s and r of (s - m) + ve, seven to eight below their largest value and raised when some
// value passes them by fifteen, so that w is at most 2^15 and the largest of a row is 2^7 or more: fp16's 11 bits (half a step is
// 2^-11 of a weight) hold for weights down to 2^-21 of the largest, and those below 2^-32 of it vanish.  (m comes off first: next
// to a large score an exponent would lose its bits.)
//
// Weights.  With one block of columns (decode, and chunks of up to eight rows) a weight enters its product in two parts, the
// fp16 and what that rounded off, as the bf16 cache's decode has it, so that little but the output's own rounding is left (against
// sums in 32 bits the results differ by 5e-5 of themselves, one part 4e-4).  128 sequences 105.9 -> 107.1 us, 61 long ones 104.9 -> 107.1, one 7.7 -> 7.9.
// With two or three blocks, rows of chunks, it is one part: the chunk kernel beside it has eight bits, and the second part costs
// 64 drafts 90 -> 100 us, 24 rows 106 -> 118.  There l sums the same eleven bits, for a row that one token outweighs then loses
// none of them (without, 9e-4; 64 drafts 90.1 -> 92.2, 24 rows 106 -> 109).  And the references are whole numbers: a power of two moves no
// significant bit, so a weight is rounded to the same eleven whatever the reference is, and a sequence's result does not depend
// on where its batch is cut.  (With the largest value itself, 3 to 7 % of the results changed by a step with the cut.)
//
// Work.  The batch's blocks form one stream of units of 32 KB of K and V, eight (block, kv head) tiles of 128 dims or sixteen
// of 64: all eight heads of a block (of two), or two (four) blocks of four heads, and so on.  The stream is cut into equal
// contiguous pieces, one a CTA (two an SM for up to eight rows), so that every CTA has the same work whatever the lengths: the
// same bytes, or, where sequences differ in their rows, units that cost by them.  Each of a CTA's eight warps takes its tile of
// every unit (two of 64 dims), which are neighbours in memory, through a ring of its own: the lanes copy it in 16-byte pieces
// (cp.async), placed so that ldmatrix reads without bank conflicts.  So no warp waits for another, but where the warps of a
// head join their states at a pair's end.  (By tensor copies, as large as a unit for eight heads, a CTA has to wait for all its
// warps at every unit, and a unit of one head is 24 copies, whose number bounds an SM: 128 sequences of 2048 tokens of one head
// took 28.7 us so, 17.7 like this; of eight heads 104 and 107.)  A (sequence, heads) pair cut by a piece's border leaves partial
// states (m, l, O) that a second kernel joins.
//
// Few pairs.  A call of few (sequence, kv head) pairs takes a thread-block cluster a pair instead: its units, of one head, are
// dealt to the cluster's CTAs in turns (so that their block ids can be asked for along with the length), whose states are
// joined through distributed shared memory.  One launch, no workspace, and no pass over the batch's lengths: one sequence of
// 4097 tokens, 16 q and 8 kv heads, takes 7.9 us a call.
//
// Measured (32 q and 8 kv heads of 128 dims; calls one after another over several inputs in turn): 128 sequences of 512..4096
// tokens 107.1 us, 5.7 TB/s with the second launch (0.85 of the copy bandwidth); 61 sequences of up to 65536 tokens, 64 q heads
// of 64 dims, 107.1 us, where the instructions count; 64 sequences with up to five tokens 92.2 us.  (Before weights came in two
// parts and with the products taken out, over one input: 98 and 94.)
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "fp8_cache.h"
#include "fp8_format.cuh"

namespace pkv {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMostCluster = 16;
constexpr float kNone = -3.0e38f;  // the reference of a row that has seen no token
constexpr float kTopLog = 7.f, kMostLog = 15.f;  // the largest of a row's weights is brought to 2^7 .. 2^8, may grow to 2^15

template <int D, int NC, bool kCluster>
struct Few {
  static constexpr int kCols = 8 * NC;
  static constexpr int kTile = kBlockTokens * D;           // bytes of one tile of K (or V)
  static constexpr int kTurns = 128 / D;                   // tiles of a unit that a warp takes, one after the other
  static constexpr int kUnitTiles = kWarps * kTurns;       // (block, kv head) tiles of a unit
  static constexpr int kCtas = NC == 1 ? 2 : 1;            // per SM
  // The next tile's scores beside this one's softmax: with so many registers a warp is alone with one other on its scheduler
  // (64 x 6 tokens 110 -> 103 us; with two column blocks 84.7 -> 86.2, with one 1000 short sequences 49.0 -> 50.8).
  static constexpr bool kAhead = D == 128 && NC == 3 && !kCluster;
  static constexpr int kParts = NC == 1 ? 2 : 1;  // fp16 parts of a weight
  static constexpr int kStages = kAhead ? 5 : 6 * kTurns / kCtas;   // tiles of a warp's ring
  static constexpr int kStage = 2 * kTile;                 // K, V
  static constexpr int kScales = 2 * kBlockTokens;         // the exponents of both
  static constexpr int kOffScales = kWarps * kStages * kStage;
  static constexpr int kOffExchange = kOffScales + kWarps * kStages * kScales;
  static constexpr int kExchange = kWarps / 2 * 32 * 32;  // 8 values a lane of four warps
  static constexpr int kOffQ = kOffExchange + kExchange;  // a warp's fragments of q
  static constexpr int kQ = kAhead ? NC * D / 16 * 2 * 32 * 4 : 0;
  static constexpr int kOffMl = kOffQ + kWarps * kQ;
  static constexpr int kMl = (kWarps + 1) * kCols * 8;  // a cluster CTA's: of every warp, and joined
  static constexpr int kOffSeq = kOffMl + kMl;  // costs before each sequence, [num_seqs + 1]; tokens, [num_seqs]
  // What a unit costs by the column blocks that its sequence fills: 6, 7 or 8 (64 sequences with one to five tokens: 89.6 us;
  // 4, 5, 6 92.2; 10, 11, 12 90.4; all the same 93.6).
  __host__ __device__ static constexpr int cost(int blocks) { return NC == 1 ? 1 : 5 + blocks; }
  __device__ static int next(int place) { return place + kTurns == kStages ? 0 : place + kTurns; }  // of a unit's first tile
  static constexpr int smem(int num_seqs) { return kOffSeq + (2 * num_seqs + 1) * 4; }
};

// ---------------------------------------------------------------------------
// PTX
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t saddr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
// 16 bytes global -> shared, past L1.
__device__ __forceinline__ void copy_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_wait() {  // all groups but the last kLeft have landed
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ void l2_prefetch(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint4 lds_128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of the same shared-memory location in CTA `rank` of the cluster, and loads from there.
__device__ __forceinline__ uint32_t remote(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 remote_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float2 remote_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_f16(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// ---------------------------------------------------------------------------
// A sequence's rows and tokens
// ---------------------------------------------------------------------------
struct Rows {
  int first;   // row of q and out
  int count;   // query tokens computed; 0: none, or the sequence is skipped
  int tokens;  // cached tokens that the last of them sees; row i sees tokens - count + i + 1
  unsigned wrong;  // error bits
};
__device__ __forceinline__ Rows rows_of(const Fp8AttentionParams& p, int b) {
  const int cap = p.max_blocks_per_seq * kBlockTokens;
  const int len = __ldg(p.context_lens + b);
  if (!p.query_start) {
    if (len < 0) return {b, 1, 0, kErrLenNegative};
    if (len > cap) return {b, 1, cap, kErrLenTooLong};
    return {b, 1, len, 0u};
  }
  const int q0 = __ldg(p.query_start + b), q1 = __ldg(p.query_start + b + 1);
  const int64_t chunk = static_cast<int64_t>(q1) - q0;
  if (chunk < 0 || len < chunk || len > cap || q0 < 0 || q1 > p.query_rows) return {0, 0, 0, kErrLenTooLong};
  const int count = min(static_cast<int>(chunk), p.max_query_len);
  return {q0, count, len - static_cast<int>(chunk) + count, count < chunk ? kErrLenTooLong : 0u};
}

// Where of the stream a thread is: sequence, group of heads, unit of the sequence's.
struct Walk {
  int b, heads, unit, units;
};

// A (sequence, kv head) in a warp's registers.
template <int D, int NC, bool kCluster>
struct Pair {
  using T = Few<D, NC, kCluster>;
  static constexpr int kTurns = T::kTurns;
  static constexpr int kSteps = D / 16;  // 16-byte chunks of a row of codes: 16 dims, the depth of a product
  // With few tiles a warp it is their latency that counts: V's codes, too, are taken into registers first, and the tiles'
  // places are free for the next copies.  With many it is registers (V's codes first: 128 sequences 107 -> 110 us, drafts of
  // up to five tokens 106 -> 128; one sequence 10.2 -> 8.9).
  static constexpr bool kEarly = kCluster;
  // Scores come in two sums where there would be a single chain of products.
  static constexpr int sums(int used) { return used * kTurns == 1 ? 2 : 1; }

  uint32_t ld_at;               // this lane's address for ldmatrix in the ring's first tile
  const unsigned char* scales;  // the ring's exponents
  uint32_t q_at;                // kAhead: this lane's fragments of q in shared memory
  int g, t;                     // lane / 4, lane % 4: row g and columns 2t, 2t + 1 of an accumulator
  int group_bits;
  int tokens, first_limit;    // tokens that the last and the first row see
  uint32_t q[NC][kSteps][2];  // B fragments of the rows
  float2 q_scale[NC];         // of columns 2t, 2t + 1: what takes a product to a score
  float2 nm[NC], nr[NC], l[NC];  // of those columns: -m, -r, and l
  float o[kSteps][NC][4];
  uint32_t vx[kTurns][kSteps / 2][4];

  // S^T = Kc q^T of the tiles at `place`.  Chunk c of a row: its 16 codes are the product's depth, in the order 4t, 4t + 1,
  // 4t + 2, 4t + 3 of a lane's four, as q's fragments are.
  template <int kUsed>
  __device__ __forceinline__ void products(int place, float (&sum)[kTurns][sums(kUsed)][kUsed][4]) {
    const uint32_t tile_at = ld_at + place * T::kStage;
    uint32_t kx[kTurns][kSteps / 2][4];
    if constexpr (kEarly) {
#pragma unroll
      for (int y = 0; y < kTurns; ++y) {
#pragma unroll
        for (int c = 0; c < kSteps / 2; ++c) ldsm_x4((tile_at + y * T::kStage) ^ (32u * c), kx[y][c]);
#pragma unroll
        for (int c = 0; c < kSteps / 2; ++c) ldsm_x4_t(((tile_at + y * T::kStage) ^ (32u * c)) + T::kTile, vx[y][c]);
      }
    }
#pragma unroll
    for (int y = 0; y < kTurns; ++y) {
#pragma unroll
      for (int x = 0; x < sums(kUsed); ++x)
#pragma unroll
        for (int nc = 0; nc < kUsed; ++nc)
#pragma unroll
          for (int k = 0; k < 4; ++k) sum[y][x][nc][k] = 0.f;
#pragma unroll
      for (int c = 0; c < kSteps / 2; ++c) {
        uint32_t a[4][2];
        if constexpr (!kEarly) ldsm_x4((tile_at + y * T::kStage) ^ (32u * c), kx[y][c]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          a[k][0] = fp8_halves(static_cast<uint16_t>(kx[y][c][k]));
          a[k][1] = fp8_halves(static_cast<uint16_t>(kx[y][c][k] >> 16));
        }
#pragma unroll
        for (int nc = 0; nc < kUsed; ++nc) {
          uint4 b = make_uint4(q[nc][2 * c][0], q[nc][2 * c][1], q[nc][2 * c + 1][0], q[nc][2 * c + 1][1]);
          if constexpr (T::kAhead)
            b = lds_128(q_at + (nc * kSteps / 2 + c) * 512);
          mma_f16(sum[y][0][nc], a[0][0], a[1][0], a[0][1], a[1][1], b.x, b.y);
          mma_f16(sum[y][sums(kUsed) - 1][nc], a[2][0], a[3][0], a[2][1], a[3][1], b.z, b.w);
        }
      }
    }
  }
  // The softmax of the tiles at `place`, from token0 on, and O^T += Vc^T W^T.
  template <int kUsed, typename Send>
  __device__ __forceinline__ void weigh(int place, int token0, const float (&sum)[kTurns][sums(kUsed)][kUsed][4], Send& send) {
    const uint32_t tile_at = ld_at + place * T::kStage;
    float v_lo[kTurns], v_hi[kTurns], s[kTurns][kUsed][4];
#pragma unroll
    for (int y = 0; y < kTurns; ++y) {
      const unsigned char* sc = scales + (place + y) * T::kScales;
      const float k_lo = fp8_scale(sc[g]), k_hi = fp8_scale(sc[g + 8]);
      v_lo[y] = fp8_power(sc[16 + g]);
      v_hi[y] = fp8_power(sc[24 + g]);
#pragma unroll
      for (int nc = 0; nc < kUsed; ++nc)
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // rows g and g + 8: tokens
          float2 x = make_float2(sum[y][0][nc][2 * h], sum[y][0][nc][2 * h + 1]);
          if (sums(kUsed) == 2) x = __fadd2_rn(x, make_float2(sum[y][sums(kUsed) - 1][nc][2 * h], sum[y][sums(kUsed) - 1][nc][2 * h + 1]));
          const float by = h ? k_hi : k_lo;
          x = __fmul2_rn(x, __fmul2_rn(q_scale[nc], make_float2(by, by)));
          s[y][nc][2 * h] = x.x;
          s[y][nc][2 * h + 1] = x.y;
        }
    }
    if constexpr (kEarly) {
      __syncwarp();  // the tiles have been read
#pragma unroll
      for (int turn = 0; turn < kTurns; ++turn) send();
    }
    const bool masked = token0 + kTurns * kBlockTokens > first_limit;
    if (masked) {
#pragma unroll
      for (int y = 0; y < kTurns; ++y)
#pragma unroll
        for (int nc = 0; nc < kUsed; ++nc)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (token0 + y * kBlockTokens + g + (k < 2 ? 0 : 8) >= first_limit + ((nc * 8 + 2 * t + (k & 1)) >> group_bits))
              s[y][nc][k] = -INFINITY;
    }
    // Of tile y, column block nc and row half h: s - m, and (s - m) + ve - r.
    auto logs = [&](int y, int nc, int h, float2& d, float2& e) {
      const float v = h ? v_hi[y] : v_lo[y];
      d = __fadd2_rn(make_float2(s[y][nc][2 * h], s[y][nc][2 * h + 1]), nm[nc]);
      e = __fadd2_rn(d, __fadd2_rn(make_float2(v, v), nr[nc]));
    };
    float most = -INFINITY;
#pragma unroll
    for (int y = 0; y < kTurns; ++y)
#pragma unroll
      for (int nc = 0; nc < kUsed; ++nc)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float2 d, e;
          logs(y, nc, h, d, e);
          most = fmaxf(fmaxf(most, fmaxf(d.x, d.y)), fmaxf(e.x, e.y));
        }
    if (__any_sync(kAll, most > kMostLog)) {  // seldom but for a pair's first block
#pragma unroll
      for (int nc = 0; nc < kUsed; ++nc)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float top = -INFINITY, top_w = -INFINITY;
#pragma unroll
          for (int y = 0; y < kTurns; ++y) top = fmaxf(top, fmaxf(s[y][nc][k], s[y][nc][k + 2]));
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, off));
          const float m = k ? -nm[nc].y : -nm[nc].x, r = k ? -nr[nc].y : -nr[nc].x;
          const float mn = fmaxf(floorf(top) - kTopLog, m), by = m - mn;
#pragma unroll
          for (int y = 0; y < kTurns; ++y) top_w = fmaxf(top_w, fmaxf(s[y][nc][k] - mn + v_lo[y], s[y][nc][k + 2] - mn + v_hi[y]));
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) top_w = fmaxf(top_w, __shfl_xor_sync(kAll, top_w, off));
          const float was = r + by;  // against the new m
          const float rn = fmaxf(floorf(top_w) - kTopLog, was), alpha = ex2(was - rn), beta = ex2(by);
          if (k) {
            nm[nc].y = -mn;
            nr[nc].y = -rn;
            l[nc].y *= beta;
          } else {
            nm[nc].x = -mn;
            nr[nc].x = -rn;
            l[nc].x *= beta;
          }
#pragma unroll
          for (int c = 0; c < kSteps; ++c) {
            o[c][nc][k] *= alpha;
            o[c][nc][k + 2] *= alpha;
          }
        }
    }
    uint32_t w[T::kParts][kTurns][kUsed][2];  // B fragments of the weights
#pragma unroll
    for (int y = 0; y < kTurns; ++y)
#pragma unroll
      for (int nc = 0; nc < kUsed; ++nc)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float2 d, e;
          logs(y, nc, h, d, e);
          const float2 p = make_float2(ex2(d.x), ex2(d.y)), x = make_float2(ex2(e.x), ex2(e.y));
          const uint32_t high = pack_f16(x.x, x.y);
          w[0][y][nc][h] = transpose8(high);
          if constexpr (T::kParts == 2) {
            const float2 of = unpack_f16(high);
            w[1][y][nc][h] = transpose8(pack_f16(x.x - of.x, x.y - of.y));
            l[nc] = __fadd2_rn(l[nc], p);
          } else {
            l[nc] = __fadd2_rn(l[nc], unpack_f16(pack_f16(p.x, p.y)));
          }
        }
    // O^T += Vc^T W^T.  A lane's four codes of a chunk: tokens 2t and 2t + 1, dims 2g and 2g + 1; dims 2g are rows g of
    // the product, dims 2g + 1 rows g + 8.
#pragma unroll
    for (int y = 0; y < kTurns; ++y) {
      // Rows that nobody sees must not reach the product (0 times no number).
      uint32_t keep_lo = kAll, keep_hi = kAll;  // of tokens 2t, 2t + 1 and of 2t + 8, 2t + 9
      if (masked) {
        const int left = tokens - token0 - y * kBlockTokens - 2 * t;
        keep_lo = left > 1 ? kAll : left > 0 ? 0xffffu : 0u;
        keep_hi = left > 9 ? kAll : left > 8 ? 0xffffu : 0u;
      }
#pragma unroll
      for (int c = 0; c < kSteps / 2; ++c) {
        uint32_t a[4][2];
        if constexpr (!kEarly) ldsm_x4_t(((tile_at + y * T::kStage) ^ (32u * c)) + T::kTile, vx[y][c]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t x = __byte_perm(masked ? vx[y][c][k] & (k & 1 ? keep_hi : keep_lo) : vx[y][c][k], 0, 0x3120);
          a[k][0] = fp8_halves(static_cast<uint16_t>(x));
          a[k][1] = fp8_halves(static_cast<uint16_t>(x >> 16));
        }
#pragma unroll
        for (int part = 0; part < T::kParts; ++part)
#pragma unroll
          for (int nc = 0; nc < kUsed; ++nc) {
            mma_f16(o[2 * c][nc], a[0][0], a[0][1], a[1][0], a[1][1], w[part][y][nc][0], w[part][y][nc][1]);
            mma_f16(o[2 * c + 1][nc], a[2][0], a[2][1], a[3][0], a[3][1], w[part][y][nc][0], w[part][y][nc][1]);
          }
      }
    }
    if constexpr (!kEarly) {
      __syncwarp();
#pragma unroll
      for (int turn = 0; turn < kTurns; ++turn) send();
    }
  }
  // The pair's units of this warp, `mine` of them from token0 on, `step` tokens apart.
  template <int kUsed, typename Send>
  __device__ __forceinline__ void units(int token0, int mine, int step, int& stage, Send& send) {
    if constexpr (T::kAhead) {
      float sum[kTurns][sums(kUsed)][kUsed][4];
      if (mine > 0) {
        copies_wait<T::kStages - kTurns>();
        __syncwarp();
        products<kUsed>(stage, sum);
      }
      for (int u = 0; u < mine; ++u, token0 += step) {
        const int place = stage;
        stage = T::next(stage);
        float next[kTurns][sums(kUsed)][kUsed][4];
        copies_wait<T::kStages - 2 * kTurns>();
        __syncwarp();
        products<kUsed>(u + 1 < mine ? stage : place, next);  // (without a branch, so that they run beside the softmax)
        weigh<kUsed>(place, token0, sum, send);
#pragma unroll
        for (int y = 0; y < kTurns; ++y)
#pragma unroll
          for (int x = 0; x < sums(kUsed); ++x)
#pragma unroll
            for (int nc = 0; nc < kUsed; ++nc)
#pragma unroll
              for (int k = 0; k < 4; ++k) sum[y][x][nc][k] = next[y][x][nc][k];
      }
    } else {
      for (int u = 0; u < mine; ++u, token0 += step) {
        const int place = stage;
        stage = T::next(stage);
        copies_wait<T::kStages - kTurns>();
        __syncwarp();
        float sum[kTurns][sums(kUsed)][kUsed][4];
        products<kUsed>(place, sum);
        weigh<kUsed>(place, token0, sum, send);
      }
    }
  }
};

template <int D, int NC, bool kCluster>
__global__ void __launch_bounds__(kThreads, Few<D, NC, kCluster>::kCtas)
    few_rows_fp8_kernel(const Fp8AttentionParams p) {
  using T = Few<D, NC, kCluster>;
  constexpr int kTurns = T::kTurns;
  constexpr int kSteps = D / 16;  // 16-byte chunks of a row of codes: 16 dims, the depth of a product
  extern __shared__ __align__(128) unsigned char smem[];
  const uint32_t base = saddr(smem);
  int* s_costs = reinterpret_cast<int*>(smem + T::kOffSeq);
  int* s_tokens = s_costs + p.num_seqs + 1;
  __shared__ int s_sum[kThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hc = kCluster ? 1 : p.unit_heads, nb = T::kUnitTiles / hc;  // heads and blocks of a unit
  const int head_groups = p.num_kv_heads / hc;
  pdl_trigger();
  pdl_wait();

  const int head_of = warp & (hc - 1), place_of = warp / hc;  // (hc is a power of two); of a unit's blocks place_of kTurns ..

  // This CTA's units are n1 of the stream from `at` on; of a cluster's pair, its rank and every stride-th from there on.
  const int piece = blockIdx.x;
  int n1 = 0, stride = 1;
  const int nb_bits = 31 - __clz(nb);
  auto units_at = [&](int b) -> int { return ((s_tokens[b] + kBlockTokens - 1) / kBlockTokens + nb - 1) >> nb_bits; };
  Rows pair{};
  Walk at{};  // the first unit
  if constexpr (kCluster) {
    stride = static_cast<int>(cluster_size());
    const int number = static_cast<int>(blockIdx.x) / stride;
    at.b = number / head_groups;
    at.heads = number - at.b * head_groups;
    at.unit = static_cast<int>(cluster_rank());
  } else {
    // What the units before each sequence cost.
    if (tid == 0) s_costs[0] = 0;
    int running = 0;
    for (int first = 0; first < p.num_seqs; first += kThreads) {
      const int b = first + tid;
      int costs = 0;
      if (b < p.num_seqs) {
        const Rows r = rows_of(p, b);
        if (r.wrong && blockIdx.x == 0) atomicOr(p.err, r.wrong);
        s_tokens[b] = r.count > 0 ? r.tokens : 0;
        const int blocks = (r.count * (p.num_q_heads / p.num_kv_heads) + 7) / 8;
        costs = units_at(b) * (NC > 1 && p.unit_costs ? T::cost(blocks) : 1);
      }
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(kAll, costs, off);
        if (lane >= off) costs += y;
      }
      if (lane == 31) s_sum[warp] = costs;
      __syncthreads();
      int before = running;
      for (int w = 0; w < warp; ++w) before += s_sum[w];
      if (b < p.num_seqs) s_costs[b + 1] = before + costs;
      for (int w = 0; w < kThreads / 32; ++w) running += s_sum[w];
      __syncthreads();
    }
    const int total = running * head_groups;
    const int pieces = total == 0 ? 0 : min(max(total / T::cost(NC), 1), p.num_pieces);  // (a unit or more each)
    if (piece >= pieces) return;
    // The sequence in which the cost x of the stream is reached, the last that begins there or before, and its unit there.
    auto find = [&](int x, int& b) -> int {
      int lo = 0, hi = p.num_seqs - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_costs[mid] <= x / head_groups) lo = mid;
        else hi = mid - 1;
      }
      b = lo;
      const int rest = x - s_costs[lo] * head_groups;
      return NC == 1 || rest == 0 ? rest : rest / ((s_costs[lo + 1] - s_costs[lo]) / units_at(lo));
    };
    const int from = static_cast<int>(static_cast<int64_t>(piece) * total / pieces);
    const int to = static_cast<int>(static_cast<int64_t>(piece + 1) * total / pieces);
    const int begin = find(from, at.b);
    n1 = to - from;
    if (NC > 1) {
      int last;
      n1 = find(to, last) - begin;
      for (int b = at.b; b < last; ++b) n1 += units_at(b) * head_groups;
    }
    at.units = units_at(at.b);
    at.heads = begin / at.units;
    at.unit = begin - at.heads * at.units;
  }
  // On to the pair that unit x.unit, past its own pair's end, lies in (there is one).
  auto carry = [&](Walk& x) {
    while (!kCluster && x.unit >= x.units) {
      x.unit -= x.units;
      if (++x.heads < head_groups) continue;
      x.heads = 0;
      do {
        ++x.b;
        x.units = units_at(x.b);
      } while (x.units == 0);
    }
  };

  // ---------------- copies: the piece's tiles of this warp, kStages of them ahead ----------------
  // Block ids come in windows of 32 tiles of a pair, one a lane; the window behind the current one is on its way.
  constexpr int kWindow = 32 / kTurns;  // units
  struct Window {
    Walk x;  // its first unit
    int n;   // that one's number of the CTA's
  };
  auto block_at = [&](const Window& w) -> int {  // of this lane's tile
    return (w.x.unit + lane / kTurns * stride) * nb + place_of * kTurns + lane % kTurns;
  };
  auto id_at = [&](const Window& w, int block) -> int {
    return __ldg(p.block_tables + static_cast<int64_t>(w.x.b) * p.max_blocks_per_seq + block);
  };
  auto checked = [&](int id) -> int {
    if (id >= 0 && id < p.num_blocks) return id;
    atomicOr(p.err, kErrBlockId);
    return 0;
  };
  Window window{at, 0}, next{};
  int ids = -1, next_ids = -1;  // -1: no tile
  int asked = 0;
  if constexpr (kCluster) {  // the first window's ids are asked for before the length is known
    const int block = block_at(window);
    if (block < p.max_blocks_per_seq) asked = id_at(window, block);
    pair = rows_of(p, at.b);
    if (pair.wrong && at.unit == 0 && at.heads == 0 && tid == 0) atomicOr(p.err, pair.wrong);
    if (pair.count == 0) return;  // (the whole cluster)
    at.units = ((pair.tokens + kBlockTokens - 1) / kBlockTokens + nb - 1) / nb;
    window.x.units = at.units;
    n1 = at.unit < at.units ? (at.units - at.unit + stride - 1) / stride : 0;
    if (n1 > 0 && block * kBlockTokens < pair.tokens) ids = checked(asked);
  }
  auto ids_of = [&](const Window& w) -> int {
    const int block = block_at(w);
    const bool in_pair = kCluster || w.x.unit + lane / kTurns < w.x.units;
    if (w.n >= n1 || !in_pair || block * kBlockTokens >= (kCluster ? pair.tokens : s_tokens[w.x.b])) return -1;
    return checked(id_at(w, block));
  };
  auto units_of = [&](const Window& w) -> int {  // up to the pair's end and the piece's
    return max(0, min(kWindow, min(kCluster ? kWindow : w.x.units - w.x.unit, n1 - w.n)));
  };
  auto behind = [&](Window w) {
    const int units = kCluster ? kWindow : min(kWindow, w.x.units - w.x.unit);
    w.n += units;
    if (w.n < n1) {
      w.x.unit += units * stride;
      carry(w.x);
      if (!kCluster && warp == 0 && w.x.unit == 0) {  // a pair's queries are on their way to L2 early
        const Rows r = rows_of(p, w.x.b);
        const int heads = hc * (p.num_q_heads / p.num_kv_heads);
        for (int i = lane; i < r.count; i += 32)
          l2_prefetch(static_cast<const __nv_bfloat16*>(p.q) +
                          (static_cast<int64_t>(r.first + i) * p.num_q_heads + w.x.heads * heads) * D,
                      heads * D * 2);
      }
    }
    return w;
  };
  auto tiles_of = [&](const Window& w) -> int { return units_of(w) * kTurns; };
  if (!kCluster) ids = ids_of(window);
  int sent = 0, tiles = tiles_of(window);  // of the window: tiles sent for, and all
  if (tiles > 0) {
    next = behind(window);
    next_ids = ids_of(next);
  }
  int to = 0;  // ring place of the next tile
  // A lane's 16-byte pieces of a tile: line i 4 + lane / 8 of 128 bytes, chunk lane % 8 of it, swizzled by the line.
  const uint32_t ring = base + warp * T::kStages * T::kStage, scales = base + T::kOffScales + warp * T::kStages * T::kScales;
  const uint32_t copy_even = (lane >> 3) * 128 + (((lane & 7) ^ (lane >> 3)) << 4), copy_odd = copy_even ^ 64;
  auto send = [&] {
    if (tiles > 0) {
      const int id = __shfl_sync(kAll, ids, sent);
      if (id >= 0) {
        const int64_t tile = static_cast<int64_t>(id) * p.num_kv_heads + window.x.heads * hc + head_of;
        const uint8_t *k = p.k_cache + tile * T::kTile + lane * 16, *v = p.v_cache + tile * T::kTile + lane * 16;
        const uint32_t dst = ring + to * T::kStage;
#pragma unroll
        for (int i = 0; i < T::kTile / 512; ++i) {
          copy_16(dst + i * 512 + (i & 1 ? copy_odd : copy_even), k + i * 512);
          copy_16(dst + T::kTile + i * 512 + (i & 1 ? copy_odd : copy_even), v + i * 512);
        }
        if (lane < 2) copy_16(scales + to * T::kScales + lane * 16, p.kv_scales + tile * 2 * kBlockTokens + lane * 16);
      }
      if (++sent == tiles) {
        window = next;
        ids = next_ids;
        sent = 0;
        tiles = tiles_of(window);
        if (tiles > 0) {
          next = behind(window);
          next_ids = ids_of(next);
        }
      }
    }
    copies_commit();  // (a group a call, whether or not there was a tile)
    if (++to == T::kStages) to = 0;
  };
#pragma unroll 1
  for (int k = 0; k < T::kStages; ++k) send();

  // ---------------- products (a tile of every unit a warp, or kTurns) ----------------
  const int g = lane >> 2, t = lane & 3;      // fragments: row g and columns 2t, 2t + 1 of an accumulator
  const int group = p.num_q_heads / p.num_kv_heads, group_bits = 31 - __clz(group);
  // ldmatrix: lane i gives the address of row i % 8 of matrix i / 8; matrices 0, 1: tokens 0..7 and 8..15 of a chunk,
  // 2, 3: of the next chunk.  A tile is lines of 128 bytes, swizzled: chunk c of line y lies at c ^ (y % 8) (two tokens of 64
  // dims share a line).  Two chunks on are 32 bytes on, through the swizzle an exclusive or.
  const int ld_row = (lane & 7) + ((lane >> 3) & 1) * 8;
  const int ld_line = ld_row * D / 128, ld_chunk = (D == 128 ? 0 : (ld_row & 1) * 4) + (lane >> 4);
  const uint32_t ld_at = ring + ld_line * 128 + ((ld_chunk ^ (ld_line & 7)) << 4);
  int stage = 0;

  // The piece's pairs of sequence and heads; a cluster's one, of which a CTA may have no unit.
  for (int n = 0; kCluster || n < n1;) {
    const Rows rows = kCluster ? pair : rows_of(p, at.b);
    const int kvh = at.heads * hc + head_of;
    const int count = kCluster ? n1 : min(at.units - at.unit, n1 - n);  // units of the pair here
    Pair<D, NC, kCluster> x;
    x.ld_at = ld_at;
    x.scales = smem + T::kOffScales + warp * T::kStages * T::kScales;
    x.q_at = base + T::kOffQ + warp * T::kQ + lane * 16;
    x.g = g;
    x.t = t;
    x.group_bits = group_bits;
    x.tokens = rows.tokens;
    x.first_limit = rows.tokens - rows.count + 1;
    auto &q = x.q;
    auto &o = x.o;
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
      const int col = nc * 8 + g, i = col >> group_bits;
      float top = 0.f;
#pragma unroll
      for (int c = 0; c < kSteps; ++c) {
        uint2 y = make_uint2(0u, 0u);
        if (i < rows.count)
          y = __ldg(reinterpret_cast<const uint2*>(
              static_cast<const __nv_bfloat16*>(p.q) +
              (static_cast<int64_t>(rows.first + i) * p.num_q_heads + kvh * group + (col & (group - 1))) * D + 16 * c + 4 * t));
        q[nc][c][0] = y.x;
        q[nc][c][1] = y.y;
      }
#pragma unroll
      for (int c = 0; c < kSteps; ++c)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          top = fmaxf(fmaxf(top, fabsf(__uint_as_float(q[nc][c][k] << 16))), fabsf(__uint_as_float(q[nc][c][k] & 0xffff0000u)));
      top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
      top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
      // To a largest value in [2^14, 2^15): by 2^up.
      const int up = min(14 + 127 - static_cast<int>(__float_as_uint(top) >> 23), 100);
      const float by = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
#pragma unroll
      for (int c = 0; c < kSteps; ++c)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          q[nc][c][k] = pack_f16(__uint_as_float(q[nc][c][k] << 16) * by, __uint_as_float(q[nc][c][k] & 0xffff0000u) * by);
      const float back = __uint_as_float(static_cast<uint32_t>(127 - up) << 23) * p.qscale;
      x.q_scale[nc] = make_float2(__shfl_sync(kAll, back, 2 * t * 4), __shfl_sync(kAll, back, (2 * t + 1) * 4));
      x.nm[nc] = x.nr[nc] = make_float2(-kNone, -kNone);
      x.l[nc] = make_float2(0.f, 0.f);
    }
#pragma unroll
    for (int c = 0; c < kSteps; ++c)
#pragma unroll
      for (int nc = 0; nc < NC; ++nc)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[c][nc][k] = 0.f;

    if constexpr (T::kAhead) {
      // The fragments of q make room for a second tile's scores.
      uint4* own = reinterpret_cast<uint4*>(smem + T::kOffQ + warp * T::kQ) + lane;
#pragma unroll
      for (int nc = 0; nc < NC; ++nc)
#pragma unroll
        for (int c = 0; c < kSteps / 2; ++c)
          own[(nc * kSteps / 2 + c) * 32] = make_uint4(q[nc][2 * c][0], q[nc][2 * c][1], q[nc][2 * c + 1][0], q[nc][2 * c + 1][1]);
    }

    // All of a warp's tiles of a unit at a time.  What lies in the second one's place past the last token is masked like the rows
    // past it.  Of the column blocks those that the sequence's rows fill (64 sequences with one to five tokens: 96.1 us with all
    // of them, 89.6 so).
    const int token0 = (at.unit * nb + place_of * kTurns) * kBlockTokens, step = stride * nb * kBlockTokens;
    const int mine = token0 < rows.tokens ? min(count, (rows.tokens - token0 - 1) / step + 1) : 0;  // units with such blocks
    const int cols = rows.count << group_bits;
    if (NC == 1 || cols <= 8) x.template units<1>(token0, mine, step, stage, send);
    else if (NC == 2 || cols <= 16) x.template units<NC < 2 ? NC : 2>(token0, mine, step, stage, send);
    else x.template units<NC>(token0, mine, step, stage, send);
    for (int u = mine; u < count; ++u) {  // at most one, the pair's last
      stage = T::next(stage);
#pragma unroll
      for (int turn = 0; turn < kTurns; ++turn) send();
    }

    // The pair's end here: O against m, l summed over the lanes that share a column.
    float m[NC][2], sum[NC][2];
#pragma unroll
    for (int nc = 0; nc < NC; ++nc)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        m[nc][k] = (k ? -x.nm[nc].y : -x.nm[nc].x) + kTopLog;  // (up to where the largest weight may be 2^8, not 2^15)
        sum[nc][k] = (k ? x.l[nc].y : x.l[nc].x) * ex2(-kTopLog);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) sum[nc][k] += __shfl_xor_sync(kAll, sum[nc][k], off);
        const float f = m[nc][k] == kNone ? 0.f : ex2((k ? -x.nr[nc].y : -x.nr[nc].x) - kTopLog);
#pragma unroll
        for (int c = 0; c < kSteps; ++c) {
          o[c][nc][k] *= f;
          o[c][nc][k + 2] *= f;
        }
      }
    if constexpr (!kCluster) {
      // The warps of a head join their states, half of them handing theirs to the other half at a time.
      float4* exchange = reinterpret_cast<float4*>(smem + T::kOffExchange);
      float2* s_ml = reinterpret_cast<float2*>(smem + T::kOffMl);
      for (int half = kWarps / hc / 2; half > 0; half >>= 1) {
        const bool gives = place_of >= half && place_of < 2 * half, takes = place_of < half;
        const int place = (place_of & (half - 1)) * hc + head_of;
        float mine[NC][2], other[NC][2];
        if (gives && g == 0)
#pragma unroll
          for (int nc = 0; nc < NC; ++nc)
#pragma unroll
            for (int k = 0; k < 2; ++k) s_ml[place * T::kCols + nc * 8 + 2 * t + k] = make_float2(m[nc][k], sum[nc][k]);
#pragma unroll
        for (int part = 0; part < kSteps * NC / 2; ++part) {
          if (gives)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float(&v)[4] = o[(2 * part + x) / NC][(2 * part + x) % NC];
              exchange[(place * 2 + x) * 32 + lane] = make_float4(v[0], v[1], v[2], v[3]);
            }
          asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
          if (takes) {
            if (part == 0)
#pragma unroll
              for (int nc = 0; nc < NC; ++nc)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const float2 y = s_ml[place * T::kCols + nc * 8 + 2 * t + k];
                  const float top = fmaxf(m[nc][k], y.x);
                  mine[nc][k] = ex2(m[nc][k] - top);
                  other[nc][k] = ex2(y.x - top);
                  sum[nc][k] = sum[nc][k] * mine[nc][k] + y.y * other[nc][k];
                  m[nc][k] = top;
                }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int nc = (2 * part + x) % NC;
              float(&v)[4] = o[(2 * part + x) / NC][nc];
              const float4 y = exchange[(place * 2 + x) * 32 + lane];
              v[0] = v[0] * mine[nc][0] + y.x * other[nc][0];
              v[1] = v[1] * mine[nc][1] + y.y * other[nc][1];
              v[2] = v[2] * mine[nc][0] + y.z * other[nc][0];
              v[3] = v[3] * mine[nc][1] + y.w * other[nc][1];
            }
          }
          asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
        }
      }
      const bool started = at.unit == 0, ended = at.unit + count == at.units;
      const int slot = n == 0 ? 0 : 1;  // of the piece's states
      if (warp == 0 && lane == 0) {
        int* record = p.ws_records + 2 * (static_cast<int64_t>(at.b) * head_groups + at.heads);
        if (started) record[0] = piece * 2 + slot;
        if (ended) record[1] = piece;
      }
      if (place_of == 0) {
#pragma unroll
        for (int nc = 0; nc < NC; ++nc)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int col = nc * 8 + 2 * t + k, i = col >> group_bits;
            if (i >= rows.count) continue;
            if (started && ended) {
              const float inv = 1.f / sum[nc][k];
              __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) +
                                   (static_cast<int64_t>(rows.first + i) * p.num_q_heads + kvh * group + (col & (group - 1))) * D;
#pragma unroll
              for (int c = 0; c < kSteps; ++c)
                *reinterpret_cast<uint32_t*>(dst + 16 * c + 2 * g) = pack_bf16(o[c][nc][k] * inv, o[c][nc][k + 2] * inv);
            } else {
              const int64_t state = (static_cast<int64_t>(piece * 2 + slot) * hc + head_of) * p.state_rows + col;
              float* dst = p.ws_states + state * D;
#pragma unroll
              for (int c = 0; c < kSteps; ++c)
                *reinterpret_cast<float2*>(dst + 16 * c + 2 * g) = make_float2(o[c][nc][k], o[c][nc][k + 2]);
              if (g == 0) p.ws_ml[state] = make_float2(m[nc][k], sum[nc][k]);
            }
          }
      }
      n += count;
      at.unit += count;
      if (n < n1) carry(at);
    } else {
      // The warps' states, each in its own ring (done with), joined to the CTA's.
      static_assert(T::kCols * D * 4 <= T::kStages * T::kStage, "a warp's state fits its ring");
      copies_wait<0>();
      float* s_o = reinterpret_cast<float*>(smem);
      constexpr int kRing = T::kStages * T::kStage / 4;  // floats
      float2* s_ml = reinterpret_cast<float2*>(smem + T::kOffMl);
      float2* s_joined = s_ml + kWarps * T::kCols;
#pragma unroll
      for (int nc = 0; nc < NC; ++nc)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int col = nc * 8 + 2 * t + k;
          if (col >> group_bits >= rows.count) continue;
#pragma unroll
          for (int c = 0; c < kSteps; ++c)
            *reinterpret_cast<float2*>(s_o + warp * kRing + col * D + 16 * c + 2 * g) = make_float2(o[c][nc][k], o[c][nc][k + 2]);
          if (g == 0) s_ml[warp * T::kCols + col] = make_float2(m[nc][k], sum[nc][k]);
        }
      __syncthreads();
      constexpr int kQuads = D / 4;
      for (int x = tid; x < cols * kQuads; x += kThreads) {
        const int dim = x % kQuads * 4, col = x / kQuads;
        float top = kNone, sum = 0.f;
#pragma unroll
        for (int y = 0; y < kWarps; ++y) top = fmaxf(top, s_ml[y * T::kCols + col].x);
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int y = 0; y < kWarps; ++y) {
          const float2 ml = s_ml[y * T::kCols + col];
          const float by = ex2(ml.x - top);
          const float4 v = *reinterpret_cast<const float4*>(s_o + y * kRing + col * D + dim);
          sum += ml.y * by;
          a.x += v.x * by;
          a.y += v.y * by;
          a.z += v.z * by;
          a.w += v.w * by;
        }
        *reinterpret_cast<float4*>(s_o + col * D + dim) = a;  // in place of the first warp's, which only this thread reads
        if (dim == 0) s_joined[col] = make_float2(top, sum);
      }
      // Then every CTA of the cluster forms its share of the outputs from the CTAs' states.
      cluster_sync();
      constexpr int kAtOnce = 8;
      const int rank = static_cast<int>(cluster_rank());
      for (int x = rank + stride * tid; x < cols * kQuads; x += stride * kThreads) {
        const int col = x / kQuads, dim = x % kQuads * 4;
        float top = kNone, sum = 0.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int y0 = 0; y0 < stride; y0 += kAtOnce) {
          float2 ml[kAtOnce];
          float4 v[kAtOnce];
          float most = top;
#pragma unroll
          for (int y = 0; y < kAtOnce; ++y) {
            ml[y] = make_float2(kNone, 0.f);
            v[y] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (y0 + y >= stride) continue;
            ml[y] = remote_f2(remote(saddr(s_joined + col), y0 + y));
            v[y] = remote_f4(remote(saddr(s_o + col * D + dim), y0 + y));
          }
#pragma unroll
          for (int y = 0; y < kAtOnce; ++y) most = fmaxf(most, ml[y].x);
          const float was = ex2(top - most);
          top = most;
          sum *= was;
          a = make_float4(a.x * was, a.y * was, a.z * was, a.w * was);
#pragma unroll
          for (int y = 0; y < kAtOnce; ++y) {
            const float by = ex2(ml[y].x - top);
            sum += ml[y].y * by;
            a.x += v[y].x * by;
            a.y += v[y].y * by;
            a.z += v[y].z * by;
            a.w += v[y].w * by;
          }
        }
        const float inv = rows.tokens > 0 ? 1.f / sum : 0.f;  // no token: zeros
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) +
                             (static_cast<int64_t>(rows.first + (col >> group_bits)) * p.num_q_heads + kvh * group + (col & (group - 1))) * D + dim;
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
      }
      cluster_sync();  // no CTA leaves while another reads its state
      break;
    }
  }
}

// Joins the states of every pair that a piece's border cuts: out = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s; zeros for a
// sequence without tokens.  A CTA per (sequence, kv head), a warp per row and slice of its states; a warp fetches kAhead
// states before it joins any.
template <int D, int kSlices>
__global__ void __launch_bounds__(kSlices == 1 ? 128 : kSlices * 32) join_fp8_kernel(const Fp8AttentionParams p) {
  constexpr int kPer = D / 32, kAhead = kSlices == 1 ? 8 : 10;
  constexpr int kRows = kSlices == 1 ? 4 : 1;  // rows of a CTA at a time
  __shared__ float2 s_ml[kSlices];
  __shared__ float s_o[kSlices][D];
  const int b = blockIdx.x / p.num_kv_heads, kvh = blockIdx.x - b * p.num_kv_heads;
  const int warp = threadIdx.x >> 5, slice = kSlices == 1 ? 0 : warp, lane = threadIdx.x & 31;
  const int hc = p.unit_heads, group = p.num_q_heads / p.num_kv_heads;
  pdl_trigger();
  pdl_wait();
  const Rows rows = rows_of(p, b);
  const int2 record = *reinterpret_cast<const int2*>(
      p.ws_records + 2 * (static_cast<int64_t>(b) * (p.num_kv_heads / hc) + kvh / hc));
  if (rows.count == 0) return;
  const int first = record.x >> 1;
  int states = rows.tokens > 0 ? record.y - first + 1 : 0;
  if (rows.tokens > 0 && (first < 0 || states < 1 || record.y >= p.num_pieces)) return;  // (the lengths were changed meanwhile)
  if (states == 1) return;  // whole in one piece, which wrote it
  for (int col = blockIdx.y * kRows + (kRows > 1 ? warp : 0); col < rows.count * group; col += gridDim.y * kRows) {
    float top = kNone, l = 0.f, acc[kPer];
#pragma unroll
    for (int x = 0; x < kPer; ++x) acc[x] = 0.f;
    for (int u0 = slice; u0 < states; u0 += kSlices * kAhead) {
      float2 ml[kAhead];
      float a[kAhead][kPer];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int u = u0 + k * kSlices;
        ml[k] = make_float2(kNone, 0.f);
#pragma unroll
        for (int x = 0; x < kPer; ++x) a[k][x] = 0.f;
        if (u >= states) continue;
        const int64_t state =
            (static_cast<int64_t>((first + u) * 2 + (u == 0 ? record.x & 1 : 0)) * hc + kvh % hc) * p.state_rows + col;
        ml[k] = p.ws_ml[state];
        const float* src = p.ws_states + state * D + lane * kPer;
        if constexpr (kPer == 4) {
          const float4 v = *reinterpret_cast<const float4*>(src);
          a[k][0] = v.x; a[k][1] = v.y; a[k][2] = v.z; a[k][3] = v.w;
        } else {
          const float2 v = *reinterpret_cast<const float2*>(src);
          a[k][0] = v.x; a[k][1] = v.y;
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const float mn = fmaxf(top, ml[k].x);
        const float alpha = ex2(top - mn), beta = ex2(ml[k].x - mn);
        l = l * alpha + ml[k].y * beta;
#pragma unroll
        for (int x = 0; x < kPer; ++x) acc[x] = acc[x] * alpha + a[k][x] * beta;
        top = mn;
      }
    }
    if constexpr (kSlices > 1) {
      __syncthreads();  // the column before has been read
      if (lane == 0) s_ml[slice] = make_float2(top, l);
#pragma unroll
      for (int x = 0; x < kPer; ++x) s_o[slice][lane * kPer + x] = acc[x];
      __syncthreads();
      if (slice > 0) continue;
#pragma unroll
      for (int k = 1; k < kSlices; ++k) {
        const float2 y = s_ml[k];
        const float mn = fmaxf(top, y.x);
        const float alpha = ex2(top - mn), beta = ex2(y.x - mn);
        l = l * alpha + y.y * beta;
#pragma unroll
        for (int x = 0; x < kPer; ++x) acc[x] = acc[x] * alpha + s_o[k][lane * kPer + x] * beta;
        top = mn;
      }
    }
    const float inv = states > 0 ? 1.f / l : 0.f;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) +
                         (static_cast<int64_t>(rows.first + col / group) * p.num_q_heads + kvh * group + col % group) * D + lane * kPer;
#pragma unroll
    for (int x = 0; x < kPer; x += 2)
      *reinterpret_cast<uint32_t*>(dst + x) = pack_bf16(acc[x] * inv, acc[x + 1] * inv);
  }
}

}  // namespace
}  // namespace pkv
