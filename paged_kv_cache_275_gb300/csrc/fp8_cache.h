// Internal interface of the kernels over an 8-bit cache, used by capi.cu.
//
// The format: a row of one kv head (head_dim values of one token's K or V) is held as e4m3 codes and one exponent byte e
// and stands for code * 2^(e - 127).  Codes: [num_blocks][num_kv_heads][16][head_dim]; exponents:
// [num_blocks][num_kv_heads][2][16], those of the block's K rows and then those of its V rows.
#pragma once

#include "pkv_internal.h"

namespace pkv {

constexpr int kFp8MaxAxes = 4;

// Quantising append, with the rotation of q and k before it if cos_sin is given (fp8_cache.cu).
struct Fp8AppendParams {
  const void* q;  // rows of [heads][head_dim] bf16, `stride` 16-byte chunks apart
  const void* k;
  const void* v;
  void* q_out;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  const int64_t* positions;  // [num_axes][num_tokens], axes axis_stride apart
  int64_t axis_stride;
  const float* cos_sin;  // fp32 [max_position][head_dim], or null: no rotation, and no q
  int64_t max_position;
  const int64_t* slot_mapping;
  uint8_t* k_cache;
  uint8_t* v_cache;
  uint8_t* kv_scales;
  unsigned* err;
  int64_t num_tokens;
  int64_t num_slots;  // 16 * num_blocks
  int num_q_heads;    // 0 without rotation
  int num_kv_heads;
  int num_axes;
  int parts;  // warps that share a token's rows
  uint8_t freq_axis[64];  // position axis of each of the head_dim / 2 frequencies
};

// Rows read back as bf16, by slot.
struct Fp8GatherParams {
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const uint8_t* kv_scales;
  const int64_t* slot_mapping;
  void* k;  // rows of [num_kv_heads][head_dim] bf16, `stride` 16-byte chunks apart
  void* v;
  int64_t k_stride, v_stride;
  unsigned* err;
  int64_t num_tokens;
  int64_t num_slots;
  int num_kv_heads;
};

struct Fp8CopyParams {
  void* k_cache;
  void* v_cache;
  void* kv_scales;
  const int64_t* src_dst;  // [num_pairs][2]
  unsigned* err;
  int64_t num_blocks;
  int64_t cache_chunks;  // 16-byte chunks of a block's codes of K (or V), all kv heads
  int64_t scale_chunks;  // and of its exponents
};

struct Fp8AttentionParams {
  const void* q;  // bf16 [query_rows][num_q_heads][head_dim]
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const uint8_t* kv_scales;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start;  // [num_seqs + 1], or null: row b is sequence b's one query token
  void* out;                   // bf16, as q
  unsigned* err;
  int64_t num_blocks;
  int64_t query_rows;
  int num_seqs;
  int num_q_heads;
  int num_kv_heads;
  int max_blocks_per_seq;
  int max_query_len;
  float scale;
  // Few rows a sequence (fp8_decode.cuh), up to kFp8LaunchSeqs sequences a launch.
  float qscale;         // scale * log2(e): scores are kept in base-2 units
  int cluster_ctas;     // CTAs a (sequence, kv head), joined through their shared memory; 0: the stream form, all below
  int unit_heads;       // kv heads of a unit: 8, 4, 2 or 1
  int num_pieces;       // most pieces that the stream of units is cut into
  int unit_costs;       // whether units cost by their rows, not all the same
  int state_rows;       // rows of a state: most query tokens * q heads per kv head
  int* ws_records;      // [num_seqs][head groups][2]: the piece of the first unit (times 2, plus its state slot), of the last
  float2* ws_ml;        // [piece][2 slots][unit_heads][state_rows]: (m in base 2, l)
  float* ws_states;     // the same, [head_dim] each: O against m
};

constexpr int kFp8LaunchSeqs = 1024;
// Above this the chunk kernel is faster, although it pads the rows to 128.  64 sequences of 512..8192 tokens, 8 kv heads, here
// and there: 128 dims, 24 rows 104 and 171 us, 32 rows 253 and 163; 64 dims, 16 rows 61 and 138, 24 rows 72 and 138.  (With few
// sequences the chunk kernel, whose splits fill the GPU, is the faster from some 16 rows on: eight of 2048 tokens, 128 dims, 24
// rows 40 and 27, 16 rows 30 and 26; one of 8192, 24 rows 20 and 22.)
constexpr int kFp8MostRows = 24;
// Tables up to here keep every position, past the last unit's end too, below 2^31.
constexpr int kFp8MostBlocks = 1 << 26;
// Blocks of eight columns that hold so many rows; 0: too many.
inline int fp8_columns(int rows) { return rows <= kFp8MostRows ? (rows + 7) / 8 : 0; }
// Its workspace and how its work is cut.
struct Fp8FewPlan {
  int unit_heads, num_pieces;
  bool unit_costs;  // (their sum fits 31 bits)
  size_t ml, states, bytes;  // byte offsets of the parts behind the records, and the sum
  Fp8FewPlan(int num_seqs, int num_kv_heads, int head_dim, int max_blocks_per_seq, int state_rows, int sms) {
    const int seqs = num_seqs < kFp8LaunchSeqs ? num_seqs : kFp8LaunchSeqs;
    unit_heads = 8;
    while (num_kv_heads % unit_heads) unit_heads /= 2;
    const int blocks = (head_dim == 128 ? 8 : 16) / unit_heads;
    const int64_t units = static_cast<int64_t>(seqs) * (num_kv_heads / unit_heads) * ((max_blocks_per_seq + blocks - 1) / blocks);
    unit_costs = units < (int64_t{1} << 27);
    const int64_t ctas = static_cast<int64_t>(sms) * (fp8_columns(state_rows) == 1 ? 2 : 1);
    num_pieces = static_cast<int>(units < 1 ? 1 : units < ctas ? units : ctas);
    const size_t rows = static_cast<size_t>(num_pieces) * 2 * unit_heads * state_rows;
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    ml = up(static_cast<size_t>(seqs) * (num_kv_heads / unit_heads) * 8);
    states = ml + up(rows * 8);
    bytes = states + rows * head_dim * 4;
  }
};

// What a chunk call unpacks to bf16 (fp8_prefill.cu).
struct Fp8Unpacked {
  void* k;  // bf16 [num_seqs][max_blocks_per_seq][num_kv_heads][16][head_dim]
  void* v;
  int32_t* block_tables;  // [num_seqs][max_blocks_per_seq]: 0, 1, 2, ...
  int32_t* context_lens;  // [num_seqs]; -1: skipped
};

cudaError_t launch_append_fp8(const Fp8AppendParams& p, int head_dim, int num_sms, cudaStream_t stream);
cudaError_t launch_gather_fp8(const Fp8GatherParams& p, int head_dim, int num_sms, cudaStream_t stream);
cudaError_t launch_copy_blocks_fp8(const Fp8CopyParams& p, int num_pairs, cudaStream_t stream);
// CTAs a pair of a call of few pairs, which needs no workspace; 0: the call takes the stream form.  *fewer: whether the calls of
// every smaller batch and narrower table need none either.
cudaError_t fp8_cluster_ctas(int head_dim, int rows, int num_seqs, int num_kv_heads, int max_blocks_per_seq, int* ctas,
                             bool* fewer);
cudaError_t launch_few_rows_fp8(const Fp8AttentionParams& p, int head_dim, cudaStream_t stream);
// Chunks on the 5th-generation tensor cores (fp8_prefill.cu); ws: prefill_workspace_bytes of num_splits > 1.
cudaError_t launch_prefill_unpacked_fp8(const Fp8AttentionParams& p, int head_dim, int num_splits, const Fp8Unpacked& to, float* ws,
                                        int num_sms, cudaStream_t stream);
cudaError_t launch_prefill_fp8(const Fp8AttentionParams& p, int head_dim, int num_splits, float* ws, cudaStream_t stream);

}  // namespace pkv
