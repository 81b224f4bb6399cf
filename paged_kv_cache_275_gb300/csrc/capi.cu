// C ABI of the paged KV-cache hot path (declared in include/pagedkv.h).
//
// Host-side only: argument validation (every host-checkable error returns
// before anything is enqueued), workspace layout, the default partition
// count, kernel dispatch on the caller's stream, the per-device sticky error
// word, and the per-thread error message.  No call allocates device memory.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "pagedkv.h"
#include "copy_blocks.h"
#include "decode_views.h"
#include "paged_prefill.h"
#include "pkv_internal.h"
#include "rope_append.h"

// Sticky device error word; one instance per device (module-scope __device__).
static __device__ unsigned int g_pkv_device_error;

namespace {

thread_local char t_message[512] = "";
std::atomic<uint64_t> g_launches{0};

constexpr int kMaxDevices = 64;
std::mutex g_device_mu;
unsigned* g_error_word[kMaxDevices] = {};
int g_sm_count[kMaxDevices] = {};

pkv_status fail(pkv_status status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(t_message, sizeof t_message, fmt, ap);
  va_end(ap);
  return status;
}

pkv_status cuda_fail(cudaError_t e, const char* what) {
  return fail(PKV_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}

pkv_status ok() {
  t_message[0] = '\0';
  return PKV_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Error word address and SM count of the current device, looked up once per device.
pkv_status device_state(unsigned** err, int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(PKV_ERR_UNSUPPORTED, "device ordinal %d out of range", dev);
  std::lock_guard<std::mutex> lock(g_device_mu);
  if (!g_error_word[dev]) {
    void* addr = nullptr;
    if ((e = cudaGetSymbolAddress(&addr, g_pkv_device_error)) != cudaSuccess)
      return cuda_fail(e, "cudaGetSymbolAddress(device error word)");
    int count = 0;
    if ((e = cudaDeviceGetAttribute(&count, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
      return cuda_fail(e, "cudaDeviceGetAttribute(multiProcessorCount)");
    g_sm_count[dev] = count;
    g_error_word[dev] = static_cast<unsigned*>(addr);
  }
  if (err) *err = g_error_word[dev];
  if (sms) *sms = g_sm_count[dev];
  return PKV_OK;
}

// Sequences of a decode call handled by one partition + merge launch pair (larger batches are
// cut on the host into consecutive slices of at most this many).
int32_t launch_seqs(int32_t num_seqs) { return num_seqs < PKV_MAX_SEQS ? num_seqs : PKV_MAX_SEQS; }

// Shape checks shared by the workspace query and the attention calls.  `per_launch` is the most
// sequences one kernel launch sees (decode slices the batch; prefill takes it whole).
pkv_status check_shapes(int32_t num_seqs, int32_t per_launch, int32_t num_q_heads, int32_t num_kv_heads,
                        int32_t head_dim, int32_t max_blocks_per_seq) {
  if (num_seqs < 0) return fail(PKV_ERR_INVALID_ARGUMENT, "num_seqs must be >= 0 (got %d)", num_seqs);
  if (num_q_heads <= 0 || num_kv_heads <= 0)
    return fail(PKV_ERR_INVALID_ARGUMENT, "head counts must be positive (q %d, kv %d)", num_q_heads, num_kv_heads);
  if (num_q_heads % num_kv_heads != 0)
    return fail(PKV_ERR_INVALID_ARGUMENT, "num_q_heads %d is not a multiple of num_kv_heads %d", num_q_heads,
                num_kv_heads);
  const int group = num_q_heads / num_kv_heads;
  if (group != 1 && group != 2 && group != 4 && group != 8)
    return fail(PKV_ERR_UNSUPPORTED, "GQA group %d not built (1, 2, 4 or 8)", group);
  if (head_dim != 64 && head_dim != 128)
    return fail(PKV_ERR_UNSUPPORTED, "head_dim %d not built (64 or 128)", head_dim);
  if (max_blocks_per_seq <= 0)
    return fail(PKV_ERR_INVALID_ARGUMENT, "max_blocks_per_seq must be positive (got %d)", max_blocks_per_seq);
  if (static_cast<int64_t>(per_launch) * max_blocks_per_seq * num_kv_heads >= (int64_t{1} << 31) ||
      static_cast<int64_t>(max_blocks_per_seq) * PKV_BLOCK_SIZE >= (int64_t{1} << 31))
    return fail(PKV_ERR_UNSUPPORTED, "sequences per launch * max_blocks_per_seq * num_kv_heads must stay below 2^31");
  return PKV_OK;
}
pkv_status check_decode_shapes(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                               int32_t max_blocks_per_seq) {
  return check_shapes(num_seqs, launch_seqs(num_seqs), num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq);
}

constexpr int32_t kMaxPartitions = 1 << 20;

// A sliding window and sinks; window 0: neither.
struct Window {
  int32_t window = 0;
  int32_t sinks = 0;
};
pkv_status check_window(int32_t window, int32_t sinks) {
  if (window <= 0) return fail(PKV_ERR_INVALID_ARGUMENT, "window must be positive (got %d)", window);
  if (sinks < 0) return fail(PKV_ERR_INVALID_ARGUMENT, "num_sink_tokens must be >= 0 (got %d)", sinks);
  return PKV_OK;
}
// Both within the table, so that the kernels' sums stay within 32 bits (a window of the table's length is
// no window, and so many sinks are every token).
Window within_table(Window w, int32_t max_blocks_per_seq) {
  const int32_t cap = max_blocks_per_seq * PKV_BLOCK_SIZE;
  if (w.window > cap) w.window = cap;
  if (w.sinks > cap) w.sinks = cap;
  return w;
}
// Window and tail streams are cut into pieces of no less than this many blocks: a piece is a state to join, and a block
// more a piece is a block's time (one sequence, window 1024, two heads: 9.3 us a call with 2, 9.4 with 1, 11.7 with 4,
// 16.2 with 8).
constexpr int32_t kMinPieceBlocks = 2;
// Least key steps of a split of a windowed prefill (one chunk of 512, window 1024: 18.6 us with 1 to 3, 19.7 with 4,
// 21.0 with 5).
constexpr int32_t kMinSplitSteps = 2;
// Blocks of one sequence that a query token can see.
int32_t visible_blocks(Window w, int32_t max_blocks_per_seq) {
  if (w.window == 0) return max_blocks_per_seq;
  w = within_table(w, max_blocks_per_seq);
  const int64_t n = (static_cast<int64_t>(w.sinks) + PKV_BLOCK_SIZE - 1) / PKV_BLOCK_SIZE +
                    (static_cast<int64_t>(w.window) + 2 * PKV_BLOCK_SIZE - 2) / PKV_BLOCK_SIZE;
  return n < max_blocks_per_seq ? static_cast<int32_t>(n) : max_blocks_per_seq;
}

// CTAs a (sequence, kv head) of a windowed call in its form for few pairs; 0: the call takes the other form, as it
// does whenever a partition count is given.
pkv_status cluster_ctas(int32_t num_seqs, int32_t num_kv_heads, int32_t head_dim, int32_t group,
                        int32_t max_blocks_per_seq, const Window& window, int32_t num_partitions, int* ctas) {
  *ctas = 0;
  if (num_partitions != 0 || num_seqs == 0 || num_seqs > PKV_MAX_SEQS) return PKV_OK;
  const cudaError_t e = pkv::window_cluster_ctas(head_dim, group, num_seqs, num_kv_heads,
                                                 visible_blocks(window, max_blocks_per_seq), ctas);
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "cluster occupancy query");
}

// Pieces of a stream, `resident` if it can have so many: never more than it can have items, or pieces of the least size.
int32_t most_partitions(int32_t num_seqs, int32_t num_kv_heads, int32_t visible, const Window& window, int resident) {
  int64_t bound = static_cast<int64_t>(num_seqs) * num_kv_heads * visible;
  if (window.window) bound = (bound + kMinPieceBlocks - 1) / kMinPieceBlocks;
  int64_t n = resident;
  if (n > bound) n = bound;
  if (n > kMaxPartitions) n = kMaxPartitions;
  return static_cast<int32_t>(n < 1 ? 1 : n);
}

pkv_status default_partitions(int32_t num_seqs, int32_t num_kv_heads, int32_t head_dim, int32_t group,
                              int32_t max_blocks_per_seq, const Window& window, int32_t* out) {
  int pieces = 0;
  const cudaError_t e = window.window ? pkv::resident_window_pieces(head_dim, group, num_seqs, &pieces)
                                      : pkv::resident_partition_pieces(head_dim, group, num_seqs, &pieces);
  if (e != cudaSuccess) return cuda_fail(e, "occupancy query");
  *out = most_partitions(num_seqs, num_kv_heads, visible_blocks(window, max_blocks_per_seq), window, pieces);
  return PKV_OK;
}

size_t workspace_bytes_for(int32_t num_seqs, int32_t num_kv_heads, int32_t head_dim, int32_t group,
                           int32_t num_partitions) {
  return pkv::workspace_header_bytes(num_seqs, num_kv_heads) +
         static_cast<size_t>(num_partitions) * 2 * pkv::piece_floats(head_dim, group) * sizeof(float);
}

// Workspace one decode call needs: the most any of its slices needs (a slice of PKV_MAX_SEQS and,
// when the batch does not divide evenly, the shorter last one; each at its own default partition
// count unless one is given).
pkv_status decode_workspace_need(int32_t num_seqs, int32_t num_kv_heads, int32_t head_dim, int32_t group,
                                 int32_t max_blocks_per_seq, const Window& window, int32_t num_partitions,
                                 size_t* need) {
  *need = 0;
  const int32_t sizes[2] = {launch_seqs(num_seqs), num_seqs > PKV_MAX_SEQS ? num_seqs % PKV_MAX_SEQS : 0};
  for (int32_t n : sizes) {
    if (n == 0) continue;
    int32_t parts = num_partitions;
    if (parts == 0)
      if (pkv_status st = default_partitions(n, num_kv_heads, head_dim, group, max_blocks_per_seq, window, &parts);
          st != PKV_OK)
        return st;
    const size_t b = workspace_bytes_for(n, num_kv_heads, head_dim, group, parts);
    if (b > *need) *need = b;
  }
  return PKV_OK;
}

}  // namespace

// Fused-step inputs of decode_impl (null for plain attention).
struct FusedStep {
  const void* k_new;
  const void* v_new;
  const float* cos_sin;
  int64_t max_position;
};

static pkv_status decode_impl(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                              int32_t max_blocks_per_seq, const int32_t* context_lens, int32_t num_seqs,
                              int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int64_t num_blocks,
                              int32_t block_size, float scale, void* out, void* workspace, size_t workspace_bytes,
                              int32_t num_partitions, int32_t phases, pkv_stream_t stream, const FusedStep* fused,
                              const Window& window) {
  if (pkv_status st = check_decode_shapes(num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq);
      st != PKV_OK)
    return st;
  if (block_size != PKV_BLOCK_SIZE)
    return fail(PKV_ERR_UNSUPPORTED, "block_size must be %d (got %d)", PKV_BLOCK_SIZE, block_size);
  if (num_blocks <= 0 || num_blocks > (int64_t{1} << 40))
    return fail(PKV_ERR_INVALID_ARGUMENT, "num_blocks out of range (got %lld)", (long long)num_blocks);
  if (!std::isfinite(scale)) return fail(PKV_ERR_INVALID_ARGUMENT, "scale must be finite");
  if (phases < 1 || phases > PKV_PHASE_ALL) return fail(PKV_ERR_INVALID_ARGUMENT, "phases must be 1, 2 or 3");
  if (num_partitions < 0 || num_partitions > kMaxPartitions)
    return fail(PKV_ERR_INVALID_ARGUMENT, "num_partitions out of range (got %d)", num_partitions);
  if (window.window && num_blocks * num_kv_heads * PKV_BLOCK_SIZE >= (int64_t{1} << 31))
    return fail(PKV_ERR_UNSUPPORTED, "num_blocks * num_kv_heads * 16 must be below 2^31 (got %lld blocks)",
                (long long)num_blocks);
  if (num_seqs == 0) return ok();
  int cluster = 0;  // CTAs a (sequence, kv head) of the form without a workspace
  if (window.window)
    if (pkv_status st = cluster_ctas(num_seqs, num_kv_heads, head_dim, num_q_heads / num_kv_heads,
                                       max_blocks_per_seq, window, num_partitions, &cluster);
        st != PKV_OK)
      return st;
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out || (!workspace && !cluster))
    return fail(PKV_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || !aligned16(workspace) ||
      (reinterpret_cast<uintptr_t>(block_tables) & 3u) || (reinterpret_cast<uintptr_t>(context_lens) & 3u))
    return fail(PKV_ERR_INVALID_ARGUMENT, "q, caches, out and workspace must be 16-byte aligned");
  const int group = num_q_heads / num_kv_heads;
  if (num_seqs > PKV_MAX_SEQS && phases != PKV_PHASE_ALL)
    return fail(PKV_ERR_UNSUPPORTED, "phases other than PKV_PHASE_ALL need num_seqs <= PKV_MAX_SEQS (%d)",
                PKV_MAX_SEQS);
  size_t need = 0;
  if (!cluster)
    if (pkv_status st = decode_workspace_need(num_seqs, num_kv_heads, head_dim, group, max_blocks_per_seq, window,
                                              num_partitions, &need);
        st != PKV_OK)
      return st;
  if (workspace_bytes < need)
    return fail(PKV_ERR_INVALID_ARGUMENT, "workspace too small: %zu bytes given, %zu needed", workspace_bytes, need);

  unsigned* err = nullptr;
  if (pkv_status st = device_state(&err, nullptr); st != PKV_OK) return st;
  // A batch larger than PKV_MAX_SEQS runs as consecutive slices of at most that many sequences,
  // each a partition + merge pair on the same stream and workspace (a slice's merge has read the
  // workspace before the next slice's partition kernel, which waits for it, writes it).
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const size_t q_row = static_cast<size_t>(num_q_heads) * head_dim * 2;  // bytes of one sequence's q / out
  const size_t kv_row = static_cast<size_t>(num_kv_heads) * head_dim * 2;
  for (int32_t s0 = 0; s0 < num_seqs; s0 += PKV_MAX_SEQS) {
    const int32_t n = launch_seqs(num_seqs - s0);
    int32_t parts = num_partitions;
    if (parts == 0 && !cluster)
      if (pkv_status st = default_partitions(n, num_kv_heads, head_dim, group, max_blocks_per_seq, window, &parts);
          st != PKV_OK)
        return st;
    pkv::DecodeParams p{};
    p.q = static_cast<const unsigned char*>(q) + s0 * q_row;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.block_tables = block_tables + static_cast<size_t>(s0) * max_blocks_per_seq;
    p.context_lens = context_lens + s0;
    p.out = static_cast<unsigned char*>(out) + s0 * q_row;
    if (workspace) {
      p.ws_prefix = static_cast<int32_t*>(workspace);
      p.ws_pairs = reinterpret_cast<int32_t*>(static_cast<unsigned char*>(workspace) + pkv::workspace_prefix_bytes(n));
      p.ws_pieces = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) +
                                             pkv::workspace_header_bytes(n, num_kv_heads));
    }
    p.err = err;
    p.num_blocks = num_blocks;
    p.num_seqs = n;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.num_partitions = parts;
    p.qscale = scale * 1.4426950408889634f;
    if (fused) {
      p.k_new = static_cast<const unsigned char*>(fused->k_new) + s0 * kv_row;
      p.v_new = static_cast<const unsigned char*>(fused->v_new) + s0 * kv_row;
      p.cos_sin = fused->cos_sin;
      p.max_position = fused->max_position;
    }
    if (window.window) {
      const Window w = within_table(window, max_blocks_per_seq);
      pkv::DecodeViewParams v{};
      static_cast<pkv::DecodeParams&>(v) = p;
      v.window = w.window;
      v.sinks = w.sinks;
      v.min_piece_blocks = num_partitions == 0 ? kMinPieceBlocks : 1;
      const cudaError_t e = cluster ? pkv::launch_window_cluster(v, head_dim, group, cluster, s)
                                    : pkv::launch_window_decode(v, head_dim, group, s);
      if (e != cudaSuccess) return cuda_fail(e, "window decode launch");
      g_launches.fetch_add(cluster ? 1 : 2);
      continue;
    }
    if (phases & PKV_PHASE_PARTITION) {
      const cudaError_t e = pkv::launch_decode_partition(p, head_dim, group, s);
      if (e != cudaSuccess) return cuda_fail(e, "partition kernel launch");
      g_launches.fetch_add(1);
    }
    if (phases & PKV_PHASE_MERGE) {
      const cudaError_t e = pkv::launch_decode_merge(p, head_dim, group, s);
      if (e != cudaSuccess) return cuda_fail(e, "merge kernel launch");
      g_launches.fetch_add(1);
    }
  }
  return ok();
}


void pkv::set_error_message(const char* message) { snprintf(t_message, sizeof t_message, "%s", message); }

extern "C" {

const char* pkv_last_error_message(void) { return t_message; }

uint64_t pkv_kernel_launch_count(void) { return g_launches.load(); }

pkv_status pkv_kv_append(const void* k, const void* v, const int64_t* slot_mapping, int64_t num_tokens,
                         int32_t num_kv_heads, int32_t head_dim, void* k_cache, void* v_cache, int64_t num_blocks,
                         int32_t block_size, pkv_stream_t stream) {
  if (num_tokens < 0) return fail(PKV_ERR_INVALID_ARGUMENT, "num_tokens must be >= 0 (got %lld)", (long long)num_tokens);
  if (num_kv_heads <= 0) return fail(PKV_ERR_INVALID_ARGUMENT, "num_kv_heads must be positive (got %d)", num_kv_heads);
  if (head_dim != 64 && head_dim != 128)
    return fail(PKV_ERR_UNSUPPORTED, "head_dim %d not built (64 or 128)", head_dim);
  if (block_size != PKV_BLOCK_SIZE)
    return fail(PKV_ERR_UNSUPPORTED, "block_size must be %d (got %d)", PKV_BLOCK_SIZE, block_size);
  if (num_blocks <= 0 || num_blocks > (int64_t{1} << 40))
    return fail(PKV_ERR_INVALID_ARGUMENT, "num_blocks out of range (got %lld)", (long long)num_blocks);
  if (num_tokens > (int64_t{1} << 32))
    return fail(PKV_ERR_UNSUPPORTED, "num_tokens %lld too large", (long long)num_tokens);
  if (num_tokens == 0) return ok();
  if (!k || !v || !slot_mapping || !k_cache || !v_cache)
    return fail(PKV_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
    return fail(PKV_ERR_INVALID_ARGUMENT, "k, v and the caches must be 16-byte aligned, slot_mapping 8-byte aligned");
  unsigned* err = nullptr;
  int sms = 0;
  if (pkv_status st = device_state(&err, &sms); st != PKV_OK) return st;
  pkv::AppendParams p{};
  p.k = k;
  p.v = v;
  p.slot_mapping = slot_mapping;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.err = err;
  p.num_tokens = num_tokens;
  p.num_slots = num_blocks * PKV_BLOCK_SIZE;
  p.num_kv_heads = num_kv_heads;
  p.head_dim = head_dim;
  const cudaError_t e = pkv::launch_kv_append(p, sms, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kv_append launch");
  g_launches.fetch_add(1);
  return ok();
}

pkv_status pkv_copy_blocks(void* k_cache, void* v_cache, const int64_t* src_dst, int32_t num_pairs,
                           int32_t num_kv_heads, int32_t head_dim, int64_t num_blocks, pkv_stream_t stream) {
  if (num_pairs < 0) return fail(PKV_ERR_INVALID_ARGUMENT, "num_pairs must be >= 0 (got %d)", num_pairs);
  if (num_pairs > (1 << 30)) return fail(PKV_ERR_UNSUPPORTED, "num_pairs %d too large", num_pairs);
  if (num_kv_heads <= 0) return fail(PKV_ERR_INVALID_ARGUMENT, "num_kv_heads must be positive (got %d)", num_kv_heads);
  if (head_dim != 64 && head_dim != 128)
    return fail(PKV_ERR_UNSUPPORTED, "head_dim %d not built (64 or 128)", head_dim);
  if (num_blocks <= 0 || num_blocks > (int64_t{1} << 40))
    return fail(PKV_ERR_INVALID_ARGUMENT, "num_blocks out of range (got %lld)", (long long)num_blocks);
  if (num_pairs == 0) return ok();
  if (!k_cache || !v_cache || !src_dst) return fail(PKV_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (!aligned16(k_cache) || !aligned16(v_cache) || (reinterpret_cast<uintptr_t>(src_dst) & 7u))
    return fail(PKV_ERR_INVALID_ARGUMENT, "caches must be 16-byte aligned, src_dst 8-byte aligned");
  unsigned* err = nullptr;
  if (pkv_status st = device_state(&err, nullptr); st != PKV_OK) return st;
  pkv::CopyParams p{};
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.src_dst = src_dst;
  p.err = err;
  p.num_blocks = num_blocks;
  p.chunks_per_block = static_cast<int64_t>(num_kv_heads) * PKV_BLOCK_SIZE * head_dim / 8;
  const cudaError_t e = pkv::launch_copy_blocks(p, num_pairs, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "copy_blocks launch");
  g_launches.fetch_add(1);
  return ok();
}

pkv_status pkv_selftest_wait_timeout(uint64_t limit_ns, pkv_stream_t stream) {
  if (limit_ns < 1000 || limit_ns > 1000000000ull)
    return fail(PKV_ERR_INVALID_ARGUMENT, "limit_ns must lie in [1e3, 1e9] (got %llu)", (unsigned long long)limit_ns);
  unsigned* err = nullptr;
  if (pkv_status st = device_state(&err, nullptr); st != PKV_OK) return st;
  const cudaError_t e =
      pkv::launch_bounded_wait_selftest(err, limit_ns, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "self-test launch");
  g_launches.fetch_add(1);
  return ok();
}

namespace {
constexpr int32_t kMaxPrefillSplits = 32;  // the merge reads one split per lane

// SMs that a windowed call counts on.
int32_t window_sms(int sms) { return sms < pkv::kWindowSplitCtas ? sms : pkv::kWindowSplitCtas; }

// The most splits that keep every CTA of the call in one wave (one CTA per SM), at most 32, and
// within the 65535 grid rows; 1 when the call already fills the GPU.
int32_t one_wave_splits(int32_t num_seqs, int32_t max_query_len, int32_t num_q_heads, int32_t num_kv_heads, int sms) {
  const int64_t cta = pkv::prefill_cta_tokens(num_q_heads / num_kv_heads);
  const int64_t ctas = static_cast<int64_t>(num_seqs) * num_kv_heads * ((max_query_len + cta - 1) / cta);
  int64_t n = ctas > 0 ? sms / ctas : 1;
  if (n > kMaxPrefillSplits) n = kMaxPrefillSplits;
  if (num_seqs > 0 && n > 65535 / num_seqs) n = 65535 / num_seqs;
  return static_cast<int32_t>(n < 1 ? 1 : n);
}

pkv_status prefill_impl(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                        int32_t max_blocks_per_seq, const int32_t* context_lens, const int32_t* query_start,
                        int32_t max_query_len, int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                        int32_t head_dim, int64_t num_blocks, int32_t block_size, float scale, void* out,
                        int32_t num_splits, void* workspace, size_t workspace_bytes, pkv_stream_t stream,
                        const Window& window, int64_t query_rows) {
  if (num_splits < 1 || num_splits > kMaxPrefillSplits)
    return fail(PKV_ERR_INVALID_ARGUMENT, "num_splits must be in [1, %d] (got %d)", kMaxPrefillSplits, num_splits);
  if (window.window && num_seqs > pkv::kPrefillRankedSeqs) num_splits = 1;  // its units are not split
  if (static_cast<int64_t>(num_seqs) * num_splits > 65535)
    return fail(PKV_ERR_UNSUPPORTED, "num_seqs * num_splits = %lld exceeds 65535 (one grid row of CTAs each)",
                static_cast<long long>(num_seqs) * num_splits);
  if (pkv_status st = check_shapes(num_seqs, num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq);
      st != PKV_OK)
    return st;
  if (block_size != PKV_BLOCK_SIZE)
    return fail(PKV_ERR_UNSUPPORTED, "block_size must be %d (got %d)", PKV_BLOCK_SIZE, block_size);
  if (num_blocks <= 0 || num_blocks * num_kv_heads * PKV_BLOCK_SIZE >= (int64_t{1} << 31))
    return fail(PKV_ERR_UNSUPPORTED, "num_blocks * num_kv_heads * 16 must be in (0, 2^31) (got %lld blocks)",
                (long long)num_blocks);
  if (!std::isfinite(scale)) return fail(PKV_ERR_INVALID_ARGUMENT, "scale must be finite");
  if (max_query_len < 0) return fail(PKV_ERR_INVALID_ARGUMENT, "max_query_len must be >= 0 (got %d)", max_query_len);
  // A CTA takes two 128-row tiles of 128 / G chunk tokens each; its sequence's tiles are one grid dimension.
  const int32_t cta_tokens = 256 / (num_q_heads / num_kv_heads);
  if ((static_cast<int64_t>(max_query_len) + cta_tokens - 1) / cta_tokens > 65535)
    return fail(PKV_ERR_UNSUPPORTED, "max_query_len %d exceeds 65535 CTAs of %d chunk tokens", max_query_len,
                cta_tokens);
  if (num_seqs == 0 || max_query_len == 0 || (window.window && query_rows == 0)) return ok();
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !query_start || !out)
    return fail(PKV_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(block_tables) & 3u) || (reinterpret_cast<uintptr_t>(context_lens) & 3u) ||
      (reinterpret_cast<uintptr_t>(query_start) & 3u))
    return fail(PKV_ERR_INVALID_ARGUMENT, "q, caches and out must be 16-byte aligned");
  const pkv::WindowSplitLayout layout(head_dim, num_splits);
  if (num_splits > 1) {
    const size_t need =
        window.window ? layout.bytes
                      : pkv::prefill_workspace_bytes(num_seqs, max_query_len, num_q_heads, num_kv_heads, head_dim, num_splits);
    if (!workspace || workspace_bytes < need)
      return fail(PKV_ERR_INVALID_ARGUMENT, "workspace too small: %zu bytes given, %zu needed", workspace_bytes, need);
    if (!aligned16(workspace)) return fail(PKV_ERR_INVALID_ARGUMENT, "workspace must be 16-byte aligned");
  }
  unsigned* err = nullptr;
  int sms = 0;
  if (pkv_status st = device_state(&err, &sms); st != PKV_OK) return st;
  pkv::PrefillParams p{};
  p.q = q;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.query_start = query_start;
  p.out = out;
  p.err = err;
  p.num_blocks = num_blocks;
  p.num_seqs = num_seqs;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_query_len = max_query_len;
  p.scale = scale;
  if (num_splits > 1) {
    p.num_splits = num_splits;
    p.ws = static_cast<float*>(workspace);
    p.ws_units = reinterpret_cast<int4*>(static_cast<unsigned char*>(workspace) + layout.units);
    p.ws_count = reinterpret_cast<int32_t*>(static_cast<unsigned char*>(workspace) + layout.count);
  }
  p.num_sms = window_sms(sms);
  const Window w = within_table(window, max_blocks_per_seq);
  p.window = w.window;
  p.sinks = w.sinks;
  p.query_rows = query_rows;
  const cudaError_t e =
      (window.window ? pkv::launch_window_prefill : pkv::launch_paged_prefill)(
          p, head_dim, num_q_heads / num_kv_heads, max_query_len, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "prefill kernel launch");
  if (window.window) {
    g_launches.fetch_add(pkv::window_splits(p, num_q_heads / num_kv_heads, max_query_len)
                             ? 2
                             : (num_seqs + pkv::kPrefillRankedSeqs - 1) / pkv::kPrefillRankedSeqs);
  } else {
    g_launches.fetch_add(num_splits > 1 ? 2 : 1);
  }
  return ok();
}
}  // namespace

pkv_status pkv_paged_prefill_attention(const void* q, const void* k_cache, const void* v_cache,
                                       const int32_t* block_tables, int32_t max_blocks_per_seq,
                                       const int32_t* context_lens, const int32_t* query_start,
                                       int32_t max_query_len, int32_t num_seqs, int32_t num_q_heads,
                                       int32_t num_kv_heads, int32_t head_dim, int64_t num_blocks, int32_t block_size,
                                       float scale, void* out, pkv_stream_t stream) {
  return prefill_impl(q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, query_start, max_query_len,
                      num_seqs, num_q_heads, num_kv_heads, head_dim, num_blocks, block_size, scale, out, 1, nullptr, 0,
                      stream, Window{}, 0);
}

pkv_status pkv_paged_prefill_attention_split(const void* q, const void* k_cache, const void* v_cache,
                                             const int32_t* block_tables, int32_t max_blocks_per_seq,
                                             const int32_t* context_lens, const int32_t* query_start,
                                             int32_t max_query_len, int32_t num_seqs, int32_t num_q_heads,
                                             int32_t num_kv_heads, int32_t head_dim, int64_t num_blocks,
                                             int32_t block_size, float scale, void* out, int32_t num_splits,
                                             void* workspace, size_t workspace_bytes, pkv_stream_t stream) {
  return prefill_impl(q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, query_start, max_query_len,
                      num_seqs, num_q_heads, num_kv_heads, head_dim, num_blocks, block_size, scale, out, num_splits,
                      workspace, workspace_bytes, stream, Window{}, 0);
}

pkv_status pkv_prefill_default_splits(int32_t num_seqs, int32_t max_query_len, int32_t num_q_heads,
                                      int32_t num_kv_heads, int32_t* num_splits) {
  if (!num_splits) return fail(PKV_ERR_INVALID_ARGUMENT, "num_splits is null");
  if (num_seqs < 0 || max_query_len < 0) return fail(PKV_ERR_INVALID_ARGUMENT, "num_seqs and max_query_len must be >= 0");
  if (pkv_status st = check_shapes(num_seqs, num_seqs, num_q_heads, num_kv_heads, 128, 1); st != PKV_OK) return st;
  int sms = 0;
  if (pkv_status st = device_state(nullptr, &sms); st != PKV_OK) return st;
  *num_splits = one_wave_splits(num_seqs, max_query_len, num_q_heads, num_kv_heads, sms);
  return ok();
}

pkv_status pkv_prefill_workspace_size(int32_t num_seqs, int32_t max_query_len, int32_t num_q_heads,
                                      int32_t num_kv_heads, int32_t head_dim, int32_t num_splits, size_t* bytes) {
  if (!bytes) return fail(PKV_ERR_INVALID_ARGUMENT, "bytes must not be null");
  if (num_seqs < 0 || max_query_len < 0) return fail(PKV_ERR_INVALID_ARGUMENT, "num_seqs and max_query_len must be >= 0");
  if (num_splits < 1 || num_splits > kMaxPrefillSplits)
    return fail(PKV_ERR_INVALID_ARGUMENT, "num_splits must be in [1, %d] (got %d)", kMaxPrefillSplits, num_splits);
  if (pkv_status st = check_shapes(num_seqs, num_seqs, num_q_heads, num_kv_heads, head_dim, 1); st != PKV_OK) return st;
  *bytes = pkv::prefill_workspace_bytes(num_seqs, max_query_len, num_q_heads, num_kv_heads, head_dim, num_splits);
  return ok();
}

pkv_status pkv_decode_default_partitions(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                         int32_t head_dim, int32_t max_blocks_per_seq, int32_t* num_partitions) {
  if (!num_partitions) return fail(PKV_ERR_INVALID_ARGUMENT, "num_partitions is null");
  if (pkv_status st = check_decode_shapes(num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq);
      st != PKV_OK)
    return st;
  if (pkv_status st = default_partitions(launch_seqs(num_seqs), num_kv_heads, head_dim, num_q_heads / num_kv_heads,
                                         max_blocks_per_seq, Window{}, num_partitions);
      st != PKV_OK)
    return st;
  return ok();
}

pkv_status pkv_decode_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                     int32_t max_blocks_per_seq, int32_t num_partitions, size_t* bytes) {
  if (!bytes) return fail(PKV_ERR_INVALID_ARGUMENT, "bytes is null");
  if (pkv_status st = check_decode_shapes(num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq);
      st != PKV_OK)
    return st;
  if (num_partitions < 0 || num_partitions > kMaxPartitions)
    return fail(PKV_ERR_INVALID_ARGUMENT, "num_partitions out of range (got %d)", num_partitions);
  size_t need = 0;
  if (pkv_status st = decode_workspace_need(num_seqs, num_kv_heads, head_dim, num_q_heads / num_kv_heads,
                                            max_blocks_per_seq, Window{}, num_partitions, &need);
      st != PKV_OK)
    return st;
  *bytes = need;
  return ok();
}

pkv_status pkv_paged_decode_attention_split(const void* q, const void* k_cache, const void* v_cache,
                                            const int32_t* block_tables, int32_t max_blocks_per_seq,
                                            const int32_t* context_lens, int32_t num_seqs, int32_t num_q_heads,
                                            int32_t num_kv_heads, int32_t head_dim, int64_t num_blocks,
                                            int32_t block_size, float scale, void* out, void* workspace,
                                            size_t workspace_bytes, int32_t num_partitions, int32_t phases,
                                            pkv_stream_t stream) {
  return decode_impl(q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, num_seqs, num_q_heads,
                     num_kv_heads, head_dim, num_blocks, block_size, scale, out, workspace, workspace_bytes,
                     num_partitions, phases, stream, nullptr, Window{});
}

pkv_status pkv_decode_step(const void* q, const void* k_new, const void* v_new, const float* cos_sin,
                           int64_t max_position, void* k_cache, void* v_cache, const int32_t* block_tables,
                           int32_t max_blocks_per_seq, const int32_t* context_lens, int32_t num_seqs,
                           int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int64_t num_blocks,
                           int32_t block_size, float scale, void* out, void* workspace, size_t workspace_bytes,
                           pkv_stream_t stream) {
  if (num_seqs > 0) {
    if (!k_new || !v_new) return fail(PKV_ERR_INVALID_ARGUMENT, "null pointer argument");
    if (!aligned16(k_new) || !aligned16(v_new) || (cos_sin && !aligned16(cos_sin)))
      return fail(PKV_ERR_INVALID_ARGUMENT, "k_new, v_new and cos_sin must be 16-byte aligned");
    if (cos_sin && max_position <= 0)
      return fail(PKV_ERR_INVALID_ARGUMENT, "max_position must be positive with a rotary table (got %lld)",
                  (long long)max_position);
  }
  const FusedStep fused{k_new, v_new, cos_sin, cos_sin ? max_position : 0};
  return decode_impl(q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, num_seqs, num_q_heads,
                     num_kv_heads, head_dim, num_blocks, block_size, scale, out, workspace, workspace_bytes, 0,
                     PKV_PHASE_ALL, stream, &fused, Window{});
}

pkv_status pkv_paged_decode_attention(const void* q, const void* k_cache, const void* v_cache,
                                      const int32_t* block_tables, int32_t max_blocks_per_seq,
                                      const int32_t* context_lens, int32_t num_seqs, int32_t num_q_heads,
                                      int32_t num_kv_heads, int32_t head_dim, int64_t num_blocks, int32_t block_size,
                                      float scale, void* out, void* workspace, size_t workspace_bytes,
                                      pkv_stream_t stream) {
  return pkv_paged_decode_attention_split(q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens,
                                          num_seqs, num_q_heads, num_kv_heads, head_dim, num_blocks, block_size,
                                          scale, out, workspace, workspace_bytes, 0, PKV_PHASE_ALL, stream);
}

pkv_status pkv_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                           int64_t v_stride, const int64_t* positions, int32_t num_axes, int64_t axis_stride,
                           const uint8_t* freq_axes, const float* cos_sin, int64_t max_position,
                           const int64_t* slot_mapping, int64_t num_tokens, int32_t num_q_heads,
                           int32_t num_kv_heads, int32_t head_dim, void* q_out, int64_t q_out_stride, void* k_cache,
                           void* v_cache, int64_t num_blocks, int32_t block_size, pkv_stream_t stream) {
  if (num_tokens < 0) return fail(PKV_ERR_INVALID_ARGUMENT, "num_tokens must be >= 0 (got %lld)", (long long)num_tokens);
  if (num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads > (1 << 20) || num_kv_heads > (1 << 20))
    return fail(PKV_ERR_INVALID_ARGUMENT, "head counts must be in [1, 2^20] (q %d, kv %d)", num_q_heads, num_kv_heads);
  if (head_dim != 64 && head_dim != 128)
    return fail(PKV_ERR_UNSUPPORTED, "head_dim %d not built (64 or 128)", head_dim);
  if (block_size != PKV_BLOCK_SIZE)
    return fail(PKV_ERR_UNSUPPORTED, "block_size must be %d (got %d)", PKV_BLOCK_SIZE, block_size);
  if (num_blocks <= 0 || num_blocks > (int64_t{1} << 40))
    return fail(PKV_ERR_INVALID_ARGUMENT, "num_blocks out of range (got %lld)", (long long)num_blocks);
  if (num_tokens > (int64_t{1} << 32))
    return fail(PKV_ERR_UNSUPPORTED, "num_tokens %lld too large", (long long)num_tokens);
  if (num_axes < 1 || num_axes > pkv::kMaxPositionAxes)
    return fail(PKV_ERR_INVALID_ARGUMENT, "num_axes must be in [1, %d] (got %d)", pkv::kMaxPositionAxes, num_axes);
  if (max_position <= 0)
    return fail(PKV_ERR_INVALID_ARGUMENT, "max_position must be positive (got %lld)", (long long)max_position);
  if (num_axes > 1) {
    if (axis_stride < 0) return fail(PKV_ERR_INVALID_ARGUMENT, "axis_stride must be >= 0 (got %lld)", (long long)axis_stride);
    if (!freq_axes) return fail(PKV_ERR_INVALID_ARGUMENT, "freq_axes is null with %d axes", num_axes);
    for (int i = 0; i < head_dim / 2; ++i)
      if (freq_axes[i] >= num_axes)
        return fail(PKV_ERR_INVALID_ARGUMENT, "freq_axes[%d] = %d, with %d axes", i, freq_axes[i], num_axes);
  }
  const struct {
    const char* name;
    int64_t stride, least;
  } strides[] = {{"q_stride", q_stride, 0},
                 {"k_stride", k_stride, 0},
                 {"v_stride", v_stride, 0},
                 {"q_out_stride", q_out_stride, static_cast<int64_t>(num_q_heads) * head_dim}};
  for (const auto& x : strides)
    if (x.stride < x.least || x.stride % 8 || x.stride > (int64_t{1} << 40))
      return fail(PKV_ERR_INVALID_ARGUMENT, "%s must be a multiple of 8 elements and at least %lld (got %lld)", x.name,
                  (long long)x.least, (long long)x.stride);
  if (num_tokens == 0) return ok();
  if (!q || !k || !v || !positions || !cos_sin || !slot_mapping || !q_out || !k_cache || !v_cache)
    return fail(PKV_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_cache) ||
      !aligned16(v_cache) || !aligned16(cos_sin) || (reinterpret_cast<uintptr_t>(positions) & 7u) ||
      (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
    return fail(PKV_ERR_INVALID_ARGUMENT,
                "q, k, v, q_out, cos_sin and the caches must be 16-byte aligned, positions and slot_mapping 8-byte");
  unsigned* err = nullptr;
  int sms = 0;
  if (pkv_status st = device_state(&err, &sms); st != PKV_OK) return st;
  pkv::RopeAppendParams p{};
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_out = q_out;
  p.q_stride = q_stride / 8;
  p.k_stride = k_stride / 8;
  p.v_stride = v_stride / 8;
  p.q_out_stride = q_out_stride / 8;
  p.positions = positions;
  p.axis_stride = axis_stride;
  p.cos_sin = cos_sin;
  p.max_position = max_position;
  p.slot_mapping = slot_mapping;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.err = err;
  p.num_tokens = num_tokens;
  p.num_slots = num_blocks * PKV_BLOCK_SIZE;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.num_axes = num_axes;
  if (num_axes > 1) memcpy(p.freq_axis, freq_axes, head_dim / 2);
  const cudaError_t e = pkv::launch_rope_append(p, head_dim, sms, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "rope_append launch");
  g_launches.fetch_add(1);
  return ok();
}

pkv_status pkv_window_decode_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                            int32_t head_dim, int32_t max_blocks_per_seq, int32_t window,
                                            int32_t num_sink_tokens, int32_t num_partitions, size_t* bytes) {
  if (!bytes) return fail(PKV_ERR_INVALID_ARGUMENT, "bytes is null");
  if (pkv_status st = check_decode_shapes(num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq);
      st != PKV_OK)
    return st;
  if (pkv_status st = check_window(window, num_sink_tokens); st != PKV_OK) return st;
  if (num_partitions < 0 || num_partitions > kMaxPartitions)
    return fail(PKV_ERR_INVALID_ARGUMENT, "num_partitions out of range (got %d)", num_partitions);
  const Window w{window, num_sink_tokens};
  const int group = num_q_heads / num_kv_heads;
  size_t need = 0;
  if (num_partitions != 0) {
    if (pkv_status st = decode_workspace_need(num_seqs, num_kv_heads, head_dim, group, max_blocks_per_seq, w, num_partitions,
                                              &need);
        st != PKV_OK)
      return st;
  } else if (num_seqs > 0) {
    // What every call of up to num_seqs sequences can do with: nothing if all of them take the form for few pairs, else the
    // most pieces that any of them is cut into, which a single sequence's shared memory leaves room for.
    const int32_t n = launch_seqs(num_seqs);
    const int32_t visible = visible_blocks(w, max_blocks_per_seq);
    bool none = false;
    if (n == num_seqs) {
      const cudaError_t e = pkv::window_cluster_takes_all(head_dim, group, n, num_kv_heads, visible, &none);
      if (e != cudaSuccess) return cuda_fail(e, "cluster occupancy query");
    }
    if (!none) {
      int pieces = 0;
      const cudaError_t e = pkv::resident_window_pieces(head_dim, group, 1, &pieces);
      if (e != cudaSuccess) return cuda_fail(e, "occupancy query");
      need = workspace_bytes_for(n, num_kv_heads, head_dim, group, most_partitions(n, num_kv_heads, visible, w, pieces));
    }
  }
  *bytes = need;
  return ok();
}

pkv_status pkv_paged_window_decode_attention(const void* q, const void* k_cache, const void* v_cache,
                                             const int32_t* block_tables, int32_t max_blocks_per_seq,
                                             const int32_t* context_lens, int32_t num_seqs, int32_t num_q_heads,
                                             int32_t num_kv_heads, int32_t head_dim, int64_t num_blocks,
                                             int32_t block_size, float scale, int32_t window, int32_t num_sink_tokens,
                                             void* out, void* workspace, size_t workspace_bytes,
                                             int32_t num_partitions, pkv_stream_t stream) {
  if (pkv_status st = check_window(window, num_sink_tokens); st != PKV_OK) return st;
  return decode_impl(q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, num_seqs, num_q_heads,
                     num_kv_heads, head_dim, num_blocks, block_size, scale, out, workspace, workspace_bytes,
                     num_partitions, PKV_PHASE_ALL, stream, nullptr, Window{window, num_sink_tokens});
}

pkv_status pkv_window_prefill_default_splits(int32_t num_seqs, int32_t max_query_len, int32_t num_q_heads,
                                             int32_t num_kv_heads, int32_t window, int32_t num_sink_tokens,
                                             int32_t* num_splits) {
  if (!num_splits) return fail(PKV_ERR_INVALID_ARGUMENT, "num_splits is null");
  if (num_seqs < 0 || max_query_len < 0) return fail(PKV_ERR_INVALID_ARGUMENT, "num_seqs and max_query_len must be >= 0");
  if (pkv_status st = check_shapes(num_seqs, num_seqs, num_q_heads, num_kv_heads, 128, 1); st != PKV_OK) return st;
  if (pkv_status st = check_window(window, num_sink_tokens); st != PKV_OK) return st;
  // At least two key steps a split: a CTA's rows see at most its tokens' windows and the sinks.
  const int64_t keys = static_cast<int64_t>(window) + num_sink_tokens + pkv::prefill_cta_tokens(num_q_heads / num_kv_heads);
  const int64_t most = (keys + 128 * kMinSplitSteps - 1) / (128 * kMinSplitSteps);
  *num_splits = num_seqs > pkv::kPrefillRankedSeqs ? 1 : static_cast<int32_t>(most < kMaxPrefillSplits ? most : kMaxPrefillSplits);
  return ok();
}

pkv_status pkv_window_prefill_splits(int64_t num_query_tokens, int32_t max_query_len, int32_t num_seqs,
                                     int32_t num_q_heads, int32_t num_kv_heads, int32_t num_splits, int32_t* used) {
  if (!used) return fail(PKV_ERR_INVALID_ARGUMENT, "used is null");
  if (num_query_tokens < 0 || max_query_len < 0 || num_seqs < 0)
    return fail(PKV_ERR_INVALID_ARGUMENT, "num_query_tokens, max_query_len and num_seqs must be >= 0");
  if (num_splits < 1 || num_splits > kMaxPrefillSplits)
    return fail(PKV_ERR_INVALID_ARGUMENT, "num_splits must be in [1, %d] (got %d)", kMaxPrefillSplits, num_splits);
  if (pkv_status st = check_shapes(num_seqs, num_seqs, num_q_heads, num_kv_heads, 128, 1); st != PKV_OK) return st;
  *used = 1;
  if (num_splits == 1 || num_seqs == 0 || num_seqs > pkv::kPrefillRankedSeqs || max_query_len == 0 || num_query_tokens == 0)
    return ok();
  int sms = 0;
  if (pkv_status st = device_state(nullptr, &sms); st != PKV_OK) return st;
  pkv::PrefillParams p{};
  p.num_seqs = num_seqs;
  p.num_kv_heads = num_kv_heads;
  p.query_rows = num_query_tokens;
  p.num_splits = num_splits;
  p.num_sms = window_sms(sms);
  if (pkv::window_splits(p, num_q_heads / num_kv_heads, max_query_len)) *used = num_splits;
  return ok();
}

pkv_status pkv_window_prefill_workspace_size(int32_t head_dim, int32_t num_splits, size_t* bytes) {
  if (!bytes) return fail(PKV_ERR_INVALID_ARGUMENT, "bytes is null");
  if (pkv_status st = check_shapes(1, 1, 1, 1, head_dim, 1); st != PKV_OK) return st;
  if (num_splits < 1 || num_splits > kMaxPrefillSplits)
    return fail(PKV_ERR_INVALID_ARGUMENT, "num_splits must be in [1, %d] (got %d)", kMaxPrefillSplits, num_splits);
  *bytes = pkv::WindowSplitLayout(head_dim, num_splits).bytes;
  return ok();
}

pkv_status pkv_paged_window_prefill_attention(const void* q, const void* k_cache, const void* v_cache,
                                              const int32_t* block_tables, int32_t max_blocks_per_seq,
                                              const int32_t* context_lens, const int32_t* query_start,
                                              int64_t num_query_tokens, int32_t max_query_len, int32_t num_seqs,
                                              int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                              int64_t num_blocks, int32_t block_size, float scale, int32_t window,
                                              int32_t num_sink_tokens, void* out, int32_t num_splits, void* workspace,
                                              size_t workspace_bytes, pkv_stream_t stream) {
  if (pkv_status st = check_window(window, num_sink_tokens); st != PKV_OK) return st;
  if (!(scale > 0.f)) return fail(PKV_ERR_INVALID_ARGUMENT, "scale must be positive");
  if (num_query_tokens < 0)
    return fail(PKV_ERR_INVALID_ARGUMENT, "num_query_tokens must be >= 0 (got %lld)", (long long)num_query_tokens);
  return prefill_impl(q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, query_start, max_query_len,
                      num_seqs, num_q_heads, num_kv_heads, head_dim, num_blocks, block_size, scale, out, num_splits,
                      workspace, workspace_bytes, stream, Window{window, num_sink_tokens}, num_query_tokens);
}

namespace {
// Shared-prefix decode: its grid, partition count and workspace (byte offsets of the parts).  The tail is cut into as many
// pieces as run at once with `sized_for` sequences: the call's own, or one for the size query (the most of any batch, so
// that what is enough for a batch is enough for smaller ones).
struct PrefixPlan {
  int cluster = 0;  // CTAs a (sequence, kv head) of the form for few pairs, which needs none of the rest
  int32_t ctas = 0, parts = 0, sms = 0;
  size_t pairs = 0, shared = 0, plan_ok = 0, records = 0, whole = 0, pieces = 0, prefix = 0, bytes = 0;
};

pkv_status plan_prefix_decode(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                              int32_t max_blocks_per_seq, int32_t num_groups, int32_t sized_for, PrefixPlan* plan) {
  if (pkv_status st = check_shapes(num_seqs, num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq);
      st != PKV_OK)
    return st;
  if (num_seqs > PKV_MAX_SEQS)
    return fail(PKV_ERR_UNSUPPORTED, "num_seqs %d exceeds PKV_MAX_SEQS (%d)", num_seqs, PKV_MAX_SEQS);
  if (num_groups < 0 || num_groups > PKV_MAX_SEQS)
    return fail(PKV_ERR_INVALID_ARGUMENT, "num_groups must be in [0, %d] (got %d)", PKV_MAX_SEQS, num_groups);
  const int group = num_q_heads / num_kv_heads;
  if (num_seqs > 0) {
    const cudaError_t e = pkv::prefix_cluster_ctas(head_dim, group, num_seqs, num_kv_heads, max_blocks_per_seq, &plan->cluster);
    if (e != cudaSuccess) return cuda_fail(e, "cluster occupancy query");
    if (plan->cluster) return PKV_OK;
  }
  int sms = 0;
  if (pkv_status st = device_state(nullptr, &sms); st != PKV_OK) return st;
  // The most (tile pair, kv head) units the groups can make, and from there whole waves of one CTA per SM.
  const int64_t tiles = (num_groups < num_seqs ? num_groups : num_seqs) +
                        static_cast<int64_t>(num_seqs) / pkv::prefill_cta_tokens(group);
  const int64_t waves = (tiles * num_kv_heads + sms - 1) / sms;
  const int64_t ctas = (waves < 1 ? 1 : waves) * sms;
  if (ctas * 256 >= (int64_t{1} << 31))
    return fail(PKV_ERR_UNSUPPORTED, "too many groups, sequences and kv heads for one launch (%lld CTAs)", (long long)ctas);
  int pieces = 0;
  const cudaError_t e = pkv::resident_tail_pieces(head_dim, group, sized_for, &pieces);
  if (e != cudaSuccess) return cuda_fail(e, "occupancy query");
  const int64_t bound = (static_cast<int64_t>(num_seqs) * num_kv_heads * max_blocks_per_seq + kMinPieceBlocks - 1) /
                        kMinPieceBlocks;
  plan->ctas = static_cast<int32_t>(ctas);
  plan->sms = sms;
  plan->parts = pieces < bound ? pieces : static_cast<int32_t>(bound < 1 ? 1 : bound);
  const size_t state = static_cast<size_t>(pkv::piece_floats(head_dim, group)) * sizeof(float);
  const size_t pair_count = static_cast<size_t>(num_seqs) * num_kv_heads;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t from = at;
    at += (bytes + 255) & ~size_t(255);
    return from;
  };
  take(pkv::workspace_prefix_bytes(num_seqs));
  plan->pairs = take(pair_count * 8);
  plan->shared = take(static_cast<size_t>(num_seqs) * 4);
  plan->plan_ok = take(4);
  plan->records = take(pair_count * 8);
  plan->whole = take(pair_count * state);
  plan->pieces = take(static_cast<size_t>(plan->parts) * 2 * state);
  plan->prefix = take(static_cast<size_t>(ctas) * 256 * (head_dim + 2) * sizeof(float));
  plan->bytes = at;
  return PKV_OK;
}
}  // namespace

pkv_status pkv_prefix_decode_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                            int32_t head_dim, int32_t max_blocks_per_seq, int32_t num_groups,
                                            size_t* bytes) {
  if (!bytes) return fail(PKV_ERR_INVALID_ARGUMENT, "bytes is null");
  PrefixPlan plan;
  if (pkv_status st = plan_prefix_decode(num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, num_groups,
                                         1, &plan);
      st != PKV_OK)
    return st;
  *bytes = plan.bytes;
  return ok();
}

pkv_status pkv_paged_prefix_decode_attention(const void* q, const void* k_cache, const void* v_cache,
                                             const int32_t* block_tables, int32_t max_blocks_per_seq,
                                             const int32_t* context_lens, const int32_t* group_start,
                                             const int32_t* prefix_lens, int32_t num_groups, int32_t num_seqs,
                                             int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                             int64_t num_blocks, int32_t block_size, float scale, void* out,
                                             void* workspace, size_t workspace_bytes, pkv_stream_t stream) {
  if (pkv_status st = check_shapes(num_seqs, num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq);
      st != PKV_OK)
    return st;
  if (block_size != PKV_BLOCK_SIZE)
    return fail(PKV_ERR_UNSUPPORTED, "block_size must be %d (got %d)", PKV_BLOCK_SIZE, block_size);
  if (num_blocks <= 0 || num_blocks > (int64_t{1} << 40) ||
      num_blocks * num_kv_heads * PKV_BLOCK_SIZE >= (int64_t{1} << 31))
    return fail(PKV_ERR_UNSUPPORTED, "num_blocks * num_kv_heads * 16 must be in (0, 2^31) (got %lld blocks)",
                (long long)num_blocks);
  if (!std::isfinite(scale) || scale <= 0.f) return fail(PKV_ERR_INVALID_ARGUMENT, "scale must be finite and positive");
  if (num_seqs > PKV_MAX_SEQS)
    return fail(PKV_ERR_UNSUPPORTED, "num_seqs %d exceeds PKV_MAX_SEQS (%d)", num_seqs, PKV_MAX_SEQS);
  if (num_groups < 0 || num_groups > PKV_MAX_SEQS)
    return fail(PKV_ERR_INVALID_ARGUMENT, "num_groups must be in [0, %d] (got %d)", PKV_MAX_SEQS, num_groups);
  if (num_seqs == 0) return ok();
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out ||
      (num_groups > 0 && (!group_start || !prefix_lens)))
    return fail(PKV_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || !aligned16(workspace) ||
      ((reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(context_lens) |
        reinterpret_cast<uintptr_t>(group_start) | reinterpret_cast<uintptr_t>(prefix_lens)) &
       3u))
    return fail(PKV_ERR_INVALID_ARGUMENT, "q, caches, out and workspace must be 16-byte aligned");
  PrefixPlan plan;
  if (pkv_status st = plan_prefix_decode(num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, num_groups,
                                         num_seqs, &plan);
      st != PKV_OK)
    return st;
  if (workspace_bytes < plan.bytes || (!workspace && plan.bytes))
    return fail(PKV_ERR_INVALID_ARGUMENT, "workspace too small: %zu bytes given, %zu needed",
                workspace ? workspace_bytes : size_t{0}, plan.bytes);
  unsigned* err = nullptr;
  if (pkv_status st = device_state(&err, nullptr); st != PKV_OK) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int group = num_q_heads / num_kv_heads;
  pkv::DecodeViewParams p{};
  p.q = q;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.out = out;
  p.err = err;
  p.num_blocks = num_blocks;
  p.num_seqs = num_seqs;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.qscale = scale * 1.4426950408889634f;
  p.group_start = group_start;
  p.prefix_lens = prefix_lens;
  p.num_groups = num_groups;
  if (plan.cluster) {
    const cudaError_t e = pkv::launch_prefix_cluster(p, head_dim, group, plan.cluster, s);
    if (e != cudaSuccess) return cuda_fail(e, "prefix decode launch");
    g_launches.fetch_add(1);
    return ok();
  }
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  pkv::PrefillParams f{};
  f.q = q;
  f.k_cache = k_cache;
  f.v_cache = v_cache;
  f.block_tables = block_tables;
  f.context_lens = context_lens;
  f.out = out;
  f.err = err;
  f.num_blocks = num_blocks;
  f.num_seqs = num_seqs;
  f.num_q_heads = num_q_heads;
  f.num_kv_heads = num_kv_heads;
  f.max_blocks_per_seq = max_blocks_per_seq;
  f.max_query_len = 1;
  f.scale = scale;
  f.ws = reinterpret_cast<float*>(ws + plan.prefix);
  f.group_start = group_start;
  f.prefix_lens = prefix_lens;
  f.num_groups = num_groups;
  f.shared_ctas = plan.ctas;
  f.num_sms = plan.sms;
  f.ws_records = reinterpret_cast<int2*>(ws + plan.records);
  f.ws_plan_ok = reinterpret_cast<int32_t*>(ws + plan.plan_ok);
  cudaError_t e = pkv::launch_shared_prefix(f, head_dim, group, s);
  if (e != cudaSuccess) return cuda_fail(e, "shared prefix launch");
  p.ws_prefix = reinterpret_cast<int32_t*>(ws);
  p.ws_pairs = reinterpret_cast<int32_t*>(ws + plan.pairs);
  p.ws_pieces = reinterpret_cast<float*>(ws + plan.pieces);
  p.num_partitions = plan.parts;
  p.min_piece_blocks = kMinPieceBlocks;
  p.ws_shared = reinterpret_cast<int32_t*>(ws + plan.shared);
  p.ws_whole = reinterpret_cast<float*>(ws + plan.whole);
  p.ws_plan_ok = f.ws_plan_ok;
  p.ws_records = f.ws_records;
  p.ws_prefix_o = f.ws;
  p.ws_prefix_ml = reinterpret_cast<const float2*>(f.ws + static_cast<size_t>(plan.ctas) * 256 * head_dim);
  if ((e = pkv::launch_tail_partition(p, head_dim, group, s)) != cudaSuccess) return cuda_fail(e, "tail partition launch");
  if ((e = pkv::launch_prefix_join(p, head_dim, group, s)) != cudaSuccess) return cuda_fail(e, "prefix join launch");
  g_launches.fetch_add(3);
  return ok();
}

pkv_status pkv_get_and_clear_device_error(uint32_t* bits, pkv_stream_t stream) {
  if (!bits) return fail(PKV_ERR_INVALID_ARGUMENT, "bits is null");
  unsigned* err = nullptr;
  if (pkv_status st = device_state(&err, nullptr); st != PKV_OK) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
  unsigned host = 0;
  if ((e = cudaMemcpyAsync(&host, err, sizeof host, cudaMemcpyDeviceToHost, s)) != cudaSuccess)
    return cuda_fail(e, "reading the device error word");
  if ((e = cudaMemsetAsync(err, 0, sizeof(unsigned), s)) != cudaSuccess)
    return cuda_fail(e, "clearing the device error word");
  if ((e = cudaStreamSynchronize(s)) != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
  *bits = host;
  return ok();
}

}  // extern "C"
