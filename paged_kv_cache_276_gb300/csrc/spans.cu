// Attention over part of a sequence's cached tokens: a sliding window with first
// tokens that stay visible (paged_attention_window), and a tree of drafted
// tokens (paged_attention_tree).
//
// The calls' checks; chunks and trees go to spans_tc.cu, single tokens to spans_step.cu.
#include <algorithm>
#include <cmath>

#include "internal.h"
#include "pkv.h"
#include "spans.cuh"

namespace pkv {
namespace spans {
namespace {

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Sizes and pointers; *work: there is something to do.
int check(const Call &a, bool *work) {
  *work = false;
  const bool single = !a.q_start;
  if (a.num_seqs < 0 || a.total_q < 0 || a.max_blocks < 0 || a.max_seq_len < 0 || a.num_q_heads < 1 ||
      a.num_kv_heads < 1 || a.num_blocks < 0 || !std::isfinite(a.scale) || a.num_q_heads % a.num_kv_heads != 0)
    return PKV_ERR_ARG;
  if ((a.head_dim != 64 && a.head_dim != 128) || a.num_q_heads / a.num_kv_heads > 16) return PKV_ERR_UNSUPPORTED;
  if (a.block_size != 16 && a.block_size != 32 && a.block_size != 64 && a.block_size != 128)
    return PKV_ERR_UNSUPPORTED;
  if (a.num_seqs > (single ? 65535 : kMaxSeqs)) return PKV_ERR_UNSUPPORTED;
  constexpr long long kLimit = (1ll << 31) - 512;
  if (static_cast<long long>(a.max_blocks) * a.block_size >= kLimit ||
      static_cast<long long>(a.num_blocks) * a.num_kv_heads * a.block_size >= kLimit)
    return PKV_ERR_UNSUPPORTED;
  if (a.num_seqs == 0 || a.total_q == 0) return PKV_OK;
  if (!a.q || !a.k_cache || !a.v_cache || !a.block_tables || !a.seq_lens || !a.out || a.num_blocks == 0)
    return PKV_ERR_ARG;
  if (!aligned16(a.q) || !aligned16(a.k_cache) || !aligned16(a.v_cache) || !aligned16(a.out) ||
      !aligned4(a.block_tables) || !aligned4(a.seq_lens) || !aligned4(a.q_start))
    return PKV_ERR_ARG;
  *work = true;
  return PKV_OK;
}

// The sizes that both calls' workspaces depend on; false: not sizes of a call that
// would run.
bool sizes(Call *a, int num_seqs, int total_q, int num_q_heads, int num_kv_heads, int head_dim, int max_seq_len) {
  a->num_seqs = num_seqs;
  a->total_q = total_q;
  a->num_q_heads = num_q_heads;
  a->num_kv_heads = num_kv_heads;
  a->head_dim = head_dim;
  a->max_seq_len = max_seq_len;
  return num_seqs > 0 && total_q > 0 && num_q_heads > 0 && num_kv_heads > 0 && num_q_heads % num_kv_heads == 0 &&
         num_q_heads / num_kv_heads <= 16 && (head_dim == 64 || head_dim == 128) && max_seq_len >= 0;
}

int run(const Call &a) {
  bool work;
  const int rc = check(a, &work);
  if (rc != PKV_OK || !work) return rc;
  return a.q_start ? tc_launch(a) : step_launch(a);
}

}  // namespace
}  // namespace spans
}  // namespace pkv

extern "C" {

size_t paged_attention_window_workspace_size(int num_seqs, int total_q, int num_q_heads, int num_kv_heads,
                                             int head_dim, int max_seq_len, int window, int sinks) {
  pkv::spans::Call a{};
  if (window < 1 || sinks < 0 ||
      !pkv::spans::sizes(&a, num_seqs, total_q, num_q_heads, num_kv_heads, head_dim, max_seq_len))
    return 0;
  a.window = window;
  a.sinks = sinks;
  return std::max(pkv::spans::step_workspace_size(a), pkv::spans::tc_workspace_size(a));
}

size_t paged_attention_tree_workspace_size(int num_seqs, int total_q, int max_nodes, int num_q_heads,
                                           int num_kv_heads, int head_dim, int max_seq_len) {
  pkv::spans::Call a{};
  if (max_nodes < 1 || max_nodes > pkv::spans::kMaxNodes ||
      !pkv::spans::sizes(&a, num_seqs, total_q, num_q_heads, num_kv_heads, head_dim, max_seq_len))
    return 0;
  static const uint64_t some = 0;  // a tree's call is one with a mask
  a.mask = &some;
  a.max_nodes = max_nodes;
  return pkv::spans::tc_workspace_size(a);
}

int paged_attention_window(const pkv_bf16 *q, const pkv_bf16 *k_cache, const pkv_bf16 *v_cache,
                           const int32_t *block_tables, int max_blocks_per_seq, const int32_t *seq_lens,
                           const int32_t *q_start, int num_seqs, int total_q, int max_seq_len, int window, int sinks,
                           int num_q_heads, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                           float scale, pkv_bf16 *out, void *workspace, size_t workspace_bytes, int32_t *d_status,
                           void *stream) {
  if (window < 1 || sinks < 0 || (!q_start && total_q != num_seqs)) return PKV_ERR_ARG;
  return pkv::spans::run({q, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens, q_start, nullptr, num_seqs,
                          total_q, max_seq_len, window, sinks, 0, num_q_heads, num_kv_heads, head_dim, block_size,
                          num_blocks, scale, out, workspace, workspace_bytes, d_status, stream});
}

int paged_attention_tree(const pkv_bf16 *q, const pkv_bf16 *k_cache, const pkv_bf16 *v_cache,
                         const int32_t *block_tables, int max_blocks_per_seq, const int32_t *seq_lens,
                         const int32_t *q_start, const uint64_t *tree_mask, int num_seqs, int total_q, int max_nodes,
                         int max_seq_len, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                         int num_blocks, float scale, pkv_bf16 *out, void *workspace, size_t workspace_bytes,
                         int32_t *d_status, void *stream) {
  if (max_nodes < 1 || max_nodes > pkv::spans::kMaxNodes) return PKV_ERR_ARG;
  if (num_seqs > 0 && total_q > 0 && (!q_start || !tree_mask || (reinterpret_cast<uintptr_t>(tree_mask) & 7u)))
    return PKV_ERR_ARG;
  return pkv::spans::run({q, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens, q_start, tree_mask,
                          num_seqs, total_q, max_seq_len, 0, 0, max_nodes, num_q_heads, num_kv_heads, head_dim,
                          block_size, num_blocks, scale, out, workspace, workspace_bytes, d_status, stream});
}

}  // extern "C"
