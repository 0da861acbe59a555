// What the windowed and the tree attention's translation units share.
#pragma once

#include <cstddef>
#include <cstdint>

#include "pkv.h"

namespace pkv {
namespace spans {

constexpr int kMaxNodes = 64;    // of a tree: a node's mask is one 64-bit word
constexpr int kMaxSeqs = 1024;   // of a call with query chunks or trees

// The arguments of paged_attention_window and paged_attention_tree.
struct Call {
  const pkv_bf16 *q, *k_cache, *v_cache;
  const int32_t *block_tables;
  int max_blocks;
  const int32_t *seq_lens, *q_start;  // q_start NULL: one row per sequence
  const uint64_t *mask;               // tree; NULL: window
  int num_seqs, total_q, max_seq_len;
  int window, sinks;                  // without a mask
  int max_nodes;                      // with one
  int num_q_heads, num_kv_heads, head_dim, block_size, num_blocks;
  float scale;
  pkv_bf16 *out;
  void *workspace;
  size_t workspace_bytes;
  int32_t *status;
  void *stream;
};

// Query chunks and trees (spans_tc.cu).  The sizes in `a` are valid; its pointers
// and stream are used by tc_launch only.
size_t tc_workspace_size(const Call &a);
int tc_launch(const Call &a);

// Single tokens, one per sequence (spans_step.cu).
size_t step_workspace_size(const Call &a);
int step_launch(const Call &a);

}  // namespace spans
}  // namespace pkv
