// Attention over part of a sequence's cached tokens: a sliding window with first
// tokens that stay visible (paged_attention_window), and a tree of drafted
// tokens (paged_attention_tree).
//
// Math: out = softmax(scale * q K^T) V over the keys that a row sees, with the
// running maximum and sum of the online softmax.
//
// One warp per (query row, query head), a lane holding D / 32 values of a row:
// a key costs a dot product over the lanes and an update of the running sums.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "internal.h"
#include "launch.cuh"
#include "pkv.h"
#include "ptx.cuh"
#include "spans.cuh"

namespace pkv {
namespace spans {
namespace {

struct SpanParams {
  const __nv_bfloat16 *q, *k_cache, *v_cache;
  const int32_t *block_tables, *seq_lens, *q_start;
  const uint64_t *mask;  // tree; NULL: window
  __nv_bfloat16 *out;
  int32_t *status;
  int num_seqs, total_q, max_blocks, max_len, num_q_heads, num_kv_heads, group, num_blocks, block_size;
  int window, sinks, max_nodes;
  float scale_log2;
};

// The sequence that owns a row (-1: none), and its chunk's first row and length.
__device__ int owner(const SpanParams &p, int row, int *first, int *count) {
  if (!p.q_start) {
    *first = row;
    *count = 1;
    return row;
  }
  int lo = 0, hi = p.num_seqs;  // the last sequence whose first row is at most `row`
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.q_start[mid] <= row) lo = mid; else hi = mid;
  }
  const int a = p.q_start[lo], b = p.q_start[lo + 1];
  *first = a;
  *count = b - a;
  if (a < 0 || b < a || b > p.total_q || row < a || row >= b) return -1;
  return p.mask && b - a > p.max_nodes ? -1 : lo;
}

template <int D>
__global__ void __launch_bounds__(128) spans_kernel(const SpanParams p) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const long long w = blockIdx.x * 4ll + (threadIdx.x >> 5);
  if (blockIdx.x == 0 && p.status) {
    const long long cap_tbl = static_cast<long long>(p.max_blocks) * p.block_size;
    for (int i = threadIdx.x; i < p.num_seqs; i += blockDim.x) {
      const int L = p.seq_lens[i];
      if (L < 0 || L > p.max_len || L > cap_tbl) atomicOr(p.status, PKV_STATUS_BAD_LEN);
      if (!p.q_start) continue;
      const int a = p.q_start[i], b = p.q_start[i + 1];
      if (a < 0 || b < a || b > p.total_q || (p.mask && b - a > p.max_nodes)) atomicOr(p.status, PKV_STATUS_BAD_QSTART);
    }
  }
  if (w >= static_cast<long long>(p.total_q) * p.num_q_heads) return;
  const int row = static_cast<int>(w / p.num_q_heads), head = static_cast<int>(w % p.num_q_heads);
  int first, count;
  const int seq = owner(p, row, &first, &count);
  if (seq < 0) return;
  const long long cap = min(static_cast<long long>(p.max_blocks) * p.block_size, static_cast<long long>(p.max_len));
  const int L = static_cast<int>(max(0ll, min(cap, static_cast<long long>(p.seq_lens[seq]))));
  const int ctx = L - count, pos = ctx + row - first;
  constexpr int PER = D / 32;
  float q[PER], o[PER], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    q[i] = __bfloat162float(p.q[w * D + lane * PER + i]);
    o[i] = 0.f;
  }
  const uint64_t word = p.mask ? p.mask[row] : 0;
  const int end = p.mask ? L : pos + 1;
  const int lo = p.mask ? 0 : max(0, pos - p.window + 1);
  for (int t = 0; t < end; ++t) {
    if (p.mask) {
      if (t >= ctx && !((word >> (t - ctx)) & 1)) continue;
    } else if (t < lo && t >= p.sinks) {
      t = lo - 1;
      continue;
    }
    const int b = p.block_tables[static_cast<size_t>(seq) * p.max_blocks + t / p.block_size];
    const bool ok = b >= 0 && b < p.num_blocks;
    if (!ok && lane == 0 && p.status) atomicOr(p.status, PKV_STATUS_BAD_BLOCK);
    const size_t at = ((static_cast<size_t>(ok ? b : 0) * p.num_kv_heads + head / p.group) * p.block_size +
                       t % p.block_size) * D + lane * PER;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) s += q[i] * (ok ? __bfloat162float(p.k_cache[at + i]) : 0.f);
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.scale_log2;
    if (s > m) {
      const float f = m == -INFINITY ? 0.f : exp2f(m - s);
      l *= f;
#pragma unroll
      for (int i = 0; i < PER; ++i) o[i] *= f;
      m = s;
    }
    const float e = s == -INFINITY ? 0.f : exp2f(s - (m == -INFINITY ? 0.f : m));
    l += e;
#pragma unroll
    for (int i = 0; i < PER; ++i) o[i] += e * (ok ? __bfloat162float(p.v_cache[at + i]) : 0.f);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < PER; ++i) p.out[w * D + lane * PER + i] = __float2bfloat16_rn(o[i] * inv);
}

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

int launch(const Call &a, SpanParams p) {
  p.q = reinterpret_cast<const __nv_bfloat16 *>(a.q);
  p.k_cache = reinterpret_cast<const __nv_bfloat16 *>(a.k_cache);
  p.v_cache = reinterpret_cast<const __nv_bfloat16 *>(a.v_cache);
  p.block_tables = a.block_tables;
  p.seq_lens = a.seq_lens;
  p.q_start = a.q_start;
  p.out = reinterpret_cast<__nv_bfloat16 *>(a.out);
  p.status = a.status;
  p.num_seqs = a.num_seqs;
  p.total_q = a.total_q;
  p.max_blocks = a.max_blocks;
  p.max_len = a.max_seq_len;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.group = a.num_q_heads / a.num_kv_heads;
  p.num_blocks = a.num_blocks;
  p.block_size = a.block_size;
  p.window = a.window;
  p.sinks = a.sinks;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  const long long grid = (static_cast<long long>(a.total_q) * a.num_q_heads + 3) / 4;
  if (grid > 0x7fffffffll) return PKV_ERR_UNSUPPORTED;
  const cudaError_t e = a.head_dim == 64 ? launch_overlapped(spans_kernel<64>, static_cast<unsigned>(grid), 128, 0,
                                                             as_stream(a.stream), p)
                                         : launch_overlapped(spans_kernel<128>, static_cast<unsigned>(grid), 128, 0,
                                                             as_stream(a.stream), p);
  return e == cudaSuccess ? PKV_OK : (set_cuda_error(e), PKV_ERR_CUDA);
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
  return a.q_start ? tc_launch(a) : launch(a, SpanParams{});
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
  return pkv::spans::tc_workspace_size(a);
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
