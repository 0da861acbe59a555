// Single-token paged attention over the 8-bit cache (paged_attention_decode_quant).
//
// Math: with key codes kc_t, value codes vc_t (e4m3) and the rows' powers of two
// 2^ke_t, 2^ve_t:  s_t = scale 2^ke_t (q . kc_t),  out = sum_t softmax_t(s) 2^ve_t vc_t.
//
// One CTA per (KV head, sequence): four warps take the tokens in turn, each with
// a running maximum and sum, and are joined in shared memory at the end.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "internal.h"
#include "pkv.h"
#include "ptx.cuh"
#include "quant.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxGroup = 16;
constexpr float kLog2e = 1.4426950408889634f;

struct Params {
  const __nv_bfloat16 *q;
  const uint8_t *k_codes, *v_codes, *k_exps, *v_exps;
  const int32_t *block_tables, *seq_lens;
  __nv_bfloat16 *out;
  int32_t *status;
  int max_blocks, max_len, num_q_heads, num_kv_heads, group, num_blocks, block_size;
  float scale_log2;
};

__device__ __forceinline__ float code_value(uint8_t c) {
  const uint32_t h = quant::e4m3x2_to_f16x2(c);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xFFFFu)));
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) decode_simple(const Params p) {
  constexpr int PER = D / 32;
  __shared__ float so[kWarps][D], sm[kWarps], sl[kWarps];
  const int h = blockIdx.x, seq = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_launch_dependents();
  grid_dependency_wait();
  int L = p.seq_lens[seq];
  const long long cap_tbl = static_cast<long long>(p.max_blocks) * p.block_size;
  const int cap = static_cast<int>(cap_tbl < p.max_len ? cap_tbl : p.max_len);
  if (L < 0 || L > cap) {
    if (h == 0 && threadIdx.x == 0 && p.status) atomicOr(p.status, PKV_STATUS_BAD_LEN);
    L = L < 0 ? 0 : cap;
  }
  for (int g = 0; g < p.group; ++g) {
    const size_t row = (static_cast<size_t>(seq) * p.num_q_heads + h * p.group + g) * D;
    float q[PER], o[PER], m = -INFINITY, l = 0.f;
    for (int i = 0; i < PER; ++i) q[i] = __bfloat162float(p.q[row + lane * PER + i]), o[i] = 0.f;
    for (int t = warp; t < L; t += kWarps) {
      const int b = p.block_tables[static_cast<size_t>(seq) * p.max_blocks + t / p.block_size];
      float s = 0.f, v[PER];
      for (int i = 0; i < PER; ++i) v[i] = 0.f;
      if (b >= 0 && b < p.num_blocks) {
        const size_t r = (static_cast<size_t>(b) * p.num_kv_heads + h) * p.block_size + t % p.block_size;
        const float kf = quant::pow2i(quant::clamp_exp(p.k_exps[r])), vf = quant::pow2i(quant::clamp_exp(p.v_exps[r]));
        for (int i = 0; i < PER; ++i) {
          s += q[i] * code_value(p.k_codes[r * D + lane * PER + i]);
          v[i] = code_value(p.v_codes[r * D + lane * PER + i]) * vf;
        }
        for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= kf * p.scale_log2;
      } else if (lane == 0 && p.status) {
        atomicOr(p.status, PKV_STATUS_BAD_BLOCK);
      }
      const float mn = fmaxf(m, s), a = m == -INFINITY ? 0.f : exp2f(m - mn), w = exp2f(s - mn);
      l = l * a + w;
      for (int i = 0; i < PER; ++i) o[i] = o[i] * a + w * v[i];
      m = mn;
    }
    for (int i = 0; i < PER; ++i) so[warp][lane * PER + i] = o[i];
    if (lane == 0) sm[warp] = m, sl[warp] = l;
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += kWarps * 32) {
      float M = -INFINITY, lt = 0.f, ot = 0.f;
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w]);
      for (int w = 0; w < kWarps; ++w) {
        const float f = sl[w] == 0.f ? 0.f : exp2f(sm[w] - M);
        lt += sl[w] * f;
        ot += so[w][i] * f;
      }
      p.out[row + i] = __float2bfloat16_rn(L > 0 ? ot / lt : 0.f);
    }
    __syncthreads();
  }
}

int check_decode(const void *q, const void *k_codes, const void *v_codes, const void *k_exps, const void *v_exps,
                 const int32_t *block_tables, int max_blocks_per_seq, const int32_t *seq_lens, int num_seqs,
                 int max_seq_len, int num_q_heads, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                 float scale, const void *out) {
  if (num_seqs < 0 || max_blocks_per_seq < 0 || max_seq_len < 0 || num_q_heads < 1 || num_kv_heads < 1 ||
      num_blocks < 0 || !std::isfinite(scale))
    return PKV_ERR_ARG;
  if (num_q_heads % num_kv_heads != 0) return PKV_ERR_ARG;
  if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (block_size != 16 && block_size != 32 && block_size != 64 && block_size != 128) return PKV_ERR_UNSUPPORTED;
  if (num_q_heads / num_kv_heads > kMaxGroup) return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PKV_OK;
  if (num_seqs > 65535 || num_kv_heads > 65535) return PKV_ERR_UNSUPPORTED;
  if (!q || !k_codes || !v_codes || !k_exps || !v_exps || !block_tables || !seq_lens || !out || num_blocks == 0)
    return PKV_ERR_ARG;
  if (!aligned16(q) || !aligned16(k_codes) || !aligned16(v_codes) || !aligned16(k_exps) || !aligned16(v_exps) ||
      !aligned16(out) || (reinterpret_cast<uintptr_t>(block_tables) & 3u) ||
      (reinterpret_cast<uintptr_t>(seq_lens) & 3u))
    return PKV_ERR_ARG;
  const long long rows = static_cast<long long>(num_blocks) * num_kv_heads * block_size;
  if (rows + block_size >= (1ll << 31)) return PKV_ERR_UNSUPPORTED;
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

extern "C" {

size_t paged_attention_decode_quant_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                                   int max_seq_len) {
  return 0;
}

int paged_attention_decode_quant(const pkv_bf16 *q, const uint8_t *k_codes, const uint8_t *v_codes,
                                 const uint8_t *k_exps, const uint8_t *v_exps, const int32_t *block_tables,
                                 int max_blocks_per_seq, const int32_t *seq_lens, int num_seqs, int max_seq_len,
                                 int num_q_heads, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                                 float scale, pkv_bf16 *out, void *workspace, size_t workspace_bytes,
                                 int32_t *d_status, void *stream) {
  const int rc = pkv::check_decode(q, k_codes, v_codes, k_exps, v_exps, block_tables, max_blocks_per_seq, seq_lens,
                                   num_seqs, max_seq_len, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                                   scale, out);
  if (rc != PKV_OK || num_seqs == 0) return rc;
  pkv::Params p{};
  p.q = reinterpret_cast<const __nv_bfloat16 *>(q);
  p.k_codes = k_codes;
  p.v_codes = v_codes;
  p.k_exps = k_exps;
  p.v_exps = v_exps;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.out = reinterpret_cast<__nv_bfloat16 *>(out);
  p.status = d_status;
  p.max_blocks = max_blocks_per_seq;
  p.max_len = max_seq_len;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = num_q_heads / num_kv_heads;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.scale_log2 = scale * pkv::kLog2e;
  const dim3 grid(num_kv_heads, num_seqs);
  if (head_dim == 128) pkv::decode_simple<128><<<grid, pkv::kWarps * 32, 0, pkv::as_stream(stream)>>>(p);
  else pkv::decode_simple<64><<<grid, pkv::kWarps * 32, 0, pkv::as_stream(stream)>>>(p);
  return pkv::check_launch();
}

}  // extern "C"
