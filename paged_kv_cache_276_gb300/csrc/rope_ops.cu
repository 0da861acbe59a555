// Rotary append: rotate the queries and keys of new tokens to their positions
// and store keys and values into their cache slots, bf16 (pkv_write_rope) or
// quantised to 8 bits on the way (pkv_write_rope_quant).
//
// Math: a rotated pair (a, b) of a row at position p becomes
//     (a c - b s, b c + a s),  c = cos(p f), s = sin(p f)
// with c and s of each pair read from a table.  Each product and the sum are
// rounded to fp32 (no contraction into an FMA), then the result once to bf16 or
// e4m3: the value is the elementary formula's, bit for bit.
//
// Data movement with three operations per value, bound by HBM: per token every
// query row is read and written, every key and value row read and stored.  A
// group of W lanes takes kRows query heads, key heads or value heads of one token.
// A lane holds 16 values of a
// row in two 16-byte chunks, each chunk contiguous over the lanes: values 8 i
// and R/2 + 8 i of the rotated part (so that a pair of either style lies in one
// lane, and a group's accesses are whole lines), or two such halves of the rest.
// The lane's cosines and sines are read once for its kRows rows, whose loads are
// all in flight together.
// Measured at 32768 tokens, 32 query and 8 KV heads of 128, rows of a fused
// projection: 119.6 us (6.9 TB/s of what is read and written, a plain copy 6.78; an eighth
// of the writes is still in L2 at the end); 8192 tokens, 64 and 8 heads, into the 8-bit
// cache: 53.4 us (6.05 TB/s; the conversions leave the loads of a warp waiting); the 256
// tokens of a decode step 3.4 us, a launch and two dependent loads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "internal.h"
#include "launch.cuh"
#include "pkv.h"
#include "ptx.cuh"
#include "quant.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
// Rows of one token per lane group, and CTAs per SM that the registers are held to
// (85 a thread).  32768 tokens, 32 + 8 + 8 heads of 128: 119.6 us; two rows and four
// CTAs 128.5, one row 171.
constexpr int kRows = 4;
constexpr int kCtas = 3;
constexpr int kMaxHeadDim = 512;  // 32 lanes x 16 values

struct RopeParams {
  const uint4 *q, *k, *v;
  uint4 *q_out;
  int64_t q_stride, k_stride, v_stride, q_out_stride;  // 16-byte chunks between tokens
  const int64_t *positions, *slots;
  const float *table;   // [max_positions][rot_dim]: cosines, then sines
  int64_t num_slots, tasks;
  int32_t *status;
  int max_positions, rot_dim, head_dim, num_q_heads, num_kv_heads, block_size;
  int q_groups, kv_groups, groups;  // lane groups of a token: for queries, for keys (and for values), together
  int narrow;  // tasks and num_slots fit 32 bits: divide in 32 bits
  // one of the two caches
  uint4 *k_cache, *v_cache;
  uint2 *k_codes, *v_codes;
  uint8_t *k_exps, *v_exps;
};

__device__ __forceinline__ void widen(const uint4 &x, float (&f)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 narrow(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ void rotate_pair(float &a, float &b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
}

// Half split: pairs (x0[i], x1[i]).  Pairs: (x[2i], x[2i + 1]); c[0..3] and
// s[0..3] belong to x0's pairs, c[4..7] and s[4..7] to x1's.
template <bool PAIRS>
__device__ __forceinline__ void rotate16(float (&x0)[8], float (&x1)[8], const float (&c)[8], const float (&s)[8]) {
  if constexpr (PAIRS) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      rotate_pair(x0[2 * i], x0[2 * i + 1], c[i], s[i]);
      rotate_pair(x1[2 * i], x1[2 * i + 1], c[4 + i], s[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) rotate_pair(x0[i], x1[i], c[i], s[i]);
  }
}

__device__ __forceinline__ void load4(const float *p, float *f) {
  const float4 x = *reinterpret_cast<const float4 *>(p);
  f[0] = x.x;
  f[1] = x.y;
  f[2] = x.z;
  f[3] = x.w;
}

// |x| as bits, 0 where x is not finite.
__device__ __forceinline__ uint32_t finite_magnitude(float x) {
  const uint32_t m = __float_as_uint(x) & 0x7FFFFFFFu;
  return m >= 0x7F800000u ? 0u : m;
}

// Exponent of a row whose largest finite magnitude has the fp32 bits `a`: the
// smallest e with a <= 448 * 2^e = 1.75 * 2^(e + 8), clamped (quant::row_exponent
// for bf16 magnitudes; a rotated value is not one).
__device__ __forceinline__ int row_exponent(uint32_t a) {
  const int e = static_cast<int>(a >> 23) - 127 - 8 + ((a & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(quant::kExpMin, min(quant::kExpMax, e));
}

__device__ __forceinline__ uint2 encode8(const float (&f)[8], float inv) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // an infinity becomes NaN (the conversion would hold it at 448)
    const float a = isinf(f[2 * i]) ? __uint_as_float(0x7FFFFFFFu) : f[2 * i] * inv;
    const float b = isinf(f[2 * i + 1]) ? __uint_as_float(0x7FFFFFFFu) : f[2 * i + 1] * inv;
    h[i] = quant::to_e4m3x2(a, b);
  }
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

template <int W, bool PAIRS, bool QUANT>
__global__ void __launch_bounds__(kThreads, kCtas) rope_kernel(const RopeParams p) {
  // the grid queued behind this one may become resident now (it waits for this
  // grid's writes before it reads them)
  grid_launch_dependents();
  grid_dependency_wait();  // the rows may come from the kernel launched just before
  const int lane = threadIdx.x % W;
  const int64_t task = static_cast<int64_t>(blockIdx.x) * (kThreads / W) + threadIdx.x / W;
  const bool real = task < p.tasks && lane < p.head_dim / 16;
  int64_t t = 0, slot = -1, at = 0;
  int g = 0;
  if (real) {
    if (p.narrow) t = static_cast<uint32_t>(task) / static_cast<uint32_t>(p.groups);
    else t = task / p.groups;
    g = static_cast<int>(task - t * p.groups);
    at = p.positions[t];
    slot = p.slots[t];
  }
  // the group's rows: kRows query heads, key heads or value heads from row0 on
  const bool is_q = g < p.q_groups, is_v = g >= p.q_groups + p.kv_groups;
  const int row0 = (is_q ? g : g - p.q_groups - (is_v ? p.kv_groups : 0)) * kRows;
  const int rows = (is_q ? p.num_q_heads : p.num_kv_heads) - row0;
  // this lane's two chunks (of 8 values) of a row, and its cosines and sines
  const int rot16 = p.rot_dim / 16, rest = p.head_dim - p.rot_dim;
  const bool turns = lane < rot16 && !is_v;
  const int c0 = lane < rot16 ? lane : p.rot_dim / 8 + (lane - rot16);
  const int apart = (lane < rot16 ? p.rot_dim : rest) / 16;
  const int chunks = p.head_dim / 8;
  // (the queries' loads wait for nothing; keys and values are read where they are stored)
  uint4 a[kRows], b[kRows];
  {
    const uint4 *src = (is_q   ? p.q + t * p.q_stride
                        : is_v ? p.v + t * p.v_stride
                               : p.k + t * p.k_stride) +
                       static_cast<int64_t>(row0) * chunks + c0;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      a[r] = b[r] = make_uint4(0u, 0u, 0u, 0u);
      if (real && r < rows && (is_q || slot >= 0)) {
        a[r] = src[r * chunks];
        b[r] = src[r * chunks + apart];
      }
    }
  }
  bool live = real && at >= 0 && at < p.max_positions;
  if (real && lane == 0 && g == 0 && p.status) {
    if (!live) atomicOr(p.status, PKV_STATUS_BAD_POS);
    else if (slot >= p.num_slots) atomicOr(p.status, PKV_STATUS_BAD_SLOT);
  }
  if (!is_q) live = live && slot >= 0 && slot < p.num_slots;
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;
  if (live && turns) {
    const float *cs = p.table + at * p.rot_dim, *sn = cs + p.rot_dim / 2;
    const int i0 = PAIRS ? 4 * lane : 8 * lane, i1 = PAIRS ? p.rot_dim / 4 + 4 * lane : 8 * lane + 4;
    load4(cs + i0, c);
    load4(cs + i1, c + 4);
    load4(sn + i0, s);
    load4(sn + i1, s + 4);
  }
  // where the first row goes, in rows of the cache or chunks of q_out, and rows between heads
  int64_t dst = 0;
  if (is_q) {
    dst = t * p.q_out_stride + static_cast<int64_t>(row0) * chunks + c0;
  } else if (live) {
    int64_t blk;
    if (p.narrow) blk = static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.block_size);
    else blk = slot / p.block_size;
    dst = (blk * p.num_kv_heads + row0) * p.block_size + (slot - blk * p.block_size);
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const bool use = live && r < rows;
    const int64_t cache_row = dst + static_cast<int64_t>(r) * p.block_size;
    if (!QUANT || is_q) {  // (queries and keys alike in the bf16 cache; a warp may hold groups of both kinds)
      if (use) {
        uint4 *to = is_q ? p.q_out + dst + r * chunks : (is_v ? p.v_cache : p.k_cache) + cache_row * chunks + c0;
        if (turns) {
          float x0[8], x1[8];
          widen(a[r], x0);
          widen(b[r], x1);
          rotate16<PAIRS>(x0, x1, c, s);
          a[r] = narrow(x0);
          b[r] = narrow(x1);
        }
        to[0] = a[r];
        to[apart] = b[r];
      }
    }
    if constexpr (QUANT) {
      // the row's largest magnitude, over its lanes: every lane of the warp takes part
      if (!__any_sync(0xffffffffu, use && !is_q)) continue;
      float x0[8], x1[8];
      widen(a[r], x0);
      widen(b[r], x1);
      if (turns && !is_q) rotate16<PAIRS>(x0, x1, c, s);
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, max(finite_magnitude(x0[i]), finite_magnitude(x1[i])));
#pragma unroll
      for (int o = W / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int e = row_exponent(top);
      if (use && !is_q) {
        uint2 *to = (is_v ? p.v_codes : p.k_codes) + cache_row * chunks + c0;
        const float inv = quant::pow2i(-e);
        to[0] = encode8(x0, inv);
        to[apart] = encode8(x1, inv);
        if (lane == 0) (is_v ? p.v_exps : p.k_exps)[cache_row] = static_cast<uint8_t>(e + quant::kExpBias);
      }
    }
  }
}

// The two caches' arguments that are alike.
struct RopeCall {
  const pkv_bf16 *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const int64_t *positions;
  const float *cos_sin;
  int max_positions, rot_dim, interleaved;
  const int64_t *slots;
  int num_tokens;
  pkv_bf16 *q_out;
  int64_t q_out_stride;
  int num_blocks, block_size, num_q_heads, num_kv_heads, head_dim;
  int32_t *status;
  void *stream;
};

int check(const RopeCall &a) {
  if (a.num_tokens < 0 || a.num_blocks < 0 || a.block_size < 1 || a.num_q_heads < 0 || a.num_kv_heads < 1 ||
      a.head_dim < 1 || a.max_positions < 0 || a.rot_dim < 1 || (a.interleaved != 0 && a.interleaved != 1))
    return PKV_ERR_ARG;
  if (a.head_dim % 16 != 0 || a.head_dim > kMaxHeadDim) return PKV_ERR_UNSUPPORTED;
  if (a.rot_dim > a.head_dim) return PKV_ERR_ARG;
  if (a.rot_dim % 16 != 0) return PKV_ERR_UNSUPPORTED;
  const int64_t kv = static_cast<int64_t>(a.num_kv_heads) * a.head_dim;
  const int64_t qw = static_cast<int64_t>(a.num_q_heads) * a.head_dim;
  if (a.k_stride < kv || a.v_stride < kv || a.k_stride % 8 != 0 || a.v_stride % 8 != 0) return PKV_ERR_ARG;
  if (a.num_q_heads > 0 &&
      (a.q_stride < qw || a.q_out_stride < qw || a.q_stride % 8 != 0 || a.q_out_stride % 8 != 0))
    return PKV_ERR_ARG;
  if (a.num_tokens == 0) return PKV_OK;
  if (!a.k || !a.v || !a.positions || !a.cos_sin || !a.slots || (a.num_q_heads > 0 && (!a.q || !a.q_out)))
    return PKV_ERR_ARG;
  if (!aligned16(a.k) || !aligned16(a.v) || !aligned16(a.cos_sin) ||
      (a.num_q_heads > 0 && (!aligned16(a.q) || !aligned16(a.q_out))) ||
      (reinterpret_cast<uintptr_t>(a.slots) & 7u) || (reinterpret_cast<uintptr_t>(a.positions) & 7u))
    return PKV_ERR_ARG;
  return PKV_OK;
}

template <bool QUANT>
int launch(const RopeCall &a, RopeParams p) {
  p.q = reinterpret_cast<const uint4 *>(a.q);
  p.k = reinterpret_cast<const uint4 *>(a.k);
  p.v = reinterpret_cast<const uint4 *>(a.v);
  p.q_out = reinterpret_cast<uint4 *>(a.q_out);
  p.q_stride = a.q_stride / 8;
  p.k_stride = a.k_stride / 8;
  p.v_stride = a.v_stride / 8;
  p.q_out_stride = a.q_out_stride / 8;
  p.positions = a.positions;
  p.slots = a.slots;
  p.table = a.cos_sin;
  p.num_slots = static_cast<int64_t>(a.num_blocks) * a.block_size;
  p.status = a.status;
  p.max_positions = a.max_positions;
  p.rot_dim = a.rot_dim;
  p.head_dim = a.head_dim;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.block_size = a.block_size;
  const int64_t rows = static_cast<int64_t>(a.num_q_heads) + 2ll * a.num_kv_heads;
  if (rows > (1 << 24)) return PKV_ERR_UNSUPPORTED;
  p.q_groups = (a.num_q_heads + kRows - 1) / kRows;
  p.kv_groups = (a.num_kv_heads + kRows - 1) / kRows;
  p.groups = p.q_groups + 2 * p.kv_groups;
  p.tasks = static_cast<int64_t>(a.num_tokens) * p.groups;
  p.narrow = p.tasks <= 0xffffffffll && p.num_slots <= 0xffffffffll;
  auto go = [&](auto w) {
    constexpr int W = decltype(w)::value;
    const int64_t per = kThreads / W, grid = (p.tasks + per - 1) / per;
    if (grid > 0x7fffffffll) return PKV_ERR_UNSUPPORTED;  // more CTAs than a grid's x dimension holds
    const unsigned n = static_cast<unsigned>(grid);
    const cudaError_t e =
        a.interleaved ? launch_overlapped(rope_kernel<W, true, QUANT>, n, kThreads, 0, as_stream(a.stream), p)
                      : launch_overlapped(rope_kernel<W, false, QUANT>, n, kThreads, 0, as_stream(a.stream), p);
    return e == cudaSuccess ? PKV_OK : (set_cuda_error(e), PKV_ERR_CUDA);
  };
  const int lanes = a.head_dim / 16;  // the power of two that covers them
  if (lanes <= 1) return go(std::integral_constant<int, 1>());
  if (lanes <= 2) return go(std::integral_constant<int, 2>());
  if (lanes <= 4) return go(std::integral_constant<int, 4>());
  if (lanes <= 8) return go(std::integral_constant<int, 8>());
  if (lanes <= 16) return go(std::integral_constant<int, 16>());
  return go(std::integral_constant<int, 32>());
}

}  // namespace
}  // namespace pkv

extern "C" {

int pkv_write_rope(const pkv_bf16 *q, const pkv_bf16 *k, const pkv_bf16 *v, int64_t q_stride, int64_t k_stride,
                   int64_t v_stride, const int64_t *positions, const float *cos_sin, int max_positions, int rot_dim,
                   int interleaved, const int64_t *slot_mapping, int num_tokens, pkv_bf16 *q_out,
                   int64_t q_out_stride, pkv_bf16 *k_cache, pkv_bf16 *v_cache, int num_blocks, int block_size,
                   int num_q_heads, int num_kv_heads, int head_dim, int32_t *d_status, void *stream) {
  const pkv::RopeCall a{q, k, v, q_stride, k_stride, v_stride, positions, cos_sin, max_positions, rot_dim, interleaved,
                        slot_mapping, num_tokens, q_out, q_out_stride, num_blocks, block_size, num_q_heads,
                        num_kv_heads, head_dim, d_status, stream};
  const int rc = pkv::check(a);
  if (rc != PKV_OK || num_tokens == 0) return rc;
  if (!k_cache || !v_cache || !pkv::aligned16(k_cache) || !pkv::aligned16(v_cache)) return PKV_ERR_ARG;
  pkv::RopeParams p{};
  p.k_cache = reinterpret_cast<uint4 *>(k_cache);
  p.v_cache = reinterpret_cast<uint4 *>(v_cache);
  return pkv::launch<false>(a, p);
}

int pkv_write_rope_quant(const pkv_bf16 *q, const pkv_bf16 *k, const pkv_bf16 *v, int64_t q_stride, int64_t k_stride,
                         int64_t v_stride, const int64_t *positions, const float *cos_sin, int max_positions,
                         int rot_dim, int interleaved, const int64_t *slot_mapping, int num_tokens, pkv_bf16 *q_out,
                         int64_t q_out_stride, uint8_t *k_codes, uint8_t *v_codes, uint8_t *k_exps, uint8_t *v_exps,
                         int num_blocks, int block_size, int num_q_heads, int num_kv_heads, int head_dim,
                         int32_t *d_status, void *stream) {
  const pkv::RopeCall a{q, k, v, q_stride, k_stride, v_stride, positions, cos_sin, max_positions, rot_dim, interleaved,
                        slot_mapping, num_tokens, q_out, q_out_stride, num_blocks, block_size, num_q_heads,
                        num_kv_heads, head_dim, d_status, stream};
  const int rc = pkv::check(a);
  if (rc != PKV_OK || num_tokens == 0) return rc;
  if (!k_codes || !v_codes || !k_exps || !v_exps || !pkv::aligned16(k_codes) || !pkv::aligned16(v_codes))
    return PKV_ERR_ARG;
  pkv::RopeParams p{};
  p.k_codes = reinterpret_cast<uint2 *>(k_codes);
  p.v_codes = reinterpret_cast<uint2 *>(v_codes);
  p.k_exps = k_exps;
  p.v_exps = v_exps;
  return pkv::launch<true>(a, p);
}

}  // extern "C"
