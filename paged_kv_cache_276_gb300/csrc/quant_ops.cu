// Quantising slot write (pkv_write_quant) and read-back (pkv_read_quant) of the
// 8-bit cache.
//
// Both are data movement with a little arithmetic, bound by HBM: per row of d
// values a write reads 2 d bytes and stores d + 1, a read-back the reverse.  A
// group of lanes takes one (token, KV head): its key row and its value row, 16
// values (32 bytes of bf16 in one access where it is aligned, 16 bytes of codes)
// per lane, so the row's maximum is a few shuffles and a row is read once.  No
// loop: a CTA per few rows lets the hardware balance a ragged end (with a grid
// of 8 CTAs per SM that walks the rows, read-back took 41.8 us instead of 32.2).
// Measured at 32768 tokens x 8 KV heads x 128: write 31.0 us (6.5 TB/s),
// read-back 31.7 us (6.4 TB/s), of 6.78 TB/s for a plain copy; the 256 tokens of
// a decode step 2.1 us, a launch's latency.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
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
constexpr int kMaxHeadDim = 512;  // 32 lanes x 16 values

struct RowParams {
  const int64_t *slots;
  int64_t num_slots;  // num_blocks * block_size
  int64_t rows;       // num_tokens * num_kv_heads
  int64_t k_stride, v_stride;  // elements between tokens (write)
  int32_t *status;
  int num_kv_heads, block_size, chunks;  // chunks: head_dim / 16
  int narrow;  // rows and num_slots fit 32 bits: divide in 32 bits
};

struct CachePtrs {
  uint4 *k_codes, *v_codes;
  uint8_t *k_exps, *v_exps;
};

// The bf16 pair's magnitudes, non-finite ones replaced by 0.
__device__ __forceinline__ uint32_t finite_magnitudes(uint32_t v) {
  const uint32_t m = v & 0x7FFF7FFFu;
  return ((m & 0xFFFFu) >= 0x7F80u ? 0u : m & 0xFFFFu) | ((m >> 16) >= 0x7F80u ? 0u : m & 0xFFFF0000u);
}

// This row's token and head, and its slot; false: nothing to do.
__device__ __forceinline__ bool locate(const RowParams &p, int64_t row, bool report, int64_t *token, int *head,
                                       int64_t *cache_row) {
  int64_t t;
  if (p.narrow) t = static_cast<uint32_t>(row) / static_cast<uint32_t>(p.num_kv_heads);
  else t = row / p.num_kv_heads;
  const int h = static_cast<int>(row - t * p.num_kv_heads);
  const int64_t slot = p.slots[t];
  if (slot < 0) return false;
  if (slot >= p.num_slots) {
    if (report && h == 0 && p.status) atomicOr(p.status, PKV_STATUS_BAD_SLOT);
    return false;
  }
  int64_t blk;
  if (p.narrow) blk = static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.block_size);
  else blk = slot / p.block_size;
  *token = t;
  *head = h;
  *cache_row = (blk * p.num_kv_heads + h) * p.block_size + (slot - blk * p.block_size);
  return true;
}

// 16 bf16 of a row (two 16-byte loads) -> 16 codes, given the row's exponent.
__device__ __forceinline__ uint4 encode(const uint4 &a, const uint4 &b, float inv) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t half[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t v = w[2 * i + j];
      half[j] = quant::to_e4m3x2(__uint_as_float(v << 16) * inv, __uint_as_float(v & 0xFFFF0000u) * inv);
    }
    c[i] = half[0] | (half[1] << 16);
  }
  return make_uint4(c[0], c[1], c[2], c[3]);
}

// The largest magnitude of a lane's 16 values, as bf16 bits in either half.
__device__ __forceinline__ uint32_t magnitude_max(const uint4 &a, const uint4 &b) {
  constexpr uint32_t M = 0x7FFF7FFFu;
  uint32_t m = __vmaxu2(__vmaxu2(a.x & M, a.y & M), __vmaxu2(a.z & M, a.w & M));
  return __vmaxu2(m, __vmaxu2(__vmaxu2(b.x & M, b.y & M), __vmaxu2(b.z & M, b.w & M)));
}

template <int W>
__device__ __forceinline__ uint32_t group_max(uint32_t m) {
#pragma unroll
  for (int off = W / 2; off; off >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, off));
  return max(m & 0xFFFFu, m >> 16);
}

// Infinities become NaN (a row that holds any is rare: only then).
__device__ __forceinline__ uint32_t infinities_to_nan(uint32_t v) {
  const uint32_t m = v & 0x7FFF7FFFu;
  return v | ((m & 0xFFFFu) == 0x7F80u ? 0x40u : 0u) | ((m >> 16) == 0x7F80u ? 0x400000u : 0u);
}
__device__ __forceinline__ uint4 infinities_to_nan(const uint4 &a) {
  return make_uint4(infinities_to_nan(a.x), infinities_to_nan(a.y), infinities_to_nan(a.z), infinities_to_nan(a.w));
}
__device__ __forceinline__ uint4 finite_magnitudes(const uint4 &a) {
  return make_uint4(finite_magnitudes(a.x), finite_magnitudes(a.y), finite_magnitudes(a.z), finite_magnitudes(a.w));
}

// One row's 16 values per lane -> codes and exponent byte, W lanes together.
template <int W>
__device__ __forceinline__ uint4 quantise(uint4 a, uint4 b, uint8_t *exp_byte) {
  uint32_t top = group_max<W>(magnitude_max(a, b));
  if (__any_sync(0xffffffffu, top >= 0x7F80u)) {  // a NaN or infinity somewhere in the warp's rows
    top = group_max<W>(magnitude_max(finite_magnitudes(a), finite_magnitudes(b)));
    a = infinities_to_nan(a);
    b = infinities_to_nan(b);
  }
  const int e = quant::row_exponent(top);
  *exp_byte = static_cast<uint8_t>(e + quant::kExpBias);
  return encode(a, b, quant::pow2i(-e));
}

// 16 values: one 32-byte load where the rows are aligned to it.
template <bool WIDE>
__device__ __forceinline__ void load16(const uint4 *src, uint4 &a, uint4 &b) {
  if constexpr (WIDE) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(src));
  } else {
    a = src[0];
    b = src[1];
  }
}
template <bool WIDE>
__device__ __forceinline__ void store16(uint4 *dst, const uint4 &a, const uint4 &b) {
  if constexpr (WIDE) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(a.x), "r"(a.y), "r"(a.z),
                 "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
  } else {
    dst[0] = a;
    dst[1] = b;
  }
}

// W lanes per (token, KV head) row pair: lane c of the group holds values 16 c ..
// 16 c + 15 of the key row and of the value row.  Eight CTAs an SM (32 registers
// a thread) keep most loads in flight.  At 262144 row pairs of 128 values:
// 31.2 us; with 40 registers 36.9; two row pairs per thread (63) 34.5; keys and
// values by different threads 37.7.  (No __restrict__ on the inputs: the kernel
// just before may still be writing them when this one becomes resident, so they
// are not read-only for this kernel's whole life.)
template <int W, bool WIDE>
__global__ void __launch_bounds__(kThreads, 8) write_kernel(const uint4 *k, const uint4 *v,
                                                            const RowParams p, const CachePtrs out) {
  // the grid queued behind this one may become resident now (it waits for this
  // grid's writes before it reads the cache)
  grid_launch_dependents();
  grid_dependency_wait();  // the rows may come from the kernel launched just before
  const int c = threadIdx.x % W;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / W) + threadIdx.x / W;
  int64_t t = 0, dst = 0;
  int h = 0;
  const bool live = row < p.rows && locate(p, row, c == 0, &t, &h, &dst) && c < p.chunks;
  uint4 ka = make_uint4(0u, 0u, 0u, 0u), kb = ka, va = ka, vb = ka;
  if (live) {
    const int64_t at = (static_cast<int64_t>(h) * p.chunks + c) * 2;
    load16<WIDE>(k + (t * p.k_stride) / 8 + at, ka, kb);
    load16<WIDE>(v + (t * p.v_stride) / 8 + at, va, vb);
  }
  uint8_t e;
  uint4 codes = quantise<W>(ka, kb, &e);
  if (live) {
    out.k_codes[dst * p.chunks + c] = codes;
    if (c == 0) out.k_exps[dst] = e;
  }
  codes = quantise<W>(va, vb, &e);
  if (live) {
    out.v_codes[dst * p.chunks + c] = codes;
    if (c == 0) out.v_exps[dst] = e;
  }
}

// 4 codes -> 4 bf16 (two words), times the row's power of two: exact.
__device__ __forceinline__ uint2 decode4(uint32_t codes, float scale) {
  const uint32_t lo = quant::e4m3x2_to_f16x2(codes), hi = quant::e4m3x2_hi_to_f16x2(codes);
  const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
  return make_uint2(pack_bf16x2(a.x * scale, a.y * scale), pack_bf16x2(b.x * scale, b.y * scale));
}

template <bool WIDE>
__device__ __forceinline__ void decode16(const uint4 &codes, float scale, uint4 *dst) {
  const uint2 a = decode4(codes.x, scale), b = decode4(codes.y, scale);
  const uint2 c = decode4(codes.z, scale), d = decode4(codes.w, scale);
  store16<WIDE>(dst, make_uint4(a.x, a.y, b.x, b.y), make_uint4(c.x, c.y, d.x, d.y));
}

// W lanes per (token, KV head) row pair, as in write_kernel.
template <int W, bool WIDE>
__global__ void __launch_bounds__(kThreads) read_kernel(uint4 *__restrict__ k, uint4 *__restrict__ v,
                                                        const RowParams p, const CachePtrs in) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int c = threadIdx.x % W;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / W) + threadIdx.x / W;
  int64_t t, src;
  int h;
  if (c >= p.chunks || row >= p.rows || !locate(p, row, c == 0, &t, &h, &src)) return;
  const uint4 kc = in.k_codes[src * p.chunks + c], vc = in.v_codes[src * p.chunks + c];
  const int ke = in.k_exps[src], ve = in.v_exps[src];
  const int64_t at = (row * p.chunks + c) * 2;
  decode16<WIDE>(kc, quant::pow2i(quant::clamp_exp(ke)), k + at);
  decode16<WIDE>(vc, quant::pow2i(quant::clamp_exp(ve)), v + at);
}

int check_rows(const void *k, const void *v, const int64_t *slots, int num_tokens, const void *k_codes,
               const void *v_codes, const void *k_exps, const void *v_exps, int num_blocks, int block_size,
               int num_kv_heads, int head_dim) {
  if (num_tokens < 0 || num_blocks < 0 || block_size < 1 || num_kv_heads < 1 || head_dim < 1) return PKV_ERR_ARG;
  if (head_dim % 16 != 0 || head_dim > kMaxHeadDim) return PKV_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PKV_OK;
  if (!k || !v || !slots || !k_codes || !v_codes || !k_exps || !v_exps) return PKV_ERR_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_codes) || !aligned16(v_codes) ||
      (reinterpret_cast<uintptr_t>(slots) & 7u))
    return PKV_ERR_ARG;
  return PKV_OK;
}

RowParams row_params(const int64_t *slots, int num_tokens, int num_blocks, int block_size, int num_kv_heads,
                     int head_dim, int32_t *status) {
  RowParams p{};
  p.slots = slots;
  p.num_slots = static_cast<int64_t>(num_blocks) * block_size;
  p.rows = static_cast<int64_t>(num_tokens) * num_kv_heads;
  p.status = status;
  p.num_kv_heads = num_kv_heads;
  p.block_size = block_size;
  p.chunks = head_dim / 16;
  p.narrow = p.rows <= 0xffffffffll && p.num_slots <= 0xffffffffll;
  return p;
}

// CTAs for so many rows of `lanes` lanes.
int64_t row_grid(int64_t rows, int lanes) {
  const int64_t per = kThreads / lanes;
  return (rows + per - 1) / per;
}

template <typename K, typename... Args>
int launch_grid(K kernel, int64_t grid, void *stream, const Args &...args) {
  if (grid > 0x7fffffffll) return PKV_ERR_UNSUPPORTED;  // more CTAs than a grid's x dimension holds
  const cudaError_t e =
      launch_overlapped(kernel, static_cast<unsigned>(grid), kThreads, 0, as_stream(stream), args...);
  return e == cudaSuccess ? PKV_OK : (set_cuda_error(e), PKV_ERR_CUDA);
}

bool aligned32(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

// f with the lanes per row (the power of two that covers head_dim / 16) and
// whether rows are aligned to 32 bytes, as types.
template <typename F>
int launch_rows(int chunks, bool wide, F &&f) {
  auto go = [&](auto w) { return wide ? f(w, std::true_type()) : f(w, std::false_type()); };
  if (chunks <= 1) return go(std::integral_constant<int, 1>());
  if (chunks <= 2) return go(std::integral_constant<int, 2>());
  if (chunks <= 4) return go(std::integral_constant<int, 4>());
  if (chunks <= 8) return go(std::integral_constant<int, 8>());
  if (chunks <= 16) return go(std::integral_constant<int, 16>());
  return go(std::integral_constant<int, 32>());
}

}  // namespace
}  // namespace pkv

extern "C" {

int pkv_write_quant(const pkv_bf16 *k, const pkv_bf16 *v, int64_t k_stride, int64_t v_stride,
                    const int64_t *slot_mapping, int num_tokens, uint8_t *k_codes, uint8_t *v_codes, uint8_t *k_exps,
                    uint8_t *v_exps, int num_blocks, int block_size, int num_kv_heads, int head_dim,
                    int32_t *d_status, void *stream) {
  const int rc = pkv::check_rows(k, v, slot_mapping, num_tokens, k_codes, v_codes, k_exps, v_exps, num_blocks,
                                 block_size, num_kv_heads, head_dim);
  if (rc != PKV_OK) return rc;
  const int64_t width = static_cast<int64_t>(num_kv_heads) * head_dim;
  if (k_stride < width || v_stride < width || k_stride % 8 != 0 || v_stride % 8 != 0) return PKV_ERR_ARG;
  if (num_tokens == 0) return PKV_OK;
  pkv::RowParams p = pkv::row_params(slot_mapping, num_tokens, num_blocks, block_size, num_kv_heads, head_dim, d_status);
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  const pkv::CachePtrs out{reinterpret_cast<uint4 *>(k_codes), reinterpret_cast<uint4 *>(v_codes), k_exps, v_exps};
  const bool wide = pkv::aligned32(k) && pkv::aligned32(v) && k_stride % 16 == 0 && v_stride % 16 == 0;
  return pkv::launch_rows(p.chunks, wide, [&](auto w, auto wd) {
    constexpr int W = decltype(w)::value;
    constexpr bool WIDE = decltype(wd)::value;
    return pkv::launch_grid(pkv::write_kernel<W, WIDE>, pkv::row_grid(p.rows, W), stream,
                            reinterpret_cast<const uint4 *>(k), reinterpret_cast<const uint4 *>(v), p, out);
  });
}

int pkv_read_quant(const uint8_t *k_codes, const uint8_t *v_codes, const uint8_t *k_exps, const uint8_t *v_exps,
                   const int64_t *slot_mapping, int num_tokens, pkv_bf16 *k, pkv_bf16 *v, int num_blocks,
                   int block_size, int num_kv_heads, int head_dim, int32_t *d_status, void *stream) {
  const int rc = pkv::check_rows(k, v, slot_mapping, num_tokens, k_codes, v_codes, k_exps, v_exps, num_blocks,
                                 block_size, num_kv_heads, head_dim);
  if (rc != PKV_OK || num_tokens == 0) return rc;
  const pkv::RowParams p =
      pkv::row_params(slot_mapping, num_tokens, num_blocks, block_size, num_kv_heads, head_dim, d_status);
  const pkv::CachePtrs in{reinterpret_cast<uint4 *>(const_cast<uint8_t *>(k_codes)),
                          reinterpret_cast<uint4 *>(const_cast<uint8_t *>(v_codes)), const_cast<uint8_t *>(k_exps),
                          const_cast<uint8_t *>(v_exps)};
  return pkv::launch_rows(p.chunks, pkv::aligned32(k) && pkv::aligned32(v), [&](auto w, auto wd) {
    constexpr int W = decltype(w)::value;
    return pkv::launch_grid(pkv::read_kernel<W, decltype(wd)::value>, pkv::row_grid(p.rows, W), stream,
                            reinterpret_cast<uint4 *>(k), reinterpret_cast<uint4 *>(v), p, in);
  });
}

}  // extern "C"
