// Softmax steps of the tensor-core attention kernels: a thread holds 64 raw scores
// of its query row, as it loads them from tensor memory.
#pragma once

#include <cfloat>
#include <cstdint>

#include "ptx.cuh"

namespace pkv {

constexpr float kLog2e = 1.4426950408889634f;

// The kernels compare raw scores before scaling them; a zero scale would turn
// the masked -inf scores into NaN, so it runs as the smallest normal float,
// whose products with finite scores round to the same weights (all 1).
inline float kernel_scale_log2(float scale) { return (scale == 0.f ? FLT_MIN : scale) * kLog2e; }

// 32 bytes from eight 32-bit registers to global memory in one request
// (256-bit store, sm_100+); the address must be 32-byte aligned.
__device__ __forceinline__ void st_global_v8(void *p, const uint32_t *w) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// The largest (smallest, for a negative scale) of 64 raw scores: eight short
// chains of 3-input maxima.
__device__ __forceinline__ float extreme64(const uint32_t (&v)[64], bool neg) {
  float e[8];
  if (!neg) {
#pragma unroll
    for (int q = 0; q < 8; ++q) e[q] = fmax3(__uint_as_float(v[q]), __uint_as_float(v[q + 8]), __uint_as_float(v[q + 16]));
#pragma unroll
    for (int q = 0; q < 8; ++q) e[q] = fmax3(e[q], __uint_as_float(v[q + 24]), __uint_as_float(v[q + 32]));
#pragma unroll
    for (int q = 0; q < 8; ++q) e[q] = fmax3(e[q], __uint_as_float(v[q + 40]), __uint_as_float(v[q + 48]));
#pragma unroll
    for (int q = 0; q < 8; ++q) e[q] = fmaxf(e[q], __uint_as_float(v[q + 56]));
    return fmax3(fmax3(e[0], e[1], e[2]), fmax3(e[3], e[4], e[5]), fmaxf(e[6], e[7]));
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) e[q] = fmin3(__uint_as_float(v[q]), __uint_as_float(v[q + 8]), __uint_as_float(v[q + 16]));
#pragma unroll
  for (int q = 0; q < 8; ++q) e[q] = fmin3(e[q], __uint_as_float(v[q + 24]), __uint_as_float(v[q + 32]));
#pragma unroll
  for (int q = 0; q < 8; ++q) e[q] = fmin3(e[q], __uint_as_float(v[q + 40]), __uint_as_float(v[q + 48]));
#pragma unroll
  for (int q = 0; q < 8; ++q) e[q] = fminf(e[q], __uint_as_float(v[q + 56]));
  return fmin3(fmin3(e[0], e[1], e[2]), fmin3(e[3], e[4], e[5]), fminf(e[6], e[7]));
}

// Weights of 64 raw scores, p = 2^(s * scale * log2e - m), two at a time with a
// packed fp32 FMA, packed to bf16 pairs; returns the sum of the weights before
// their rounding to bf16.  They are rounded because a matrix instruction takes
// both operands in one 16-bit type and the values are bf16 (fp16 does not hold
// their range); weights as two bf16 terms would double the P V products.  The
// rounding errors, at most 2^-8 of each weight and of either sign, leave the sum's
// relative error far below the output's bf16 step.  Masked keys hold -inf (or
// +inf for a negative scale): their weight is 2^-inf = 0.
__device__ __forceinline__ float weights64(const uint32_t (&v)[64], uint64_t ks2, uint64_t nm2, uint32_t (&pk)[32]) {
  uint64_t ls[4] = {0ull, 0ull, 0ull, 0ull};  // four packed partial sums (0 bits = +0.0)
#pragma unroll
  for (int c = 0; c < 32; ++c) {
    float x0, x1;
    f32x2_split(ffma2(f32x2_bits(v[2 * c], v[2 * c + 1]), ks2, nm2), x0, x1);
    const float e0 = fast_exp2(x0), e1 = fast_exp2(x1);
    pk[c] = pack_bf16x2(e0, e1);
    ls[c & 3] = fadd2(ls[c & 3], f32x2_bits(__float_as_uint(e0), __float_as_uint(e1)));
  }
  float a0, a1, b0, b1, c0, c1, d0, d1;
  f32x2_split(ls[0], a0, a1);
  f32x2_split(ls[1], b0, b1);
  f32x2_split(ls[2], c0, c1);
  f32x2_split(ls[3], d0, d1);
  return ((a0 + a1) + (b0 + b1)) + ((c0 + c1) + (d0 + d1));
}

// Bounded wait whose outcome every lane of the warp agrees on; try_wait
// parks the warp until the phase completes (or a short hardware window ends).
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

}  // namespace pkv
