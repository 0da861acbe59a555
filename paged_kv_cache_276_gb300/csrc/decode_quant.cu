// Single-token paged attention over the 8-bit cache (paged_attention_decode_quant).
//
// Math: with key codes kc_t, value codes vc_t (e4m3) and the rows' powers of two
// 2^ke_t, 2^ve_t:  s_t = scale 2^ke_t (q . kc_t),  out = sum_t softmax_t(s) 2^ve_t vc_t.
// In log2 units x_t = log2(e) s_t + ve_t, with any reference R:
//   w_t = 2^(x_t - R)  (the weight with the value row's scale folded in),
//   O = sum_t w_t vc_t,  l = sum_t w_t 2^-ve_t,  out = O / l,
// so codes enter the products as they are stored and a scale costs one FMA per
// score.  e4m3 values are exact in fp16, so both products run on fp16 MMA with
// fp32 accumulators; the queries are scaled by a power of two per head to use
// fp16's range (bf16 has fewer significant bits: exact but for values 2^-31
// and more below the head's largest).  The weights' rounding to fp16 (2^-11)
// enters O only; l sums them unrounded, since a key whose value row is tiny can
// hold most of the softmax at a negligible w.
//
// Work: the cache is read once, so the kernel is bound by HBM; it has to keep
// every SM streaming however the lengths are spread.  All (sequence, KV head)
// runs are cut into units of kUnitBytes of keys (32 tokens at head_dim 128, 64
// at 64) and laid end to end; every warp of a grid of one CTA per SM takes an
// equal, contiguous range of units (short batches: make_plan).  The lengths'
// prefix sums are taken by every CTA at its start, so there is no host-built
// list and a captured graph follows its lengths.  A warp streams its units
// through a ring of its own (TMA with the 128-byte swizzle for the codes,
// cp.async for the exponents, one mbarrier per stage) and refills a stage right
// after it has used it: no barrier between warps until the end.  A run that a
// warp holds whole is written at once; pieces of a run are joined in shared
// memory at the CTA's end, and runs that span CTAs through the workspace by a
// second kernel.  Joins take the pieces in an order that the sizes fix: results
// repeat bit for bit.
//
// Measured (both kernels, back to back in a graph; in brackets per call in a row
// of calls): 16 x 32768 tokens, 64 q / 8 KV heads of 128, block 32: 174 us (176),
// 6.2 TB/s of 6.78 for a plain copy; 256 mixed lengths, 32 / 8, block 16: 76.5 us
// (78.4), 5.8 TB/s; one sequence of 32768: 20.2 us (20.5), of which the copies
// take 12.6, start and joins the rest.  Units of half or twice the size, or more
// stages with fewer warps, were 1 % faster on the first at best and 7 to 28 %
// slower on the second.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "internal.h"
#include "launch.cuh"
#include "pkv.h"
#include "ptx.cuh"
#include "quant.cuh"

namespace pkv {
namespace {

constexpr int kMaxGroup = 16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kUnitBytes = 4096;  // key codes of one unit; the value codes take as many
// A weight is 2^(x - R): R is set 7 below the largest x when it moves, and moves
// when an x exceeds it by more than 15, so weights stay below 2^15 (fp16 holds
// 65504) and most units skip the rescale.
constexpr float kHeadroom = 7.f, kSlack = 15.f;
// R before any x: every x moves it, and 2^(-inf - R) is still 0.
constexpr float kNoRef = -1e38f;
constexpr int kDirectUnits = 2;   // runs of at most so many units may go to a warp whole
constexpr int kDirectRounds = 2;  // ... of so many per warp to a CTA

struct Params {
  const __nv_bfloat16 *q;
  const uint8_t *k_exps, *v_exps;
  const int32_t *block_tables, *seq_lens;
  __nv_bfloat16 *out;
  float *ws;      // [grid][2] pieces of runs that span CTAs, then [grid] descriptors; NULL: no run does
  int4 *ws_desc;  // {sequence | KV head << 16, -, last CTA of the run, 1} of the run that leaves CTA c, or .w = 0
  int32_t *status;
  int num_seqs, max_blocks, max_len, num_q_heads, num_kv_heads, group, num_blocks;
  int direct;  // 1: whole runs go round the warps; k > 1: k warps of a CTA share a run; 0: equal ranges of units
  float scale_log2;
};

template <int D, int NT>
struct Shape {
  static constexpr int kTokens = kUnitBytes / D;  // tokens of a unit
  static constexpr int kStages = 2;
  // tokens of one softmax step: the whole unit where registers allow (168 a thread with more than 8 warps, 255 with 8)
  static constexpr int kStep = NT == 1 || D == 128 ? kTokens : kTokens / 2;
  static constexpr int kTileFloats = NT * 8 * D;  // O of one piece, in accumulator order
  static constexpr int kPieceFloats = kTileFloats + 2 * NT * 8;  // ..., R[cols], l[cols]
  static constexpr int kRingBytes = kStages * 2 * kUnitBytes;
  static constexpr int kExpBytes = kStages * 2 * kTokens;
  static constexpr int kMetaBytes = kStages * (16 + 8);  // an int4 and a barrier per stage
  static constexpr int kWarpBytes = kRingBytes + kExpBytes + kMetaBytes + kPieceFloats * 4;
  // as many warps as shared memory (227 KB a CTA) holds rings and pieces for; 8
  // of them where two tiles at head_dim 128 need 255 registers a thread
  static constexpr int kWarps = D == 128 ? (NT == 1 ? 11 : 8) : (NT == 1 ? 12 : 10);
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kSmemBytes = 1024 + kWarps * kWarpBytes;
  static_assert(kPieceFloats * 4 <= kRingBytes, "a warp's last piece goes over its ring");
  static_assert(kSmemBytes + kThreads * 8 + kWarps * 40 + 64 <= 227 * 1024, "shared memory of one CTA");
};

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ int lds_u8(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(a) : "memory");
  return static_cast<int>(r);
}

// 16 bytes global -> shared by this thread, asynchronously, past L1: the bytes
// are read once and need no line there.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// One arrival on `bar` once this thread's cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Shared-memory address of byte `off` of a unit staged with the 128-byte swizzle.
__device__ __forceinline__ uint32_t swz(uint32_t base, uint32_t off) { return base + (off ^ ((off >> 3) & 0x70u)); }

__device__ __forceinline__ int capped_len(const Params &p, int bs) {
  const long long cap = static_cast<long long>(p.max_blocks) * bs;
  return static_cast<int>(cap < p.max_len ? cap : p.max_len);
}

// The running softmax of one warp's piece: its columns are the query heads.
template <int D, int NT>
struct Acc {
  float r[NT][2];  // reference R per column (the thread's two columns of each 8)
  float l[NT][2];  // this thread's part of the sum
  float o[D / 16][NT][4];
  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      r[nt][0] = r[nt][1] = kNoRef;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int md = 0; md < D / 16; ++md) o[md][nt][0] = o[md][nt][1] = o[md][nt][2] = o[md][nt][3] = 0.f;
    }
  }
};

// The group's queries as B fragments.  The product over head_dim takes its
// terms in the order a key row's bytes are read in: lane t of a quad holds
// values [t D/4, (t + 1) D/4) of each row, four to a k-step.  cf: per column of
// the accumulators, the factor that undoes the queries' power of two and
// applies the scale (in log2 units).
template <int D, int NT>
__device__ __forceinline__ void load_queries(const Params &p, int seq, int h, uint32_t (&qf)[NT][D / 16][2],
                                             float (&cf)[NT][2], int lane) {
  const int g4 = lane >> 2, c4 = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int col = nt * 8 + g4;
    const bool real = col < p.group;
    const uint4 *src = reinterpret_cast<const uint4 *>(
        p.q + (static_cast<size_t>(seq) * p.num_q_heads + static_cast<size_t>(h) * p.group + (real ? col : 0)) * D +
        c4 * (D / 4));
    uint32_t w[D / 8];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint4 x = real ? src[i] : make_uint4(0u, 0u, 0u, 0u);
      w[4 * i] = x.x;
      w[4 * i + 1] = x.y;
      w[4 * i + 2] = x.z;
      w[4 * i + 3] = x.w;
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) top = __vmaxu2(top, w[i] & 0x7FFF7FFFu);
    top = max(top & 0xFFFFu, top >> 16);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // largest magnitude to [2^14, 2^15); queries below 2^-86 keep a smaller one
    const int shift = min(100, 14 + 127 - static_cast<int>(top >> 7));
    const float up = quant::pow2i(shift);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const uint32_t v = w[ks * 2 + b];
        qf[nt][ks][b] = pack_f16x2(__uint_as_float(v << 16) * up, __uint_as_float(v & 0xFFFF0000u) * up);
      }
    const float f = p.scale_log2 * quant::pow2i(-shift);
    cf[nt][0] = __shfl_sync(0xffffffffu, f, 8 * c4);
    cf[nt][1] = __shfl_sync(0xffffffffu, f, 8 * c4 + 4);
  }
}

// 16 MT staged tokens: scores, running softmax, product with the values.
//   valid: those of them before the sequence's end (at least 1); staged bytes
//          behind them may be anything.
template <int D, int NT, int MT>
__device__ __forceinline__ void attend_tokens(Acc<D, NT> &acc, const uint32_t (&qf)[NT][D / 16][2],
                                            const float (&cf)[NT][2], uint32_t kb, uint32_t vb, uint32_t keb,
                                            uint32_t veb, int valid, int lane) {
  constexpr int W = D / 64;  // 16-byte chunks of a key row per lane
  const int g4 = lane >> 2, c4 = lane & 3;

  // S^T[token][head]: A rows are tokens, read 16 bytes at a time as they lie
  float s[MT][NT][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    float s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[mt][nt][i] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const uint32_t off = (mt * 16 + g4) * D + (c4 * W + j) * 16;
      const uint4 lo = lds128(swz(kb, off)), hi = lds128(swz(kb, off + 8 * D));
      const uint32_t a[4] = {lo.x, lo.y, lo.z, lo.w}, b[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a0 = quant::e4m3x2_to_f16x2(a[i]), a2 = quant::e4m3x2_hi_to_f16x2(a[i]);
        const uint32_t a1 = quant::e4m3x2_to_f16x2(b[i]), a3 = quant::e4m3x2_hi_to_f16x2(b[i]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {  // two chains of products, so that they overlap
          const int ks = j * 4 + i;
          if (NT == 1 && (i & 1)) mma_f16_16816(s2, a0, a1, a2, a3, qf[nt][ks][0], qf[nt][ks][1]);
          else mma_f16_16816(s[mt][nt], a0, a1, a2, a3, qf[nt][ks][0], qf[nt][ks][1]);
        }
      }
    }
    if (NT == 1)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[mt][0][i] += s2[i];
  }

  // The tokens' scales, one lane per token of 32: {2^ke in the low half, 2^-ve in
  // the high one} (powers of two are the upper 16 bits of an fp32), and ve.
  uint32_t pow[MT / 2];
  float add[MT / 2];
#pragma unroll
  for (int k = 0; k < MT / 2; ++k) {
    const int ke = quant::clamp_exp(lds_u8(keb + k * 32 + lane)), ve = quant::clamp_exp(lds_u8(veb + k * 32 + lane));
    pow[k] = static_cast<uint32_t>(ke + 127) << 7 | static_cast<uint32_t>(127 - ve) << 23;
    add[k] = static_cast<float>(ve);
  }
  // x = log2(e) s + ve; the columns' largest
  float top[NT][2], inv[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int src = (mt & 1) * 16 + 8 * hf + g4;
      const uint32_t pw = __shfl_sync(0xffffffffu, pow[mt >> 1], src);
      const float vf = __shfl_sync(0xffffffffu, add[mt >> 1], src);
      const float kf = __uint_as_float(pw << 16);
      inv[mt][hf] = __uint_as_float(pw & 0xFFFF0000u);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) s[mt][nt][2 * hf + e] = fmaf(s[mt][nt][2 * hf + e] * kf, cf[nt][e], vf);
    }
  if (valid < 16 * MT) {  // warp-uniform
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (mt * 16 + g4 + 8 * (i >> 1) >= valid) s[mt][nt][i] = -INFINITY;
  }
  bool moves = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float t = fmaxf(s[0][nt][e], s[0][nt][2 + e]);
#pragma unroll
      for (int mt = 1; mt < MT; ++mt) t = fmax3(t, s[mt][nt][e], s[mt][nt][2 + e]);
      t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
      t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
      t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
      top[nt][e] = t;
      moves |= t > acc.r[nt][e] + kSlack;
    }
  if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float r = acc.r[nt][e], n = top[nt][e] > r + kSlack ? top[nt][e] - kHeadroom : r;
        const float alpha = fast_exp2(r - n);
        acc.r[nt][e] = n;
        acc.l[nt][e] *= alpha;
#pragma unroll
        for (int md = 0; md < D / 16; ++md) {
          acc.o[md][nt][e] *= alpha;
          acc.o[md][nt][e + 2] *= alpha;
        }
      }
  }

  // weights -> fp16 -> B fragments of P^T (movmatrix turns the accumulator layout)
  uint32_t pb[MT][NT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const float w0 = fast_exp2(s[mt][nt][2 * hf] - acc.r[nt][0]);
        const float w1 = fast_exp2(s[mt][nt][2 * hf + 1] - acc.r[nt][1]);
        acc.l[nt][0] = fmaf(w0, inv[mt][hf], acc.l[nt][0]);
        acc.l[nt][1] = fmaf(w1, inv[mt][hf], acc.l[nt][1]);
        pb[mt][nt][hf] = movmatrix_trans(pack_f16x2(w0, w1));
      }

  // O^T[value][head] += V^T P^T.  A rows are values: accumulator rows g and
  // g + 8 of step md stand for values g D/8 + 2 md and + 2 md + 1, so a lane
  // reads D/8 consecutive bytes of each of its four tokens; a byte permute pairs
  // two tokens' codes of the same value.
#pragma unroll
  for (int kt = 0; kt < MT; ++kt) {
    uint32_t v[4][D / 32];
    const int t0 = kt * 16 + 2 * c4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = t0 + (i & 1) + 8 * (i >> 1);
      const uint32_t a = swz(vb, tok * D + g4 * (D / 8));
      if constexpr (D == 128) {
        const uint4 x = lds128(a);
        v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
      } else {
        const uint2 x = lds64(a);
        v[i][0] = x.x, v[i][1] = x.y;
      }
    }
    if (valid < (kt + 1) * 16) {  // warp-uniform; a NaN code behind the end must not meet its zero weight
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (t0 + (i & 1) + 8 * (i >> 1) >= valid)
#pragma unroll
          for (int c = 0; c < D / 32; ++c) v[i][c] = 0u;
    }
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t sel = half ? 0x7362u : 0x5140u;
        const uint32_t lo = __byte_perm(v[0][c], v[1][c], sel), hi = __byte_perm(v[2][c], v[3][c], sel);
        const uint32_t a0 = quant::e4m3x2_to_f16x2(lo), a1 = quant::e4m3x2_hi_to_f16x2(lo);
        const uint32_t a2 = quant::e4m3x2_to_f16x2(hi), a3 = quant::e4m3x2_hi_to_f16x2(hi);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma_f16_16816(acc.o[c * 2 + half][nt], a0, a1, a2, a3, pb[kt][nt][0], pb[kt][nt][1]);
      }
  }
}

// Values g D/8 + 2 md and + 1 of heads col and col + 1 from their joined accumulators.
// A run has a key at least and its largest weight is not lost, so a sum of 0 means
// scores of -inf throughout (an infinite query): 0 / 0, as the formula has it.
template <int D>
__device__ __forceinline__ void store_quad(const Params &p, uint32_t run, int col, int g4, int md, const float4 &o,
                                           float l0, float l1) {
  const size_t seq = run & 0xFFFFu, h = run >> 16;
  uint32_t *row = reinterpret_cast<uint32_t *>(p.out + (seq * p.num_q_heads + h * p.group + col) * D + g4 * (D / 8) +
                                               2 * md);
  const float i0 = 1.f / l0, i1 = 1.f / l1;
  if (col < p.group) row[0] = pack_bf16x2(o.x * i0, o.z * i0);
  if (col + 1 < p.group) row[D / 2] = pack_bf16x2(o.y * i1, o.w * i1);
}

// Weight of a piece with reference r in a join to the largest reference R.
__device__ __forceinline__ float piece_factor(float r, float R) { return fast_exp2(r - R); }

// Join of one run's pieces in shared memory, tile nt, by one warp.  The whole
// run goes to the output, a part of one to the workspace.
//   g: {bits of the pieces' places, run, 2 began at the run's start | 4 ends it, -}
template <int D, int NT>
__device__ __forceinline__ void join_pieces(const Params &p, const uint4 g, int nt, const uint8_t *smem,
                                            const uint8_t *rest, int lane) {
  using Sh = Shape<D, NT>;
  constexpr int COLS = NT * 8;
  const int col = nt * 8 + 2 * (lane & 3);
  auto place = [&](int k) {
    return reinterpret_cast<const float *>((k & 1) ? smem + (k >> 1) * Sh::kRingBytes
                                                   : rest + (k >> 1) * (Sh::kPieceFloats * 4));
  };
  float2 R = make_float2(kNoRef, kNoRef);
#pragma unroll 1
  for (unsigned left = g.x; left; left &= left - 1) {
    const float2 r = *reinterpret_cast<const float2 *>(place(__ffs(left) - 1) + Sh::kTileFloats + col);
    R.x = fmaxf(R.x, r.x);
    R.y = fmaxf(R.y, r.y);
  }
  float4 o[D / 16];
#pragma unroll
  for (int md = 0; md < D / 16; ++md) o[md] = make_float4(0.f, 0.f, 0.f, 0.f);
  float2 l = make_float2(0.f, 0.f);
#pragma unroll 1
  for (unsigned left = g.x; left; left &= left - 1) {
    const float *x = place(__ffs(left) - 1);
    const float2 r = *reinterpret_cast<const float2 *>(x + Sh::kTileFloats + col);
    const float2 pl = *reinterpret_cast<const float2 *>(x + Sh::kTileFloats + COLS + col);
    const float f0 = piece_factor(r.x, R.x), f1 = piece_factor(r.y, R.y);
    l.x += pl.x * f0;
    l.y += pl.y * f1;
#pragma unroll
    for (int md = 0; md < D / 16; ++md) {
      const float4 v = reinterpret_cast<const float4 *>(x)[(md * NT + nt) * 32 + lane];
      o[md].x += v.x * f0;
      o[md].y += v.y * f1;
      o[md].z += v.z * f0;
      o[md].w += v.w * f1;
    }
  }
  if ((g.z & 6u) == 6u) {
#pragma unroll
    for (int md = 0; md < D / 16; ++md) store_quad<D>(p, g.y, col, lane >> 2, md, o[md], l.x, l.y);
    return;
  }
  float *dst = p.ws + (static_cast<size_t>(blockIdx.x) * 2 + (g.z & 2u ? 1 : 0)) * Sh::kPieceFloats;
#pragma unroll
  for (int md = 0; md < D / 16; ++md) reinterpret_cast<float4 *>(dst)[(md * NT + nt) * 32 + lane] = o[md];
  if (lane < 4) {
    *reinterpret_cast<float2 *>(dst + Sh::kTileFloats + col) = R;
    *reinterpret_cast<float2 *>(dst + Sh::kTileFloats + COLS + col) = l;
  }
}

// Where a warp's producer stands: run (seq, h) of n units, its next unit j.
struct Cursor {
  int seq, h, j, n, len;
  int wbase, window;  // 32 table entries from wbase on, one per lane
  bool from0;         // the current piece began at its run's first unit
  bool done;          // nothing is left to issue
};

template <int D, int BS, int NT>
__global__ void __launch_bounds__(Shape<D, NT>::kThreads, 1)
    decode_quant_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                        const Params p) {
  using Sh = Shape<D, NT>;
  constexpr int UT = Sh::kTokens, S = Sh::kStages, NW = Sh::kWarps, COLS = NT * 8, TH = Sh::kThreads;
  constexpr int BR = BS < UT ? BS : UT;   // tokens of one copy
  constexpr int BOXES = UT / BR;          // copies per unit and tensor
  constexpr int BOX_BYTES = BR * D;
  constexpr int EXP_LANES = 2 * UT / 16;  // 16 exponent bytes each
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t warp_sum[NW];
  __shared__ __align__(16) uint32_t chunk_start[TH];  // first unit of each thread's sequences
  __shared__ int chunk_len[TH];         // their length, where a thread has one sequence
  __shared__ uint4 pieces[2 * NW];      // each warp's incomplete pieces: from another warp's run, and of a run it starts
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  uint8_t *ring_ptr = smem + warp * Sh::kRingBytes;
  uint8_t *rest = smem + NW * Sh::kRingBytes;
  float *piece_ptr = reinterpret_cast<float *>(rest) + warp * Sh::kPieceFloats;
  uint8_t *exp_ptr = rest + NW * Sh::kPieceFloats * 4 + warp * Sh::kExpBytes;
  uint8_t *meta_ptr = rest + NW * (Sh::kPieceFloats * 4 + Sh::kExpBytes) + warp * (S * 16);
  uint8_t *bar_ptr = rest + NW * (Sh::kPieceFloats * 4 + Sh::kExpBytes + S * 16) + warp * (S * 8);
  const uint32_t ring = smem_u32(ring_ptr), exps = smem_u32(exp_ptr), full = smem_u32(bar_ptr);
  int4 *meta = reinterpret_cast<int4 *>(meta_ptr);

  grid_launch_dependents();
  if (lane == 0) {
    for (int s = 0; s < S; ++s) mbar_init(full + 8 * s, 1 + EXP_LANES);
    mbar_init_fence();
  }
  // A warp clears its own two entries: where runs are shared by a CTA's warps
  // (direct > 1) nothing orders one warp's clearing before another's record.
  if (lane < 2) pieces[2 * warp + lane] = make_uint4(0u, 0u, 0u, 0u);
  __syncwarp();  // a warp's barriers and entries are its own
  if (tid == 0) {
    tma_prefetch_desc(&tmk);
    tma_prefetch_desc(&tmv);
  }
  grid_dependency_wait();  // the inputs may come from the kernel launched just before

  const int cap = capped_len(p, BS);
  const int CH = (p.num_seqs + TH - 1) / TH;
  auto length = [&](int seq) {
    const int L = p.seq_lens[seq];
    return L < 0 ? 0 : min(L, cap);
  };
  auto units = [&](int L) { return (static_cast<uint32_t>(L) + UT - 1) / UT; };
  Cursor c{};
  uint32_t u0 = 0, u1 = 0;      // this warp's units of the batch's; direct: [0, whatever its runs have)
  uint32_t cq = 0, crem = 0;    // units of a CTA, and how many CTAs have one more
  int any_empty = 0;            // a sequence without keys
  // Direct, 1: warp i takes the runs i, i + (number of warps), ...; the next one
  // with keys (the others' outputs are zeros).  Direct, k > 1: k consecutive
  // warps of a CTA share one run.  The table entries load beside a run's length.
  const uint32_t runs = static_cast<uint32_t>(p.num_seqs) * static_cast<uint32_t>(p.num_kv_heads);
  const uint32_t warps = gridDim.x * NW;
  int part = 0;
  uint32_t run = blockIdx.x * NW + warp;
  if (p.direct > 1) {
    const int together = NW / p.direct, mine = warp / p.direct;
    part = warp - mine * p.direct;
    run = mine < together ? blockIdx.x * together + mine : runs;
  }
  auto take_run = [&]() {
    for (;; run += warps) {
      if (run >= runs) {
        c.done = true;
        return;
      }
      c.seq = static_cast<int>(run / static_cast<uint32_t>(p.num_kv_heads));
      c.h = static_cast<int>(run - static_cast<uint32_t>(c.seq) * p.num_kv_heads);
      const int L = p.seq_lens[c.seq];
      c.window = lane < p.max_blocks ? p.block_tables[static_cast<size_t>(c.seq) * p.max_blocks + lane] : -1;
      c.len = L < 0 ? 0 : min(L, cap);
      c.n = static_cast<int>(units(c.len));
      c.wbase = 0;
      if (p.direct > 1) {
        const int q = c.n / p.direct, r = c.n - q * p.direct;
        c.j = part * q + min(part, r);
        u1 = q + (part < r ? 1 : 0);
      }
      c.from0 = c.j == 0;
      if (L != c.len && c.h == 0 && part == 0 && lane == 0 && p.status) atomicOr(p.status, PKV_STATUS_BAD_LEN);
      if (c.n > 0) {
        c.done = u1 == 0;
        return;
      }
      if (part == 0) {
        uint4 *dst = reinterpret_cast<uint4 *>(
            p.out + (static_cast<size_t>(c.seq) * p.num_q_heads + static_cast<size_t>(c.h) * p.group) * D);
        for (int k = lane; k < p.group * (D / 8); k += 32) dst[k] = make_uint4(0u, 0u, 0u, 0u);
      }
      if (p.direct > 1 || runs - run <= warps) {  // (the sum may pass 32 bits)
        c.done = true;
        return;
      }
    }
  };
  if (p.direct) {
    u1 = 0xffffffffu;
    take_run();
  } else {
    // ---- prefix sums of the runs' units: thread i holds sequences [i CH, (i + 1) CH)
    uint32_t mine = 0;
    for (int k = 0; k < CH; ++k) {
      const int seq = tid * CH + k;
      if (seq >= p.num_seqs) break;
      int L = p.seq_lens[seq];
      if (L < 0 || L > cap) {
        if (blockIdx.x == 0 && p.status) atomicOr(p.status, PKV_STATUS_BAD_LEN);
        L = L < 0 ? 0 : cap;
      }
      mine += units(L);
      any_empty |= L == 0;
      if (k == 0) chunk_len[tid] = L;
    }
    uint32_t incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t t = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += t;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    uint32_t before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const uint32_t x = warp_sum[w];
      if (w < warp) before += x;
      total += x;
    }
    chunk_start[tid] = (before + incl - mine) * p.num_kv_heads;
    any_empty = __syncthreads_or(any_empty);
    const uint32_t U = total * p.num_kv_heads;  // below 2^31 (checked on the host)
    // as many CTAs as give every warp a unit; the others have none.  CTA c's
    // range, then the warp's part of it: equal to within a unit.  Where no run has
    // more units than a CTA has warps (no workspace), a CTA's range is moved to
    // the runs' borders: no run spans CTAs.
    const uint32_t nc = max(1u, min(gridDim.x, (U + NW - 1) / NW));
    cq = U / nc;
    crem = U - cq * nc;
    const bool whole = p.ws == nullptr && nc > 1;
    if (blockIdx.x < nc) {
      uint32_t cs = blockIdx.x * cq + min(blockIdx.x, crem), ce = cs + cq + (blockIdx.x < crem ? 1 : 0);
#pragma unroll 1
      for (int step = whole ? 0 : 2; step < 3; ++step) {  // the run at cs, at ce, at this warp's start
        if (step == 2) {
          const uint32_t size = ce - cs, wq = size / NW, wrem = size - wq * NW, w = warp;
          u0 = cs + w * wq + min(w, wrem);
          u1 = u0 + wq + (w < wrem ? 1 : 0);
          if (u0 == u1) break;
        }
        const uint32_t u = step == 0 ? cs : step == 1 ? ce : u0;
        if (u >= U) continue;  // ce of the last CTA
        // the last chunk that starts at or before u
        int at = 0;
#pragma unroll
        for (int k = 0; k < NW; ++k) at += chunk_start[k * 32 + lane] <= u ? 1 : 0;
        at = __reduce_add_sync(0xffffffffu, at) - 1;
        uint32_t base = chunk_start[at];
        c.seq = at;
        c.len = chunk_len[at];
        if (CH > 1) {  // walk the chunk, 32 sequences at a time
          for (int seq = at * CH;; seq += 32) {
            const int s = seq + lane, L = s < p.num_seqs ? length(s) : 0;
            uint32_t pre = units(L) * p.num_kv_heads;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
              const uint32_t t = __shfl_up_sync(0xffffffffu, pre, off);
              if (lane >= off) pre += t;
            }
            const unsigned in = __ballot_sync(0xffffffffu, u < base + pre);
            if (in || seq + 32 >= p.num_seqs) {
              const int src = in ? __ffs(in) - 1 : 31;
              c.seq = min(seq + src, p.num_seqs - 1);
              c.len = __shfl_sync(0xffffffffu, L, src);
              base += src > 0 ? __shfl_sync(0xffffffffu, pre, src - 1) : 0;
              break;
            }
            base += __shfl_sync(0xffffffffu, pre, 31);
          }
        }
        c.n = max(1, static_cast<int>(units(c.len)));
        c.h = static_cast<int>((u - base) / static_cast<uint32_t>(c.n));
        c.j = static_cast<int>(u - base) - c.h * c.n;
        const uint32_t border = c.j == 0 ? u : u + (c.n - c.j);  // the first run that starts at or behind u
        if (step == 0) cs = border;
        if (step == 1) ce = border;
      }
    }
    c.wbase = -32;
    c.window = -1;
    c.from0 = c.j == 0;
    c.done = u0 == u1;
  }

  bool ok = true;
  if (!c.done) {
    const uint64_t pol = l2_policy_evict_first();
    uint32_t next = u0;  // next unit to issue
    // Issue the cursor's unit into stage s and move the cursor on (whole warp).
    // meta[s]: {sequence, KV head, valid tokens | flags, units of the run behind this one};
    // flags: 16 first unit of a piece, 17 last of a piece, 18 the piece began at its run's start, 19 it ends the run
    auto issue = [&](int s) {
      const int valid = min(UT, c.len - c.j * UT);
      const bool ends = c.j + 1 == c.n;
      const int first_entry = BS <= UT ? c.j * BOXES : c.j / (BS / UT);
      const int piece_row = BS <= UT ? 0 : (c.j % (BS / UT)) * UT;  // token of the block where the unit starts
      if ((first_entry & ~31) != c.wbase) {
        c.wbase = first_entry & ~31;
        const int e = c.wbase + lane;
        c.window =
            static_cast<long long>(e) * BS < c.len ? p.block_tables[static_cast<size_t>(c.seq) * p.max_blocks + e] : -1;
      }
      const int nbox = BS <= UT ? (valid + BR - 1) / BR : 1;
      const uint32_t bar = full + 8 * s, kdst = ring + s * 2 * kUnitBytes, vdst = kdst + kUnitBytes;
      if (lane == 0) {
        meta[s] = make_int4(c.seq, c.h,
                            valid | (next == u0 || c.j == 0 ? 1 << 16 : 0) | (ends || next + 1 == u1 ? 1 << 17 : 0) |
                                (c.from0 ? 1 << 18 : 0) | (ends ? 1 << 19 : 0),
                            c.n - 1 - c.j);
        mbar_arrive_expect_tx(bar, 2 * nbox * BOX_BYTES);
      }
      int erow = -1;  // this lane's 16 exponents: their first row, or none
#pragma unroll
      for (int k = 0; k < BOXES; ++k) {
        if (k < nbox) {
          const int b = __shfl_sync(0xffffffffu, c.window, (first_entry + k) & 31);
          const bool good = b >= 0 && b < p.num_blocks;
          if (!good && lane == 0 && p.status) atomicOr(p.status, PKV_STATUS_BAD_BLOCK);
          const int row = good ? (b * p.num_kv_heads + c.h) * BS + piece_row : 0;
          if (lane == 0) {  // a bad block: a box wholly outside the tensor reads zeros
            const int y = good ? static_cast<int>(static_cast<long long>(row) * D / 128) : 0x7fffff00;
            tma_load_2d(kdst + k * BOX_BYTES, &tmk, 0, y, bar, pol);
            tma_load_2d(vdst + k * BOX_BYTES, &tmv, 0, y, bar, pol);
          }
          const int chunk = lane % (UT / 16);
          if (lane < EXP_LANES && chunk / (BR / 16) == k) erow = row + (chunk % (BR / 16)) * 16;
        }
      }
      if (lane < EXP_LANES) {
        const bool value = lane >= UT / 16;
        if (erow >= 0)
          cp_async16(exps + (s * 2 + value) * UT + (lane % (UT / 16)) * 16, (value ? p.v_exps : p.k_exps) + erow);
        cp_async_arrive(bar);
      }
      if (c.j == 0 && lane * 64 < p.group * D)  // the run's queries, 128 bytes a lane
        asm volatile("prefetch.global.L2 [%0];" ::"l"(
            p.q + (static_cast<size_t>(c.seq) * p.num_q_heads + static_cast<size_t>(c.h) * p.group) * D + lane * 64));
      __syncwarp();  // meta[s] is there for every lane
      ++next;
      if (next == u1) c.done = true;
      if (!ends) {
        ++c.j;
        return;
      }
      c.j = 0;
      c.from0 = true;
      if (p.direct == 1) {
        if (runs - run <= warps) {
          c.done = true;
        } else {
          run += warps;
          take_run();
        }
        return;
      }
      if (next >= u1 || ++c.h < p.num_kv_heads) return;
      c.h = 0;
      do {
        c.len = c.seq + 1 < p.num_seqs ? length(++c.seq) : 1;  // (the range ends before the last sequence does)
      } while (c.len == 0);
      c.n = static_cast<int>(units(c.len));
      c.wbase = -32;
    };

    for (int s = 0; s < S && !c.done; ++s) issue(s);

    Acc<D, NT> acc;
    uint32_t qf[NT][D / 16][2];
    float cf[NT][2];
    const int g4 = lane >> 2, c4 = lane & 3;
    int i = 0;
    for (; i < static_cast<int>(next - u0); ++i) {
      const int s = i % S;
      const int4 m = meta[s];
      if (m.z & (1 << 16)) {  // while the unit is on its way
        load_queries<D, NT>(p, m.x, m.y, qf, cf, lane);
        acc.reset();
      }
      if (!mbar_wait(full + 8 * s, static_cast<uint32_t>(i / S) & 1)) ok = false;
      if (!__all_sync(0xffffffffu, ok)) {
        if (lane == 0 && p.status) atomicOr(p.status, PKV_STATUS_TIMEOUT);
        ok = false;
        break;
      }
      const uint32_t kb = ring + s * 2 * kUnitBytes, eb = exps + s * 2 * UT;
      const int valid = m.z & 0xFFFF;
      if constexpr (Sh::kStep == UT) {
        attend_tokens<D, NT, UT / 16>(acc, qf, cf, kb, kb + kUnitBytes, eb, eb + UT, valid, lane);
      } else {
#pragma unroll 1
        for (int t = 0; t < valid; t += Sh::kStep)
          attend_tokens<D, NT, Sh::kStep / 16>(acc, qf, cf, kb + t * D, kb + kUnitBytes + t * D, eb + t, eb + UT + t,
                                               valid - t, lane);
      }
      __syncwarp();
      if (!c.done) issue(s);
      if (m.z & (1 << 17)) {  // the piece ends here
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float l = acc.l[nt][e];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            acc.l[nt][e] = l;
          }
        const bool from0 = m.z & (1 << 18), ends = m.z & (1 << 19);
        if (from0 && ends) {
          // the whole run: values g D/8 .. of this lane's two heads per tile
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int col = nt * 8 + 2 * c4 + e;
              if (col >= p.group) continue;
              const float inv = 1.f / acc.l[nt][e];  // (store_quad)
              uint32_t w[D / 16];
#pragma unroll
              for (int md = 0; md < D / 16; ++md)
                w[md] = pack_bf16x2(acc.o[md][nt][e] * inv, acc.o[md][nt][e + 2] * inv);
              uint4 *dst = reinterpret_cast<uint4 *>(
                  p.out + (static_cast<size_t>(m.x) * p.num_q_heads + static_cast<size_t>(m.y) * p.group + col) * D +
                  g4 * (D / 8));
#pragma unroll
              for (int k = 0; k < D / 64; ++k)
                dst[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
            }
        } else {
          // a first piece goes to its own place, a last one (from a run's start) over the drained ring
          float *dst = from0 ? reinterpret_cast<float *>(ring_ptr) : piece_ptr;
          float4 *o4 = reinterpret_cast<float4 *>(dst) + lane;
#pragma unroll
          for (int md = 0; md < D / 16; ++md)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              o4[(md * NT + nt) * 32] =
                  make_float4(acc.o[md][nt][0], acc.o[md][nt][1], acc.o[md][nt][2], acc.o[md][nt][3]);
          if (g4 == 0)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                dst[Sh::kTileFloats + nt * 8 + 2 * c4 + e] = acc.r[nt][e];
                dst[Sh::kTileFloats + COLS + nt * 8 + 2 * c4 + e] = acc.l[nt][e];
              }
          // {sequence | KV head << 16, 1 | began at the run's start << 1 | ends it << 2, the run's last unit}
          if (lane == 0)
            pieces[2 * warp + (from0 ? 1 : 0)] =
                make_uint4(static_cast<uint32_t>(m.x) | (static_cast<uint32_t>(m.y) << 16),
                           1u | (from0 ? 2u : 0u) | (ends ? 4u : 0u), u0 + i + m.w, 0u);
        }
      }
    }
    // after a timeout: leave no copy in flight into this CTA's shared memory
    if (!ok)
      for (int k = i + 1; k < static_cast<int>(next - u0); ++k) mbar_wait(full + 8 * (k % S), (k / S) & 1);
  }
  if (p.direct == 1) return;
  const bool failed = __syncthreads_or(!ok);

  // ---- join the pieces of each run
  if (!failed) {
    // the pieces of one run each: {their places, run, flags, its last unit}
    uint4 *groups = reinterpret_cast<uint4 *>(chunk_start);
    static_assert(2 * NW * sizeof(uint4) <= sizeof chunk_start, "the table goes over the prefix sums");
    const unsigned below = (1u << lane) - 1;
    const uint4 info = lane < 2 * NW ? pieces[lane] : make_uint4(0u, 0u, 0u, 0u);
    const unsigned all = __ballot_sync(0xffffffffu, info.y & 1u);
    // a piece opens a group where the one before it is another run's
    const uint32_t before_it = __shfl_sync(0xffffffffu, info.x, 31 - __clz(all & below | 1u));
    const bool opens = (info.y & 1u) && (!(all & below) || before_it != info.x);
    const unsigned starts = __ballot_sync(0xffffffffu, opens);
    const unsigned later = starts & ~below & ~(1u << lane);
    const unsigned same = all & ~below & (later ? (later & -later) - 1 : ~0u);
    const uint32_t end_flags = __shfl_sync(0xffffffffu, info.y, same ? 31 - __clz(same) : 0);
    // every warp writes the same table, and reads what it wrote
    if (opens)
      groups[__popc(starts & below)] = make_uint4(same, info.x, (info.y & 2u) | (end_flags & 4u), info.z);
    __syncwarp();
    const int count = __popc(starts);
    if (tid == TH - 1 && p.ws_desc) {  // the run that leaves this CTA, if any, and the CTA that holds its last unit
      const uint4 g = count ? groups[count - 1] : make_uint4(0u, 0u, 4u, 0u);
      const uint32_t big = crem * (cq + 1);
      int4 desc = make_int4(0, 0, 0, 0);
      if ((g.z & 6u) == 2u)
        desc = make_int4(g.y, 0, static_cast<int>(g.w < big ? g.w / (cq + 1) : crem + (g.w - big) / cq), 1);
      p.ws_desc[blockIdx.x] = desc;
    }
    for (int t = warp; t < count * NT; t += NW) join_pieces<D, NT>(p, groups[t / NT], t % NT, smem, rest, lane);
  } else if (tid == 0 && p.ws_desc) {
    p.ws_desc[blockIdx.x] = make_int4(0, 0, 0, 0);
  }

  // ---- sequences without keys: zeros
  if (!any_empty) return;
  for (int s = blockIdx.x + gridDim.x * warp; s < p.num_seqs; s += gridDim.x * NW) {
    if (length(s) != 0) continue;
    uint4 *dst = reinterpret_cast<uint4 *>(p.out + static_cast<size_t>(s) * p.num_q_heads * D);
    for (int k = lane; k < p.num_q_heads * D / 8; k += 32) dst[k] = make_uint4(0u, 0u, 0u, 0u);
  }
}

// A thread's share of the join of a run's pieces: one accumulator quad.
struct Joined {
  float2 R = make_float2(kNoRef, kNoRef), l = make_float2(0.f, 0.f);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  __device__ __forceinline__ void refer_to(const float2 &M) {
    const float f0 = piece_factor(R.x, M.x), f1 = piece_factor(R.y, M.y);
    l.x *= f0, l.y *= f1, o.x *= f0, o.y *= f1, o.z *= f0, o.w *= f1;
    R = M;
  }
  __device__ __forceinline__ void add(const float2 &r, const float2 &pl, const float4 &v) {
    const float f0 = piece_factor(r.x, R.x), f1 = piece_factor(r.y, R.y);
    l.x += pl.x * f0, l.y += pl.y * f1, o.x += v.x * f0, o.y += v.y * f1, o.z += v.z * f0, o.w += v.w * f1;
  }
  // Pieces i0, i0 + step, ... of the n that follow each other from `first` on
  // (CTA c0's last piece, then the first ones of the CTAs behind it), FLY of
  // them in flight; quad `t` of head column `col`.
  template <int D, int NT, int FLY>
  __device__ __forceinline__ void take(const float *first, int n, int i0, int step, int t, int col, int lane) {
    using Sh = Shape<D, NT>;
#pragma unroll 1
    for (int base = i0; base < n; base += FLY * step) {
      float2 r[FLY], pl[FLY];
      float4 v[FLY];
#pragma unroll
      for (int k = 0; k < FLY; ++k) {
        const int i = base + k * step;
        const float *x = first + (i == 0 ? 0 : i * 2 - 1) * static_cast<size_t>(Sh::kPieceFloats);
        r[k] = i < n ? *reinterpret_cast<const float2 *>(x + Sh::kTileFloats + col) : make_float2(kNoRef, kNoRef);
        pl[k] = i < n ? *reinterpret_cast<const float2 *>(x + Sh::kTileFloats + NT * 8 + col) : make_float2(0.f, 0.f);
        v[k] = i < n ? reinterpret_cast<const float4 *>(x)[t * 32 + lane] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float2 M = R;
#pragma unroll
      for (int k = 0; k < FLY; ++k) M.x = fmaxf(M.x, r[k].x), M.y = fmaxf(M.y, r[k].y);
      refer_to(M);
#pragma unroll
      for (int k = 0; k < FLY; ++k) add(r[k], pl[k], v[k]);
    }
  }
  // Another thread's share of the same quad, through shared memory.
  __device__ __forceinline__ void give(float4 *slot) const {
    slot[0] = o;
    slot[1] = make_float4(R.x, R.y, l.x, l.y);
  }
  __device__ __forceinline__ void get(const float4 *slot) {
    const float4 x = slot[1];
    refer_to(make_float2(fmaxf(R.x, x.x), fmaxf(R.y, x.y)));
    add(make_float2(x.x, x.y), make_float2(x.z, x.w), slot[0]);
  }
};

// The run that starts in CTA c and spans more (blockIdx.x = c), by one block:
// every kSplit-th piece goes to one group of threads, five in flight, and the
// groups are joined in shared memory.
template <int D, int NT>
struct JoinShape {
  static constexpr int kLanes = D * NT * 2;
  static constexpr int kSplit = kLanes <= 256 ? 4 : 2;
  static constexpr int kThreads = kLanes * kSplit;
};

template <int D, int NT>
__global__ void __launch_bounds__(JoinShape<D, NT>::kThreads) join_kernel(const Params p) {
  using J = JoinShape<D, NT>;
  __shared__ float4 part[J::kSplit - 1][J::kLanes][2];
  grid_launch_dependents();
  const int c0 = blockIdx.x, grp = threadIdx.x / J::kLanes, quad = threadIdx.x % J::kLanes;
  const int t = quad >> 5, lane = quad & 31, md = t / NT, col = (t - md * NT) * 8 + 2 * (lane & 3);
  grid_dependency_wait();  // the pieces come from the grid launched just before
  const int4 desc = p.ws_desc[c0];
  if (desc.w == 0) return;
  const int n = desc.z - c0 + 1;
  Joined acc;
  acc.take<D, NT, 5>(p.ws + (static_cast<size_t>(c0) * 2 + 1) * Shape<D, NT>::kPieceFloats, n, grp, J::kSplit, t, col, lane);
  if (grp > 0) acc.give(part[grp - 1][quad]);
  __syncthreads();
  if (grp > 0) return;
  for (int k = 1; k < min(n, J::kSplit); ++k) acc.get(part[k - 1][quad]);
  store_quad<D>(p, static_cast<uint32_t>(desc.x), col, lane >> 2, md, acc.o, acc.l.x, acc.l.y);
}

// For few runs, which span many CTAs each: block (x, t) joins quad row t of the
// x-th run that spans CTAs, every 32nd piece by one warp, three in flight.
constexpr int kFewWarps = 32;

template <int D, int NT>
__global__ void __launch_bounds__(kFewWarps * 32) join_few_kernel(const Params p, int ctas) {
  constexpr int kLast = 4;  // warps of the last but one step
  __shared__ float4 part[kFewWarps][32][2];
  __shared__ int leaving[kFewWarps], found[3];
  grid_launch_dependents();
  const int t = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int md = t / NT, col = (t - md * NT) * 8 + 2 * (lane & 3);
  if (threadIdx.x == 0) found[0] = -1;
  grid_dependency_wait();
  // thread c stands for CTA c: the one whose run is the x-th to leave
  const int4 d = static_cast<int>(threadIdx.x) < ctas ? p.ws_desc[threadIdx.x] : make_int4(0, 0, 0, 0);
  const unsigned leaves = __ballot_sync(0xffffffffu, d.w != 0);
  if (lane == 0) leaving[warp] = __popc(leaves);
  __syncthreads();
  if (d.w != 0) {
    int before = __popc(leaves & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) before += leaving[w];
    if (before == static_cast<int>(blockIdx.x)) {
      found[0] = threadIdx.x;
      found[1] = d.z;
      found[2] = d.x;
    }
  }
  __syncthreads();
  const int c0 = found[0], n = found[1] - c0 + 1;
  if (c0 < 0) return;
  Joined acc;
  acc.take<D, NT, 3>(p.ws + (static_cast<size_t>(c0) * 2 + 1) * Shape<D, NT>::kPieceFloats, n, warp, kFewWarps, t, col, lane);
  acc.give(part[warp][lane]);
  __syncthreads();
  if (warp < kLast) {
    for (int k = warp + kLast; k < min(n, kFewWarps); k += kLast) acc.get(part[k][lane]);
    acc.give(part[warp][lane]);
  }
  __syncthreads();
  if (warp > 0) return;
  for (int k = 1; k < min(n, kLast); ++k) acc.get(part[k][lane]);
  store_quad<D>(p, static_cast<uint32_t>(found[2]), col, lane >> 2, md, acc.o, acc.l.x, acc.l.y);
}

// ------------------------------------------------------------------------ host
struct Plan {
  int grid = 1;
  size_t piece_bytes = 0;
  bool whole = false;   // runs are not split between CTAs
  int direct = 0;       // as Params::direct
  size_t ws_bytes() const { return grid > 1 && !whole ? grid * (2 * piece_bytes + sizeof(int4)) : 0; }
};

// The grid: one CTA per SM, fewer when the longest possible batch has fewer
// than a unit per warp.  One CTA needs no workspace and no second kernel, and so
// do short sequences.
Plan make_plan(int num_seqs, int num_kv_heads, int group, int head_dim, int max_seq_len) {
  const int nt = group > 8 ? 2 : 1, tokens = kUnitBytes / head_dim;
  const int warps = head_dim == 128 ? (nt == 1 ? Shape<128, 1>::kWarps : Shape<128, 2>::kWarps)
                                    : (nt == 1 ? Shape<64, 1>::kWarps : Shape<64, 2>::kWarps);
  const double units = static_cast<double>(num_seqs) * num_kv_heads * ((max_seq_len + (tokens - 1ll)) / tokens);
  Plan plan;
  plan.grid = static_cast<int>(std::max(1.0, std::min<double>(num_sms(), std::ceil(units / warps))));
  const long long longest = (max_seq_len + (tokens - 1ll)) / tokens;
  // Runs of a unit or two go to the warps whole, without prefix sums or joins,
  // where each warp gets one at most, or so many that uneven numbers do not
  // matter.  Measured, this way / by equal units: 3 sequences 3.6 / 4.6 us, 1688
  // runs of up to 2 units 7.1 / 10.6, 4096 of 2 (2.2 a warp) 22.0 / 20.5.  Where
  // there are few longer ones, a run gets as many warps of one CTA as the longest
  // has units, and only a join: 22 x up to 120 tokens x 8 heads 5.4 / 8.4 us,
  // 18 x up to 380 8.1 / 10.1, 8 x 704 9.4 / 11.2; at four units a warp it is
  // even (8 x 1400 13.1 / 13.5, 2 x 1400 12.6 / 10.5).
  const double runs = static_cast<double>(num_seqs) * num_kv_heads, slots = static_cast<double>(num_sms()) * warps;
  const int share = static_cast<int>(std::min<long long>(warps, std::max(1ll, longest))), together = warps / share;
  if (longest <= kDirectUnits && (runs <= slots || runs >= 8 * slots)) {
    plan.direct = 1;
    plan.grid = static_cast<int>(std::min<double>(num_sms(), std::ceil(runs / warps)));
  } else if (longest <= kDirectRounds * warps && runs <= static_cast<double>(num_sms()) * together) {
    plan.direct = share;
    plan.grid = static_cast<int>(std::ceil(runs / together));
  }
  // A run of at most a unit per warp is not worth splitting between CTAs: the
  // second kernel costs more (about 3 us) than the runs' uneven ends.
  plan.whole = longest <= warps || plan.direct;
  plan.piece_bytes = (static_cast<size_t>(nt) * 8 * head_dim + 2 * nt * 8) * sizeof(float);
  return plan;
}

bool sizes_valid(int num_seqs, int max_seq_len, int num_q_heads, int num_kv_heads) {
  return num_seqs >= 0 && max_seq_len >= 0 && num_q_heads >= 1 && num_kv_heads >= 1 && num_q_heads % num_kv_heads == 0;
}

bool sizes_supported(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim) {
  return (head_dim == 64 || head_dim == 128) && num_q_heads / num_kv_heads <= kMaxGroup && num_seqs <= 65535 &&
         num_kv_heads <= 65535;
}

int check_decode(const void *q, const void *k_codes, const void *v_codes, const void *k_exps, const void *v_exps,
                 const int32_t *block_tables, int max_blocks_per_seq, const int32_t *seq_lens, int num_seqs,
                 int max_seq_len, int num_q_heads, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                 float scale, const void *out) {
  if (!sizes_valid(num_seqs, max_seq_len, num_q_heads, num_kv_heads) || max_blocks_per_seq < 0 || num_blocks < 0 ||
      !std::isfinite(scale))
    return PKV_ERR_ARG;
  if (!sizes_supported(num_seqs, num_q_heads, num_kv_heads, head_dim)) return PKV_ERR_UNSUPPORTED;
  if (block_size != 16 && block_size != 32 && block_size != 64 && block_size != 128) return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PKV_OK;
  if (!q || !k_codes || !v_codes || !k_exps || !v_exps || !block_tables || !seq_lens || !out || num_blocks == 0)
    return PKV_ERR_ARG;
  if (!aligned16(q) || !aligned16(k_codes) || !aligned16(v_codes) || !aligned16(k_exps) || !aligned16(v_exps) ||
      !aligned16(out) || (reinterpret_cast<uintptr_t>(block_tables) & 3u) ||
      (reinterpret_cast<uintptr_t>(seq_lens) & 3u))
    return PKV_ERR_ARG;
  const long long rows = static_cast<long long>(num_blocks) * num_kv_heads * block_size;
  if (rows + block_size >= 0x7fffff00ll) return PKV_ERR_UNSUPPORTED;
  // the batch's units are counted in 31 bits
  const long long len = std::min<long long>(max_seq_len, static_cast<long long>(max_blocks_per_seq) * block_size);
  const int tokens = kUnitBytes / head_dim;
  if (static_cast<double>(num_seqs) * num_kv_heads * ((len + tokens - 1) / tokens) >= 2147483648.0)
    return PKV_ERR_UNSUPPORTED;
  return PKV_OK;
}

template <int D, int BS, int NT>
cudaError_t launch(const CUtensorMap &tmk, const CUtensorMap &tmv, const Params &p, int grid, cudaStream_t stream) {
  using Sh = Shape<D, NT>;
  auto k = decode_quant_kernel<D, BS, NT>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmemBytes);
  if (e == cudaSuccess) e = launch_overlapped(k, grid, Sh::kThreads, Sh::kSmemBytes, stream, tmk, tmv, p);
  if (e != cudaSuccess || !p.ws) return e;
  // Runs of eight pieces and more, of which there are few, go to more blocks.
  // Measured, join_kernel / join_few_kernel: 1 run of 131072 tokens 23.3 / 16.9
  // us, 2 of 65536 19.8 / 16.7, 8 of 32768 21.0 / 20.3, 16 of 20000 22.2 / 22.1.
  const long long runs = static_cast<long long>(p.num_seqs) * p.num_kv_heads;
  if (grid > 8 * runs && grid <= kFewWarps * 32)
    e = launch_overlapped(join_few_kernel<D, NT>, dim3(static_cast<unsigned>(runs), D / 16 * NT), kFewWarps * 32, 0, stream, p, grid);
  else
    e = launch_overlapped(join_kernel<D, NT>, grid, JoinShape<D, NT>::kThreads, 0, stream, p);
  return e;
}

template <int D, int NT>
cudaError_t by_block(const CUtensorMap &tmk, const CUtensorMap &tmv, const Params &p, int grid, int block_size,
                     cudaStream_t stream) {
  switch (block_size) {
    case 16: return launch<D, 16, NT>(tmk, tmv, p, grid, stream);
    case 32: return launch<D, 32, NT>(tmk, tmv, p, grid, stream);
    case 64: return launch<D, 64, NT>(tmk, tmv, p, grid, stream);
    default: return launch<D, 128, NT>(tmk, tmv, p, grid, stream);
  }
}

}  // namespace
}  // namespace pkv

extern "C" {

size_t paged_attention_decode_quant_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                                   int max_seq_len) {
  if (!pkv::sizes_valid(num_seqs, max_seq_len, num_q_heads, num_kv_heads) ||
      !pkv::sizes_supported(num_seqs, num_q_heads, num_kv_heads, head_dim) || num_seqs == 0)
    return 0;
  return pkv::make_plan(num_seqs, num_kv_heads, num_q_heads / num_kv_heads, head_dim, max_seq_len).ws_bytes();
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
  const int group = num_q_heads / num_kv_heads;
  const pkv::Plan plan = pkv::make_plan(num_seqs, num_kv_heads, group, head_dim, max_seq_len);
  if (plan.ws_bytes() > 0 && (!workspace || workspace_bytes < plan.ws_bytes() || !pkv::aligned16(workspace)))
    return PKV_ERR_WORKSPACE;

  // the code arrays as rows of 128 bytes, copied a block (or a unit's part of one) at a time
  const int unit_tokens = pkv::kUnitBytes / head_dim, box_tokens = std::min(block_size, unit_tokens);
  const long long rows = static_cast<long long>(num_blocks) * num_kv_heads * block_size * head_dim / 128;
  CUtensorMap tmk, tmv;
  if (!pkv::make_tensor_map_bytes(&tmk, k_codes, rows, box_tokens * head_dim / 128) ||
      !pkv::make_tensor_map_bytes(&tmv, v_codes, rows, box_tokens * head_dim / 128))
    return PKV_ERR_CUDA;

  pkv::Params p{};
  p.q = reinterpret_cast<const __nv_bfloat16 *>(q);
  p.k_exps = k_exps;
  p.v_exps = v_exps;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.out = reinterpret_cast<__nv_bfloat16 *>(out);
  if (plan.ws_bytes() > 0) {
    p.ws = static_cast<float *>(workspace);
    p.ws_desc = reinterpret_cast<int4 *>(static_cast<char *>(workspace) + plan.grid * 2 * plan.piece_bytes);
  }
  p.status = d_status;
  p.direct = plan.direct;
  p.num_seqs = num_seqs;
  p.max_blocks = max_blocks_per_seq;
  p.max_len = max_seq_len;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = group;
  p.num_blocks = num_blocks;
  p.scale_log2 = scale * pkv::kLog2e;
  cudaStream_t st = pkv::as_stream(stream);
  const cudaError_t e =
      head_dim == 128 ? (group > 8 ? pkv::by_block<128, 2>(tmk, tmv, p, plan.grid, block_size, st)
                                   : pkv::by_block<128, 1>(tmk, tmv, p, plan.grid, block_size, st))
                      : (group > 8 ? pkv::by_block<64, 2>(tmk, tmv, p, plan.grid, block_size, st)
                                   : pkv::by_block<64, 1>(tmk, tmv, p, plan.grid, block_size, st));
  if (e != cudaSuccess) return pkv::set_cuda_error(e), PKV_ERR_CUDA;
  return PKV_OK;
}

}  // extern "C"
