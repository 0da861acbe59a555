// Windowed attention of single tokens: paged_attention_window without q_start.
//
// Math: out = softmax(scale * q K^T) V over the keys of the window and the sinks,
// with the running maximum and sum of the online softmax.  All query heads of a
// group see the same keys.
//
// The keys and values that are seen are read once, so the kernel is bound by HBM
// and has to keep every SM streaming.  The runs, one per (sequence, KV head), are
// cut into units of 32 keys (those of the sinks, then those of the window) and
// laid end to end; every warp of a grid of one CTA per SM takes an equal,
// contiguous range of units and streams it through two stages of its own: TMA
// copies of the unit's keys and values (with the 128-byte swizzle) and, with the
// first unit of a run, of its queries.  A stage is filled again as soon as it has
// been used, so no warp waits for another.  Per unit: S^T = K Q^T and O^T += V^T
// P^T on bf16 MMA (m16n8k16), keys as the M dimension, the group's query heads as
// N, fp32 softmax in between.
//
// A run that lies in one warp's range is written at once.  The pieces of one that
// does not (at most two per warp) go to the workspace, and a second kernel joins
// them in the order of the warps: results repeat bit for bit.  Where no run has
// more than kDirectUnits units, whole runs go to the warps instead, and there is
// neither workspace nor second kernel.
//
// Measured (clocks at 2070 MHz, of a copy's 6.78 TB/s): 256 sequences of mixed lengths,
// window 1024 and 4 sinks, 32 / 8 heads of 128: 103 to 105 us, 5.8 TB/s; 16 sequences of
// 32768 tokens, window 4096, 64 / 8 heads: 48 to 49 us, 5.5 TB/s.  On the tensor cores' kernel
// (spans_tc.cu with tiles of one token) they take 142 and 60 us: a tile of 128 rows holds
// G that are used, and one CTA keeps fewer copies in flight than these warps' rings.
// What is left is the start (dependent loads of lengths and tables, about 3 us) and the
// second kernel (about 4 us).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "attend.cuh"
#include "internal.h"
#include "launch.cuh"
#include "pkv.h"
#include "ptx.cuh"
#include "spans.cuh"

namespace pkv {
namespace spans {
namespace {

using attend::kLog2e;
using attend::swz;

constexpr int kUnit = 32;        // keys
constexpr int kStages = 2;
constexpr int kDirectUnits = 4;  // runs of at most so many units go to a warp whole
constexpr int kMinUnits = 4;     // of a warp's range

struct StepParams {
  const __nv_bfloat16 *q;
  const int32_t *block_tables, *seq_lens;
  __nv_bfloat16 *out;
  float4 *ws_o;    // [2 warps][D / 16][NT][32 lanes], in accumulator order
  float2 *ws_ml;   // [2 warps][NT * 8]
  int4 *ws_desc;   // [warps]: {sequence, KV head, flags, -}; NULL: whole runs only
  int32_t *status;
  int num_seqs, max_blocks, max_len, num_q_heads, num_kv_heads, group, num_blocks, oob_row;
  int window, sinks;
  float scale_log2;
};

constexpr int kLeaves = 1;  // the warp's last run goes on in the next warp (piece 1 holds its start)
constexpr int kEnds = 2;    // the run that the warp goes on with (piece 0) ends here

template <int D, int NT, int BS>
struct Shape {
  static constexpr int kBoxRows = BS < kUnit ? BS : kUnit;  // rows of one copy
  static constexpr int kBoxes = kUnit / kBoxRows;
  static constexpr int kBoxBytes = kBoxRows * D * 2;
  static constexpr int kTile = kUnit * D * 2;               // keys (or values) of a unit
  static constexpr int kQBytes = NT * 8 * D * 2;
  static constexpr int kStage = 2 * kTile + kQBytes;
  // as many warps as 227 KB of shared memory hold two stages of each for
  static constexpr int kWarps = D == 128 ? (NT == 1 ? 6 : 5) : (NT == 1 ? 12 : 11);
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kSmem = 1024 + kWarps * kStages * kStage + kWarps * kStages * 8;
  static_assert(kStage % 1024 == 0, "swizzle atoms");
  static_assert(kSmem + kThreads * 8 + 64 <= 227 * 1024, "shared memory");
};

// The units of a sequence of L tokens: [0, ns) the sinks', then from t_lo on.
struct Keys {
  int L, lo, sink_end, ns, t_lo, n;
  __device__ __forceinline__ Keys() {}
  __device__ __forceinline__ Keys(const StepParams &p, int len) : L(len) {
    lo = max(0, L - p.window);
    sink_end = min(p.sinks, lo);
    t_lo = lo / kUnit;
    ns = min((sink_end + kUnit - 1) / kUnit, t_lo);
    n = max(1, ns + (L + kUnit - 1) / kUnit - t_lo);  // an empty sequence: one unit without keys
  }
  __device__ __forceinline__ int key0(int u) const { return kUnit * (u < ns ? u : u - ns + t_lo); }
  // what the row sees of the 32 keys from k0 on
  __device__ __forceinline__ uint32_t seen(int k0) const {
    return (below(L - k0) & ~below(lo - k0)) | below(sink_end - k0);
  }
  static __device__ __forceinline__ uint32_t below(int x) { return x <= 0 ? 0u : x >= 32 ? ~0u : (1u << x) - 1; }
};

template <int BS>
__device__ __forceinline__ int length(const StepParams &p, int seq, bool report) {
  const long long cap_tbl = static_cast<long long>(p.max_blocks) * BS;
  const int cap = static_cast<int>(cap_tbl < p.max_len ? cap_tbl : p.max_len);
  int L = p.seq_lens[seq];
  if (L < 0 || L > cap) {
    if (report && p.status) atomicOr(p.status, PKV_STATUS_BAD_LEN);
    L = L < 0 ? 0 : cap;
  }
  return L;
}

// A position in the row of all units.
struct Cursor {
  int seq, head, u;  // u: unit of the run
  Keys k;
  template <int BS>
  __device__ void enter(const StepParams &p, int s) {
    seq = s;
    if (seq < p.num_seqs) k = Keys(p, length<BS>(p, seq, false));
  }
  // the next unit; true: of another run
  template <int BS>
  __device__ bool advance(const StepParams &p) {
    if (++u < k.n) return false;
    u = 0;
    if (++head == p.num_kv_heads) {
      head = 0;
      enter<BS>(p, seq + 1);
    }
    return true;
  }
};

template <int D, int NT>
struct Acc {
  float m[NT][2], l[NT][2];  // the lane's two columns of each 8: reference (log2 units), its part of the sum
  float o[D / 16][NT][4];
  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int md = 0; md < D / 16; ++md) o[md][nt][0] = o[md][nt][1] = o[md][nt][2] = o[md][nt][3] = 0.f;
    }
  }
};

// One staged unit.  see: bit per key.
template <int D, int NT, int R>
__device__ __forceinline__ void attend_unit(Acc<D, NT> &acc, const uint32_t (&qf)[NT][D / 16][2], uint32_t kb, uint32_t vb,
                                            uint32_t see, float scale_log2, int lane) {
  constexpr int MT = kUnit / 16;
  const int r8 = lane & 7, mi = lane >> 3, g4 = lane >> 2, c4 = lane & 3;
  // S^T[key][head]: even and odd steps in registers of their own, so that two chains of products overlap
  float sc[MT][NT][4], sc2[MT][NT][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[mt][nt][i] = sc2[mt][nt][i] = 0.f;
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      uint32_t a[4];
      ldsm_x4(swz<R, D / 64>(kb, mt * 16 + r8 + (mi & 1) * 8, ks * 2 + (mi >> 1)), a);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma_bf16_16816(ks & 1 ? sc2[mt][nt] : sc[mt][nt], a, qf[nt][ks][0], qf[nt][ks][1]);
    }
  float top[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) top[nt][0] = top[nt][1] = -INFINITY;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float s = (sc[mt][nt][i] + sc2[mt][nt][i]) * scale_log2;
        sc[mt][nt][i] = (see >> (mt * 16 + g4 + (i >> 1) * 8)) & 1 ? s : -INFINITY;
        top[nt][i & 1] = fmaxf(top[nt][i & 1], sc[mt][nt][i]);
      }
  // the reference moves only where a score passes it by more than the slack
  bool moved = false;
  float alpha[NT][2], ref[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float t = top[nt][e];
      t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
      t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
      t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
      const float m = acc.m[nt][e];
      alpha[nt][e] = 1.f;
      if (t > m + attend::kRescaleSlack) {
        alpha[nt][e] = m == -INFINITY ? 0.f : exp2f(m - t);
        acc.m[nt][e] = t;
        moved = true;
      }
      ref[nt][e] = acc.m[nt][e] == -INFINITY ? 0.f : acc.m[nt][e];
    }
  if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        acc.l[nt][e] *= alpha[nt][e];
#pragma unroll
        for (int md = 0; md < D / 16; ++md) {
          acc.o[md][nt][e] *= alpha[nt][e];
          acc.o[md][nt][e + 2] *= alpha[nt][e];
        }
      }
  }
  // weights: summed in fp32 as they are, rounded to bf16 for the product with the values (both
  // operands of a matrix instruction have one 16-bit type, and fp16 does not hold bf16 values)
  uint32_t pb[MT][NT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = fast_exp2(sc[mt][nt][i] - ref[nt][i & 1]);
        acc.l[nt][i & 1] += w[i];
      }
      pb[mt][nt][0] = movmatrix_trans(pack_bf16x2(w[0], w[1]));
      pb[mt][nt][1] = movmatrix_trans(pack_bf16x2(w[2], w[3]));
    }
  // O^T[d][head] += V^T[d][key] P^T[key][head]; values that are not seen are cleared (0 times NaN is NaN)
#pragma unroll
  for (int kt = 0; kt < MT; ++kt) {
    const uint32_t s = see >> (kt * 16 + 2 * c4);
    const bool all = ((see >> (kt * 16)) & 0xFFFFu) == 0xFFFFu;
    const uint32_t m0 = (s & 1u ? 0x0000FFFFu : 0u) | (s & 2u ? 0xFFFF0000u : 0u);
    const uint32_t m1 = ((s >> 8) & 1u ? 0x0000FFFFu : 0u) | ((s >> 8) & 2u ? 0xFFFF0000u : 0u);
#pragma unroll
    for (int md = 0; md < D / 16; ++md) {
      uint32_t a[4];
      ldsm_x4_trans(swz<R, D / 64>(vb, kt * 16 + r8 + (mi >> 1) * 8, md * 2 + (mi & 1)), a);
      if (!all) {
        a[0] &= m0;
        a[1] &= m0;
        a[2] &= m1;
        a[3] &= m1;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma_bf16_16816(acc.o[md][nt], a, pb[kt][nt][0], pb[kt][nt][1]);
    }
  }
}

template <int D, int NT, int BS>
__global__ void __launch_bounds__(Shape<D, NT, BS>::kThreads, 1)
    step_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const StepParams p) {
  using Sh = Shape<D, NT, BS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ long long sums[Sh::kThreads];  // units before each thread's stretch of sequences
  __shared__ long long warp_sums[Sh::kWarps + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = smem_u32(smem) + warp * kStages * Sh::kStage;
  const uint32_t bars = smem_u32(smem) + Sh::kWarps * kStages * Sh::kStage + warp * kStages * 8;
  grid_launch_dependents();
  grid_dependency_wait();

  // units (or runs) before each thread's stretch of sequences
  const int per = (p.num_seqs + Sh::kThreads - 1) / Sh::kThreads;
  const int s0 = min(p.num_seqs, static_cast<int>(threadIdx.x) * per), s1 = min(p.num_seqs, s0 + per);
  const bool direct = p.ws_desc == nullptr;
  long long mine = 0;
  for (int i = s0; i < s1; ++i) {
    const int L = length<BS>(p, i, blockIdx.x == 0);
    mine += direct ? 1 : Keys(p, L).n;
  }
  mine *= p.num_kv_heads;
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sums[warp + 1] = incl;
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < kStages; ++s) mbar_init(bars + 8 * s, 1);
    mbar_init_fence();
    if (warp == 0) {
      warp_sums[0] = 0;
      tma_prefetch_desc(&tmk);
      tma_prefetch_desc(&tmv);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0)
    for (int w = 0; w < Sh::kWarps; ++w) warp_sums[w + 1] += warp_sums[w];
  __syncthreads();
  sums[threadIdx.x] = warp_sums[warp] + incl - mine;
  __syncthreads();
  const long long total = warp_sums[Sh::kWarps];

  // this warp's range
  const int me = blockIdx.x * Sh::kWarps + warp;
  long long warps = static_cast<long long>(gridDim.x) * Sh::kWarps;
  if (!direct) warps = min(warps, max(1ll, total / kMinUnits));
  const long long xa = me < warps ? total * me / warps : total, xb = me < warps ? total * (me + 1) / warps : total;
  int4 desc = make_int4(0, 0, 0, 0);
  if (xa < xb) {
    // its first unit: the thread stretch, the sequence, the head
    int lo = 0, hi = Sh::kThreads;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sums[mid] <= xa) lo = mid; else hi = mid;
    }
    // (empty stretches at the end share their sum with the total, which xa is below)
    Cursor at;
    long long off = xa - sums[lo];
    at.enter<BS>(p, min(p.num_seqs - 1, lo * per));
    while (true) {
      const long long n = static_cast<long long>(direct ? 1 : at.k.n) * p.num_kv_heads;
      if (off < n) break;
      off -= n;
      at.enter<BS>(p, at.seq + 1);
    }
    long long count = xb - xa;  // units, or runs
    at.head = static_cast<int>(off / (direct ? 1 : at.k.n));
    at.u = direct ? 0 : static_cast<int>(off - static_cast<long long>(at.head) * at.k.n);

    const uint64_t pol = l2_policy_evict_first();
    // ---- copies: `next` runs kStages units ahead of `at`
    Cursor next = at;
    long long left = count;  // of `next`'s units (direct: runs)
    int issued = 0;
    bool fresh = true;       // its unit is the first of a run here
    int window = 0, window0 = -1;  // 32 table entries of next's sequence from window0 on
    auto issue = [&](int stage) {
      if (left <= 0) return;
      ++issued;
      const uint32_t full = bars + 8 * stage, kd = ring + stage * Sh::kStage, vd = kd + Sh::kTile, qd = vd + Sh::kTile;
      const int k0 = next.k.key0(next.u), e0 = k0 / BS;
      if (window0 < 0 || e0 < window0 || e0 + Sh::kBoxes > window0 + 32) {
        window0 = e0;
        const int e = e0 + lane;
        window = e < p.max_blocks ? p.block_tables[static_cast<size_t>(next.seq) * p.max_blocks + e] : -1;
      }
      const uint32_t see = next.k.seen(k0);
      if (lane == 0) mbar_arrive_expect_tx(full, 2 * Sh::kTile + (fresh ? p.group * D * 2 : 0));
#pragma unroll
      for (int j = 0; j < Sh::kBoxes; ++j) {
        const int kb = k0 + j * Sh::kBoxRows;
        const int b = __shfl_sync(0xffffffffu, window, (kb / BS - window0) & 31);
        // a box of which nothing is seen, or a bad id: zeros
        const bool some = ((see >> (j * Sh::kBoxRows)) & (Sh::kBoxRows == 32 ? ~0u : (1u << (Sh::kBoxRows & 31)) - 1)) != 0;
        int row = p.oob_row;
        if (some && b >= 0 && b < p.num_blocks) row = (b * p.num_kv_heads + next.head) * BS + kb % BS;
        else if (some && lane == 0 && p.status) atomicOr(p.status, PKV_STATUS_BAD_BLOCK);
        if (lane == 0) {
          if constexpr (D == 128) {
            tma_load_3d(kd + j * Sh::kBoxBytes, &tmk, 0, row, 0, full, pol);
            tma_load_3d(vd + j * Sh::kBoxBytes, &tmv, 0, row, 0, full, pol);
          } else {
            tma_load_2d(kd + j * Sh::kBoxBytes, &tmk, 0, row, full, pol);
            tma_load_2d(vd + j * Sh::kBoxBytes, &tmv, 0, row, full, pol);
          }
        }
      }
      if (fresh && lane == 0)
        bulk_load(qd, p.q + (static_cast<size_t>(next.seq) * p.num_q_heads + static_cast<size_t>(next.head) * p.group) * D,
                  p.group * D * 2, full);
      const int was = next.seq;
      fresh = next.advance<BS>(p);
      if (next.seq != was) window0 = -1;
      if (!direct || fresh) --left;
    };
    for (int s = 0; s < kStages; ++s) issue(s);

    // ---- units
    Acc<D, NT> acc;
    uint32_t qf[NT][D / 16][2];
    bool starts = true;  // the unit is the first of a run here
    const int g4 = lane >> 2, c4 = lane & 3;
    int i = 0;
    for (; count > 0; ++i) {
      const int stage = i % kStages;
      if (!__all_sync(0xffffffffu, mbar_wait(bars + 8 * stage, (i / kStages) & 1))) {
        if (lane == 0 && p.status) atomicOr(p.status, PKV_STATUS_TIMEOUT);
        break;
      }
      const uint32_t kb = ring + stage * Sh::kStage, vb = kb + Sh::kTile, qb = vb + Sh::kTile;
      const bool begins = at.u == 0;  // the run itself begins here
      if (starts) {
        acc.reset();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const bool real = nt * 8 + g4 < p.group;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t w;
              asm volatile("ld.shared.b32 %0, [%1];"
                           : "=r"(w)
                           : "r"(qb + (nt * 8 + g4) * D * 2 + (ks * 8 + e * 4 + c4) * 4)
                           : "memory");
              qf[nt][ks][e] = real ? w : 0u;
            }
        }
        if (!begins) desc.w = 1;  // (the piece goes on with a run: slot 0)
      }
      const uint32_t see = at.k.seen(at.k.key0(at.u));
      if (see) attend_unit<D, NT, Sh::kBoxRows>(acc, qf, kb, vb, see, p.scale_log2, lane);
      const int seq = at.seq, head = at.head;
      const bool ends = at.advance<BS>(p);  // the run ends with this unit
      __syncwarp();
      issue(stage);
      if (!direct || ends) --count;
      starts = ends;
      if (!ends && count > 0) continue;
      // ---- the piece's end
      float l[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = acc.l[nt][e];
          x += __shfl_xor_sync(0xffffffffu, x, 4);
          x += __shfl_xor_sync(0xffffffffu, x, 8);
          x += __shfl_xor_sync(0xffffffffu, x, 16);
          l[nt][e] = x;
        }
      if (ends && desc.w == 0) {  // the whole run: normalise and store
        __nv_bfloat16 *dst = p.out + (static_cast<size_t>(seq) * p.num_q_heads + static_cast<size_t>(head) * p.group) * D;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float i0 = l[nt][0] > 0.f ? 1.f / l[nt][0] : 0.f, i1 = l[nt][1] > 0.f ? 1.f / l[nt][1] : 0.f;
#pragma unroll
          for (int md = 0; md < D / 16; ++md)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {  // [d][head] fragments -> two values of one head per lane
              const uint32_t w = movmatrix_trans(pack_bf16x2(acc.o[md][nt][2 * hf] * i0, acc.o[md][nt][2 * hf + 1] * i1));
              if (nt * 8 + g4 < p.group)
                *reinterpret_cast<uint32_t *>(dst + (nt * 8 + g4) * D + md * 16 + hf * 8 + 2 * c4) = w;
            }
        }
      } else {
        const int slot = desc.w ? 0 : 1;
        const size_t piece = 2 * static_cast<size_t>(me) + slot;
#pragma unroll
        for (int md = 0; md < D / 16; ++md)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            p.ws_o[((piece * (D / 16) + md) * NT + nt) * 32 + lane] =
                make_float4(acc.o[md][nt][0], acc.o[md][nt][1], acc.o[md][nt][2], acc.o[md][nt][3]);
        if (g4 == 0)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) p.ws_ml[piece * NT * 8 + nt * 8 + 2 * c4 + e] = make_float2(acc.m[nt][e], l[nt][e]);
        if (slot == 1) {
          desc.x = seq;
          desc.y = head;
          desc.z |= kLeaves;
        } else if (ends) {
          desc.z |= kEnds;
        }
      }
      desc.w = 0;
    }
    // never leave a copy in flight into this CTA's shared memory (there is one only where a wait gave up)
    for (; i < issued; ++i) mbar_wait(bars + 8 * (i % kStages), (i / kStages) & 1);
  }
  if (!direct && lane == 0) p.ws_desc[me] = desc;
}

// One block per warp whose last run leaves it: the exact merge of the run's pieces,
// a warp for every 16 values of the head dim (in accumulator order).
template <int D, int NT>
__global__ void __launch_bounds__(D / 16 * 32) step_join_kernel(const StepParams p, int warps) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int4 d = p.ws_desc[blockIdx.x];
  if (!(d.z & kLeaves)) return;
  const int md = threadIdx.x >> 5, lane = threadIdx.x & 31, g4 = lane >> 2, c4 = lane & 3;
  int last = -1;  // the first warp after this one in which the run ends
  for (int base = blockIdx.x + 1; base < warps && last < 0; base += 32) {
    const unsigned ends = __ballot_sync(0xffffffffu, base + lane < warps && (p.ws_desc[base + lane].z & kEnds));
    if (ends) last = base + __ffs(ends) - 1;
  }
  if (last < 0) return;  // only where a bounded wait gave up
  const int pieces = last - static_cast<int>(blockIdx.x) + 1;
  auto slot = [&](int i) { return 2 * (static_cast<size_t>(blockIdx.x) + i) + (i == 0 ? 1 : 0); };
  __nv_bfloat16 *dst = p.out + (static_cast<size_t>(d.x) * p.num_q_heads + static_cast<size_t>(d.y) * p.group) * D;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int col = nt * 8 + 2 * c4;
    constexpr int kAhead = 8;  // pieces whose loads are in flight together
    float M[2] = {-INFINITY, -INFINITY}, den[2] = {0.f, 0.f}, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int b = 0; b < pieces; b += kAhead) {
      float4 ml[kAhead], x[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        ml[i] = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
        x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (b + i < pieces) {
          ml[i] = *reinterpret_cast<const float4 *>(p.ws_ml + slot(b + i) * NT * 8 + col);
          x[i] = p.ws_o[((slot(b + i) * (D / 16) + md) * NT + nt) * 32 + lane];
        }
      }
      float top[2] = {M[0], M[1]};
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        top[0] = fmaxf(top[0], ml[i].x);
        top[1] = fmaxf(top[1], ml[i].z);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float keep = M[e] == -INFINITY ? 0.f : exp2f(M[e] - top[e]);
        M[e] = top[e];
        den[e] *= keep;
        o[e] *= keep;
        o[e + 2] *= keep;
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        // a piece without keys (max -inf) holds zeros and weighs nothing
        const float f0 = ml[i].x == -INFINITY ? 0.f : exp2f(ml[i].x - M[0]);
        const float f1 = ml[i].z == -INFINITY ? 0.f : exp2f(ml[i].z - M[1]);
        den[0] += ml[i].y * f0;
        den[1] += ml[i].w * f1;
        o[0] += f0 * x[i].x;
        o[1] += f1 * x[i].y;
        o[2] += f0 * x[i].z;
        o[3] += f1 * x[i].w;
      }
    }
    const float i0 = den[0] > 0.f ? 1.f / den[0] : 0.f, i1 = den[1] > 0.f ? 1.f / den[1] : 0.f;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const uint32_t w = movmatrix_trans(pack_bf16x2(o[2 * hf] * i0, o[2 * hf + 1] * i1));
      if (nt * 8 + g4 < p.group) *reinterpret_cast<uint32_t *>(dst + (nt * 8 + g4) * D + md * 16 + hf * 8 + 2 * c4) = w;
    }
  }
}

// ------------------------------------------------------------------ host
struct StepPlan {
  bool direct;
  int warps;  // of the grid
  size_t o_bytes, ml_bytes, desc_bytes;
  size_t bytes() const { return direct ? 0 : o_bytes + ml_bytes + desc_bytes; }
};

StepPlan make_step_plan(const Call &a) {
  StepPlan plan{};
  // the longest run: its keys' units, one more at either end of the window, the sinks'
  long long keys = std::min<long long>(a.max_seq_len, static_cast<long long>(a.window) + a.sinks + 3 * kUnit);
  plan.direct = (keys + kUnit - 1) / kUnit <= kDirectUnits;
  const int nt = a.num_q_heads / a.num_kv_heads <= 8 ? 1 : 2;
  const int per_cta = a.head_dim == 128 ? (nt == 1 ? Shape<128, 1, 16>::kWarps : Shape<128, 2, 16>::kWarps)
                                        : (nt == 1 ? Shape<64, 1, 16>::kWarps : Shape<64, 2, 16>::kWarps);
  plan.warps = num_sms() * per_cta;
  const size_t pieces = 2 * static_cast<size_t>(plan.warps);
  plan.o_bytes = pieces * nt * 8 * a.head_dim * sizeof(float);
  plan.ml_bytes = pieces * nt * 8 * sizeof(float2);
  plan.desc_bytes = static_cast<size_t>(plan.warps) * sizeof(int4);
  return plan;
}

template <int D, int NT, int BS>
int launch(const CUtensorMap &tmk, const CUtensorMap &tmv, const StepParams &p, const StepPlan &plan, cudaStream_t stream) {
  using Sh = Shape<D, NT, BS>;
  const auto kernel = step_kernel<D, NT, BS>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
  // as many CTAs as their warps have a run (direct) or every SM
  long long grid = plan.warps / Sh::kWarps;
  if (plan.direct)
    grid = std::min(grid, (static_cast<long long>(p.num_seqs) * p.num_kv_heads + Sh::kWarps - 1) / Sh::kWarps);
  if (e == cudaSuccess)
    e = launch_overlapped(kernel, static_cast<unsigned>(grid), Sh::kThreads, Sh::kSmem, stream, tmk, tmv, p);
  if (e == cudaSuccess && !plan.direct)
    e = launch_overlapped(step_join_kernel<D, NT>, static_cast<unsigned>(plan.warps), D / 16 * 32, 0, stream, p, plan.warps);
  return e == cudaSuccess ? PKV_OK : (set_cuda_error(e), PKV_ERR_CUDA);
}

template <int D, int NT>
int launch_bs(const CUtensorMap &tmk, const CUtensorMap &tmv, const StepParams &p, const StepPlan &plan, int block_size,
              cudaStream_t stream) {
  switch (block_size) {
    case 16: return launch<D, NT, 16>(tmk, tmv, p, plan, stream);
    case 32: return launch<D, NT, 32>(tmk, tmv, p, plan, stream);
    case 64: return launch<D, NT, 64>(tmk, tmv, p, plan, stream);
    default: return launch<D, NT, 128>(tmk, tmv, p, plan, stream);
  }
}

}  // namespace

size_t step_workspace_size(const Call &a) { return make_step_plan(a).bytes(); }

int step_launch(const Call &a) {
  const StepPlan plan = make_step_plan(a);
  if (plan.bytes() > 0 && (!a.workspace || a.workspace_bytes < plan.bytes() || !aligned16(a.workspace)))
    return PKV_ERR_WORKSPACE;
  // a warp's range is found with products of all units and the warps in 64 bits
  if (static_cast<double>(a.num_seqs) * a.num_kv_heads * (a.max_seq_len / kUnit + 4) * plan.warps > 4e18)
    return PKV_ERR_UNSUPPORTED;
  const long long rows = static_cast<long long>(a.num_blocks) * a.num_kv_heads * a.block_size;
  CUtensorMap tmk, tmv;
  const int box = std::min(a.block_size, kUnit);
  if (!make_tensor_map_rows(&tmk, a.k_cache, a.head_dim, box, rows) ||
      !make_tensor_map_rows(&tmv, a.v_cache, a.head_dim, box, rows))
    return PKV_ERR_CUDA;
  StepParams p{};
  p.q = reinterpret_cast<const __nv_bfloat16 *>(a.q);
  p.block_tables = a.block_tables;
  p.seq_lens = a.seq_lens;
  p.out = reinterpret_cast<__nv_bfloat16 *>(a.out);
  if (!plan.direct) {
    char *ws = static_cast<char *>(a.workspace);
    p.ws_o = reinterpret_cast<float4 *>(ws);
    p.ws_ml = reinterpret_cast<float2 *>(ws + plan.o_bytes);
    p.ws_desc = reinterpret_cast<int4 *>(ws + plan.o_bytes + plan.ml_bytes);
  }
  p.status = a.status;
  p.num_seqs = a.num_seqs;
  p.max_blocks = a.max_blocks;
  p.max_len = a.max_seq_len;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.group = a.num_q_heads / a.num_kv_heads;
  p.num_blocks = a.num_blocks;
  p.oob_row = static_cast<int>(rows);
  p.window = a.window;
  p.sinks = a.sinks;
  p.scale_log2 = a.scale * kLog2e;
  const cudaStream_t st = as_stream(a.stream);
  if (a.head_dim == 128)
    return p.group <= 8 ? launch_bs<128, 1>(tmk, tmv, p, plan, a.block_size, st)
                        : launch_bs<128, 2>(tmk, tmv, p, plan, a.block_size, st);
  return p.group <= 8 ? launch_bs<64, 1>(tmk, tmv, p, plan, a.block_size, st)
                      : launch_bs<64, 2>(tmk, tmv, p, plan, a.block_size, st);
}

}  // namespace spans
}  // namespace pkv
