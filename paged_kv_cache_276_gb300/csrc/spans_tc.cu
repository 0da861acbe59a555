// Windowed attention of query chunks and attention of drafted trees on the
// 5th-generation tensor cores.
//
// For one KV head, a query tile of 128 rows holds up to 128 / G tokens x the G
// query heads of the group (row r = token r / G, head r % G).  Over each tile of
// 64 keys that some row sees:
//     S  = Q K^T                     tcgen05.mma, M 128 x N 64 x K d -> TMEM
//     P  = exp2(S * scale*log2e - m)  softmax warps, one query row per thread,
//                                    bf16 in TMEM
//     O += P V                       tcgen05.mma, M 128 x N d x K 64 -> TMEM
// with the running max / sum of the online softmax.  What a row sees of a tile is
// a 64-bit word, from the window's bounds or from the tree's mask: a key whose
// bit is clear gets the score -inf.
//
// Runs and ranges.  A run is one (sequence, KV head, query tile or pair of query
// tiles) with the key tiles it needs: of a tree every tile of the sequence, of a
// window those between its first row's window and its last row's position, and
// the sinks' before them.  The runs of the batch are laid end to end, each with a
// weight of its keys plus kRunCost, and every CTA of a persistent grid (one per
// SM) takes an equal, contiguous range of the weight: a border inside a run falls
// on a key tile, or on the run's end if that is near.  So all SMs end together
// whatever the lengths are, with no host-built list.  The weights have closed
// forms, so a CTA finds its first run by a few searches.  (Where windows give every
// CTA several runs, whole ones go round the CTAs first: neighbours then read the same
// keys at the same time, 0.4 GB of HBM traffic instead of 1.5 for four prompts of 8192
// tokens.  Where no run is long enough to be cut, all go round whole.)  A run that lies in one
// range is written at once; the pieces of one that does not (at most two per CTA:
// the first and the last of its range) go to the workspace as (max, sum,
// unnormalised O), and a second kernel joins them in the order of the CTAs:
// results repeat bit for bit.
//
// A slot is what works on one query tile: its queries' buffer, softmax warps,
// scores, weights and accumulator.  Batches of long chunks and of large trees run
// with two slots in a CTA, one CTA per SM: both query tiles of a pair are multiplied
// against each key and value tile, half the traffic per product (a query tile
// without a partner goes to the slots in turn).  Batches of one query tile per
// sequence, and long chunks at head_dim 64, run with one slot in a CTA, two CTAs per
// SM, each over runs of its own: while one starts or ends a run the other streams.
//
// Values that a row does not see must not reach it, and 0 times NaN or infinity is
// NaN: in a tile that is not seen whole, the P V issuer's warp clears the values no
// row of the run sees and those that are not finite, in shared memory, while the
// tile's weights are computed; a tile with any of the latter is noted, and the rows
// that do see one add it when they are written out (rare).
//
// Warp roles: four softmax warps per slot (thread = row), then a TMA producer of
// queries and keys, which also finds the CTA's runs and hands them to the others
// through a ring of descriptors in shared memory, the score-product issuer (one
// lane) and tensor-memory owner, the P V product issuer (one lane), and the TMA
// producer of values.
//
// What bounds it.  A key tile of a pair is 1280 clocks of matrix instructions (a
// score product of 64 keys reads the queries from shared memory again: 384 clocks where
// the arithmetic is 256; P V 256) against about 1650 measured: products and softmax
// overlap, and what they wait for each other is the rest.  A run's end takes a slot about
// 7000 clocks (the last product, the rows' output, the next descriptor).
// Measured (clocks at 2070 MHz): four prompts of 8192 tokens, 32 / 8 heads of 128, window
// 1024: 492 to 502 us by the card, 1.03 to 1.05 PFLOP/s of the visible products; a tree of
// 64 nodes on 32768 tokens, 64 / 8 heads: 66 to 67 us, 1.02 PFLOP/s; 256 trees of 8 nodes on
// 215 k tokens, 32 / 8 heads: 157 to 158 us, 5.7 TB/s.  In a tree's batch the products fit
// beside the copies while a node's G heads fill few rows, and HBM is the bound.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "internal.h"
#include "launch.cuh"
#include "pkv.h"
#include "ptx.cuh"
#include "spans.cuh"
#include "tc.cuh"
#include "tc_softmax.cuh"

namespace pkv {
namespace spans {
namespace {

constexpr int kRows = 128;       // query rows per tile
constexpr int kTK = 64;          // keys per tile
// The reference of the weights moves when a score passes it by more than this (log2
// units): weights stay below 2^20, which fp32 sums and bf16 hold with the same
// relative rounding (sums overflow for values above 2^107 / keys).  With 8, a warp
// of 32 rows rescaled its accumulator at every third tile of a window that starts
// with the sinks' four keys (571 us for the four prompts of 8192 tokens).
constexpr float kSlack = 20.f;
// A run's start and end, in keys.  256 trees of 8 nodes and mixed lengths take 157 us,
// 32 trees of 26 nodes 64; with 128 they take 154 and 65, with 448 165 and 64.5.
constexpr int kRunCost = 256;
constexpr int kMinRange = 512;   // least weight of a CTA's range, in keys
constexpr int kRoundsFrom = 4;   // runs per CTA from which most go round the CTAs whole
// Key tiles that a border leaves on either side of it: with 2, 158 and 64 us, with 8, 159
// and 66.
constexpr int kMinPiece = 4;
constexpr int kJoinShares = 8;   // blocks of the join that share a run's head dim
constexpr int kPairedSeqs = 512;  // sequences up to which two CTAs of one slot fit an SM
constexpr int kRunRing = 4;      // descriptors of runs ahead
constexpr long long kMaxRuns = (1ll << 31) - (1 << 20);  // of a call: they are counted in 32 bits

template <int D, int S>
struct Layout {
  static_assert(D == 64 || D == 128, "head dim");
  static_assert(S == 1 || S == 2, "slots");
  static constexpr int kKWarp = 4 * S, kMmaWarp = kKWarp + 1, kPvWarp = kKWarp + 2, kVWarp = kKWarp + 3;
  static constexpr int kThreads = (kKWarp + 4) * 32, kCtasPerSm = 3 - S;
  static constexpr int kHalves = D / 64;            // 64-column (128-byte) halves of a row
  static constexpr int kQHalf = kRows * 128;        // one half of a query tile
  static constexpr int kQTile = kHalves * kQHalf;   // [half][128 rows][128 B]
  static constexpr int kHalf = kTK * 128;           // one half of a key or value tile
  static constexpr int kTile = kHalves * kHalf;     // [half][64 rows][128 B]
  static constexpr int kStages = S * 256 / D;       // of keys, and of values: 32 KB per slot each
  static constexpr int kSmemK = S * kQTile;         // after the query tiles
  static constexpr int kSmemV = kSmemK + kStages * kTile;
  static constexpr int kSmemBars = kSmemV + kStages * kTile;
  // tensor memory: the slots' accumulators, then their scores, then two P of each
  static constexpr int kTmemCols = S * 256;
  static constexpr int kTmemS = S * D, kTmemP = kTmemS + S * kTK;
  static_assert(kTmemP + 2 * S * (kTK / 2) <= kTmemCols, "tensor memory");
  // barrier indices (8 bytes each)
  static constexpr int kQFull = 0, kQFree = kQFull + S, kOFull = kQFree + S, kOFree = kOFull + S, kSFull = kOFree + S,
                       kSFree = kSFull + S,                                // [slot]
                       kPFull = kSFree + S, kPvDone = kPFull + 2 * S,      // [slot][buffer of P]
                       kRunFull = kPvDone + 2 * S, kRunFree = kRunFull + kRunRing,
                       kKFull = kRunFree + kRunRing, kKEmpty = kKFull + kStages, kVFull = kKEmpty + kStages,
                       kVEmpty = kVFull + kStages, kBars = (kVEmpty + kStages + 1) / 2 * 2;
};

// A run's descriptor: the fields of Run in this order.
constexpr int kRunInts = 12;

template <int D, int S>
constexpr size_t smem_bytes(int num_seqs) {
  using Lay = Layout<D, S>;
  return 1024 + Lay::kSmemBars + Lay::kBars * 8 + 16 + kRunRing * kRunInts * 4 + static_cast<size_t>(num_seqs + 1) * 12 +
         static_cast<size_t>(num_seqs) * 12;
}
static_assert(smem_bytes<128, 2>(kMaxSeqs) <= 227 * 1024, "shared memory");
// two CTAs (and 1 KB that the system takes of each) in an SM's 228 KB
static_assert(smem_bytes<128, 1>(kPairedSeqs) <= 113 * 1024, "shared memory");

struct Params {
  const int32_t *block_tables, *seq_lens, *q_start;
  const uint64_t *mask;        // tree; NULL: window
  const __nv_bfloat16 *v_cache;
  __nv_bfloat16 *out;
  float4 *ws_o;                // [2 grid][D / 4][piece_rows]
  float2 *ws_ml;               // [2 grid][piece_rows]
  int4 *ws_desc;               // [grid]: {first query row, KV head, flags, tokens} of a CTA's pieces; NULL: none is cut
  int32_t *status;
  int bs_log2, num_seqs, max_blocks, num_q_heads, num_kv_heads, num_blocks, total_q, max_len, oob_row;
  int group, tile_tok, span;   // tokens of a query tile (floor(128 / G) or the tree's) and of a run
  int window, sinks, max_nodes, piece_rows;
  float scale_log2;            // of the scale's magnitude; negate: it is negative
  int negate;
};

// flags of a descriptor
constexpr int kLeaves = 1;  // the CTA's last run goes on in the next CTA (piece 1 holds its start)
constexpr int kEnds = 2;    // the run that the CTA goes on with (piece 0) ends here
// in the place of a piece's sum: it holds no key tile, and its O was not written
constexpr float kNoTile = -1.f;

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// a / b for a >= 0, b > 0 and a quotient below 2^31, in few instructions: an estimate
// and single steps.
__device__ __forceinline__ int divide(long long a, long long b) {
  int q = static_cast<int>(__fdividef(static_cast<float>(a), static_cast<float>(b)));
#pragma unroll 1
  while (q * b > a) --q;
#pragma unroll 1
  while ((q + 1ll) * b <= a) ++q;
  return q;
}

// Per-sequence values kept in shared memory.
struct SeqTab {
  const long long *prefix;  // [B + 1] weight before each sequence
  const int *first;           // [B + 1] runs before each sequence
  const int *lens, *qs, *qc;  // [B] clamped length, first query row, query tokens (0: none or a bad q_start)
};

// The weights of a sequence's runs (of one KV head), in keys: run i has
//   i < bent:  base + span (i + 1)     (its window still reaches the first token)
//   else       flat
struct Weights {
  long long base, flat;
  int bent, span, runs;
  __device__ Weights() {}
  __device__ __forceinline__ Weights(const Params &p, int L, int c) {
    span = p.span;
    runs = ceil_div(c, span);
    if (p.mask) {
      bent = 0;
      base = 0;
      flat = kRunCost + max(L, 1);
    } else {
      const long long ctx = max(0, L - c);
      const long long sunk = (static_cast<long long>(p.sinks) + kTK - 1) / kTK * kTK, reach = p.window - 1ll + sunk;
      // at most runs, so that the division fits 32 bits
      const long long room = min(reach - ctx, static_cast<long long>(runs) * span);
      bent = room < 0 ? 0 : min(runs, static_cast<int>(static_cast<uint32_t>(room) / static_cast<uint32_t>(span)) + 1);
      base = kRunCost + ctx;
      flat = kRunCost + span + reach;
    }
  }
  __device__ __forceinline__ long long of(int i) const { return i < bent ? base + span * (i + 1ll) : flat; }
  __device__ __forceinline__ long long sum(int m) const {  // of the first m runs
    const long long b = min(m, bent);
    return b * base + span * (b * (b + 1) / 2) + (m - b) * flat;
  }
  // the run that holds weight x, 0 <= x < sum(runs)
  __device__ __forceinline__ int find(long long x) const {
    const long long s = sum(bent);
    if (x >= s) return bent + divide(x - s, flat);
    int lo = 0, hi = bent;
#pragma unroll 1
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sum(mid) <= x) lo = mid; else hi = mid;
    }
    return lo;
  }
};

// A CTA's piece of a run: key tiles [t0, t1) of its n.  Tile v starts at key
// 64 v (the sinks', v < ns) or 64 (v - ns + t_lo).
struct Run {
  int seq, head, r0, ntq;  // first query token, query tiles (0: no further run)
  int lo, hi, sink_end;    // the run sees nothing outside [lo, hi) and [0, sink_end)
  int ns, t_lo, n, t0, t1;
  __device__ bool whole() const { return t0 == 0 && t1 == n; }
  __device__ int key0(int v) const { return kTK * (v < ns ? v : v - ns + t_lo); }
  __device__ void put(volatile int *d) const {
    d[0] = seq, d[1] = head, d[2] = r0, d[3] = ntq, d[4] = lo, d[5] = hi, d[6] = sink_end, d[7] = ns, d[8] = t_lo;
    d[9] = n, d[10] = t0, d[11] = t1;
  }
  __device__ void get(const volatile int *d) {
    seq = d[0], head = d[1], r0 = d[2], ntq = d[3], lo = d[4], hi = d[5], sink_end = d[6], ns = d[7], t_lo = d[8];
    n = d[9], t0 = d[10], t1 = d[11];
  }
};

// The keys that every one of some rows sees, tokens first .. last of a sequence's
// chunk (of a tree: any tokens): [lo, hi) and [0, sinks).
template <bool Tree>
struct Common {
  int lo, hi, sinks;
  __device__ __forceinline__ Common(const Params &p, int ctx, int first, int last) {
    if (Tree) {
      lo = sinks = 0;
      hi = ctx;
    } else {
      hi = ctx + first + 1;
      lo = max(0, max(0, ctx + last + 1) - p.window);  // (a row may stand before the first token)
      sinks = min(p.sinks, hi);
    }
  }
  __device__ __forceinline__ Common(const Params &p, const Run &x, int L, int c)  // the rows of a run
      : Common(p, L - c, x.r0, min(c, x.r0 + p.span) - 1) {}
  // all of a key tile
  __device__ bool has(int k0) const { return (k0 >= lo && k0 + kTK <= hi) || k0 + kTK <= sinks; }
};

// The runs of this CTA in order: first whole rounds (run c, c + grid, ... for CTA
// c), then its range of the weight of the rest.  One call site and little code: the
// roles share the SM's instruction cache.
struct Sched {
  long long xa, xb, s;  // the CTA's range; the current run's start
  int seq, head, i, round, rounds;
  Weights w;  // of the current sequence
  Run x;

  __device__ __forceinline__ Sched(const Params &p, const SeqTab &t) {
    const int runs = t.first[p.num_seqs], grid = gridDim.x;
    // where no run is cut, they all go round whole
    rounds = !p.ws_desc ? (runs + grid - 1) / grid : !p.mask && runs >= kRoundsFrom * grid ? runs / grid - 1 : 0;
    round = -1;
  }

  // the next run into x; false: there is none
  __device__ __forceinline__ bool next(const Params &p, const SeqTab &t) {
    const int grid = gridDim.x;
    ++round;
    if (!p.ws_desc && round * static_cast<long long>(grid) + blockIdx.x >= t.first[p.num_seqs]) return false;
    if (round <= rounds) {
      // a whole round's run, or the first run behind the rounds
      const int run = round * grid + (round < rounds ? blockIdx.x : 0);
      long long lo = search(t.first, p.num_seqs, run);
      if (rounds > 0) {
        enter(p, t, static_cast<int>(lo));
        const int off = run - t.first[seq];
        head = static_cast<unsigned>(off) / static_cast<unsigned>(w.runs);
        i = off - head * w.runs;
      }
      if (round == rounds) {  // this CTA's range of the rest
        const long long start = rounds > 0 ? t.prefix[seq] + head * w.sum(w.runs) + w.sum(i) : 0;
        const long long rest = t.prefix[p.num_seqs] - start;
        const int c = blockIdx.x, ctas = static_cast<int>(max(1ll, min(static_cast<long long>(grid), rest / kMinRange)));
        const long long each = rest / ctas;
        const unsigned more = static_cast<unsigned>(rest - each * ctas);
        xa = start + each * c + more * c / ctas;
        xb = start + each * (c + 1) + more * (c + 1) / ctas;
        if (c >= ctas || xa >= xb) return false;
        enter(p, t, search(t.prefix, p.num_seqs, xa));
        const long long per_head = w.sum(w.runs), off = xa - t.prefix[seq];
        head = divide(off, per_head);
        i = w.find(off - head * per_head);
        s = t.prefix[seq] + head * per_head + w.sum(i);
      }
    } else {
      step(p, t);
    }
#pragma unroll 1
    for (;; step(p, t)) {  // from this run on: the first that the CTA has a piece of
      const bool whole = round < rounds;
      if (!whole && (s >= xb || seq >= p.num_seqs)) return false;
      geometry(p, t.lens[seq], t.qc[seq]);
      x.t0 = 0;
      x.t1 = x.n;
      if (whole) return true;
      const long long weight = w.of(i);
      if (xa > s) x.t0 = border(xa - s, weight);
      if (xb < s + weight) x.t1 = border(xb - s, weight);
      // a run without keys belongs to the CTA that holds its start; a range inside a
      // tile is an empty piece, which the join expects
      if (x.n == 0 ? xa <= s : x.t0 < x.t1 || (x.t0 > 0 && x.t0 < x.n)) return true;
    }
  }

 private:
  // the last of the n sequences that begins at or before x
  template <typename T>
  static __device__ __forceinline__ int search(const T *before, int n, T x) {
    int lo = 0, hi = n;
#pragma unroll 1
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (before[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
  }
  __device__ __forceinline__ void enter(const Params &p, const SeqTab &t, int sequence) {
    seq = sequence;
    w = Weights(p, t.lens[seq], t.qc[seq]);
  }
  __device__ __forceinline__ void step(const Params &p, const SeqTab &t) {
    s += w.of(i);
    if (++i < w.runs) return;
    i = 0;
    if (++head < p.num_kv_heads) return;
    head = 0;
#pragma unroll 1
    do ++seq;
    while (seq < p.num_seqs && t.qc[seq] == 0);
    if (seq < p.num_seqs) enter(p, t, seq);
  }
  // the key tile that a border at this weight of the run falls on: every CTA that asks gets the same
  __device__ __forceinline__ int border(long long at, long long weight) const {
    const int o = static_cast<int>(__fdividef(static_cast<float>(at), static_cast<float>(weight)) * static_cast<float>(x.n));
    return o < kMinPiece ? 0 : o > x.n - kMinPiece ? x.n : o;
  }
  __device__ __forceinline__ void geometry(const Params &p, int L, int c) {
    x.seq = seq;
    x.head = head;
    x.r0 = i * p.span;
    const int ctx = L - c, end = min(c, x.r0 + p.span);
    x.ntq = end - x.r0 > p.tile_tok ? 2 : 1;
    if (p.mask) {
      x.lo = 0;
      x.hi = L;
      x.sink_end = 0;
    } else {
      x.hi = max(0, ctx + end);
      x.lo = max(0, max(0, ctx + x.r0) - p.window + 1);
      x.sink_end = min(p.sinks, x.lo);
    }
    x.t_lo = x.lo / kTK;
    x.ns = min(ceil_div(x.sink_end, kTK), x.t_lo);
    x.n = x.hi > 0 ? x.ns + ceil_div(x.hi, kTK) - x.t_lo : 0;
  }
};

// Bits below x of a 64-bit word.
__device__ __forceinline__ uint64_t below(int x) { return x <= 0 ? 0ull : x >= 64 ? ~0ull : (1ull << x) - 1; }

// What a row sees of 64 keys from h0 on.
template <bool Tree>
struct RowSight {
  int lo, hi, sinks;   // window: [lo, hi) and [0, sinks)
  int ctx;             // tree: [0, ctx) and bit j of word for key ctx + j
  uint64_t word;       // (bits of the tree only: keep)
  uint64_t keep;
  __device__ __forceinline__ uint64_t of(int h0) const {
    if (!Tree) return (below(hi - h0) & ~below(lo - h0)) | below(sinks - h0);
    const int sh = ctx - h0;
    const uint64_t w = word & keep, own = sh >= 64 || sh <= -64 ? 0ull : sh >= 0 ? w << sh : w >> -sh;
    return below(sh) | own;
  }
};

// mbar_wait (bounded by kWaitLimitNs too) in few instructions: this kernel's roles
// share the SM's instruction cache, and a wait is in every one of their steps.  A
// waiting warp sleeps between its looks, which leaves the issue slots to the softmax
// (four prompts of 8192 tokens: 514 us without the sleeps, 503 with).
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_timer_ns();
  bool ok;
#pragma unroll 1
  do {
    __nanosleep(20);
    ok = mbar_try_wait(bar, parity);
  } while (!ok && global_timer_ns() - t0 < kWaitLimitNs);
  return ok;
}
__device__ __forceinline__ bool wait_warp(uint32_t b, uint32_t parity) {
  return __all_sync(0xffffffffu, wait(b, parity));
}

// Shared-memory matrix descriptors (tc::desc_sw128, groups of 8 rows 1024 bytes
// apart) in two words: the first holds the address (in 16 bytes), so that a product's
// steps differ by an addition to it; few instructions between the issues matter, as
// one thread issues them.
constexpr uint32_t kSpanHi = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_word(uint32_t saddr) { return (saddr >> 4) & 0x3FFFu; }
__device__ __forceinline__ uint64_t desc_of(uint32_t lo, uint32_t hi) { return f32x2_bits(lo, hi); }

// 0 * x + acc for two bf16: NaN where x is not finite.
__device__ __forceinline__ uint32_t poison2(uint32_t x, uint32_t acc) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(x), "r"(0u), "r"(acc));
  return d;
}
__device__ __forceinline__ bool any_nan2(uint32_t x) {
  const uint32_t m = x & 0x7FFF7FFFu;
  return (m & 0xFFFFu) > 0x7F80u || (m >> 16) > 0x7F80u;
}

// One warp: the value rows of a staged tile from key k0 on that no row of the run
// sees become zeros, and so do values that are not finite; true: there were some.
template <int D>
__device__ __forceinline__ bool clear_values(uint32_t tile, const Run &x, int k0, int lane) {
  constexpr int kHalves = D / 64, kHalf = kTK * 128, kPerRow = kHalves * 8;  // 16-byte chunks of a row
  auto at = [&](int e) {
    const int row = e / kPerRow, rem = e % kPerRow;
    return tile + (rem / 8) * kHalf + row * 128 + (rem % 8) * 16;
  };
  auto zero = [&](int key0, int key1) {  // rows of keys [key0, key1)
    const int a = max(0, key0 - k0) * kPerRow, b = min(kTK, key1 - k0) * kPerRow;
#pragma unroll 1
    for (int e = a + lane; e < b; e += 32)
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at(e)), "r"(0u) : "memory");
  };
  zero(x.sink_end, x.lo);
  zero(x.hi, k0 + kTK);
  __syncwarp();
  uint32_t acc[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
  for (int e = lane; e < kTK * kPerRow; e += 32 * 8) {
    uint32_t w[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3])
                   : "r"(at(e + 32 * i))
                   : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[k] = poison2(w[i][k], acc[k]);
  }
  const bool bad = any_nan2(acc[0]) || any_nan2(acc[1]) || any_nan2(acc[2]) || any_nan2(acc[3]);
  const bool odd = __any_sync(0xffffffffu, bad);
  if (odd) {
#pragma unroll 1
    for (int e = lane; e < kTK * kPerRow * 8; e += 32) {  // single values
      const uint32_t a = at(e / 8) + (e % 8) * 2;
      uint16_t v;
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
      if ((v & 0x7F80u) == 0x7F80u)
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"(static_cast<uint16_t>(0)) : "memory");
    }
  }
  fence_proxy_async_shared();
  __syncwarp();
  return odd;
}

template <bool Tree, int D, int S>
__global__ void __launch_bounds__(Layout<D, S>::kThreads, Layout<D, S>::kCtasPerSm)
    spans_tc_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                    const __grid_constant__ CUtensorMap tmv, const Params p) {
  using Lay = Layout<D, S>;
  using BI = Lay;
  constexpr int kStages = Lay::kStages, kHalves = Lay::kHalves, kTile = Lay::kTile, kQTile = Lay::kQTile;
  constexpr int kKWarp = Lay::kKWarp, kMmaWarp = Lay::kMmaWarp, kPvWarp = Lay::kPvWarp, kVWarp = Lay::kVWarp;
  constexpr int kTmemCols = Lay::kTmemCols, kThreads = Lay::kThreads;
  // the slot of the n-th query tile, and how many tiles the slot had before it
  auto slot_of = [](int n) { return S == 2 ? n & 1 : 0; };
  auto use_of = [](int n) { return S == 2 ? n >> 1 : n; };
  // one TMA box per block of the tile (a block longer than the tile: the tile's piece of it)
  const int box_rows = min(1 << p.bs_log2, kTK), boxes = kTK / box_rows;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Lay::kSmemBars);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + BI::kBars);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  // 1 + the last key tile (counted over the CTA) whose values were not all finite
  int *odd_tile = reinterpret_cast<int *>(tmem_slot + 2);
  volatile int *runs = reinterpret_cast<volatile int *>(bars + BI::kBars + 2);  // [kRunRing][kRunInts]
  long long *prefix = reinterpret_cast<long long *>(bars + BI::kBars + 2 + kRunRing * kRunInts / 2);  // [B + 1]
  int *first = reinterpret_cast<int *>(prefix + p.num_seqs + 1);             // [B + 1]
  int *lens = first + p.num_seqs + 1;                                        // [B]
  int *qs = lens + p.num_seqs, *qc = qs + p.num_seqs;                        // [B] each
  const SeqTab tab{prefix, first, lens, qs, qc};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int B = p.num_seqs, hkv = p.num_kv_heads;
  auto bar = [&](int i) { return smem_u32(bars + i); };

  grid_launch_dependents();
  // what the kernel before does not touch
  if (threadIdx.x == 32 * kKWarp) {
    for (int i = 0; i < S; ++i) {  // one per slot
      mbar_init(bar(BI::kQFull + i), 1);
      mbar_init(bar(BI::kQFree + i), 1);
      mbar_init(bar(BI::kOFull + i), 1);
      mbar_init(bar(BI::kOFree + i), kRows);
      mbar_init(bar(BI::kSFull + i), 1);
      mbar_init(bar(BI::kSFree + i), kRows);
      for (int h = 2 * i; h < 2 * i + 2; ++h) {  // one per slot and buffer of P
        mbar_init(bar(BI::kPFull + h), kRows);
        mbar_init(bar(BI::kPvDone + h), 1);
      }
    }
    for (int i = 0; i < kRunRing; ++i) {
      mbar_init(bar(BI::kRunFull + i), 1);
      mbar_init(bar(BI::kRunFree + i), 4 * S + 3);  // the softmax warps, two issuers, the value producer
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(BI::kKFull + s), 1);
      mbar_init(bar(BI::kKEmpty + s), 1);
      mbar_init(bar(BI::kVFull + s), 1);
      mbar_init(bar(BI::kVEmpty + s), 1);
    }
    *abort_flag = 0;
    *odd_tile = 0;
    mbar_init_fence();
  }
  if (p.tile_tok * p.group < kRows) {
    // the loads fill the tile's first tile_tok * G rows only: the rest stay zero
#pragma unroll 1
    for (int i = threadIdx.x; i < S * kQTile / 16; i += kThreads)
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(smem_u32(smem) + i * 16), "r"(0u) : "memory");
    fence_proxy_async_shared();
  }
  if (threadIdx.x == 32 * kKWarp + 1) {
    tma_prefetch_desc(&tmq);
    tma_prefetch_desc(&tmk);
    tma_prefetch_desc(&tmv);
  }
  grid_dependency_wait();
  // (tensor memory after the wait: a CTA of that kernel may not have taken its own yet)
  if (warp == kMmaWarp) {
    tc::alloc(smem_u32(tmem_slot), kTmemCols);
    tc::relinquish();
  }
  if (warp == 0) {  // weight and runs per sequence -> exclusive prefixes
    const int per = (B + 31) / 32;
    const int lo = min(B, lane * per), hi = min(B, lo + per);
    const int cap = min(p.max_blocks << p.bs_log2, p.max_len);
    long long sum = 0, count = 0;
#pragma unroll 1
    for (int i = lo; i < hi; ++i) {
      int L = p.seq_lens[i];
      if (L < 0 || L > cap) {
        if (blockIdx.x == 0 && p.status) atomicOr(p.status, PKV_STATUS_BAD_LEN);
        L = L < 0 ? 0 : cap;
      }
      const int a = p.q_start[i], b = p.q_start[i + 1];
      int c = b - a;
      if (a < 0 || b < a || b > p.total_q || (Tree && c > p.max_nodes)) {
        if (blockIdx.x == 0 && p.status) atomicOr(p.status, PKV_STATUS_BAD_QSTART);
        c = 0;
      }
      lens[i] = L;
      qs[i] = a;
      qc[i] = c;
      const Weights w(p, L, c);
      sum += w.sum(w.runs) * hkv;
      count += static_cast<long long>(w.runs) * hkv;
      prefix[i + 1] = sum;  // within the lane's stretch
      first[i + 1] = static_cast<int>(count);
    }
    long long incl = sum, before = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o), n = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) incl += v, before += n;
    }
#pragma unroll 1
    for (int i = lo; i < hi; ++i) prefix[i + 1] += incl - sum, first[i + 1] += static_cast<int>(before - count);
    if (lane == 0) prefix[0] = 0, first[0] = 0;
    // starts that go back and forth give sequences rows in common, and so more runs
    // than the call was sized for: none is taken
    if (__shfl_sync(0xffffffffu, before, 31) >= kMaxRuns) {
      if (blockIdx.x == 0 && lane == 0 && p.status) atomicOr(p.status, PKV_STATUS_BAD_QSTART);
      __syncwarp();
#pragma unroll 1
      for (int i = lo; i < hi; ++i) prefix[i + 1] = 0, first[i + 1] = 0;
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t sQ = smem_u32(smem), sK = smem_u32(smem + Lay::kSmemK), sV = smem_u32(smem + Lay::kSmemV);
  const uint32_t tS = tmem + Lay::kTmemS, tP = tmem + Lay::kTmemP;
  auto timed_out = [&] {
    if (p.status) atomicOr(p.status, PKV_STATUS_TIMEOUT);
    *abort_flag = 1;
  };
  // the CTA's j-th run, once its descriptor is there; ntq 0: there is none (or a wait gave up)
  auto run_at = [&](int j, Run &x) {
    if (wait(bar(BI::kRunFull + j % kRunRing), (j / kRunRing) & 1)) x.get(runs + (j % kRunRing) * kRunInts);
    else x.ntq = 0;
  };
  auto run_done = [&](int j) { mbar_arrive(bar(BI::kRunFree + j % kRunRing)); };

  // one slot: 128 registers a thread at launch (256 threads, two CTAs) do not hold a
  // softmax; 128 (160 + 96) are as many
  if (warp >= kKWarp) {
    if constexpr (S == 1) asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    if (warp == kKWarp || warp == kVWarp) {
      // ------------------------------------- producers: runs, K (+ Q); V
      const bool is_v = warp == kVWarp;
      const CUtensorMap *tm = is_v ? &tmv : &tmk;
      const uint32_t ring = is_v ? sV : sK;
      const int full0 = is_v ? BI::kVFull : BI::kKFull, empty0 = is_v ? BI::kVEmpty : BI::kKEmpty;
      // a tree of one run per KV head reads every key once; other runs share theirs
      const uint64_t pol = Tree && p.max_nodes <= p.span ? l2_policy_evict_first() : l2_policy_evict_normal();
      int g = 0, nq = 0;  // key tiles and query tiles so far
      int tw_seq = -1, tw_base = 0, tw_val = -1;
      Sched sc(p, tab);
      int4 desc = make_int4(0, 0, 0, 0);  // this CTA's pieces, for the join
#pragma unroll 1
      for (int j = 0; !*abort_flag; ++j) {
        Run x;
        if (is_v) {
          run_at(j, x);
          __syncwarp();
        } else {
          const bool got = sc.next(p, tab);
          x = sc.x;
          if (!got) x.ntq = 0;
          if (j >= kRunRing && !wait_warp(bar(BI::kRunFree + j % kRunRing), (j / kRunRing - 1) & 1)) {
            if (lane == 0) timed_out();
            break;
          }
          if (lane == 0) {
            x.put(runs + (j % kRunRing) * kRunInts);
            mbar_arrive(bar(BI::kRunFull + j % kRunRing));
          }
        }
        if (x.ntq == 0) break;
        if (!is_v && !x.whole()) {
          if (x.t0 > 0 && x.t1 == x.n) desc.z |= kEnds;
          if (x.t0 == 0) {
            desc.x = qs[x.seq] + x.r0;
            desc.y = x.head;
            desc.w = min(p.span, qc[x.seq] - x.r0);
            desc.z |= kLeaves;
          }
        }
        if (!is_v && x.t0 < x.t1) {
          bool ok = true;
#pragma unroll 1
          for (int q = 0; q < x.ntq && ok; ++q, ++nq) {
            const int slot = slot_of(nq), use = use_of(nq);
            if (use > 0 && !wait_warp(bar(BI::kQFree + slot), (use - 1) & 1)) ok = false;
            if (ok && lane == 0) {
              mbar_arrive_expect_tx(bar(BI::kQFull + slot), p.tile_tok * p.group * D * 2);  // the boxes' bytes
              for (int hf = 0; hf < kHalves; ++hf)
                asm volatile(
                    "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
                    " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(sQ + slot * kQTile + hf * Lay::kQHalf),
                    "l"(reinterpret_cast<uint64_t>(&tmq)), "r"(hf * 64), "r"(x.head * p.group),
                    "r"(qs[x.seq] + x.r0 + q * p.tile_tok), "r"(bar(BI::kQFull + slot))
                    : "memory");
            }
          }
          if (!ok) {
            if (lane == 0) timed_out();
            break;
          }
        }
#pragma unroll 1
        for (int t = x.t0; t < x.t1; ++t, ++g) {
          const int s = g % kStages;
          if (g >= kStages && !wait_warp(bar(empty0 + s), ((g / kStages) - 1) & 1)) {
            if (lane == 0) timed_out();
            break;
          }
          const int k0 = x.key0(t), blk = k0 >> p.bs_log2;
          if (x.seq != tw_seq || blk < tw_base || blk + boxes > tw_base + 32) {
            tw_seq = x.seq;
            tw_base = blk;
            const int e = blk + lane;
            tw_val = e < p.max_blocks ? p.block_tables[static_cast<size_t>(x.seq) * p.max_blocks + e] : -1;
          }
          if (lane == 0) mbar_arrive_expect_tx(bar(full0 + s), kTile);
          // one lane per (box, half): the box copies go out in parallel
          const int jb = lane / kHalves, hf = lane % kHalves;
          const int b = __shfl_sync(0xffffffffu, tw_val, (blk + min(jb, boxes - 1) - tw_base) & 31);
          if (jb < boxes) {
            const int kb = k0 + jb * box_rows;  // the box's first key
            const bool seen = kb < x.hi && (kb + box_rows > x.lo || kb < x.sink_end);
            int row = p.oob_row;  // no row of the run sees any of it, or a bad id: zeros
            if (seen && b >= 0 && b < p.num_blocks) row = ((b * hkv + x.head) << p.bs_log2) + (kb & ((1 << p.bs_log2) - 1));
            else if (seen && p.status && !is_v && hf == 0) atomicOr(p.status, PKV_STATUS_BAD_BLOCK);
            tma_load_2d(ring + s * kTile + hf * Lay::kHalf + jb * box_rows * 128, tm, hf * 64, row, bar(full0 + s), pol);
          }
        }
        if (is_v && lane == 0) run_done(j);
      }
      // never leave a copy in flight into this CTA's shared memory
      if (lane == 0) {
#pragma unroll 1
        for (int y = g > kStages ? g - kStages : 0; y < g; ++y)
          mbar_wait_sleep(bar(full0 + (y % kStages)), (y / kStages) & 1);
        if (!is_v) {
#pragma unroll 1
          for (int y = nq > S ? nq - S : 0; y < nq; ++y) mbar_wait_sleep(bar(BI::kQFull + slot_of(y)), use_of(y) & 1);
          if (p.ws_desc) p.ws_desc[blockIdx.x] = desc;
        }
      }
    } else if (warp == kMmaWarp) {
      // ------------------------------------------------- S = Q K^T issuer
      // A product goes out once the slot's softmax has read the one before it (its
      // weights have their own columns), so the next product of a slot runs while
      // the weights of this one are computed.  One thread issues, and the softmax warps
      // keep its code out of the nearest instruction cache: few instructions per tile.
      // (A wait for the phase before a barrier's first, parity 1, returns at once.)
      if (tc::elect_one()) {
        // a negative scale is taken as the negated queries' product (bit 13: negate A)
        const uint32_t kIdS = tc::idesc_bf16(kRows, kTK, false, false) | (p.negate ? 1u << 13 : 0u);
        const uint32_t kd0 = desc_word(sK);
        uint32_t k_phase = 0, free_phase = 3, pv_phase = 15, buf = 0;  // of the stage; bits: [slot]; [slot][buffer]; [slot]
        int s = 0, nq = 0;  // stage; query tiles so far
        bool ok = true;
        auto product = [&](int slot) {
          if (!wait(bar(BI::kSFree + slot), (free_phase >> slot) & 1)) return false;
          free_phase ^= 1u << slot;
          // the weights that the softmax makes of this product go where those of the slot's
          // tile before the last were: their product must be complete
          const uint32_t b = 2 * slot + ((buf >> slot) & 1);
          if (!wait(bar(BI::kPvDone) + 8 * b, (pv_phase >> b) & 1)) return false;
          pv_phase ^= 1u << b;
          buf ^= 1u << slot;
          tc::fence_after();
          const uint32_t qd = desc_word(sQ + slot * kQTile), kd = kd0 + s * (kTile >> 4);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            tc::mma(tS + slot * kTK, desc_of(qd + (((ks >> 2) * Lay::kQHalf + (ks & 3) * 32) >> 4), kSpanHi),
                    desc_of(kd + (((ks >> 2) * Lay::kHalf + (ks & 3) * 32) >> 4), kSpanHi), kIdS, ks > 0);
          tc::commit(bar(BI::kSFull + slot));
          return true;
        };
#pragma unroll 1
        for (int j = 0; ok; ++j) {
          Run x;
          run_at(j, x);
          if (x.ntq == 0) break;
          run_done(j);
          if (x.t0 >= x.t1) continue;
          const int a = slot_of(nq), b = slot_of(nq + 1);
          const bool two = S == 2 && x.ntq == 2;
          ok = wait(bar(BI::kQFull + a), use_of(nq) & 1) && (!two || wait(bar(BI::kQFull + b), use_of(nq + 1) & 1));
#pragma unroll 1
          for (int left = x.t1 - x.t0; left > 0 && ok; --left) {
            ok = wait(bar(BI::kKFull) + 8 * s, k_phase) && product(a) && (!two || product(b));
            tc::commit(bar(BI::kKEmpty) + 8 * s);  // the keys are read by these products only
            if (++s == kStages) s = 0, k_phase ^= 1;
          }
          tc::commit(bar(BI::kQFree + a));
          if (two) tc::commit(bar(BI::kQFree + b));
          nq += x.ntq;
        }
        if (!ok) timed_out();
      }
    } else if (warp == kPvWarp) {
      // ------------------------------------------------ O += P V issuer
      // The whole warp goes through the tiles, for the values that must be cleared;
      // one lane issues.
      constexpr uint32_t kIdO = tc::idesc_bf16(kRows, D, false, true);
      constexpr int kSteps = kTK / 16;  // 16 keys = 8 packed columns of P
      const uint32_t vd0 = desc_word(sV) | (Lay::kHalf >> 4) << 16;
      uint32_t v_phase = 0, p_phase = 0, free_phase = 3, buf = 0;  // bits: [slot][buffer]; [slot]; [slot]
      int s = 0, g = 0, nq = 0;  // stage, key tiles, query tiles
      bool ok = true;
      const bool leader = tc::elect_one();
      auto product = [&](int slot, bool first, bool last) {
        const uint32_t b = 2 * slot + ((buf >> slot) & 1);
        if (!wait(bar(BI::kPFull) + 8 * b, (p_phase >> b) & 1)) return false;
        p_phase ^= 1u << b;
        buf ^= 1u << slot;
        tc::fence_after();
        const uint32_t pa = tP + b * (kTK / 2), vd = vd0 + s * (kTile >> 4);
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks)
          tc::mma_ta(tmem + slot * D, pa + ks * 8, desc_of(vd + (ks * 2048 >> 4), kSpanHi), kIdO, !(first && ks == 0));
        tc::commit(bar(BI::kPvDone) + 8 * b);
        if (last) tc::commit(bar(BI::kOFull + slot));
        return true;
      };
#pragma unroll 1
      for (int j = 0;; ++j) {
        Run x;
        run_at(j, x);
        __syncwarp();
        if (lane == 0) run_done(j);
        if (x.ntq == 0) break;
        if (x.t0 >= x.t1) continue;
        const Common<Tree> seen(p, x, lens[x.seq], qc[x.seq]);
        const int a = slot_of(nq), b = slot_of(nq + 1);
        const bool two = S == 2 && x.ntq == 2;
        // the first product overwrites the accumulator: its last run must have been read
        ok = wait(bar(BI::kOFree + a), (free_phase >> a) & 1) && (!two || wait(bar(BI::kOFree + b), (free_phase >> b) & 1));
        free_phase ^= (1u << a) | (two ? 1u << b : 0u);
#pragma unroll 1
        for (int t = x.t0, k0 = x.key0(t); t < x.t1; ++g) {
          ok = ok && wait(bar(BI::kVFull) + 8 * s, v_phase);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }  // the other lanes wait for the issues here
          if (!seen.has(k0) && clear_values<D>(sV + s * kTile, x, k0, lane) && lane == 0) *odd_tile = g + 1;
          const bool first = t == x.t0;
          k0 = ++t == x.ns ? x.t_lo * kTK : k0 + kTK;
          if (leader) {
            ok = product(a, first, t == x.t1) && (!two || product(b, first, t == x.t1));
            tc::commit(bar(BI::kVEmpty) + 8 * s);
          }
          if (++s == kStages) s = 0, v_phase ^= 1;
        }
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        nq += x.ntq;
      }
      if (!ok && lane == 0) timed_out();
    }
  } else {
    // ------------------------------------------------------ softmax warps
    if constexpr (S == 1) asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
    {
      const int slot = warp >> 2;
      const int r = threadIdx.x & (kRows - 1);  // query row = TMEM lane
      const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t tO = tmem + slot * D + lane_off, tSr = tS + slot * kTK + lane_off, tPr = tP + slot * kTK + lane_off;
      int g = 0, nq = 0, n = 0;  // key tiles and query tiles of the CTA, key tiles of this slot
      bool ok = true;
#pragma unroll 1
      for (int j = 0; ok; ++j) {
        Run x;
        run_at(j, x);
        __syncwarp();
        if (x.ntq == 0) break;
        const bool any = x.t0 < x.t1;
        // the run's query tile in this slot: without keys (nothing goes through the
        // slots) tile `slot` of the run
        const int q = S == 1 ? 0 : any ? (slot - nq) & 1 : slot, use = use_of(nq + q);
        if (any) nq += x.ntq;
        if (q >= x.ntq) {
          g += x.t1 - x.t0;
          if (lane == 0) run_done(j);
          continue;
        }
        const int c = qc[x.seq], ctx = lens[x.seq] - c;
        const int tok = r / p.group, token = x.r0 + q * p.tile_tok + tok;
        const bool row_valid = tok < p.tile_tok && token < c;
        RowSight<Tree> sight;
        sight.ctx = ctx;
        sight.word = sight.keep = 0;
        sight.lo = sight.hi = sight.sinks = 0;
        if (Tree) {
          if (row_valid) {
            sight.word = p.mask[qs[x.seq] + token];
            sight.keep = below(c);
          } else {
            sight.ctx = 0;
          }
        } else if (row_valid) {
          sight.hi = max(0, ctx + token + 1);
          sight.lo = max(0, sight.hi - p.window);
          sight.sinks = min(p.sinks, sight.hi);
        }
        // of the warp's rows, so that few of its tiles need a mask
        const int tile0 = x.r0 + q * p.tile_tok, row0 = (warp & 3) * 32;
        const int end = min(c, tile0 + p.tile_tok), row31 = tile0 + (row0 + 31) / p.group;
        const Common<Tree> seen(p, ctx, tile0 + row0 / p.group, min(end - 1, row31));
        const bool idle = __all_sync(0xffffffffu, !row_valid);  // spare rows only
        float m = -INFINITY, l = 0.f;
        const int g0 = g;
        g += x.t1 - x.t0;
#pragma unroll 1
        for (int t = x.t0, k0 = x.key0(t); t < x.t1; ++n) {
          const int buf = n & 1;
          const bool full = seen.has(k0);
          uint64_t see = ~0ull;
          bool none = idle;  // no row of the warp sees any of the tile
          if (!full) {
            see = sight.of(k0);
            none = __all_sync(0xffffffffu, see == 0);
          }
          k0 = ++t == x.ns ? x.t_lo * kTK : k0 + kTK;
          if (!wait_warp(bar(BI::kSFull + slot), n & 1)) { ok = false; break; }
          tc::fence_after();
          uint32_t pk[32];
          bool scale_o = false;
          float alpha = 1.f;
          if (none) {
            mbar_arrive(bar(BI::kSFree + slot));
#pragma unroll
            for (int k = 0; k < 32; ++k) pk[k] = 0u;
          } else {
            uint32_t sv[64];
            tc::ld32(tSr, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
            tc::ld32(tSr + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
            tc::wait_ld();
            tc::fence_before();
            mbar_arrive(bar(BI::kSFree + slot));  // the next product may take their place
            if (!full) {
              const uint32_t a = static_cast<uint32_t>(see), b = static_cast<uint32_t>(see >> 32);
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                if (!(a & (1u << k))) sv[k] = __float_as_uint(-INFINITY);
                if (!(b & (1u << k))) sv[32 + k] = __float_as_uint(-INFINITY);
              }
            }
            // move the reference max only when a score passes it by more than kSlack
            // (rare after a run's first tile); exact, since O and l share it
            const float bm = extreme64(sv, false) * p.scale_log2;
            if (bm > m + kSlack) {
              scale_o = m != -INFINITY;
              alpha = scale_o ? fast_exp2(m - bm) : 1.f;
              l *= alpha;
              m = bm;
            }
            const float msub = m == -INFINITY ? 0.f : m;
            const uint64_t ks2 = f32x2_bits(__float_as_uint(p.scale_log2), __float_as_uint(p.scale_log2));
            const uint64_t nm2 = f32x2_bits(__float_as_uint(-msub), __float_as_uint(-msub));
            l += weights64(sv, ks2, nm2, pk);
          }
          // the last product from this buffer is complete (the score product waited for it);
          // all must be before the accumulator is written
          if (__any_sync(0xffffffffu, scale_o)) {  // warp-uniform: tcgen05.ld/st are warp-wide
            if (!wait_warp(bar(BI::kPvDone + 2 * slot + (buf ^ 1)), ((n - 1) >> 1) & 1)) { ok = false; break; }
            tc::fence_after();
#pragma unroll 1
            for (int ch = 0; ch < D / 32; ++ch) {
              uint32_t ov[32];
              tc::ld32(tO + ch * 32, ov);
              tc::wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) ov[k] = __float_as_uint(__uint_as_float(ov[k]) * alpha);
              tc::st32(tO + ch * 32, ov);
            }
          }
          tc::fence_after();
          tc::st32(tPr + buf * (kTK / 2), pk);
          tc::wait_st();
          tc::fence_before();
          mbar_arrive(bar(BI::kPFull + 2 * slot + buf));
        }
        if (!ok) break;
        // ---- end of the piece: normalise and store the rows, or store the partial
        if (any) {
          if (!wait_warp(bar(BI::kOFull + slot), use & 1)) { ok = false; break; }
          tc::fence_after();
        }
        const float inv = any && l > 0.f ? 1.f / l : 0.f;
        const bool whole = x.whole();
        const size_t orow = (static_cast<size_t>(qs[x.seq]) + token) * p.num_q_heads + x.head * p.group + (r - tok * p.group);
        const size_t piece = 2 * static_cast<size_t>(blockIdx.x) + (x.t0 == 0 ? 1 : 0);
        const int prow = q * kRows + r;
        const bool odd = any && *reinterpret_cast<volatile int *>(odd_tile) > g0;
        auto store = [&](int ch, const uint32_t (&ov)[32]) {
          if (!whole) {
#pragma unroll
            for (int c4 = 0; c4 < 8; ++c4)
              p.ws_o[(piece * (D / 4) + ch * 8 + c4) * p.piece_rows + prow] =
                  make_float4(__uint_as_float(ov[c4 * 4]), __uint_as_float(ov[c4 * 4 + 1]), __uint_as_float(ov[c4 * 4 + 2]),
                              __uint_as_float(ov[c4 * 4 + 3]));
            return;
          }
          // a thread writes its own row: 32-byte stores (when the output allows) halve the requests
          __nv_bfloat16 *dst = p.out + orow * D + ch * 32;
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) w[k] = pack_bf16x2(__uint_as_float(ov[2 * k]) * inv, __uint_as_float(ov[2 * k + 1]) * inv);
          if ((reinterpret_cast<uintptr_t>(p.out) & 31) == 0) {
#pragma unroll
            for (int h8 = 0; h8 < 2; ++h8) st_global_v8(dst + h8 * 16, &w[8 * h8]);
          } else {
#pragma unroll
            for (int c8 = 0; c8 < 4; ++c8)
              reinterpret_cast<uint4 *>(dst)[c8] = make_uint4(w[4 * c8], w[4 * c8 + 1], w[4 * c8 + 2], w[4 * c8 + 3]);
          }
        };
        if (!any) {
          if (row_valid) {
            uint32_t ov[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) ov[k] = 0u;
#pragma unroll 1
            for (int ch = 0; whole && ch < D / 32; ++ch) store(ch, ov);  // an empty piece's O is not read
          }
        } else {
#pragma unroll 1
          for (int ch = 0; ch < D / 32; ++ch) {
            __syncwarp();
            uint32_t ov[32];
            tc::ld32(tO + ch * 32, ov);
            tc::wait_ld();
            if (!row_valid) continue;
            // add the values that were cleared because they are not finite, where this row sees them
#pragma unroll 1
            for (int t = x.t0; odd && t < x.t1; ++t) {
              const int k0 = x.key0(t);
              if (Common<Tree>(p, x, lens[x.seq], c).has(k0)) continue;  // (was not cleared)
#pragma unroll 1
              for (int k = 0; k < kTK; ++k) {
                if (!((sight.of(k0) >> k) & 1)) continue;
                const int b = p.block_tables[static_cast<size_t>(x.seq) * p.max_blocks + ((k0 + k) >> p.bs_log2)];
                if (b < 0 || b >= p.num_blocks) continue;
                const size_t at = ((static_cast<size_t>(b) * hkv + x.head) << p.bs_log2) + ((k0 + k) & ((1 << p.bs_log2) - 1));
                const uint32_t *row = reinterpret_cast<const uint32_t *>(p.v_cache + at * D + ch * 32);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const uint32_t w = row[i];
                  if ((w & 0x7F80u) == 0x7F80u)
                    ov[2 * i] = __float_as_uint(__uint_as_float(ov[2 * i]) + __uint_as_float(w << 16));
                  if ((w & 0x7F800000u) == 0x7F800000u)
                    ov[2 * i + 1] = __float_as_uint(__uint_as_float(ov[2 * i + 1]) + __uint_as_float(w & 0xFFFF0000u));
                }
              }
            }
            store(ch, ov);
          }
          __syncwarp();
          tc::fence_before();
          mbar_arrive(bar(BI::kOFree + slot));
        }
        if (!whole && row_valid) p.ws_ml[piece * p.piece_rows + prow] = make_float2(m, any ? l : kNoTile);
        __syncwarp();
        if (lane == 0) run_done(j);
      }
      if (!ok) timed_out();
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after();
    tc::dealloc(tmem, kTmemCols);
  }
}

// One block per CTA whose last run leaves it and per share of the head dim: the
// exact merge of the run's pieces, a thread per query row.
//   out = sum_p O_p 2^(m_p - M) / sum_p l_p 2^(m_p - M),  M = max_p m_p
template <int D>
__global__ void __launch_bounds__(2 * kRows) spans_join_kernel(const Params p, int grid) {
  grid_launch_dependents();
  grid_dependency_wait();  // the pieces come from the grid launched just before
  const int4 d = p.ws_desc[blockIdx.x];
  if (!(d.z & kLeaves)) return;
  int last = -1;  // the first CTA after this one in which the run ends
  for (int base = blockIdx.x + 1; base < grid && last < 0; base += 32) {
    const int c = base + (threadIdx.x & 31);
    const unsigned ends = __ballot_sync(0xffffffffu, c < grid && (p.ws_desc[c].z & kEnds));
    if (ends) last = base + __ffs(ends) - 1;
  }
  if (last < 0) return;  // only where a bounded wait gave up
  const int pieces = last - static_cast<int>(blockIdx.x) + 1;
  const int prow = threadIdx.x, q = prow / kRows, r = prow % kRows, tok = r / p.group, gh = r - tok * p.group;
  const int token = q * p.tile_tok + tok;
  if (tok >= p.tile_tok || token >= d.w) return;
  constexpr int kCols = D / 4 / kJoinShares;  // float4 columns of this block
  constexpr int kAhead = 4;                   // pieces whose loads are in flight together
  float4 acc[kCols];
#pragma unroll
  for (int k = 0; k < kCols; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  float M = -INFINITY, den = 0.f;
#pragma unroll 1
  for (int i0 = 0; i0 < pieces; i0 += kAhead) {
    float2 ml[kAhead];
    float4 o[kAhead][kCols];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      // piece 1 of the first CTA, piece 0 of the others
      const int c = i0 + i;
      const size_t at = 2 * (static_cast<size_t>(blockIdx.x) + c) + (c == 0 ? 1 : 0);
      ml[i] = make_float2(-INFINITY, kNoTile);
      if (c < pieces) {
        ml[i] = p.ws_ml[at * p.piece_rows + prow];
#pragma unroll
        for (int k = 0; k < kCols; ++k) o[i][k] = p.ws_o[(at * (D / 4) + blockIdx.y * kCols + k) * p.piece_rows + prow];
      }
    }
    float top = M;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) top = fmaxf(top, ml[i].x);
    const float keep = M == -INFINITY ? 0.f : exp2f(M - top);
    M = top;
    den *= keep;
#pragma unroll
    for (int k = 0; k < kCols; ++k) acc[k].x *= keep, acc[k].y *= keep, acc[k].z *= keep, acc[k].w *= keep;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      // Every piece with a tile takes part, also at a factor of 0: one whose scores are all
      // NaN has the maximum -inf too, and its sum and O (NaN) must reach the row, as must
      // what is not finite in a piece far below the maximum.
      if (ml[i].y == kNoTile) continue;
      const float f = ml[i].x == -INFINITY ? 0.f : exp2f(ml[i].x - M);
      den += ml[i].y * f;
#pragma unroll
      for (int k = 0; k < kCols; ++k) {
        acc[k].x += f * o[i][k].x;
        acc[k].y += f * o[i][k].y;
        acc[k].z += f * o[i][k].z;
        acc[k].w += f * o[i][k].w;
      }
    }
  }
  const float inv = den > 0.f ? 1.f / den : 0.f;
  uint2 *dst = reinterpret_cast<uint2 *>(p.out + ((static_cast<size_t>(d.x) + token) * p.num_q_heads + d.y * p.group + gh) * D) +
               blockIdx.y * kCols;
#pragma unroll
  for (int k = 0; k < kCols; ++k)
    dst[k] = make_uint2(pack_bf16x2(acc[k].x * inv, acc[k].y * inv), pack_bf16x2(acc[k].z * inv, acc[k].w * inv));
}

// ------------------------------------------------------------------ host
struct Plan {
  int group, tile_tok, span, piece_rows, slots, grid;
  bool split;  // some run may be cut
  size_t o_bytes, ml_bytes, desc_bytes;
  size_t bytes() const { return split ? o_bytes + ml_bytes + desc_bytes : 0; }
};

Plan make_plan(const Call &a) {
  Plan plan{};
  plan.group = a.num_q_heads / a.num_kv_heads;
  plan.tile_tok = kRows / plan.group;
  const int longest = a.mask ? a.max_nodes : a.total_q;  // tokens of a chunk or tree, at most
  plan.tile_tok = std::min(plan.tile_tok, std::max(1, longest));
  // Pairs of query tiles where the trees may have two, or the chunks have on average.
  // At head_dim 64 a pair's products are too short to hide two slots' softmax behind
  // one issuer, and longer chunks read their keys again in any case (through L2): one
  // slot, twice per SM, takes 410 us instead of 449 for four prompts of 8192 tokens
  // with 32 / 8 heads, and 337 instead of 371 for 4096 tokens of 64 / 8 heads.  Chunks
  // of one pair stay with pairs, which read their keys once: 191 us instead of 200 for
  // 64 chunks of 64 tokens with windows of 4096; trees too, 106 instead of 116 for 32
  // trees of 64 nodes on 4096 keys.
  const long long tile = static_cast<long long>(plan.tile_tok) * a.num_seqs;
  const bool one = a.head_dim == 64 && a.num_seqs <= kPairedSeqs && a.total_q > 2 * tile;
  const bool pairs = a.mask ? a.max_nodes > plan.tile_tok : a.total_q > tile && !one;
  plan.slots = pairs || a.num_seqs > kPairedSeqs ? 2 : 1;
  plan.span = pairs ? 2 * plan.tile_tok : plan.tile_tok;
  plan.grid = num_sms() * (3 - plan.slots);
  plan.piece_rows = pairs ? 2 * kRows : kRows;
  // A run of fewer tiles than two least pieces is never cut.  This and the sizes below
  // go by the longest runs that any batch of these heads and lengths has, so that one
  // workspace serves every batch: two pieces per CTA, 2 x 256 rows of them per SM.
  long long keys = a.max_seq_len;
  if (!a.mask) {
    const long long sunk = (static_cast<long long>(a.sinks) + kTK - 1) / kTK * kTK;
    keys = std::min(keys, static_cast<long long>(a.window) + 2 * kRows + 2 * kTK + sunk);
  }
  plan.split = (keys + kTK - 1) / kTK >= 2 * kMinPiece;
  const size_t rows = static_cast<size_t>(num_sms()) * 4 * kRows;
  plan.o_bytes = rows * a.head_dim * sizeof(float);
  plan.ml_bytes = rows * sizeof(float2);
  plan.desc_bytes = static_cast<size_t>(num_sms()) * 2 * sizeof(int4);
  return plan;
}

using KernelFn = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, Params);

template <int D, int S>
int launch(const CUtensorMap &tmq, const CUtensorMap &tmk, const CUtensorMap &tmv, const Params &p, const Plan &plan,
           cudaStream_t stream) {
  const KernelFn kernel = p.mask ? spans_tc_kernel<true, D, S> : spans_tc_kernel<false, D, S>;
  const size_t smem = smem_bytes<D, S>(p.num_seqs);
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem_bytes<D, S>(S == 2 ? kMaxSeqs : kPairedSeqs)));
  const unsigned grid = static_cast<unsigned>(plan.grid);
  if (e == cudaSuccess) e = launch_overlapped(kernel, grid, Layout<D, S>::kThreads, smem, stream, tmq, tmk, tmv, p);
  if (e == cudaSuccess && plan.split)
    e = launch_overlapped(spans_join_kernel<D>, dim3(grid, kJoinShares), plan.piece_rows, 0, stream, p, plan.grid);
  return e == cudaSuccess ? PKV_OK : (set_cuda_error(e), PKV_ERR_CUDA);
}

}  // namespace

size_t tc_workspace_size(const Call &a) { return make_plan(a).bytes(); }

int tc_launch(const Call &a) {
  const Plan plan = make_plan(a);
  if (plan.bytes() > 0 && (!a.workspace || a.workspace_bytes < plan.bytes() || !aligned16(a.workspace)))
    return PKV_ERR_WORKSPACE;
  const long long rows = static_cast<long long>(a.num_blocks) * a.num_kv_heads * a.block_size;
  if ((a.total_q / plan.span + static_cast<long long>(a.num_seqs)) * a.num_kv_heads >= kMaxRuns) return PKV_ERR_UNSUPPORTED;
  CUtensorMap tmq, tmk, tmv;
  // q viewed as [total_q][Hq][d]: a box is 64 columns x G heads x the tile's tokens
  const int box = std::min(a.block_size, kTK);
  if (!make_tensor_map_3d(&tmq, a.q, a.head_dim, a.num_q_heads, a.total_q, 64, plan.group, plan.tile_tok) ||
      !make_tensor_map_2d(&tmk, a.k_cache, a.head_dim, rows, 64, box) ||
      !make_tensor_map_2d(&tmv, a.v_cache, a.head_dim, rows, 64, box))
    return PKV_ERR_CUDA;
  Params p{};
  p.block_tables = a.block_tables;
  p.seq_lens = a.seq_lens;
  p.q_start = a.q_start;
  p.mask = a.mask;
  p.v_cache = reinterpret_cast<const __nv_bfloat16 *>(a.v_cache);
  p.out = reinterpret_cast<__nv_bfloat16 *>(a.out);
  if (plan.split) {
    char *ws = static_cast<char *>(a.workspace);
    p.ws_o = reinterpret_cast<float4 *>(ws);
    p.ws_ml = reinterpret_cast<float2 *>(ws + plan.o_bytes);
    p.ws_desc = reinterpret_cast<int4 *>(ws + plan.o_bytes + plan.ml_bytes);
  }
  p.status = a.status;
  while ((1 << p.bs_log2) < a.block_size) ++p.bs_log2;
  p.num_seqs = a.num_seqs;
  p.max_blocks = a.max_blocks;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.num_blocks = a.num_blocks;
  p.total_q = a.total_q;
  p.max_len = a.max_seq_len;
  p.oob_row = static_cast<int>(rows);
  p.group = plan.group;
  p.tile_tok = plan.tile_tok;
  p.span = plan.span;
  p.window = a.window;
  p.sinks = a.sinks;
  p.max_nodes = a.max_nodes;
  p.piece_rows = plan.piece_rows;
  p.scale_log2 = kernel_scale_log2(std::fabs(a.scale));
  p.negate = a.scale < 0.f;
  const cudaStream_t st = as_stream(a.stream);
  if (plan.slots == 1)
    return a.head_dim == 64 ? launch<64, 1>(tmq, tmk, tmv, p, plan, st)
                            : launch<128, 1>(tmq, tmk, tmv, p, plan, st);
  return a.head_dim == 64 ? launch<64, 2>(tmq, tmk, tmv, p, plan, st)
                          : launch<128, 2>(tmq, tmk, tmv, p, plan, st);
}

}  // namespace spans
}  // namespace pkv
