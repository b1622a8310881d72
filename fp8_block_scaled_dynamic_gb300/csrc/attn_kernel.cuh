// attn_kernel.cuh -- attention of packed prompts, and of drafted token trees over
// a paged cache -- all of it, a prefix that sequences share, or selected pages --
// on tcgen05 tensor cores.
//
// What is computed, per query row (a token or node and one of its heads):
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - m)
// over the keys j the row sees, in one pass over the keys with a running
// reference m (a running maximum, moved only when it falls behind by more
// than 2^8: the weights then stay below 2^8, and fp32 sums lose nothing by it).
// The weights are rounded to bf16 for their product with v (the tensor core's
// operand type).  Those roundings are independent of one another and weigh as
// much as the result's own: a row of random values is off by 0.0020 to 0.0024
// of its length, of which 0.0017 are the result's rounding.
//
// Tiles.  The G = Hq / Hkv query heads that share a kv head are rows of one
// tile: 128 / G tokens x G heads (so a decode step fills rows with heads, and
// k and v are read once for all of them), against 128 keys.  Two row tiles
// are in flight as two streams, so that the tensor core multiplies for one
// while the other takes its exponentials.  A single row tile has its scores
// doubly buffered instead: the next key tile's are there when one's are done.
//
// Warps of a CTA: 0-3 and 4-7 the softmax of stream 0 and 1 (a thread is a
// row: its 128 scores come from TMEM into registers), 8 issues the MMAs, 9
// loads by TMA, 10 guards the v tiles that not every row sees in full, 11
// works out the CTA's items and hands them to the others.
// TMEM: scores of a stream 128 columns, the bf16 weights over the first 64 of
// them once they are read, accumulators D columns a stream.
// Hand-offs are mbarriers; every wait is bounded.
//
// What bounds it, and what was measured (GB300; a copy runs at 6.8 TB/s, a
// bf16 library product at 1.90 PFLOP/s):
// - Long prompts of heads of 128: the two streams' chains and power.  8192 tokens
//   of 64 / 8 heads take 672-683 us at 2070 MHz (1.63 PFLOP/s): 1.53 us, 3200
//   cycles, for each pair of row tiles and 128 keys, of which the products are
//   2048 (64 for each 128 x 128 x 16; the tensor pipe is active 62 % of the time)
//   and the exponentials, beside them, 1024.  In a run of seconds the power limit
//   (1364 W) takes the clock to 1942 MHz and the time to 732 us.
// - Prompts of heads of 64: a stream's chain of scores, softmax and product
//   (about 2500 cycles a tile of which the products are 512), which two streams
//   cover to half: 8192 tokens of 64 / 8 heads 569 us, 0.97 PFLOP/s, at 2070 MHz.  A tile's
//   exponentials take 512 cycles of a scheduler, its tensor work as many.
//   Tried and slower: the weights in TMEM columns of their own with the next
//   scores under way during the softmax (585 us: the streams fall into step and
//   want the exponential unit together), two threads a row in 16 warps (732 us).
// - Trees over a long cache: HBM for one node a sequence (16 x 16384 cached
//   tokens, 8 kv heads of 128: 164-167 us, 6.4-6.5 TB/s), the softmax beside it
//   for many (32 nodes: 218-222 us, 1.26 PFLOP/s).
// - Short calls: latency.  One token over 1500 cached ones takes 12 us with
//   8 us in this kernel: reading the lists, the items, page table and first
//   load, first scores, first softmax and the result are about 1 us each.
#pragma once
#include <cstdint>
#include <cstring>
#include <mutex>
#include <type_traits>
#include <cudaTypedefs.h>
#include <cuda.h>
#include <cuda_runtime.h>

#include "attn.h"
#include "attn_ptx.cuh"
#include "kernels.h"

namespace mxg {
namespace {

// What a kernel attends to.  Shared and sparse: the sequences are the records that
// a plan kernel has written (attn_long.cu).
enum Mode { kPrompt, kTree, kShared, kSparse };
constexpr bool paged(int mode) { return mode != kPrompt; }
constexpr bool planned(int mode) { return mode >= kShared; }

constexpr int kBadIndex = 0x2;    // MXG_DEV_BAD_INDEX
constexpr int kSmemLayout = 0x4;  // MXG_DEV_SMEM_LAYOUT
constexpr int kThreads = 384;
constexpr int kKeys = 128;  // keys of a tile
constexpr int kRowsT = 128; // rows of a tile
constexpr int kHead = 3 * 1024;  // bytes of shared memory before the tiles
// Registers a thread: a softmax thread holds a row of 128 scores; the two
// softmax warpgroups take what the third gives up.  The three shares are the
// 168 a thread that the kernel is launched with.
constexpr int kRegs = 168, kRegsSoftmax = 200, kRegsRest = 104;
static_assert(2 * kRegsSoftmax + kRegsRest == 3 * kRegs, "register split");
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kFallBehind = 8.0f;  // log2 of how far the reference may lag the maximum

constexpr int kMaxCtas = 256;                       // of the paged kernels
constexpr long long kJoinFloats = kMaxCtas * 8;     // JoinItem of each CTA at the workspace's start

template <int D, int MODE>
struct Cfg {
  static constexpr int kHalves = D / 64;  // 128-byte columns of a row
  static constexpr int kTile = kKeys * D * 2;
  // A result goes to memory through a tile of its own, so that the next item's
  // q can come early.  (A tree's through its q tile, with a fifth slot for k
  // and v instead: 16 x 16384 cached tokens 166.5 us instead of 167.7, a
  // verify step's 20.0 either way.)
  static constexpr int kSlots = D == 64 ? 8 : 4;
  static constexpr int kSmem = kHead + (2 + kSlots + 1) * kTile;
  // a CTA's partial result of an item: two row tiles of [row][D] sums, then
  // their references and weight sums
  static constexpr long long kSlotFloats = 2LL * kRowsT * (D + 2);
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

// Flags of a plan's record.
constexpr int kHasNodes = 1;  // its sequence's nodes are keys too (the last tile)
constexpr int kJoined = 2;    // shared: its rows are in another record as well
constexpr int kLists = 4;     // sparse: several nodes, which name different pages

// a / b for a >= 0, b > 0 and a quotient below 2^22, in fp32 and one correction
// (the full integer division took a few hundred cycles of the item warp's way
// to the first load).
__device__ __forceinline__ int div_small(int a, int b) {
  const int q = (int)__fdividef((float)a, (float)b), r = a - q * b;
  return q + (r >= b) - (r < 0);
}

// ------------------------------------------------------------ work of a call
// Sequences in order; of each its kv heads, its row groups (pairs of row
// tiles), and -- tree -- its key tiles, all units numbered through (the host
// has checked that their number fits 31 bits).  The coarse prefix holds the
// number of units before every block of sequences and the offset that the
// block's first sequence may not start below.
constexpr int kBlocks = 64;
constexpr int kBlocksLane = kBlocks / 32;
struct Prefix {
  int units[kBlocks + 1];
  int start[kBlocks];
};

struct Seq {
  int a0, n;    // first token (node), tokens (nodes)
  int ctx;      // paged: cached tokens
  int per;      // key tiles of a row group that count as units (prompt: 1)
  int rows;     // row groups x kv heads
  int units;    // their product
  int hk, flags;  // planned: the only kv head or -1, the record's flags
  long long list; // planned: where the page numbers begin
};

struct Raw {
  int c0, c1, ctx;
  int hk, flags;
  long long list;
};
template <int MODE>
__device__ __forceinline__ Raw raw_seq(const AttnParams &p, int b) {
  if constexpr (planned(MODE)) {
    const int4 *r = reinterpret_cast<const int4 *>(p.plan.rec + b);
    const int4 x = __ldg(r), y = __ldg(r + 1);
    return {x.x, x.x + x.y, x.z, x.w, y.z, (long long)(((unsigned long long)(uint32_t)y.y << 32) | (uint32_t)y.x)};
  } else {
    return {__ldg(p.cu + b), __ldg(p.cu + b + 1), paged(MODE) ? __ldg(p.ctx + b) : 0, -1, 0, 0};
  }
}

// Sequences, or records of the plan.
template <int MODE>
__device__ __forceinline__ int seqs(const AttnParams &p) {
  return planned(MODE) ? p.plan.n : p.B;
}

template <int MODE>
__device__ __forceinline__ Seq seq_of(const AttnParams &p, const Raw &r, int tq2, int &running, bool *bad) {
  Seq s;
  if constexpr (planned(MODE)) {  // (within its bounds: the plan has seen to it)
    s.a0 = r.c0;
    s.n = r.c1 - r.c0;
    s.ctx = r.ctx;
    s.hk = r.hk;
    s.flags = r.flags;
    s.list = r.list;
    s.per = (s.ctx + kKeys - 1) / kKeys + (s.flags & kHasNodes);
    s.rows = div_small(s.n + tq2 - 1, tq2) * (s.hk < 0 ? p.Hkv : 1);
    s.units = s.rows * s.per;
    return s;
  }
  s.hk = -1;
  s.flags = kHasNodes;
  s.list = 0;
  s.a0 = max(min(max(r.c0, 0), p.T), running);
  const int a1 = max(min(max(r.c1, 0), p.T), s.a0);
  if (bad && (r.c0 != s.a0 || r.c1 != a1)) *bad = true;
  running = s.a0;
  s.n = a1 - s.a0;
  s.ctx = 0;
  s.per = 1;
  if (paged(MODE)) {
    if (s.n > kAttnMaxNodes) {
      s.n = kAttnMaxNodes;
      if (bad) *bad = true;
    }
    s.ctx = min(max(r.ctx, 0), p.table_cols * p.cache.page_size);
    if (bad && r.ctx != s.ctx) *bad = true;
    s.per = (s.ctx + kKeys - 1) / kKeys + 1;
  }
  s.rows = div_small(s.n + tq2 - 1, tq2) * p.Hkv;
  s.units = s.rows * s.per;
  return s;
}

// One warp fills the prefix.  tq2: tokens of a row group.
template <int MODE>
__device__ __forceinline__ void fill_prefix(const AttnParams &p, Prefix &pre, int tq2, int lane, bool report) {
  constexpr unsigned kFull = 0xFFFFFFFFu;
  const int B = seqs<MODE>(p), per = (B + kBlocks - 1) / kBlocks;
  const int own = kBlocksLane * per, b0 = min(lane * own, B), b1 = min(b0 + own, B);
  Raw first = {};  // (a small batch is read once)
  if (b0 < b1) first = raw_seq<MODE>(p, b0);
  int top = min(max(first.c0, 0), p.T);  // largest offset of this lane's sequences, then of those before
#pragma unroll 8
  for (int b = b0 + 1; b < b1; ++b) top = max(top, min(max(__ldg(p.cu + b), 0), p.T));
  int incl = top;
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl = max(incl, x);
  }
  int running = __shfl_up_sync(kFull, incl, 1);
  if (lane == 0) running = 0;
  bool bad = false;
  int mine = 0, part[kBlocksLane];
#pragma unroll
  for (int k = 0; k < kBlocksLane; ++k) {
    const int s0 = min(b0 + k * per, B), s1 = min(s0 + per, B);
    pre.start[lane * kBlocksLane + k] = running;
    part[k] = mine;
#pragma unroll 4
    for (int b = s0; b < s1; ++b)
      mine += seq_of<MODE>(p, b == b0 ? first : raw_seq<MODE>(p, b), tq2, running, &bad).units;
  }
  int sum = mine;
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kFull, sum, o);
    if (lane >= o) sum += x;
  }
#pragma unroll
  for (int k = 0; k < kBlocksLane; ++k) pre.units[lane * kBlocksLane + k] = sum - mine + part[k];
  if (lane == 31) pre.units[kBlocks] = sum;
  if (bad && report && p.status) atomicOr(p.status, kBadIndex);
  __syncwarp();
}

// A sequence found, and the unit at which it begins.
struct Found {
  Seq s;
  int b = -1, base = 0;
};

// The sequence that unit u is of, and u's number in it.  The units asked for
// mostly follow one another (tree), so it goes on from the last one found.
template <int MODE>
__device__ __forceinline__ Seq find_seq(const AttnParams &p, const Prefix &pre, int tq2, int &u, int &b, Found &last) {
  const int B = seqs<MODE>(p);
  if (paged(MODE) && last.b >= 0 && u >= last.base) {
    while (u >= last.base + last.s.units && last.b + 1 < B) {
      int running = last.s.a0;
      last.base += last.s.units;
      last.s = seq_of<MODE>(p, raw_seq<MODE>(p, ++last.b), tq2, running, nullptr);
    }
    b = last.b;
    u -= last.base;
    return last.s;
  }
  const int u0 = u;
  int lo = 0, hi = kBlocks - 1;
  while (lo < hi) {  // the last block that starts at or before u
    const int mid = (lo + hi + 1) >> 1;
    if (pre.units[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  u -= pre.units[lo];
  const int per = (B + kBlocks - 1) / kBlocks;
  int running = pre.start[lo];
  b = lo * per;
  Seq s = seq_of<MODE>(p, raw_seq<MODE>(p, b), tq2, running, nullptr);
  while (u >= s.units && b + 1 < B) {
    u -= s.units;
    s = seq_of<MODE>(p, raw_seq<MODE>(p, ++b), tq2, running, nullptr);
  }
  last.s = s;
  last.b = b;
  last.base = u0 - u;
  return s;
}

// The records of a plan by their units, of which the plan kernel has left a list:
// a lane adds up `per` of them, zeros behind the last one.  (Worked out from the
// records themselves, 256 of them took a CTA 4 us before its first load.)
__host__ __device__ __forceinline__ int units_per_lane(int records) { return ((records + 31) / 32 + 3) / 4 * 4; }
constexpr uint32_t kStrips = 0x80000000u;  // bit of a record's units: not one strip (row group of a kv head), but several
template <int MODE>
struct PlanUnits {
  int before, sum, total;  // of this lane's records
  int4 own;                // its records' units, if there are four a lane, and whether that is so and each is a strip
  bool alone;
  int b = -1, base = 0, units = 0;  // the record found last
  __device__ __forceinline__ void read(const AttnParams &p, int lane) {
    const int per = units_per_lane(p.plan.n);
    const int4 *at = reinterpret_cast<const int4 *>(p.plan.units + lane * per);
    sum = 0;
    uint32_t some = 0;
    int4 x;
#pragma unroll 4
    for (int i = 0; i < per / 4; ++i) {
      x = __ldg(at + i);
      some |= (uint32_t)(x.x | x.y | x.z | x.w);
      x.x &= ~kStrips, x.y &= ~kStrips, x.z &= ~kStrips, x.w &= ~kStrips;
      sum += (x.x + x.y) + (x.z + x.w);
    }
    own = x;
    alone = !__any_sync(0xFFFFFFFFu, some & kStrips) && per == 4;
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += x;
    }
    before = incl - sum;
    total = __shfl_sync(0xFFFFFFFFu, incl, 31);
  }
  // the record of unit u (u < total), and u's number in it
  __device__ __forceinline__ Seq find(const AttnParams &p, int tq2, int &u, int &of) {
    if (b < 0 || u < base) {
      const int lane = __ffs(__ballot_sync(0xFFFFFFFFu, u >= before && u < before + sum)) - 1;
      base = __shfl_sync(0xFFFFFFFFu, before, lane);
      b = lane * units_per_lane(p.plan.n);
      units = __ldg(p.plan.units + b) & ~kStrips;
    }
    while (u >= base + units) {
      base += units;
      units = __ldg(p.plan.units + ++b) & ~kStrips;
    }
    of = b;
    u -= base;
    int running = 0;
    return seq_of<MODE>(p, raw_seq<MODE>(p, b), tq2, running, nullptr);
  }
};

struct PlainItem {
  int b, hk;
  int a0, n;   // the sequence's first token (node) and count
  int r0;      // first token (node) of the first row tile, in the sequence
  int cnt[2];  // tokens (nodes) of the two row tiles
  int t0, t1;  // key tiles [t0, t1); t1 == t0: there is no item any more
  int end[2];  // a row tile's key tiles are [t0, end)
  int ctx, nct;
  int single;  // one row tile, its scores doubly buffered
  int part;    // -1 = the whole item, else the CTA's partial slot (0: the item began before, 1: it goes on);
               // 2: the whole item, of rows that another record has a part of (shared)
};
// With what a planned kernel's items have besides.
struct PlannedItem : PlainItem {
  int flags;             // the record's
  int list_lo, list_hi;  // where its page numbers begin
};
template <int MODE>
using Item = std::conditional_t<planned(MODE), PlannedItem, PlainItem>;
template <class I>
__device__ __forceinline__ void set_plan(I &it, int flags, long long list) {
  if constexpr (std::is_same_v<I, PlannedItem>) {
    it.flags = flags;
    it.list_lo = (int)(uint32_t)list;
    it.list_hi = (int)(list >> 32);
  }
}
template <class I>
__device__ __forceinline__ int flags_of(const I &it) {
  if constexpr (std::is_same_v<I, PlannedItem>) return it.flags;
  return kHasNodes;
}
template <class I>
__device__ __forceinline__ long long list_of(const I &it) {
  if constexpr (std::is_same_v<I, PlannedItem>)
    return (long long)((unsigned long long)(uint32_t)it.list_hi << 32 | (uint32_t)it.list_lo);
  return 0;
}

// What attn_join_kernel reads of a CTA's item that goes on in the next ones.
struct JoinItem {
  int rows0, rows;  // valid rows of the first row tile, of both (0: no such item)
  int tok, cnt0;    // first token of the rows, tokens of the first row tile
  int head;         // first query head
  int last;         // last CTA that holds a part
  int word;         // bits of a mask word that count; shared: 0 of a prefix, 1 of own keys
  int ctx;          // cached tokens
};

static_assert(sizeof(JoinItem) == 32, "workspace header");

// The CTAs' shares of U units: CTA c has [c q + min(c, r), ...), q = U / G, r = U % G.
__device__ __forceinline__ int share_begin(int c, int q, int r) { return c * q + min(c, r); }
__device__ __forceinline__ int share_owner(int u, int q, int r) {
  return u < r * (q + 1) ? u / (q + 1) : r + (u - r * (q + 1)) / q;
}

// A batch of at most 32 sequences in the registers of one warp, a sequence a
// lane: no prefix in shared memory, no search (0.8 us less before the first
// load of a decode step).
template <int MODE>
struct Small {
  Seq s;
  int before, total;  // units before this lane's sequence, of all
  __device__ __forceinline__ void read(const AttnParams &p, int tq2, int lane, bool report) {
    constexpr unsigned kFull = 0xFFFFFFFFu;
    Raw r = {};
    if (lane < seqs<MODE>(p)) r = raw_seq<MODE>(p, lane);
    int running = min(max(r.c0, 0), p.T);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(kFull, running, o);
      if (lane >= o) running = max(running, x);
    }
    running = __shfl_up_sync(kFull, running, 1);
    if (lane == 0) running = 0;
    bool bad = false;
    s = seq_of<MODE>(p, r, tq2, running, &bad);
    if (lane >= seqs<MODE>(p)) s.rows = s.units = 0;
    if (bad && lane < seqs<MODE>(p) && report && p.status) atomicOr(p.status, kBadIndex);
  }
  // Trees in order, prompts with the longest last (whose last units are dealt
  // first: six ragged prompts whose longest is the first of the batch 30.8 us
  // -> 27.1, as if it were the fourth).
  __device__ __forceinline__ void number(const AttnParams &p, int lane) {
    constexpr unsigned kFull = 0xFFFFFFFFu;
    total = __reduce_add_sync(kFull, s.units);
    if (paged(MODE)) {
      int sum = s.units;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kFull, sum, o);
        if (lane >= o) sum += x;
      }
      before = sum - s.units;
    } else {
      before = 0;
#pragma unroll 4
      for (int i = 0; i < p.B; ++i) {
        const int n = __shfl_sync(kFull, s.n, i), units = __shfl_sync(kFull, s.units, i);
        if (n < s.n || (n == s.n && i < lane)) before += units;
      }
    }
  }
  // Prompts: row groups of one row tile instead of two, where even then the
  // longest has more key tiles than a CTA's share of all.  The longest row
  // group's key tiles follow one another, and a lone row tile takes 0.6 to 0.7
  // of a pair's time for each: 1024 tokens of 16 / 16 heads 22.8 us -> 16.1,
  // 2048 of 16 / 2 heads 29.5 -> 23.5; but 512 of 64 / 8 heads, whose longest
  // is no longer than the share, would go from 13.8 to 16.2.  Returns the tokens
  // of a row group.
  __device__ __forceinline__ int choose_span(const AttnParams &p, int tq, int lane) {
    constexpr unsigned kFull = 0xFFFFFFFFu;
    const int ctas = gridDim.x;
    // (with two rounds of pairs the share is longer, and what follows fits 32 bits)
    if (__reduce_add_sync(kFull, s.units) >= 2 * ctas) return 2 * tq;
    const int tiles = lane < p.B ? min((s.n + kKeys - 1) / kKeys, 1 << 16) : 0;
    // key tiles of all lone row tiles, on average half the last one's
    const int work = __reduce_add_sync(kFull, s.rows * (tiles + 1));
    if (__reduce_max_sync(kFull, tiles) * ctas <= work) return 2 * tq;
    s.units = s.rows = lane < p.B ? div_small(s.n + tq - 1, tq) * p.Hkv : 0;
    return tq;
  }
  // the sequence of unit u (u < total), and u's number in it
  __device__ __forceinline__ Seq find(int &u, int &b) const {
    constexpr unsigned kFull = 0xFFFFFFFFu;
    b = __ffs(__ballot_sync(kFull, u >= before && u < before + s.units)) - 1;
    Seq r;
    r.a0 = __shfl_sync(kFull, s.a0, b);
    r.n = __shfl_sync(kFull, s.n, b);
    r.ctx = __shfl_sync(kFull, s.ctx, b);
    r.per = __shfl_sync(kFull, s.per, b);
    r.rows = r.units = 0;
    r.hk = -1;
    r.flags = kHasNodes;
    r.list = 0;
    if constexpr (planned(MODE)) {
      r.hk = __shfl_sync(kFull, s.hk, b);
      r.flags = __shfl_sync(kFull, s.flags, b);
      r.list = __shfl_sync(kFull, s.list, b);
    }
    u -= __shfl_sync(kFull, before, b);
    return r;
  }
};

// Strips (at most 128, a lane has the tiles of four and the units before them) cut
// into chunks of at least `least` tiles, at most four more, such that all have a CTA:
// this one's chunk as units x <= u < y, the CTA z of its strip's last chunk, and w = 0
// if no such length is.  A second item costs a CTA of the kernel of few rows 3 to 6 us:
// 64 strips of 19 tiles, two chunks each, 35.4 us instead of 36.5 as equal shares, 64
// of 9 18.4 instead of 20.1.  (Out of line: most calls have no use for it, and fetching
// its code cost them 0.7 us.)
__device__ __noinline__ int4 chunk_of_strips(int4 own, int before, int least, int ctas) {
  constexpr unsigned kFull = 0xFFFFFFFFu;
  const int lane = threadIdx.x & 31, c = blockIdx.x;
  const int tiles[4] = {own.x, own.y, own.z, own.w};
  for (int chunk = least; chunk < least + 5; ++chunk) {
    int pieces[4], mine = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) mine += pieces[k] = div_small(tiles[k] + chunk - 1, chunk);
    if (__reduce_add_sync(kFull, mine) > ctas) continue;
    int at = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(kFull, at, o);
      if (lane >= o) at += x;
    }
    at -= mine;
    int4 r = make_int4(0, 0, 0, 1);
    bool has = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = c - at, n = pieces[k];
      if (i >= 0 && i < n) {
        const int q = div_small(tiles[k], n), rest = tiles[k] - q * n;
        has = true;
        r.x = before + share_begin(i, q, rest);
        r.y = before + share_begin(i + 1, q, rest);
        r.z = at + n - 1;
      }
      at += n;
      before += tiles[k];
    }
    const unsigned who = __ballot_sync(kFull, has);
    const int from = who ? __ffs(who) - 1 : 0;  // (none: an empty range)
    r.x = __shfl_sync(kFull, r.x, from);
    r.y = __shfl_sync(kFull, r.y, from);
    r.z = __shfl_sync(kFull, r.z, from);
    return r;
  }
  return make_int4(0, 0, 0, 0);
}

// Walks the items of one CTA.
// Prompt: row groups from the last number to the first, dealt over the CTAs there
// and back.  A sequence's later row groups have more keys, so that within a long
// sequence who gets a heavy one in one round gets a light one in the next; in a
// small batch the longest sequence is numbered last and comes first (Small).
// Tree: the units are cut into equal ranges over the CTAs, an item is the part
// of one row group's key tiles that lies in this CTA's range -- or, where that
// costs at most two tiles a CTA more, every row group's key tiles are cut into
// equal chunks and a CTA takes one chunk: a second item costs a CTA more than
// two tiles (its result, the next q).
template <int MODE>
struct Walk {
  int cur, end, q, r;  // tree: this CTA's units, the shares; prompt: the round, the number of items
  int chunk;           // tree: most key tiles of a chunk, 0: equal ranges
  int last;            // planned: the range is a chunk, and this the CTA of the strip's last one; -1: equal ranges
  int span;            // tokens (nodes) of a row group
  int ctas;            // that share the work
  __device__ __forceinline__ Walk(int U, int span, int ctas) : chunk(0), last(-1), span(span), ctas(ctas) {
    if (paged(MODE)) {
      q = U / ctas;
      r = U - q * ctas;
      cur = share_begin(blockIdx.x, q, r);
      end = (int)blockIdx.x < ctas ? share_begin(blockIdx.x + 1, q, r) : cur;
    } else {
      cur = 0;
      end = U;
      q = r = 0;
    }
  }
  // the chunk length for which all chunks have a CTA, if there is a short one
  __device__ __forceinline__ void choose_chunk(const Small<MODE> &b) {
    if (q == 0) return;  // fewer units than CTAs: the ranges are single units
    const int least = q + (r > 0);
    int chunks[3];
#pragma unroll
    for (int i = 0; i < 3; ++i)
      chunks[i] = __reduce_add_sync(0xFFFFFFFFu, b.s.rows * div_small(b.s.per + least + i - 1, least + i));
#pragma unroll
    for (int i = 2; i >= 0; --i)
      if (chunks[i] <= ctas) chunk = least + i;
  }
  // The same for a plan's records, where they are a strip each and four a lane: a chunk
  // instead of the range.
  __device__ __forceinline__ void choose_chunk(const PlanUnits<MODE> &b) {
    if (q == 0 || !b.alone) return;
    const int4 x = chunk_of_strips(b.own, b.before, q + (r > 0), ctas);
    if (x.w) cur = x.x, end = x.y, last = x.z;
  }
  // this CTA's only item, a chunk; returns the last CTA of the row group's chunks
  __device__ __forceinline__ int one_chunk(const AttnParams &p, const Small<MODE> &b, int tq, Item<MODE> &it) {
    constexpr unsigned kFull = 0xFFFFFFFFu;
    const int lane = threadIdx.x & 31, c = blockIdx.x;
    const int pieces = div_small(b.s.per + chunk - 1, chunk);
    const int mine = b.s.rows * pieces;
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(kFull, sum, o);
      if (lane >= o) sum += x;
    }
    const unsigned has = __ballot_sync(kFull, c >= sum - mine && c < sum);
    it.t0 = it.t1 = 0;
    cur = end;
    if (!has) return 0;
    it.b = __ffs(has) - 1;
    it.a0 = __shfl_sync(kFull, b.s.a0, it.b);
    it.n = __shfl_sync(kFull, b.s.n, it.b);
    it.ctx = __shfl_sync(kFull, b.s.ctx, it.b);
    int hk = -1, flags = kHasNodes;
    long long list = 0;
    if constexpr (planned(MODE)) {
      hk = __shfl_sync(kFull, b.s.hk, it.b);
      flags = __shfl_sync(kFull, b.s.flags, it.b);
      list = __shfl_sync(kFull, b.s.list, it.b);
    }
    const int per = __shfl_sync(kFull, b.s.per, it.b), k = __shfl_sync(kFull, pieces, it.b);
    const int x = c - __shfl_sync(kFull, sum - mine, it.b), gh = div_small(x, k), piece = x - gh * k;
    const int cut = div_small(per, k), rest = per - cut * k;
    it.t0 = share_begin(piece, cut, rest);
    it.t1 = share_begin(piece + 1, cut, rest);
    rows_of(p, tq, gh, per, hk, flags, list, it);
    return c + k - 1 - piece;
  }
  // tree: kv head and rows of row group x kv head gh, what its end is
  __device__ __forceinline__ void rows_of(const AttnParams &p, int tq, int gh, int per, int hk, int flags,
                                          long long list, Item<MODE> &it) {
    const int g = planned(MODE) && hk >= 0 ? gh : div_small(gh, p.Hkv);
    it.hk = planned(MODE) && hk >= 0 ? hk : gh - g * p.Hkv;
    it.nct = planned(MODE) ? per - (flags & kHasNodes) : per - 1;
    it.part = it.t0 > 0 ? 0 : it.t1 < per ? 1 : MODE == kShared && (flags & kJoined) ? 2 : -1;
    set_plan(it, flags, list);
    it.r0 = g * span;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      it.cnt[k] = min(max(it.n - it.r0 - k * tq, 0), tq);
      it.end[k] = it.cnt[k] == 0 ? it.t0 : it.t1;
    }
    it.single = it.cnt[1] == 0;
  }
  template <class Find>
  __device__ __forceinline__ void next(const AttnParams &p, int tq, Item<MODE> &it, Find find) {
    it.t0 = it.t1 = 0;
    if (paged(MODE)) {
      if (cur >= end) return;
      int u = cur;
      const Seq s = find(u, it.b);
      it.a0 = s.a0;
      it.n = s.n;
      it.ctx = s.ctx;
      const int gh = div_small(u, s.per);
      it.t0 = u - gh * s.per;
      it.t1 = min(s.per, it.t0 + (end - cur));
      cur += it.t1 - it.t0;
      rows_of(p, tq, gh, s.per, s.hk, s.flags, s.list, it);
    } else {
      const int G = gridDim.x, x = cur * G + (cur & 1 ? G - 1 - (int)blockIdx.x : (int)blockIdx.x);
      if (cur * G >= end) return;
      ++cur;
      if (x >= end) {  // (the last round may be there or not)
        it.t1 = -1;
        return;
      }
      int u = end - 1 - x;
      const Seq s = find(u, it.b);
      it.a0 = s.a0;
      it.n = s.n;
      it.ctx = it.nct = 0;
      const int g = div_small(u, p.Hkv);
      it.hk = u - g * p.Hkv;
      it.part = -1;
      it.r0 = g * span;
      const int n = min(s.n, it.r0 + span);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        it.cnt[k] = min(max(n - it.r0 - k * tq, 0), tq);
        it.end[k] = it.cnt[k] == 0 ? 0 : (it.r0 + k * tq + it.cnt[k] + kKeys - 1) / kKeys;
      }
      it.single = it.cnt[1] == 0;
      it.t1 = max(it.end[0], it.end[1]);
    }
  }
};

// V rows of key tile j that some row of the item sees, and the first of them
// that not every row does.
template <int MODE>
__device__ __forceinline__ int v_valid(const Item<MODE> &it, int j) {
  if (paged(MODE)) return j < it.nct ? min(kKeys, it.ctx - j * kKeys) : it.n;
  return min(kKeys, it.r0 + it.cnt[0] + it.cnt[1] - j * kKeys);
}
template <int MODE>
__device__ __forceinline__ int v_shared(const Item<MODE> &it, int j) {
  if (paged(MODE)) return j < it.nct ? kKeys : 0;
  return min(max(it.r0 + 1 - j * kKeys, 0), kKeys);
}
template <int MODE>
__device__ __forceinline__ bool guarded(const Item<MODE> &it, int j) {
  return min(v_valid<MODE>(it, j), v_shared<MODE>(it, j)) < kKeys;
}
// The first guarded tile at or after t0 (they are the item's last ones).
template <int MODE>
__device__ __forceinline__ int first_guarded(const Item<MODE> &it) {
  const int j = paged(MODE) ? it.ctx / kKeys : (it.r0 + 1) / kKeys;
  return max(j, it.t0);
}

constexpr int kItemReaders = 11;  // warps 0 to 10, an arrival each

template <int D, int MODE>
struct Smem {
  using C = Cfg<D, MODE>;
  // (8-byte barriers first)
  uint64_t q_full[2], q_empty[2], kv_full[C::kSlots], kv_empty[C::kSlots];
  uint64_t v_issued[C::kSlots], kv_clean[C::kSlots];  // the guard's
  // scores, weights and products: of the two streams, then of the two buffers
  // of a single row tile (each has its own phases, since the second stream's
  // warps have no part in a single tile)
  uint64_t s_full[4], p_half[4], p_ready[4], pv_done[4], o_free[2];
  uint64_t item_full[2], item_free[2], guard_item[2], mma_done, stall;
  uint32_t tmem;
  int abort_flag;
  uint32_t poison[2][3][4];  // rows of the guarded tiles that hold a NaN or an infinity, by item parity
  Item<MODE> items[2];
  Prefix pre;
};

__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const WaitCtl &ctl) {
  const bool ok = mbar_wait_quick(smem_addr(bar), parity, ctl);
  return __all_sync(0xFFFFFFFFu, ok);
}
// The same for the warps that hold few registers, the loop out of line: some
// forty copies of it would be a fifth of the code.
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int *abort_flag, int *status,
                                     unsigned long long timeout_ns) {
  return mbar_wait_quick(bar, parity, WaitCtl{abort_flag, status, timeout_ns});
}
__device__ __forceinline__ bool lane_wait(uint64_t *bar, uint32_t parity, const WaitCtl &ctl) {
  return mbar_try_wait(smem_addr(bar), parity) ||
         wait_on(smem_addr(bar), parity, ctl.abort_flag, ctl.status, ctl.timeout_ns);
}
__device__ __forceinline__ bool warp_wait_far(uint64_t *bar, uint32_t parity, const WaitCtl &ctl) {
  return __all_sync(0xFFFFFFFFu, lane_wait(bar, parity, ctl));
}
// Bounded wait that ignores the abort flag: lets what is in flight land.
__device__ __forceinline__ void drain(uint64_t *bar, uint32_t parity, uint64_t timeout_ns) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(smem_addr(bar), parity))
    if (global_timer_ns() - t0 > timeout_ns) return;
}
__device__ __forceinline__ void warp_arrive(uint64_t *bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(smem_addr(bar));
}

__device__ __forceinline__ bool not_finite2(uint32_t w) {
  return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}

// The same two values, zeros for what is not finite.
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
  if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
  if ((w & 0x7F800000u) == 0x7F800000u) w &= 0xFFFFu;
  return w;
}

// A row written by a warp, a lane V channels: the result (0 of a row that sees nothing), a part's sums.
template <int V>
__device__ __forceinline__ void store_row(uint16_t *out, const float (&o)[V], float inv, bool any, int lane) {
#pragma unroll
  for (int e = 0; e < V; e += 2)
    reinterpret_cast<uint32_t *>(out + lane * V)[e / 2] = any ? pack_bf16x2(o[e] * inv, o[e + 1] * inv) : 0u;
}
template <int V>
__device__ __forceinline__ void store_part(float *part, const float (&o)[V], int lane) {
#pragma unroll
  for (int e = 0; e < V; e += 2)
    reinterpret_cast<float2 *>(part + lane * V)[e / 2] = make_float2(o[e], o[e + 1]);
}

// The lanes' values v[N] joined by op over a warp: lane i gets number i / (32 / N) of them.
template <int N, class Op>
__device__ __forceinline__ float over_lanes(float (&v)[N], int lane, Op op) {
  int bit = 16;
#pragma unroll
  for (int half = N / 2; half > 0; half >>= 1, bit >>= 1)
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float keep = lane & bit ? v[i + half] : v[i], send = lane & bit ? v[i] : v[i + half];
      v[i] = op(keep, __shfl_xor_sync(0xFFFFFFFFu, send, bit));
    }
#pragma unroll
  for (int rest = 16 / N; rest > 0; rest >>= 1) v[0] = op(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], rest));
  return v[0];
}

// A part's sums are taken for too large from here on.  Weights of up to 2^30 (few rows) or
// 2^8 then keep them and, joined from all CTAs, their total below fp32's largest.
constexpr uint32_t kTooLarge = 0x7A800000u;  // 2^118; NaN and infinities are above it
__device__ __forceinline__ bool too_large(uint32_t x) { return (x & 0x7FFFFFFFu) >= kTooLarge; }
__device__ const uint4 kNoKey[16] = {};  // of a page outside the cache

// R rows of a part summed again by a warp, each from what it sees: their accumulators
// held a NaN or an infinity, which may be another row's (a weight of zero times an
// infinity is a NaN), or were too large for their reference, which is the row's maximum
// here.  Lanes 32 / R * i ... give row i, its number in the row tile whose first node is
// tok0 (-1: none), and get its reference and sum of weights (as rounded); its sums go to
// to[i * stride ...].
// U keys at a time, of the pages that one of the rows sees, of which a warp finds 32 at
// once: their products with the rows' q are added up so that a lane has one row's and
// key's.  Latency bounds it.  Other warps wait meanwhile, and may for a second: four rows
// and keys at once take a warp with 32 rows 1.5 to 2 us a key (D = 128; 131072 keys, the
// most that 512 pages hold, 0.25 s), one row and key at once 0.5 us a key and row.  (A
// row's thread by itself took 16 us a key.)
template <int D, int MODE, int R, int U>
__device__ __noinline__ float2 sum_again(const AttnParams &p, const Item<MODE> &it, int tok0, int row, float *to, int stride) {
  constexpr int V = D / 32, L = 32 / R;  // channels of a lane, lanes of a row
  constexpr unsigned kFull = 0xFFFFFFFFu;
  const int lane = threadIdx.x & 31, shift = 31 - __clz(p.cache.page_size), G = p.Hq / p.Hkv;
  const float c = p.scale * kLog2e;
  struct Row {  // this lane's channels, as they are in memory
    uint32_t w[V / 2];
    __device__ __forceinline__ float operator[](int i) const {
      return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    }
  };
  auto load = [&](const uint16_t *x) {
    Row r;
    if constexpr (V == 4) {
      const uint2 z = *reinterpret_cast<const uint2 *>(x + lane * V);
      r.w[0] = z.x, r.w[1] = z.y;
    } else {
      r.w[0] = *reinterpret_cast<const uint32_t *>(x + lane * V);
    }
    return r;
  };
  const bool is = row >= 0;
  const int nd = div_small(max(row, 0), G), tok = tok0 + nd;  // this lane's row's node in the sequence
  const int my_key = lane % L / (L / U);
  Row q[R];
  float o[R][V] = {}, m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int t = __shfl_sync(kFull, tok, L * i), h = __shfl_sync(kFull, max(row, 0) - nd * G, L * i);
    q[i] = load(p.q.ptr + (long long)(it.a0 + t) * p.q.tok + (it.hk * G + h) * p.q.head);
  }
  // U keys, at k_of(u) and v_of(u); see: this lane's row sees this lane's key
  auto take = [&](bool see, auto k_of, auto v_of) {
    Row k[U], v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      k[u] = load(k_of(u));
      v[u] = load(v_of(u));
    }
    float s[R * U];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float &x = s[U * i + u];
        x = 0.0f;
#pragma unroll
        for (int d = 0; d < V; ++d) x = fmaf(q[i][d], k[u][d], x);
      }
    const float sum = over_lanes(s, lane, [](float a, float b) { return a + b; });
    const unsigned who = __ballot_sync(kFull, see && is);
    // the row's maximum: where it rises, the sums so far are scaled down
    float top = see ? sum : -INFINITY;
#pragma unroll
    for (int x = L / U; x < L; x <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, x));
    const bool rises = top > m;
    if (__any_sync(kFull, rises)) {
      const float f = rises ? ex2((m - top) * c) : 1.0f;
      m = fmaxf(m, top);
      l *= f;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float fi = __shfl_sync(kFull, f, L * i);
#pragma unroll
        for (int d = 0; d < V; ++d) o[i][d] *= fi;
      }
    }
    const uint32_t w = pack_bf16x2(0.0f, ex2(fmaf(sum, c, m == -INFINITY ? 0.0f : -m * c))) & 0xFFFF0000u;
    if (see) l += __uint_as_float(w);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int from = L * i + L / U * u;
        const float wu = __uint_as_float(__shfl_sync(kFull, w, from));
        if (!(who >> from & 1u)) continue;  // (not even a zero times v)
#pragma unroll
        for (int d = 0; d < V; ++d) o[i][d] = fmaf(wu, v[u][d], o[i][d]);
      }
  };
  // bits of the rows' nodes, or of their words
  auto of_all = [&](unsigned long long x) {
#pragma unroll
    for (int i = L; i < 32; i <<= 1) x |= __shfl_xor_sync(kFull, x, i);
    return x;
  };
  const unsigned long long toks = of_all(is ? 1ull << (tok & 63) : 0ull);
  const long long list = list_of(it);
  const int *pages = (MODE == kSparse ? p.plan.list : p.table) + list;
  const bool lists = MODE == kSparse && (flags_of(it) & kLists);
  const int begin = it.t0 * kKeys, end = min(it.ctx, it.t1 * kKeys), pe = (end + p.cache.page_size - 1) >> shift;
  for (int p0 = begin >> shift; p0 < pe; p0 += 32) {
    const int mine = p0 + lane;
    unsigned long long names = 0;
    if (mine < pe) names = lists ? p.plan.names[list + mine] : ~0ull;
    const int id = (names & toks) ? pages[mine] : 0;
    for (unsigned who = __ballot_sync(kFull, (names & toks) != 0ull); who; who &= who - 1) {
      const int x = __ffs(who) - 1, page = __shfl_sync(kFull, id, x), first = (p0 + x) << shift;
      const bool sees = __shfl_sync(kFull, names, x) >> (tok & 63) & 1ull;
      const bool in = (uint32_t)page < (uint32_t)p.cache.pages;
      const long long at = page * p.cache.page + it.hk * p.cache.head, slot = in ? p.cache.slot : 0;
      const uint16_t *const none = reinterpret_cast<const uint16_t *>(kNoKey);
      const uint16_t *const k0 = in ? p.cache.k + at : none, *const v0 = in ? p.cache.v + at : none;
      const int n = min(end - first, p.cache.page_size);
      for (int t = max(begin - first, 0); t < n; t += U)  // (past the last one: that one, which does not count)
        take(sees && t + my_key < n, [&](int u) { return k0 + min(t + u, n - 1) * slot; },
             [&](int u) { return v0 + min(t + u, n - 1) * slot; });
    }
  }
  if (it.t1 > it.nct) {
    unsigned long long word = 0;
    if (is) word = p.mask[it.a0 + tok] & (it.n >= 64 ? ~0ull : (1ull << it.n) - 1ull);
    for (unsigned long long rest = of_all(word); rest;) {
      int node[U];
      unsigned long long mine = 0;  // this lane's key's bit
#pragma unroll
      for (int u = 0; u < U; ++u) {
        node[u] = max(__ffsll((long long)rest) - 1, 0);  // (none left: the first one, which does not count)
        if (u == my_key) mine = rest & (0ull - rest);
        rest &= rest - 1ull;
      }
      take((word & mine) != 0ull, [&](int u) { return p.k.ptr + (long long)(it.a0 + node[u]) * p.k.tok + it.hk * p.k.head; },
           [&](int u) { return p.v.ptr + (long long)(it.a0 + node[u]) * p.v.tok + it.hk * p.v.head; });
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (__shfl_sync(kFull, row, L * i) >= 0) store_part(to + i * stride, o[i], lane);
  __syncwarp();
#pragma unroll
  for (int x = L / U; x < L; x <<= 1) l += __shfl_xor_sync(kFull, l, x);
  return make_float2(m, l);
}

template <int D, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmKC,
                const __grid_constant__ CUtensorMap tmVC, const __grid_constant__ AttnParams p) {
  using C = Cfg<D, MODE>;
  constexpr bool TREE = paged(MODE);
  constexpr int S = C::kSlots;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  static_assert(sizeof(Smem<D, MODE>) <= kHead, "shared memory head");
  Smem<D, MODE> &sm = *reinterpret_cast<Smem<D, MODE> *>(smem_raw);
  const uint32_t base = smem_addr(smem_raw);
  if (base & 1023u) {  // the swizzled tiles need it (uniform over the grid)
    if (threadIdx.x == 0) {
      pdl_wait();
      if (TREE) reinterpret_cast<JoinItem *>(p.ws)[blockIdx.x].rows = 0;
      if (p.status) atomicOr(p.status, kSmemLayout);
    }
    return;
  }
  const uint32_t q_smem = base + kHead, kv_smem = q_smem + 2 * C::kTile;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv, TQ = kRowsT / G;
  if (MODE != kShared) pdl_trigger();

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&sm.q_full[i]), 1);
      mbar_init(smem_addr(&sm.q_empty[i]), 4);
      mbar_init(smem_addr(&sm.o_free[i]), 4);
      mbar_init(smem_addr(&sm.guard_item[i]), 1);
      mbar_init(smem_addr(&sm.item_full[i]), 1);
      mbar_init(smem_addr(&sm.item_free[i]), kItemReaders);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_addr(&sm.s_full[i]), 1);
      mbar_init(smem_addr(&sm.p_half[i]), 4);
      mbar_init(smem_addr(&sm.p_ready[i]), 4);
      mbar_init(smem_addr(&sm.pv_done[i]), 1);
    }
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_addr(&sm.kv_full[i]), 1);
      mbar_init(smem_addr(&sm.kv_empty[i]), 1);
      mbar_init(smem_addr(&sm.v_issued[i]), 1);
      mbar_init(smem_addr(&sm.kv_clean[i]), 1);
    }
    mbar_init(smem_addr(&sm.mma_done), 1);
    mbar_init(smem_addr(&sm.stall), 1);
    sm.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(smem_addr(&sm.tmem), 512);
    tmem_relinquish();
  }
  if (warp == 9 && lane == 0) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
    if (TREE) {
      prefetch_tmap(&tmKC);
      prefetch_tmap(&tmVC);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(&sm.tmem);
  const WaitCtl ctl{&sm.abort_flag, p.status, p.timeout_ns};
  pdl_wait();
  if (MODE == kShared) pdl_trigger();  // (the plan is there for whoever starts now)
  Item<MODE> it;
  // item k of the CTA; false when there is none (or a wait ran out)
  auto next_item = [&](int k) {
    if (!warp_wait(&sm.item_full[k & 1], (k >> 1) & 1, ctl)) return false;
    it = sm.items[k & 1];
    return it.t1 > it.t0;
  };
  auto done_item = [&](int k) { warp_arrive(&sm.item_free[k & 1], lane); };

  if (warp >= 8) {
    regs_less<kRegsRest>();
    if (warp == 9) {
      // ------------------------------------------------------------- loads
      // The loader has to keep pace with 64 KB a key tile beside busy softmax
      // warps (at pages of 16, 32 copies), so: no divisions, the ring's place
      // and phase carried along, pages read from the table two to three tiles
      // ahead, and the copies issued by one elected lane from warp-uniform
      // operands.
      uint32_t n = 0, nq[2] = {0, 0}, slot = 0, turn = 0;
      bool ok = true;
      const bool el = elect_one();
      const uint32_t kvb = uniform(kv_smem), full0 = uniform(smem_addr(&sm.kv_full[0])), qb = uniform(q_smem);
      const int page_shift = TREE ? 31 - __clz(p.cache.page_size) : 0, box_shift = TREE ? min(page_shift, 7) : 7;
      if (TREE && MODE != kSparse) {
        // a small batch's page table into L1, while the items are worked out
        // (a line a lane: the first load then does not wait for L2 twice; a table
        // of no columns has a row stride of 0, and nothing is prefetched)
        const long long ints = (long long)(p.B - 1) * p.ld_table + p.table_cols;
        if (lane * 32LL < ints) prefetch_l1(p.table + lane * 32);
      }
      for (int k = 0; ok && next_item(k); ++k) {
        const int t0 = (int)uniform(it.t0), t1 = (int)uniform(it.t1), nct = (int)uniform(it.nct);
        const int hk = (int)uniform(it.hk), a0 = (int)uniform(it.a0), ctx = (int)uniform(it.ctx);
        // lane b: the page of box b (a page of up to 128 keys) of tile j
        const int *row = MODE == kSparse   ? p.plan.list + list_of(it)
                         : MODE == kShared ? p.table + list_of(it)
                                           : p.table + (long long)it.b * p.ld_table;
        auto page_of = [&](int j) {
          const int key = (j << 7) + (lane << box_shift);
          if (!TREE || j >= nct || j >= t1 || (lane << box_shift) >= kKeys || key >= ctx) return 0;
          return __ldg(row + (key >> page_shift));
        };
        auto load_kv = [&](int j, bool is_v, int pg) {
          if (!warp_wait_far(&sm.kv_empty[slot], turn ^ 1, ctl)) return false;  // (free at first)
          const uint32_t us = uniform(slot), bar = full0 + 8 * us, dst = kvb + us * C::kTile;
          if (TREE && j < nct) {
            const int boxes = (min(kKeys, ctx - (j << 7)) + (1 << box_shift) - 1) >> box_shift;
            if ((uint32_t)pg >= (uint32_t)p.cache.pages) {
              pg = p.cache.pages;  // out of the map's bounds: zeros
              if (p.status) atomicOr(p.status, kBadIndex);
            }
            int page[8];
            page[0] = (int)__shfl_sync(0xFFFFFFFFu, pg, 0);
            if (box_shift < 7) page[1] = (int)__shfl_sync(0xFFFFFFFFu, pg, 1);
            if (box_shift < 6) {
#pragma unroll
              for (int b = 2; b < 8; ++b) page[b] = (int)__shfl_sync(0xFFFFFFFFu, pg, b);
            }
            if (el) {
              mbar_arrive_expect_tx(bar, (uint32_t)boxes << (box_shift + 7) << (C::kHalves - 1));
#pragma unroll
              for (int b = 0; b < 8; ++b) {
                if (b >= boxes) break;
#pragma unroll
                for (int h = 0; h < C::kHalves; ++h)
                  tma_load_4d(dst + h * 16384 + (b << box_shift) * 128, is_v ? &tmVC : &tmKC, h * 64, hk,
                              (j << 7) & ((1 << page_shift) - 1), page[b], bar);
              }
            }
          } else if (el) {
            // keys of the packed tensors: a prompt's tile, or the nodes (64 rows)
            mbar_arrive_expect_tx(bar, (uint32_t)((TREE ? kAttnMaxNodes : kKeys) * 128 * C::kHalves));
#pragma unroll
            for (int h = 0; h < C::kHalves; ++h)
              tma_load_3d(dst + h * 16384, is_v ? &tmV : &tmK, h * 64, hk, a0 + (TREE ? 0 : j * kKeys), bar);
          }
          __syncwarp();
          if (is_v && guarded<MODE>(it, j)) warp_arrive(&sm.v_issued[slot], lane);
          ++n;
          if (++slot == S) slot = 0, turn ^= 1;
          return true;
        };
        int pg[4];  // this lane's pages of tiles j .. j + 3
#pragma unroll
        for (int x = 0; x < 3; ++x) pg[x] = page_of(t0 + x);
        ok = load_kv(t0, false, pg[0]);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          // (single row tiles take the two q tiles in turn)
          if (!ok || (it.single ? s != (k & 1) : it.end[s] <= t0)) continue;
          if (nq[s] > 0) ok = warp_wait_far(&sm.q_empty[s], (nq[s] - 1) & 1, ctl);
          if (!ok) break;
          ++nq[s];
          const int tok = (int)uniform(it.a0 + it.r0 + (it.single ? 0 : s * TQ));
          if (el) {
            const uint32_t bar = smem_addr(&sm.q_full[s]);
            mbar_arrive_expect_tx(bar, (uint32_t)(TQ * G * 128 * C::kHalves));
#pragma unroll
            for (int h = 0; h < C::kHalves; ++h)
              tma_load_3d(qb + s * C::kTile + h * 16384, &tmQ, h * 64, hk * G, tok, bar);
          }
          __syncwarp();
        }
        const bool two = it.single;  // K runs two tiles ahead of V
        if (ok && two && t0 + 1 < t1) ok = load_kv(t0 + 1, false, pg[1]);
        for (int j = t0; ok && j < t1; ++j) {
          pg[3] = page_of(j + 3);
          ok = load_kv(j, true, pg[0]);
          const int jk = j + (two ? 2 : 1);
          if (ok && jk < t1) ok = load_kv(jk, false, two ? pg[2] : pg[1]);
#pragma unroll
          for (int x = 0; x < 3; ++x) pg[x] = pg[x + 1];
        }
        done_item(k);
      }
      // nothing may land in shared memory once the CTA is gone (a timeout)
      for (uint32_t k = n > S ? n - S : 0; k < n; ++k) drain(&sm.kv_full[k % S], (k / S) & 1, p.timeout_ns);
      for (int s = 0; s < 2; ++s)
        if (nq[s] > 0) drain(&sm.q_full[s], (nq[s] - 1) & 1, p.timeout_ns);
    } else if (warp == 8) {
      // ------------------------------------------------------------- MMAs
      // One elected lane waits and issues, with operands that are warp-uniform
      // values made by the whole warp: they then live in uniform registers.
      // Held in ordinary ones, as in a single-lane loop, each MMA cost a dozen
      // instructions that compete with the softmax warps for issue slots: 102
      // cycles an MMA of 128 x 128 x 16 instead of 64.
      const bool el = elect_one();
      const uint32_t tm = uniform(tmem), qb = uniform(q_smem), kb = uniform(kv_smem);
      uint32_t rn = 0;                                   // tiles of the ring used so far
      uint32_t q_ph = 0, p_ph = 0, o_ph = 0, clean = 0;  // phases, a bit for each stream, buffer or slot
      uint32_t started = 0;
      constexpr uint32_t kIdQK = idesc_bf16(128, kKeys, false), kIdPV = idesc_bf16(128, D, true);
      auto wait = [&](uint64_t *bar, uint32_t parity) { return lane_wait(bar, parity, ctl); };
      // (what follows runs in the elected lane alone)
      auto ring = [&](uint32_t k) { return wait(&sm.kv_full[k % S], (k / S) & 1); };
      auto ring_v = [&](uint32_t k, bool guard) {
        return ring(k) && (!guard || wait(&sm.kv_clean[k % S], (clean >> k % S) & 1));
      };
      // scores = Q . K^T; x: the stream, or 2 + the buffer of a single row tile
      auto qk = [&](int x4, uint64_t a, uint64_t b) {
        const uint32_t d = tm + (x4 & 1) * 128;
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < C::kHalves; ++h)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            mma_bf16_ss(d, a + h * 1024 + x * 2, b + h * 1024 + x * 2, kIdQK, (h | x) != 0);
        tc_commit(smem_addr(&sm.s_full[x4]));
      };
      // accumulator (+)= P . V, for the first half of the keys as soon as their
      // weights are there (8192 tokens 671 us; at a quarter of them 675, at
      // three quarters 693, when all are there 681)
      auto pv = [&](int x4, uint64_t b, uint32_t acc) {
        const uint32_t ph = (p_ph >> x4) & 1, o = tm + 256 + (x4 == 1 ? 128 : 0), w = tm + (x4 & 1) * 128;
        if (!wait(&sm.p_half[x4], ph)) return false;
        tc_fence_after();
#pragma unroll
        for (int x = 0; x < 4; ++x) mma_bf16_ts(o, w + 8 * x, b + x * 128, kIdPV, x > 0 ? 1u : acc);
        if (!wait(&sm.p_ready[x4], ph)) return false;
        tc_fence_after();
#pragma unroll
        for (int x = 4; x < 8; ++x) mma_bf16_ts(o, w + 8 * x, b + x * 128, kIdPV, 1u);
        tc_commit(smem_addr(&sm.pv_done[x4]));
        return true;
      };
      auto release = [&](uint32_t k) { tc_commit(smem_addr(&sm.kv_empty[k % S])); };
      // (the whole warp)
      auto kdesc = [&](uint32_t k) { return sdesc_kmajor_sw128(kb + uniform(k % S) * C::kTile); };
      auto vdesc = [&](uint32_t k) { return sdesc_mnmajor_sw128(kb + uniform(k % S) * C::kTile, 16384); };
      auto all_ok = [&](bool ok) { return __all_sync(0xFFFFFFFFu, ok) != 0; };
      // before an item's first product into a stream's accumulator the last item's has been read
      auto o_read = [&](int s) { return !(started >> s & 1) || wait(&sm.o_free[s], (o_ph >> s) & 1); };
      auto o_took = [&](int s) {
        o_ph ^= started & (1u << s);
        started |= 1u << s;
      };
      bool ok = true;
      for (int k = 0; ok && next_item(k); ++k) {
        const int t0 = (int)uniform(it.t0), t1 = (int)uniform(it.t1);
        const int end[2] = {(int)uniform(it.end[0]), (int)uniform(it.end[1])};
        const uint32_t q0 = qb + uniform(it.single ? (uint32_t)(k & 1) * C::kTile : 0u);
        const uint64_t q[2] = {sdesc_kmajor_sw128(q0), sdesc_kmajor_sw128(qb + C::kTile)};
        done_item(k);
        if (uniform(it.single)) {
          // K runs two tiles ahead of V
          const int nt = t1 - t0;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (!ok || s >= nt) continue;
            const uint64_t kd = kdesc(rn);
            if (el) {
              ok = ring(rn) && (s > 0 || wait(&sm.q_full[k & 1], (q_ph >> (k & 1)) & 1));
              if (ok) {
                qk(2 + s, q[0], kd);
                release(rn);
              }
            }
            ok = all_ok(ok);
            if (s == 0) q_ph ^= 1u << (k & 1);
            ++rn;
          }
          for (int i = 0; ok && i < nt; i += 2) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              if (!ok || i + s >= nt) continue;
              const bool more = i + s + 2 < nt, guard = guarded<MODE>(it, t0 + i + s);
              const uint64_t vd = vdesc(rn), kd = kdesc(rn + 1);
              const uint32_t acc = uniform(i + s > 0);
              if (el) {
                ok = ring_v(rn, guard) && (i + s > 0 || o_read(0)) && pv(2 + s, vd, acc);
                if (ok) release(rn);
                if (ok && more) {
                  ok = ring(rn + 1);
                  if (ok) {
                    qk(2 + s, q[0], kd);
                    release(rn + 1);
                  }
                }
              }
              ok = all_ok(ok);
              p_ph ^= 4u << s;
              if (i + s == 0) o_took(0);
              if (guard) clean ^= 1u << rn % S;
              rn += more ? 2 : 1;
            }
          }
        } else {
          const uint64_t kd0 = kdesc(rn);
          if (el) {
            ok = ring(rn);
#pragma unroll
            for (int s = 0; s < 2; ++s)
              if (ok && end[s] > t0) {
                ok = wait(&sm.q_full[s], (q_ph >> s) & 1);
                if (ok) qk(s, q[s], kd0);
              }
            if (ok) release(rn);
          }
          ok = all_ok(ok);
#pragma unroll
          for (int s = 0; s < 2; ++s)
            if (end[s] > t0) q_ph ^= 1u << s;
          ++rn;
          for (int j = t0; ok && j < t1; ++j) {
            const bool more = j + 1 < t1, guard = guarded<MODE>(it, j);
            const uint64_t vd = vdesc(rn), kd = kdesc(rn + 1);
            const uint32_t acc = uniform(j > t0);
            if (el) {
              ok = ring_v(rn, guard);
#pragma unroll
              for (int s = 0; s < 2; ++s) {
                if (!ok || j >= end[s]) continue;
                ok = (j > t0 || o_read(s)) && pv(s, vd, acc);
                if (ok && j + 1 < end[s]) {
                  ok = ring(rn + 1);
                  if (ok) qk(s, q[s], kd);
                }
              }
              if (ok) release(rn);
              if (ok && more) release(rn + 1);
            }
            ok = all_ok(ok);
#pragma unroll
            for (int s = 0; s < 2; ++s)
              if (j < end[s]) {
                p_ph ^= 1u << s;
                if (j == t0) o_took(s);
              }
            if (guard) clean ^= 1u << rn % S;
            rn += more ? 2 : 1;
          }
        }
      }
      // every MMA has completed before the CTA leaves its shared memory and TMEM
      if (el) {
        tc_commit(smem_addr(&sm.mma_done));
        drain(&sm.mma_done, 0, p.timeout_ns);
      }
      __syncwarp();
    } else if (warp == 10) {
      // -------------------------------------------------------------- guard
      // A weight of zero times a NaN is a NaN: before a v tile that not every
      // row sees in full is multiplied, its rows that no row sees are zeroed,
      // and so are the NaN and infinities of a row that only some see, which is
      // noted: who sees it adds them at the end.
      // (item k + 2 is only handed out when the softmax is through with item k
      // and with what is noted of it)
      uint32_t n = 0, issued = 0;
      bool ok = true;
      for (int k = 0; ok && next_item(k); ++k) {
        if (lane < 12) (&sm.poison[k & 1][0][0])[lane] = 0;
        __syncwarp();
        const int nt = it.t1 - it.t0, lead = min(it.single ? 2 : 1, nt);
        const int g0 = first_guarded<MODE>(it);
        for (int j = g0; ok && j < it.t1; ++j) {
          if (!guarded<MODE>(it, j)) continue;
          const int i = j - it.t0;
          const uint32_t at = n + lead + i + min(i, nt - lead), slot = at % S;  // the v tile's place in the ring
          // (once the load is issued, the slot's earlier phases are over)
          ok = warp_wait_far(&sm.v_issued[slot], (issued >> slot) & 1, ctl) &&
               warp_wait_far(&sm.kv_full[slot], (at / S) & 1, ctl);
          if (!ok) break;
          issued ^= 1u << slot;
          const uint32_t tile = kv_smem + slot * C::kTile;
          const int valid = v_valid<MODE>(it, j), shared = v_shared<MODE>(it, j);
          for (int r = shared + lane; r < kKeys; r += 32) {
            const bool wipe = r >= valid;
            if (!wipe) {
              bool bad = false;
#pragma unroll
              for (int h = 0; h < C::kHalves; ++h)
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                  const uint4 w = ld_shared_v4(tile + h * 16384 + r * 128 + ((x + lane) & 7) * 16);
                  bad |= not_finite2(w.x) || not_finite2(w.y) || not_finite2(w.z) || not_finite2(w.w);
                }
              if (bad) {
                atomicOr(&sm.poison[k & 1][j - g0][r >> 5], 1u << (r & 31));
#pragma unroll 1
                for (int x = 0; x < 8 * C::kHalves; ++x) {
                  const uint32_t to = tile + (x >> 3) * 16384 + r * 128 + (x & 7) * 16;
                  const uint4 w = ld_shared_v4(to);
                  st_shared_v4(to, finite2(w.x), finite2(w.y), finite2(w.z), finite2(w.w));
                }
              }
            }
            if (wipe) {
#pragma unroll
              for (int h = 0; h < C::kHalves; ++h)
#pragma unroll
                for (int x = 0; x < 8; ++x) st_shared_v4(tile + h * 16384 + r * 128 + ((x + lane) & 7) * 16, 0, 0, 0, 0);
            }
          }
          // (a tile that all rows see as far as it goes: only its tail)
          for (int r = max(valid, 0) + lane; r < min(shared, kKeys); r += 32)
#pragma unroll
            for (int h = 0; h < C::kHalves; ++h)
#pragma unroll
              for (int x = 0; x < 8; ++x) st_shared_v4(tile + h * 16384 + r * 128 + ((x + lane) & 7) * 16, 0, 0, 0, 0);
          fence_proxy_async_smem();
          warp_arrive(&sm.kv_clean[slot], lane);
        }
        n += 2 * nt;
        if (ok) warp_arrive(&sm.guard_item[k & 1], lane);
        done_item(k);
      }
    } else if (warp == 11) {
      // -------------------------------------------------------------- items
      const bool few = seqs<MODE>(p) <= 32;
      Small<MODE> small;
      PlanUnits<MODE> planned_units;
      if (few) small.read(p, 2 * TQ, lane, blockIdx.x == 0);
      else if constexpr (planned(MODE)) planned_units.read(p, lane);
      else fill_prefix<MODE>(p, sm.pre, 2 * TQ, lane, blockIdx.x == 0);
      const int span = !TREE && few ? small.choose_span(p, TQ, lane) : 2 * TQ;
      if (few) small.number(p, lane);
      int ctas = gridDim.x;
      if constexpr (MODE == kShared) ctas = __ldg(p.plan.ctas);
      Walk<MODE> walk(few ? small.total : planned(MODE) ? planned_units.total : sm.pre.units[kBlocks], span, ctas);
      Found found;
      bool going_on = false;
      if constexpr (TREE) {
        if (few) walk.choose_chunk(small);
        else if constexpr (planned(MODE)) walk.choose_chunk(planned_units);
      }
      for (int k = 0;; ++k) {
        Item<MODE> w;
        int last = 0;  // the last CTA that has a part of the row group
        if constexpr (TREE) {
          if (walk.chunk > 0 && k == 0) {
            last = walk.one_chunk(p, small, TQ, w);
          } else {
            walk.next(p, TQ, w, [&](int &u, int &b) {
              if (few) return small.find(u, b);
              if constexpr (planned(MODE)) return planned_units.find(p, 2 * TQ, u, b);
              else return find_seq<MODE>(p, sm.pre, 2 * TQ, u, b, found);
            });
            if (w.t1 > w.t0 && w.part == 1)
              last = planned(MODE) && walk.last >= 0
                         ? walk.last
                         : share_owner(share_begin(blockIdx.x + 1, walk.q, walk.r) + w.nct + (flags_of(w) & kHasNodes) - 1 - w.t1,
                                       walk.q, walk.r);
          }
        } else {
          walk.next(p, TQ, w, [&](int &u, int &b) {
            return few ? small.find(u, b) : find_seq<MODE>(p, sm.pre, 2 * TQ, u, b, found);
          });
          if (w.t1 < 0) w.t1 = 0;  // (no item in the last round, and none after it)
        }
        if (k >= 2 && !warp_wait_far(&sm.item_free[k & 1], ((k >> 1) - 1) & 1, ctl)) break;
        if (lane == 0) sm.items[k & 1] = w;
        warp_arrive(&sm.item_full[k & 1], lane);
        if (w.t1 == w.t0) break;
        if (TREE && w.part == 1) {
          going_on = true;
          if (lane == 0) {
            JoinItem j;
            j.rows0 = w.cnt[0] * G;
            j.rows = j.rows0 + w.cnt[1] * G;
            j.tok = w.a0 + w.r0;
            j.cnt0 = w.cnt[0];
            j.head = w.hk * G;
            j.last = last;
            j.word = MODE == kShared ? flags_of(w) & kHasNodes : w.n;
            j.ctx = w.ctx;
            reinterpret_cast<JoinItem *>(p.ws)[blockIdx.x] = j;
          }
        }
      }
      if (TREE && !going_on && lane == 0) reinterpret_cast<JoinItem *>(p.ws)[blockIdx.x].rows = 0;
    }
  } else {
    regs_more<kRegsSoftmax>();
    // ------------------------------------------------------------ softmax
    const int st = warp >> 2;                       // stream
    const int row = (warp & 3) * 32 + lane;         // row of the tile
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t o_t = tmem + lanes + 256 + st * 128;
    const float c = p.scale * kLog2e;
    const int rt = row / G, rg = row - rt * G;      // token of the tile, head of the group
    uint32_t ph = 0;  // phases of the streams and buffers, a bit each
    bool ok = true;
    if (p.debug_stall) ok = warp_wait(&sm.stall, 0, ctl);
    for (int k = 0; ok && next_item(k); ++k) {
      const int tok = it.r0 + st * TQ + rt;  // in the sequence
      const bool valid_row = rt < (st ? it.cnt[1] : it.cnt[0]);
      const bool warp_rows = __any_sync(0xFFFFFFFFu, valid_row);
      const int last = st ? it.end[1] : it.end[0];
      // tiles from here on are not seen in full
      const bool lists = MODE == kSparse && (flags_of(it) & kLists);  // the rows see different pages
      const int ragged = lists ? it.t0 : TREE ? it.ctx / kKeys : (it.r0 + st * TQ + 1) / kKeys;
      bool saw = false;  // planned: the row sees a key of this item
      // lists: the node's bit in the words of a tile's pages, each 16 keys of the tile a bit
      unsigned long long who = 0;
      auto names_of = [&](int j) {  // lane u: the nodes that name the page of keys 16 u ... of tile j
        const int key = (j << 7) + lane * 16;
        if (lists && lane < 8 && j < it.nct && key < it.ctx)
          who = __ldg(p.plan.names + list_of(it) + (key >> (31 - __clz(p.cache.page_size))));
      };
      unsigned long long word = 0;
      bool any = true;
      if (TREE) {
        if (valid_row) word = p.mask[it.a0 + tok] & (it.n >= 64 ? ~0ull : (1ull << it.n) - 1ull);
        any = it.ctx > 0 || word != 0ull;
      }
      float m = -INFINITY, l = 0.0f;
      uint32_t x4 = it.single ? 3 : st;  // stream, or 2 + buffer
      if (lists) names_of(it.t0);
      for (int j = it.t0; j < last; ++j) {
        if (it.single) x4 ^= 1;
        uint32_t units = 0xFFu;
        if (MODE == kSparse) {
          if (lists && j < it.nct) {
            units = 0;
#pragma unroll
            for (int u = 0; u < 8; ++u) units |= (uint32_t)(__shfl_sync(0xFFFFFFFFu, who, u) >> (tok & 63) & 1ull) << u;
            if (it.ctx - j * kKeys < kKeys) units &= (1u << ((it.ctx - j * kKeys + 15) >> 4)) - 1u;
            names_of(j + 1);
          }
          saw |= j < it.nct ? units != 0 : word != 0ull;
        } else if (MODE == kShared) {
          saw |= j < it.nct || word != 0ull;
        }
        ok = warp_wait(&sm.s_full[x4], (ph >> x4) & 1, ctl);
        if (!ok) break;
        const uint32_t s_t = tmem + lanes + (x4 & 1) * 128;
        if (warp_rows) {
          tc_fence_after();
          uint32_t s[4][32];
          tmem_ld32(s_t, s[0]);
          tmem_ld32(s_t + 32, s[1]);
          tmem_ld_wait();
          tmem_landed(s[0]);
          tmem_landed(s[1]);
          tmem_ld32(s_t + 64, s[2]);
          tmem_ld32(s_t + 96, s[3]);
          if (j >= ragged) {
            // what the row does not see is -inf
            uint32_t see[4];
            const int n = TREE ? (j < it.nct ? it.ctx - j * kKeys : 0) : tok + 1 - j * kKeys;
#pragma unroll
            for (int x = 0; x < 4; ++x)
              see[x] = n >= 32 * x + 32 ? 0xFFFFFFFFu : n > 32 * x ? (1u << (n - 32 * x)) - 1u : 0u;
            if (MODE == kSparse) {
#pragma unroll
              for (int x = 0; x < 4; ++x)
                see[x] &= (units >> 2 * x & 1u ? 0xFFFFu : 0u) | (units >> 2 * x & 2u ? 0xFFFF0000u : 0u);
            }
            if (TREE && j >= it.nct) see[0] = (uint32_t)word, see[1] = (uint32_t)(word >> 32);
            tmem_ld_wait();
            tmem_landed(s[2]);
            tmem_landed(s[3]);
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(see[x] >> e & 1u)) s[x][e] = 0xFF800000u;
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            if (x == 2) {
              tmem_ld_wait();
              tmem_landed(s[2]);
              tmem_landed(s[3]);
            }
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              mx[e / 2 & 3] = max3(mx[e / 2 & 3], __uint_as_float(s[x][e]), __uint_as_float(s[x][e + 1]));
          }
          const float top = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
          if (j == it.t0) {
            m = top;
          } else if (__any_sync(0xFFFFFFFFu, valid_row && (top - m) * c > kFallBehind)) {
            // the reference has fallen behind: move it, and with it the sum and the accumulator
            const float mn = fmaxf(m, top);
            const float f = mn == -INFINITY ? 1.0f : ex2((m - mn) * c);
            l *= f;
            m = mn;
            const uint32_t prev = it.single ? x4 ^ 1 : x4;  // the last product: one phase back
            ok = warp_wait(&sm.pv_done[prev], (ph >> prev & 1) ^ 1, ctl);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int x = 0; x < D / 16; ++x) {
              uint32_t o[16];
              tmem_ld16(o_t + x * 16, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st16(o_t + x * 16, o);
            }
          }
          const float ref = m == -INFINITY ? 0.0f : -m * c;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float a, b;
              fma2(a, b, __uint_as_float(s[x][e]), __uint_as_float(s[x][e + 1]), c, ref);
              a = ex2(a);
              b = ex2(b);
              w[e / 2] = pack_bf16x2(a, b);
              s[x][e] = __float_as_uint(a);
              s[x][e + 1] = __float_as_uint(b);
            }
            tmem_st16(s_t + x * 16, w);
            if (x == 1) {
              tmem_st_wait();
              tc_fence_before();
              warp_arrive(&sm.p_half[x4], lane);
            }
          }
          tmem_st_wait();
          tc_fence_before();
          warp_arrive(&sm.p_ready[x4], lane);
          // The sum, while the weights are multiplied: of the weights in fp32, but
          // of the tile's largest as the product has it, rounded.  Where one key
          // has most of a row, its rounding then cancels: with a reference 2^4.3
          // behind, such a row's error falls from 0.0030 of its length to 0.0018.
          // 8192 tokens take 672 us, 669 without this; the sum of all the rounded
          // weights gains nothing more and takes 702.
          const float most = ex2(fmaf(top, c, ref));
          float sum[4] = {l + (__uint_as_float(pack_bf16x2(0.0f, most)) - most), 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              add2(sum[0], sum[1], __uint_as_float(s[x][e]), __uint_as_float(s[x][e + 1]));
              add2(sum[2], sum[3], __uint_as_float(s[x][e + 2]), __uint_as_float(s[x][e + 3]));
            }
          l = (sum[0] + sum[1]) + (sum[2] + sum[3]);
        } else {
          warp_arrive(&sm.p_half[x4], lane);
          warp_arrive(&sm.p_ready[x4], lane);
        }
        ph ^= 1u << x4;
      }
      if (!ok) break;
      const bool active = it.t0 < last;
      const int qt = it.single ? k & 1 : st;  // the q tile, multiplied for the last time
      if (active) warp_arrive(&sm.q_empty[qt], lane);
      ok = warp_wait(&sm.guard_item[k & 1], (k >> 1) & 1, ctl);
      if (!ok) break;
      if (active) {
        ok = warp_wait(&sm.pv_done[x4], (ph >> x4 & 1) ^ 1, ctl);
        if (!ok) break;
        tc_fence_after();
        const int g0 = first_guarded<MODE>(it);
        uint32_t anyp = 0;
#pragma unroll
        for (int x = 0; x < 12; ++x) anyp |= (&sm.poison[k & 1][0][0])[x];
        // a part's row of sums, its reference and the sum of its weights
        float *part = nullptr, *part_m = nullptr;
        if (MODE == kShared && it.part == 2) {
          const long long r = ((long long)(flags_of(it) & kHasNodes) * p.T + it.a0 + tok) * p.Hq + it.hk * G + rg;
          part = p.plan.rows + r * D;
          part_m = p.plan.stats + r * 2;
        } else if (TREE && it.part >= 0) {
          part = p.ws + p.slots + ((long long)blockIdx.x * 2 + it.part) * C::kSlotFloats + st * (kRowsT * (D + 2));
          part_m = part + D * kRowsT + row;
          part += row * D;
        }
        // A thread holds a row, and rows are far apart in memory: the result
        // goes through shared memory (half the channels at a time, each warp
        // its own rows, the 16-byte units of row r at unit ^ r), so that a store
        // writes whole halves of rows.  Straight from the rows' threads, 32
        // lines a store, this took 5000 cycles.
        constexpr int kUnits = D / 16;           // 16-byte units of a staged half row
        constexpr int kRowsStore = 32 / kUnits;  // rows a warp stores at once
        const uint32_t stage = kv_smem + S * C::kTile + st * (C::kTile / 2) + (warp & 3) * 32 * kUnits * 16;
        const uint32_t mine = stage + lane * kUnits * 16;
        const int unit = lane % kUnits, sub = lane / kUnits;
        const int rows = __popc(__ballot_sync(0xFFFFFFFFu, valid_row));  // (the first ones)
        if (planned(MODE)) {
          any = saw;
          // (a part's sum of 0 says that the row sees nothing of it)
          if (part) l = !saw ? 0.0f : m == -INFINITY ? 1.0f : l;
        }
        const float inv = any ? 1.0f / l : 0.0f;
        uint16_t *out = p.out.ptr + (long long)(it.a0 + tok) * p.out.tok + (it.hk * G + rg) * p.out.head;
        // A weight of zero times a NaN or an infinity of a page that other rows see: such
        // rows are summed again, from what they see, and written before the others (a row's q
        // may be where its result goes).
        unsigned redone = 0;
        if (lists && warp_rows) {
          bool fine = true;
#pragma unroll 1
          for (int x = 0; x < D / 32; ++x) {
            uint32_t o[32];
            tmem_ld32(o_t + x * 32, o);
            tmem_ld_wait();
            tmem_landed(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) fine &= !too_large(o[e]);
          }
          redone = __ballot_sync(0xFFFFFFFFu, valid_row && !fine);
          float *const sums = reinterpret_cast<float *>(smem_raw + (stage - base));
#pragma unroll 1
          for (unsigned rest = redone; rest;) {
            int r[4], mine = -1;  // lanes of four rows, of this lane's
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              r[i] = __ffs(rest) - 1;
              rest &= rest - 1;
              if (lane >> 3 == i) mine = r[i];
            }
            const float2 stat = sum_again<D, MODE, 4, 4>(p, sm.items[k & 1], it.r0 + st * TQ,
                                                         mine < 0 ? -1 : (warp & 3) * 32 + mine, sums, D);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (r[i] < 0) break;
              auto of = [&](auto x) { return __shfl_sync(0xFFFFFFFFu, x, r[i]); };
              float y[D / 32];
#pragma unroll
              for (int e = 0; e < D / 32; ++e) y[e] = sums[i * D + lane * (D / 32) + e];
              const unsigned long long at = of(reinterpret_cast<unsigned long long>(part ? (void *)part : (void *)out));
              const float li = __shfl_sync(0xFFFFFFFFu, stat.y, 8 * i), mi = __shfl_sync(0xFFFFFFFFu, stat.x, 8 * i);
              if (lane == r[i]) m = mi, l = part && any && m == -INFINITY ? 1.0f : li;
              if (part) store_part(reinterpret_cast<float *>(at), y, lane);
              else store_row(reinterpret_cast<uint16_t *>(at), y, 1.0f / li, of((int)any), lane);
            }
            __syncwarp();
          }
        }
        const bool again = redone >> lane & 1u;
        const unsigned long long row0 = valid_row && !again ? reinterpret_cast<unsigned long long>(out) : 0ull;
        unsigned long long to[32 / kRowsStore];  // the rows that this lane stores a unit of
#pragma unroll
        for (int i = 0; i < 32 / kRowsStore; ++i) to[i] = __shfl_sync(0xFFFFFFFFu, row0, i * kRowsStore + sub);
        if (!warp_rows) warp_arrive(&sm.o_free[st], lane);
#pragma unroll 1
        for (int h = warp_rows ? 0 : 2; h < 2; ++h) {
          uint32_t o[D / 64][32];
#pragma unroll
          for (int x = 0; x < D / 64; ++x) tmem_ld32(o_t + h * (D / 2) + x * 32, o[x]);
          tmem_ld_wait();
#pragma unroll
          for (int x = 0; x < D / 64; ++x) tmem_landed(o[x]);
          if (h == 1) {
            tc_fence_before();
            warp_arrive(&sm.o_free[st], lane);  // (the next item's products may begin)
          }
          if (anyp) {
            // what the guard has taken out of v rows, added by those who see them
#pragma unroll 1
            for (int x = 0; x < 12; ++x) {
              uint32_t bits = (&sm.poison[k & 1][0][0])[x];
              const int j = g0 + x / 4;
#pragma unroll 1
              while (bits) {
                const int r = (x & 3) * 32 + __ffs(bits) - 1;
                bits &= bits - 1;
                const int key = TREE ? r : j * kKeys + r;
                if (!valid_row || again || !(TREE ? (bool)(word >> key & 1ull) : key <= tok)) continue;
                const uint16_t *v = p.v.ptr + (long long)(it.a0 + key) * p.v.tok + it.hk * p.v.head + h * (D / 2);
#pragma unroll
                for (int c0 = 0; c0 < D / 64; ++c0)
#pragma unroll
                  for (int e = 0; e < 32; ++e) {
                    const uint32_t y = v[c0 * 32 + e];
                    if ((y & 0x7F80u) == 0x7F80u)
                      o[c0][e] = __float_as_uint(__uint_as_float(o[c0][e]) + __uint_as_float(y << 16));
                  }
              }
            }
          }
          if (part) {
            // (a part's rows are fp32, a whole line for every 32 values of a
            // thread, and often few: straight from the threads)
            if (valid_row && !again) {
#pragma unroll
              for (int x = 0; x < D / 64; ++x)
#pragma unroll
                for (int e = 0; e < 32; e += 8) st_global_v8(part + h * (D / 2) + x * 32 + e, o[x] + e);
            }
            continue;
          }
#pragma unroll
          for (int u = 0; u < kUnits; ++u) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a = __uint_as_float(o[u / 4][u % 4 * 8 + 2 * i]) * inv;
              const float b = __uint_as_float(o[u / 4][u % 4 * 8 + 2 * i + 1]) * inv;
              w[i] = any ? pack_bf16x2(a, b) : 0u;
            }
            st_shared_v4(mine + ((u ^ lane) & (kUnits - 1)) * 16, w[0], w[1], w[2], w[3]);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 32 / kRowsStore; ++i) {
            if (i * kRowsStore >= rows) break;
            const int r = i * kRowsStore + sub;
            const uint4 v = ld_shared_v4(stage + r * kUnits * 16 + ((unit ^ r) & (kUnits - 1)) * 16);
            if (to[i]) *reinterpret_cast<uint4 *>(to[i] + (h * kUnits + unit) * 16) = v;
          }
          __syncwarp();
        }
        if (part && valid_row) {
          part_m[0] = m;
          part_m[MODE == kShared && it.part == 2 ? 1 : kRowsT] = l;
        }
      }
      done_item(k);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of the items that several CTAs shared, in the order of the
// keys: a warp takes a row of an item that began in one CTA and went on.
// Latency bounds it.  Every block reads the whole list of items and deals the
// rows of all of them over the grid's warps (a block an item and 8 rows, most
// of them empty, took 6.5 us for a verify step); the references and sums of 32
// parts come in one load a lane, the parts themselves 8 in flight.
constexpr int kJoinWarps = 8, kJoinBlocksSm = 2, kJoinRowsBlocksSm = 3;
// Up to eight parts of a row at once (zeros for those past n), V values a
// lane.  One statement: left to itself, the compiler put each part's sums
// before the next part's load, eight round trips to L2 instead of one.
__device__ __forceinline__ void load_parts(const float *const (&p)[8], int n, uint32_t (&y)[8][4]) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.gt.s32 q, %40, 0; mov.b32 %0, 0; mov.b32 %1, 0; mov.b32 %2, 0; mov.b32 %3, 0;\n\t@q ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%32];\n\t"
      "setp.gt.s32 q, %40, 1; mov.b32 %4, 0; mov.b32 %5, 0; mov.b32 %6, 0; mov.b32 %7, 0;\n\t@q ld.global.cg.v4.u32 {%4, %5, %6, %7}, [%33];\n\t"
      "setp.gt.s32 q, %40, 2; mov.b32 %8, 0; mov.b32 %9, 0; mov.b32 %10, 0; mov.b32 %11, 0;\n\t@q ld.global.cg.v4.u32 {%8, %9, %10, %11}, [%34];\n\t"
      "setp.gt.s32 q, %40, 3; mov.b32 %12, 0; mov.b32 %13, 0; mov.b32 %14, 0; mov.b32 %15, 0;\n\t@q ld.global.cg.v4.u32 {%12, %13, %14, %15}, [%35];\n\t"
      "setp.gt.s32 q, %40, 4; mov.b32 %16, 0; mov.b32 %17, 0; mov.b32 %18, 0; mov.b32 %19, 0;\n\t@q ld.global.cg.v4.u32 {%16, %17, %18, %19}, [%36];\n\t"
      "setp.gt.s32 q, %40, 5; mov.b32 %20, 0; mov.b32 %21, 0; mov.b32 %22, 0; mov.b32 %23, 0;\n\t@q ld.global.cg.v4.u32 {%20, %21, %22, %23}, [%37];\n\t"
      "setp.gt.s32 q, %40, 6; mov.b32 %24, 0; mov.b32 %25, 0; mov.b32 %26, 0; mov.b32 %27, 0;\n\t@q ld.global.cg.v4.u32 {%24, %25, %26, %27}, [%38];\n\t"
      "setp.gt.s32 q, %40, 7; mov.b32 %28, 0; mov.b32 %29, 0; mov.b32 %30, 0; mov.b32 %31, 0;\n\t@q ld.global.cg.v4.u32 {%28, %29, %30, %31}, [%39];\n\t"
      "}"
      : "=&r"(y[0][0]), "=&r"(y[0][1]), "=&r"(y[0][2]), "=&r"(y[0][3]), "=&r"(y[1][0]),
        "=&r"(y[1][1]), "=&r"(y[1][2]), "=&r"(y[1][3]), "=&r"(y[2][0]), "=&r"(y[2][1]),
        "=&r"(y[2][2]), "=&r"(y[2][3]), "=&r"(y[3][0]), "=&r"(y[3][1]), "=&r"(y[3][2]),
        "=&r"(y[3][3]), "=&r"(y[4][0]), "=&r"(y[4][1]), "=&r"(y[4][2]), "=&r"(y[4][3]),
        "=&r"(y[5][0]), "=&r"(y[5][1]), "=&r"(y[5][2]), "=&r"(y[5][3]), "=&r"(y[6][0]),
        "=&r"(y[6][1]), "=&r"(y[6][2]), "=&r"(y[6][3]), "=&r"(y[7][0]), "=&r"(y[7][1]),
        "=&r"(y[7][2]), "=&r"(y[7][3])
      : "l"(p[0]), "l"(p[1]), "l"(p[2]), "l"(p[3]), "l"(p[4]), "l"(p[5]), "l"(p[6]), "l"(p[7]), "r"(n));
}
__device__ __forceinline__ void load_parts(const float *const (&p)[8], int n, uint32_t (&y)[8][2]) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.gt.s32 q, %24, 0; mov.b32 %0, 0; mov.b32 %1, 0;\n\t@q ld.global.cg.v2.u32 {%0, %1}, [%16];\n\t"
      "setp.gt.s32 q, %24, 1; mov.b32 %2, 0; mov.b32 %3, 0;\n\t@q ld.global.cg.v2.u32 {%2, %3}, [%17];\n\t"
      "setp.gt.s32 q, %24, 2; mov.b32 %4, 0; mov.b32 %5, 0;\n\t@q ld.global.cg.v2.u32 {%4, %5}, [%18];\n\t"
      "setp.gt.s32 q, %24, 3; mov.b32 %6, 0; mov.b32 %7, 0;\n\t@q ld.global.cg.v2.u32 {%6, %7}, [%19];\n\t"
      "setp.gt.s32 q, %24, 4; mov.b32 %8, 0; mov.b32 %9, 0;\n\t@q ld.global.cg.v2.u32 {%8, %9}, [%20];\n\t"
      "setp.gt.s32 q, %24, 5; mov.b32 %10, 0; mov.b32 %11, 0;\n\t@q ld.global.cg.v2.u32 {%10, %11}, [%21];\n\t"
      "setp.gt.s32 q, %24, 6; mov.b32 %12, 0; mov.b32 %13, 0;\n\t@q ld.global.cg.v2.u32 {%12, %13}, [%22];\n\t"
      "setp.gt.s32 q, %24, 7; mov.b32 %14, 0; mov.b32 %15, 0;\n\t@q ld.global.cg.v2.u32 {%14, %15}, [%23];\n\t"
      "}"
      : "=&r"(y[0][0]), "=&r"(y[0][1]), "=&r"(y[1][0]), "=&r"(y[1][1]), "=&r"(y[2][0]),
        "=&r"(y[2][1]), "=&r"(y[3][0]), "=&r"(y[3][1]), "=&r"(y[4][0]), "=&r"(y[4][1]),
        "=&r"(y[5][0]), "=&r"(y[5][1]), "=&r"(y[6][0]), "=&r"(y[6][1]), "=&r"(y[7][0]),
        "=&r"(y[7][1])
      : "l"(p[0]), "l"(p[1]), "l"(p[2]), "l"(p[3]), "l"(p[4]), "l"(p[5]), "l"(p[6]), "l"(p[7]), "r"(n));
}

// A row joined by a warp: at(k) is part k's row of sums, stat(k, m, l) its
// reference and sum of weights.  A lane gets columns lane * V ... of the sums.
template <int V>
struct Joined {
  float l = 0.0f, o[V] = {};
  bool saw = false;  // some part's sum of weights is not 0
};
template <int V, class At, class Stat>
__device__ __forceinline__ Joined<V> join_parts(int parts, int lane, float c, At at_of, Stat stat) {
  constexpr unsigned kFull = 0xFFFFFFFFu;
  Joined<V> r;
  float m = -INFINITY;
  for (int k0 = 0; k0 < parts; k0 += 32) {
    const int n = min(32, parts - k0);
    float mk = -INFINITY, lk = 0.0f, f = 0.0f;
    if (lane < n) stat(k0 + lane, mk, lk);
    for (int k = 0; k < n; k += 8) {
      const float *at[8];
      uint32_t y[8][V];
#pragma unroll
      for (int i = 0; i < 8; ++i) at[i] = at_of(k0 + k + i) + lane * V;
      load_parts(at, n - k, y);
      if (k == 0) {  // (with the first parts under way)
        r.saw |= __any_sync(kFull, lk != 0.0f);
        float top = mk;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, x));
        const float mn = fmaxf(m, top);
        const float old = m == -INFINITY ? 0.0f : ex2((m - mn) * c);  // (more than 32 parts)
        f = mk == -INFINITY ? 0.0f : ex2((mk - mn) * c);
        m = mn;
        r.l *= old;
#pragma unroll
        for (int e = 0; e < V; ++e) r.o[e] *= old;
        lk *= f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float fk = __shfl_sync(kFull, f, (k + i) & 31), la = __shfl_sync(kFull, lk, (k + i) & 31);
        r.l += k + i < n ? la : 0.0f;  // (lanes past n hold a factor of 0)
#pragma unroll
        for (int e = 0; e < V; ++e) r.o[e] = fmaf(fk, __uint_as_float(y[i][e]), r.o[e]);
      }
    }
  }
  return r;
}

template <int V>
__device__ __forceinline__ void store_joined(const AttnParams &p, const Joined<V> &r, bool any, int node, int head,
                                             int lane) {
  store_row(p.out.ptr + (long long)node * p.out.tok + head * p.out.head, r.o, 1.0f / r.l, any, lane);
}

template <int D, int MODE>
__global__ void __launch_bounds__(32 * kJoinWarps, kJoinBlocksSm) attn_join_kernel(const AttnParams p, int ctas) {
  using C = Cfg<D, MODE>;
  constexpr int V = D / 32;  // columns a lane
  constexpr unsigned kFull = 0xFFFFFFFFu;
  static_assert(32 * kJoinWarps == kMaxCtas, "a thread reads an item");
  __shared__ JoinItem s_item[kMaxCtas];
  __shared__ int s_end[kMaxCtas], s_warp[kJoinWarps];  // rows of the items up to and with one
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv;
  const float c = p.scale * kLog2e;
  pdl_wait();
  JoinItem mine = {};
  if ((int)threadIdx.x < ctas) mine = reinterpret_cast<const JoinItem *>(p.ws)[threadIdx.x];
  int sum = mine.rows;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kFull, sum, o);
    if (lane >= o) sum += x;
  }
  if (lane == 31) s_warp[warp] = sum;
  s_item[threadIdx.x] = mine;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) sum += w < warp ? s_warp[w] : 0;
  s_end[threadIdx.x] = sum;
  __syncthreads();
  const int total = s_end[kMaxCtas - 1];
  for (int x = blockIdx.x + gridDim.x * warp; x < total; x += gridDim.x * kJoinWarps) {
    int c0 = 0;  // the first item whose rows end after x
#pragma unroll
    for (int o = kMaxCtas / 2; o > 0; o >>= 1)
      if (s_end[c0 + o - 1] <= x) c0 += o;
    const JoinItem it = s_item[c0];
    const int r = x - (s_end[c0] - it.rows);
    const int tile = r >= it.rows0, row = r - tile * it.rows0;
    const int rt = row / G, node = it.tok + tile * it.cnt0 + rt, head = it.head + row - rt * G;
    // CTA c0's part is in its second slot, the others' in their first
    const float *base = p.ws + p.slots + (long long)c0 * 2 * C::kSlotFloats + tile * (kRowsT * (D + 2));
    auto slot = [&](int k) { return base + (long long)(k == 0 ? 1 : 2 * k) * C::kSlotFloats; };
    bool any = true;
    if (!planned(MODE)) {
      const unsigned long long word = p.mask[node] & (it.word >= 64 ? ~0ull : (1ull << it.word) - 1ull);
      any = it.ctx > 0 || word != 0ull;
    }
    const Joined<V> j = join_parts<V>(
        it.last - c0 + 1, lane, c, [&](int k) { return slot(k) + row * D; },
        [&](int k, float &m, float &l) {
          const float *q = slot(k) + D * kRowsT + row;
          m = __ldcg(q);
          l = __ldcg(q + kRowsT);
        });
    store_joined<V>(p, j, planned(MODE) ? j.saw : any, node, head, lane);
  }
}

// The same for groups that share a prefix: a warp takes a row of the call, whose
// parts are those of its group's prefix, in the order of the keys, and those of
// its sequence's own keys.  Either is one part in the row's own place, or the
// slots of the CTAs that shared it.  Prefixes and own keys were two launches, each
// with its list of items that went on and its slots, or one with a list of both; of a
// kind the list is in the order of (first node, kv head), so the row's item is found by
// bisection.
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps, kJoinRowsBlocksSm) attn_join_rows_kernel(const AttnParams p, int ctas) {
  using C = Cfg<D, kShared>;
  constexpr int V = D / 32;
  constexpr unsigned kFull = 0xFFFFFFFFu;
  __shared__ JoinItem s_item[2][kMaxCtas];
  __shared__ unsigned long long s_key[2][kMaxCtas];
  __shared__ int s_cta[2][kMaxCtas], s_warp[2][kJoinWarps];
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv;
  const float c = p.scale * kLog2e;
  s_key[0][threadIdx.x] = s_key[1][threadIdx.x] = ~0ull;
  pdl_wait();
  JoinItem mine[2] = {};
  unsigned has[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if ((int)threadIdx.x < ctas && p.plan.part_ws[i])
      mine[i] = reinterpret_cast<const JoinItem *>(p.plan.part_ws[i])[threadIdx.x];
    if (mine[i].word != i) mine[i].rows = 0;  // (one list of both)
    has[i] = __ballot_sync(kFull, mine[i].rows > 0);
    if (lane == 0) s_warp[i][warp] = __popc(has[i]);
  }
  __syncthreads();
  auto key_of = [&](int node, int hk) { return ((unsigned long long)(uint32_t)node << 24) | (unsigned long long)hk; };
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (mine[i].rows > 0) {
      int at = __popc(has[i] & ((1u << lane) - 1u));
      for (int w = 0; w < warp; ++w) at += s_warp[i][w];
      s_item[i][at] = mine[i];
      s_cta[i][at] = threadIdx.x;
      s_key[i][at] = key_of(mine[i].tok, mine[i].head / G);
    }
  __syncthreads();
  auto last_at = [&](int list, unsigned long long key) {  // the last item whose key is not above this one, or -1
    int i = -1;
#pragma unroll
    for (int o = kMaxCtas / 2; o > 0; o >>= 1)
      if (s_key[list][i + o] <= key) i += o;
    return i;
  };
  const long long total = (long long)p.T * p.Hq;
  for (long long x = blockIdx.x + (long long)gridDim.x * warp; x < total; x += (long long)gridDim.x * kJoinWarps) {
    const int node = (int)(x / p.Hq), head = (int)(x - (long long)node * p.Hq), hk = head / G;
    const int info = __ldg(p.plan.info + node);  // -1: no sequence's, 0: nothing shared, 1: with a prefix
    if (info < 0) continue;
    const float *base[2] = {nullptr, nullptr};  // first part's row of sums, the prefix's and its own
    int parts[2] = {info, info}, row[2] = {0, 0};
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      if (kind >= 1 - info) {
        // the first node of the last row group that begins at or before this one, then its item of this kv head
        int i = last_at(kind, key_of(node, (1 << 24) - 1));
        if (i >= 0) i = last_at(kind, key_of(s_item[kind][i].tok, hk));
        if (i >= 0) {
          const JoinItem it = s_item[kind][i];
          const int d = node - it.tok, tile = d >= it.cnt0;
          if (it.head == hk * G && d >= 0 && d * G < it.rows) {
            row[kind] = (d - tile * it.cnt0) * G + head - it.head;
            parts[kind] = it.last - s_cta[kind][i] + 1;
            base[kind] = p.plan.part_ws[kind] + p.slots + ((long long)s_cta[kind][i] * 2 + 1) * C::kSlotFloats +
                         tile * (kRowsT * (D + 2));
          }
        }
      }
    }
    if (!info && !base[1]) continue;  // (already written)
    if (!info) parts[0] = 0;
    // slot k of a chain: the first CTA's second, then the others' first
    auto slot = [&](int kind, int k) { return base[kind] + (long long)(k == 0 ? 0 : 2 * k - 1) * C::kSlotFloats; };
    const Joined<V> j = join_parts<V>(
        parts[0] + parts[1], lane, c,
        [&](int k) {
          const int kind = k >= parts[0];
          k -= kind * parts[0];
          return base[kind] ? slot(kind, k) + row[kind] * D : p.plan.rows + ((long long)kind * total + x) * D;
        },
        [&](int k, float &m, float &l) {
          const int kind = k >= parts[0];
          k -= kind * parts[0];
          const float *q = base[kind] ? slot(kind, k) + D * kRowsT + row[kind] : p.plan.stats + ((long long)kind * total + x) * 2;
          m = __ldcg(q);
          l = __ldcg(q + (base[kind] ? kRowsT : 1));
        });
    store_joined<V>(p, j, j.saw, node, head, lane);
  }
}

// ------------------------------------------------------------------- host
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// bf16, 128-byte swizzle; dims[0] = D, strides (bytes) of the others; a
// dimension of one entry gets a stride the encoder accepts whatever the
// caller's is.
bool make_map(CUtensorMap *m, const void *ptr, int rank, const cuuint64_t *dims, const long long *elem_strides,
              const cuuint32_t *box) {
  auto enc = encoder();
  if (!enc) return false;
  cuuint64_t strides[4];
  for (int i = 0; i < rank - 1; ++i)
    strides[i] = dims[i + 1] == 1 ? dims[0] * 2 : (cuuint64_t)elem_strides[i] * 2;
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void *>(ptr), dims, strides, box, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool heads_map(CUtensorMap *m, const Heads &h, int heads, int T, int D, int box_heads, int box_toks) {
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)T};
  const long long st[2] = {h.head, h.tok};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_toks};
  return make_map(m, h.ptr, 3, dims, st, box);
}

bool cache_maps(CUtensorMap *k, CUtensorMap *v, const AttnParams &p) {
  const cuuint64_t dims[4] = {(cuuint64_t)p.D, (cuuint64_t)p.Hkv, (cuuint64_t)p.cache.page_size, (cuuint64_t)p.cache.pages};
  const long long st[3] = {p.cache.head, p.cache.slot, p.cache.page};
  const cuuint32_t box[4] = {64, 1, (cuuint32_t)(p.cache.page_size < kKeys ? p.cache.page_size : kKeys), 1};
  return make_map(k, p.cache.k, 4, dims, st, box) && make_map(v, p.cache.v, 4, dims, st, box);
}

// The grid of a paged kernel: what a part's slot is numbered by.
int paged_ctas(int sm_count) { return sm_count < kMaxCtas ? sm_count : kMaxCtas; }

template <int D, int MODE>
cudaError_t launch_join(const AttnParams &p, int sm_count, cudaStream_t stream) {
  const int per_sm = MODE == kShared ? kJoinRowsBlocksSm : kJoinBlocksSm;
  cudaLaunchConfig_t jc = pdl_config(dim3((unsigned)(per_sm * sm_count)), dim3(32 * kJoinWarps), 0, stream);
  cudaLaunchAttribute attr[1];
  attach_pdl(jc, attr);
  if constexpr (MODE == kShared) return cudaLaunchKernelEx(&jc, attn_join_rows_kernel<D>, p, paged_ctas(sm_count));
  else return cudaLaunchKernelEx(&jc, attn_join_kernel<D, MODE>, p, paged_ctas(sm_count));
}

template <int D, int MODE>
cudaError_t launch_t(const AttnParams &p, int sm_count, cudaStream_t stream) {
  using C = Cfg<D, MODE>;
  auto kern = attn_kernel<D, MODE>;
  static DeviceOnce once;
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!once.done(dev)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    // the warpgroups' register shares must be what the launch brings
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
    if (fa.numRegs != kRegs) return cudaErrorInvalidConfiguration;
    once.set(dev);
  }
  const int G = p.Hq / p.Hkv, TQ = kRowsT / G;
  CUtensorMap q, k, v, kc, vc;
  std::memset(&kc, 0, sizeof(kc));
  std::memset(&vc, 0, sizeof(vc));
  constexpr bool TREE = paged(MODE);
  const int rows = TREE ? kAttnMaxNodes : kKeys;
  if (!heads_map(&q, p.q, p.Hq, p.T, D, G, TQ) || !heads_map(&k, p.k, p.Hkv, p.T, D, 1, rows) ||
      !heads_map(&v, p.v, p.Hkv, p.T, D, 1, rows))
    return cudaErrorInvalidValue;
  long long ctas = paged_ctas(sm_count);
  if (TREE) {
    if (!cache_maps(&kc, &vc, p)) return cudaErrorInvalidValue;
  } else {
    // no more than there can be row groups (each sequence rounds up)
    const long long items = ((long long)p.T / TQ + p.B) * p.Hkv;
    if (items < ctas) ctas = items;
  }
  cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)ctas), dim3(kThreads), C::kSmem, stream);
  cudaLaunchAttribute attr[1];
  attach_pdl(cfg, attr);
  return cudaLaunchKernelEx(&cfg, kern, q, k, v, kc, vc, p);
}

}  // namespace
}  // namespace mxg

