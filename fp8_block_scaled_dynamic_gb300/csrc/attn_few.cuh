// attn_few.cuh -- attention of few rows a sequence and kv head over a plan's
// records: decoding and small trees, where attn_kernel.cuh's tiles would be mostly
// empty.
//
// The same sums with the operands exchanged, so that keys and channels, not rows,
// fill the tensor core's 128 lanes:
//   S^T (keys x rows)     = K (128 keys x D) . Q^T (D x NR rows)
//   O^T (channels x rows) += V^T (channels x 128 keys) . P^T (128 keys x NR rows)
// A softmax thread is a key of the tile (its NR scores), at the end a channel (NR
// results).  A row's exponentials are spread over 128 threads: a tile of 8 rows
// takes a warp 0.3 us of instructions where a thread a row took 1.6, and so an item of
// a few tiles, whose parts follow one another, a third of the time.
//
// One pass with a reference a row, as there.  It need not be near the maximum: weights
// have fp32's and bf16's range of exponents, and a reference that some key of the row
// has is never above it.  So the first key's score serves where all rows see it (else
// the first tile's maximum, 0.9 us more), and it is moved to the maximum only when a
// weight is past 2^30 (one vote a tile).  Weights are rounded to bf16 and summed as
// rounded, so that what one key's rounding adds above it also adds below.
//
// Rows see different keys: a key has a word of the rows that see it (mask words for
// nodes, a page's word for lists).  A key that no row sees has its v set to zero in
// shared memory.  A NaN or an infinity in the v of a key that some rows see makes an
// accumulator that is not finite; such a row is summed again from what it sees, and so is
// one whose values are too large for a reference so far below its maximum.
//
// Warps: four of softmax for each 16 rows (a thread with 64 rows had 24 KB of code a
// tile, whose fetching took 3.4 us), then one each for MMAs, loads and items.
// TMEM columns: two buffers of scores, two of results (of items in turn), 64 each.
//
// What bounds it, and what was measured (GB300; a copy runs at 6.8 TB/s): an item's
// chain.  The first comes 2.3 us after the plan, its first scores 2 us later; a tile
// follows the last after 0.6 (16 rows) to 1.4 us (64), where memory keeps up (64 KB a
// tile and SM take 1.5 us); the last product, the results' turn and their way out 2 us.
// - 32 requests over 32 pages of 64 each (64 / 8 heads of 128, 269 MB): 52 us, 5.1 TB/s
//   in this kernel, 58 with plan and join.
// - 8 trees of 8 nodes over 16 pages a node (74 MB in all): 35.5 us; one node a request:
//   18.6.
// Left out: a decoded token's own key added after its last part instead of a tile of its
// own (64 requests 98 -> 106 us: the loads and the product are in the item's chain, the
// tile is not); results of four rows unrolled (20.3 -> 21.2 us for short requests: more
// code to fetch).
#pragma once
#include "attn_kernel.cuh"

namespace mxg {
namespace {

constexpr int kFewRows = 16;  // rows of a softmax thread
constexpr int kFewHead = 6 * 1024;  // bytes of shared memory before the tiles

template <int D, int NR>
struct FewCfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kTile = kKeys * D * 2;
  static constexpr int kQ = NR * 128 * kHalves;  // a q tile: NR rows of 128 bytes for each 64 channels
  static constexpr int kGroups = NR / kFewRows;  // of four softmax warps
  static constexpr int kThreads = 128 * kGroups + 96;
  static constexpr int kP = kFewRows * 256;      // weights of a group: its rows of 128 bytes for each 64 keys
  static constexpr int kW = 2 * kGroups * kP;    // two buffers of them a group
  static constexpr int kEnd = 16 * 1024;         // (with D = 64 the lanes past the channels read on behind a v tile)
  static constexpr int kFit = (227 * 1024 - kFewHead - 2 * kQ - (kW < kEnd ? kEnd : kW)) / kTile;
  static constexpr int kSlots = kFit < 12 ? kFit : 12;
  static constexpr int kSmem = kFewHead + kSlots * kTile + 2 * kQ + (kW < kEnd ? kEnd : kW);
  static_assert(kSlots >= 4 && kQ % 1024 == 0 && kP % 1024 == 0, "shared memory");
};

// A weight above this moves the reference.  What a row adds up is at most so much larger
// than with its maximum; where that makes it too large, the row is summed again.
constexpr float kFewPast = 0x1p30f;

template <int D, int NR, int MODE>
struct FewSmem {
  using C = FewCfg<D, NR>;
  uint64_t kv_full[C::kSlots], kv_empty[C::kSlots], q_full[2], q_empty[2], s_full[2], p_ready[2], pv_done[2];
  uint64_t o_free[2], item_full[2], item_free[2], mma_done, stall;
  // of a row: its reference m, -m in units of the exponent (infinite: none yet), what the sums are scaled by
  alignas(16) float ref[NR], neg[NR], fac[NR];
  float part[C::kGroups][4][kFewRows];  // of a group's warps: the rows' maxima or sums over their keys
  uint32_t seen[C::kGroups][4];  // of a warp's keys: the rows of its group that see one
  uint32_t bad[C::kGroups];      // rows whose accumulator is not finite, or too large
  uint32_t tmem;
  int abort_flag;
  Item<MODE> items[2];
};

// D fp32, A (N-major or not) and B K-major.
__host__ __device__ constexpr uint32_t idesc_few(int n, bool a_mn) {
  return idesc_bf16(128, n, false) | ((a_mn ? 1u : 0u) << 15);
}

// Common barriers of a group's four warps.
__device__ __forceinline__ bool any_of_four(int group, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbarrier.cta.red.or.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(1 + group), "r"((uint32_t)x)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void sync_four(int group) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + group) : "memory"); }
__device__ __forceinline__ void st_shared_u16(uint32_t to, uint32_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(to), "h"((uint16_t)v) : "memory");
}
__device__ __forceinline__ void tmem_ld_rows(uint32_t at, uint32_t (&r)[kFewRows]) {
  tmem_ld16(at, r);
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < kFewRows; ++i) asm volatile("" : "+r"(r[i]));
}

template <int D, int NR, int MODE>
__global__ void __launch_bounds__(FewCfg<D, NR>::kThreads, 1)
    attn_few_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmKC,
                    const __grid_constant__ CUtensorMap tmVC, const __grid_constant__ AttnParams p) {
  using C = FewCfg<D, NR>;
  constexpr int S = C::kSlots, kSoft = 4 * C::kGroups;  // softmax warps
  constexpr unsigned kFull = 0xFFFFFFFFu;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  static_assert(sizeof(FewSmem<D, NR, MODE>) <= kFewHead, "shared memory head");
  FewSmem<D, NR, MODE> &sm = *reinterpret_cast<FewSmem<D, NR, MODE> *>(smem_raw);
  const uint32_t base = smem_addr(smem_raw);
  if (base & 1023u) {  // the swizzled tiles need it (uniform over the grid)
    if (threadIdx.x == 0) {
      pdl_wait();
      reinterpret_cast<JoinItem *>(p.ws)[blockIdx.x].rows = 0;
      if (p.status) atomicOr(p.status, kSmemLayout);
    }
    return;
  }
  const uint32_t kv_smem = base + kFewHead, q_smem = kv_smem + S * C::kTile, p_smem = q_smem + 2 * C::kQ;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv, TQ = NR / G;  // (the host sees to G <= NR)
  pdl_trigger();
  // (attn_shared: the launch before this one, which has not waited for anything else
  // when it lets this one start, works on the prefixes: what this one reads is older,
  // so it waits at its end, for the join's sake)
  const bool late = MODE == kShared && p.plan.beside;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_addr(&sm.kv_full[i]), 1);
      mbar_init(smem_addr(&sm.kv_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&sm.q_full[i]), 1);
      mbar_init(smem_addr(&sm.q_empty[i]), 1);
      mbar_init(smem_addr(&sm.s_full[i]), 1);
      mbar_init(smem_addr(&sm.p_ready[i]), kSoft);
      mbar_init(smem_addr(&sm.pv_done[i]), 1);
      mbar_init(smem_addr(&sm.o_free[i]), kSoft);
      mbar_init(smem_addr(&sm.item_full[i]), 1);
      mbar_init(smem_addr(&sm.item_free[i]), kSoft + 2);
    }
    mbar_init(smem_addr(&sm.mma_done), 1);
    mbar_init(smem_addr(&sm.stall), 1);
    sm.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kSoft) {
    tmem_alloc(smem_addr(&sm.tmem), 256);
    tmem_relinquish();
  }
  if (warp == kSoft + 1 && lane == 0) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
    prefetch_tmap(&tmKC);
    prefetch_tmap(&tmVC);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(&sm.tmem);
  const WaitCtl ctl{&sm.abort_flag, p.status, p.timeout_ns};
  if (!late) pdl_wait();
  Item<MODE> it;
  auto next_item = [&](int k) {
    if (!warp_wait(&sm.item_full[k & 1], (k >> 1) & 1, ctl)) return false;
    it = sm.items[k & 1];
    return it.t1 > it.t0;
  };
  auto done_item = [&](int k) { warp_arrive(&sm.item_free[k & 1], lane); };

  if (warp == kSoft + 1) {
    // --------------------------------------------------------------- loads
    uint32_t n = 0, nq = 0, slot = 0, turn = 0;
    bool ok = true;
    const bool el = elect_one();
    const uint32_t kvb = uniform(kv_smem), full0 = uniform(smem_addr(&sm.kv_full[0])), qb = uniform(q_smem);
    const int page_shift = 31 - __clz(p.cache.page_size), box_shift = min(page_shift, 7);
    for (int k = 0; ok && next_item(k); ++k) {
      const int t0 = (int)uniform(it.t0), t1 = (int)uniform(it.t1), nct = (int)uniform(it.nct);
      const int hk = (int)uniform(it.hk), a0 = (int)uniform(it.a0), ctx = (int)uniform(it.ctx);
      const int *row = (MODE == kSparse ? p.plan.list : p.table) + list_of(it);
      // lane b: the page of box b (a page of up to 128 keys) of tile j
      auto page_of = [&](int j) {
        const int key = (j << 7) + (lane << box_shift);
        if (j >= nct || j >= t1 || (lane << box_shift) >= kKeys || key >= ctx) return 0;
        return __ldg(row + (key >> page_shift));
      };
      auto load_kv = [&](int j, bool is_v, int pg) {
        if (!warp_wait_far(&sm.kv_empty[slot], turn ^ 1, ctl)) return false;  // (free at first)
        const uint32_t us = uniform(slot), bar = full0 + 8 * us, dst = kvb + us * C::kTile;
        if (j < nct) {
          const int boxes = (min(kKeys, ctx - (j << 7)) + (1 << box_shift) - 1) >> box_shift;
          if ((uint32_t)pg >= (uint32_t)p.cache.pages) {
            pg = p.cache.pages;  // out of the map's bounds: zeros
            if (p.status) atomicOr(p.status, kBadIndex);
          }
          int page[8];
#pragma unroll
          for (int b = 0; b < 8; ++b) page[b] = (int)__shfl_sync(kFull, pg, b);
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
          mbar_arrive_expect_tx(bar, (uint32_t)(kAttnMaxNodes * 128 * C::kHalves));
#pragma unroll
          for (int h = 0; h < C::kHalves; ++h) tma_load_3d(dst + h * 16384, is_v ? &tmV : &tmK, h * 64, hk, a0, bar);
        }
        __syncwarp();
        ++n;
        if (++slot == S) slot = 0, turn ^= 1;
        return true;
      };
      int pg[4];  // this lane's pages of tiles j .. j + 3
#pragma unroll
      for (int x = 0; x < 3; ++x) pg[x] = page_of(t0 + x);
      // q (the q tiles in turn)
      if (nq >= 2) ok = warp_wait_far(&sm.q_empty[nq & 1], ((nq >> 1) - 1) & 1, ctl);
      if (!ok) break;
      if (el) {
        const uint32_t bar = smem_addr(&sm.q_full[nq & 1]);
        mbar_arrive_expect_tx(bar, (uint32_t)(TQ * G * 128 * C::kHalves));
#pragma unroll
        for (int h = 0; h < C::kHalves; ++h)
          tma_load_3d(qb + (nq & 1) * C::kQ + h * NR * 128, &tmQ, h * 64, hk * G, a0 + (int)it.r0, bar);
      }
      __syncwarp();
      ++nq;
      ok = load_kv(t0, false, pg[0]);
      if (ok && t0 + 1 < t1) ok = load_kv(t0 + 1, false, pg[1]);
      for (int j = t0; ok && j < t1; ++j) {  // (k two tiles ahead of v)
        pg[3] = page_of(j + 3);
        ok = load_kv(j, true, pg[0]);
        if (ok && j + 2 < t1) ok = load_kv(j + 2, false, pg[2]);
#pragma unroll
        for (int x = 0; x < 3; ++x) pg[x] = pg[x + 1];
      }
      done_item(k);
    }
    // nothing may land in shared memory once the CTA is gone (a timeout)
    for (uint32_t k = n > S ? n - S : 0; k < n; ++k) drain(&sm.kv_full[k % S], (k / S) & 1, p.timeout_ns);
    for (uint32_t k = nq > 2 ? nq - 2 : 0; k < nq; ++k) drain(&sm.q_full[k & 1], (k >> 1) & 1, p.timeout_ns);
  } else if (warp == kSoft) {
    // ---------------------------------------------------------------- MMAs
    const bool el = elect_one();
    const uint32_t tm = uniform(tmem), qb = uniform(q_smem), kb = uniform(kv_smem), pb = uniform(p_smem);
    constexpr uint32_t kIdQK = idesc_few(NR, false), kIdPV = idesc_few(kFewRows, true);
    uint32_t rn = 0, tile = 0;  // tiles of the ring, tiles of keys so far
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) { return lane_wait(bar, parity, ctl); };
    auto ring = [&](uint32_t k) { return wait(&sm.kv_full[k % S], (k / S) & 1); };
    auto all_ok = [&](bool x) { return __all_sync(kFull, x) != 0; };
    // scores of tile number t of all (buffer t & 1); its k is ring tile r
    auto qk = [&](uint32_t t, uint64_t kd, uint64_t qd, uint32_t r) {
      tc_fence_after();
#pragma unroll
      for (int h = 0; h < C::kHalves; ++h)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          mma_bf16_ss(tm + (t & 1) * 64, kd + h * 1024 + x * 2, qd + h * (NR * 8) + x * 2, kIdQK, (h | x) != 0);
      tc_commit(smem_addr(&sm.s_full[t & 1]));
      tc_commit(smem_addr(&sm.kv_empty[r % S]));
    };
    auto kdesc = [&](uint32_t r) { return sdesc_kmajor_sw128(kb + uniform(r % S) * C::kTile); };
    auto vdesc = [&](uint32_t r) { return sdesc_mnmajor_sw128(kb + uniform(r % S) * C::kTile, 16384); };
    for (int k = 0; ok && next_item(k); ++k) {
      const int nt = (int)uniform(it.t1 - it.t0);
      done_item(k);
      const uint64_t qd = sdesc_kmajor_sw128(qb + uniform(k & 1) * C::kQ);
      const uint32_t o = tm + 128 + (k & 1) * 64;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (!ok || s >= nt) continue;
        const uint64_t kd = kdesc(rn);
        if (el) {
          // (the weights of two tiles back are there: their scores have been read)
          const uint32_t t = tile + s;
          ok = ring(rn) && (s > 0 || wait(&sm.q_full[k & 1], (k >> 1) & 1));
          if (ok) qk(t, kd, qd, rn);
        }
        ok = all_ok(ok);
        ++rn;
      }
      for (int i = 0; ok && i < nt; ++i) {
        const bool more = i + 2 < nt;
        const uint64_t vd = vdesc(rn), kd = kdesc(rn + 1);
        const uint32_t t = tile + i;
        if (el) {
          const uint64_t pd = sdesc_kmajor_sw128(pb + (t & 1) * C::kP);  // the first group's
          ok = ring(rn) && (i > 0 || k < 2 || wait(&sm.o_free[k & 1], ((k >> 1) - 1) & 1)) &&
               wait(&sm.p_ready[t & 1], (t >> 1) & 1);
          if (ok) {
            tc_fence_after();
#pragma unroll
            for (int x = 0; x < 8; ++x)
#pragma unroll
              for (int g = 0; g < C::kGroups; ++g)
                mma_bf16_ss(o + g * kFewRows, vd + x * 128, pd + g * (2 * C::kP / 16) + (x >> 2) * (kFewRows * 8) + (x & 3) * 2,
                            kIdPV, i > 0 || x > 0);
            tc_commit(smem_addr(&sm.pv_done[t & 1]));
            tc_commit(smem_addr(&sm.kv_empty[rn % S]));
            if (i + 1 == nt) tc_commit(smem_addr(&sm.q_empty[k & 1]));
          }
          if (ok && more) {
            ok = ring(rn + 1);
            if (ok) qk(t + 2, kd, qd, rn + 1);
          }
        }
        ok = all_ok(ok);
        rn += more ? 2 : 1;
      }
      tile += nt;
    }
    // every MMA has completed before the CTA leaves its shared memory and TMEM
    if (el) {
      tc_commit(smem_addr(&sm.mma_done));
      drain(&sm.mma_done, 0, p.timeout_ns);
    }
    __syncwarp();
  } else if (warp == kSoft + 2) {
    // --------------------------------------------------------------- items
    const bool few = seqs<MODE>(p) <= 32;
    Small<MODE> small;
    PlanUnits<MODE> units;
    if (few) {
      small.read(p, TQ, lane, false);
      small.number(p, lane);
    } else {
      units.read(p, lane);
    }
    Walk<MODE> walk(few ? small.total : units.total, TQ, p.plan.ctas ? __ldg(p.plan.ctas) : (int)gridDim.x);
    bool going_on = false;
    if (few) walk.choose_chunk(small);
    else walk.choose_chunk(units);
    for (int k = 0;; ++k) {
      Item<MODE> w;
      int last = 0;  // the last CTA that has a part of the row group
      if (walk.chunk > 0 && k == 0) {
        last = walk.one_chunk(p, small, TQ, w);
      } else {
        walk.next(p, TQ, w, [&](int &u, int &b) { return few ? small.find(u, b) : units.find(p, TQ, u, b); });
        if (w.t1 > w.t0 && w.part == 1)
          last = walk.last >= 0 ? walk.last
                                : share_owner(share_begin(blockIdx.x + 1, walk.q, walk.r) + w.nct +
                                                  (flags_of(w) & kHasNodes) - 1 - w.t1,
                                              walk.q, walk.r);
      }
      if (k >= 2 && !warp_wait_far(&sm.item_free[k & 1], ((k >> 1) - 1) & 1, ctl)) break;
      if (lane == 0) sm.items[k & 1] = w;
      warp_arrive(&sm.item_full[k & 1], lane);
      if (w.t1 == w.t0) break;
      if (w.part == 1) {
        going_on = true;
        if (lane == 0) {
          JoinItem j;
          j.rows0 = j.rows = w.cnt[0] * G;
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
    if (!going_on && lane == 0) reinterpret_cast<JoinItem *>(p.ws)[blockIdx.x].rows = 0;
  } else {
    // ------------------------------------------------------------- softmax
    // (A wait that runs out lets a warp go on without what it waited for, to the
    // next common barrier: a group's four warps leave together.)
    constexpr int R = kFewRows;
    const int grp = warp >> 2, wi = warp & 3, first = grp * R;  // the group's first row
    const uint32_t lanes = (uint32_t)(wi * 32) << 16;
    const int key = wi * 32 + lane;  // of a tile; at the end the channel
    const float c = p.scale * kLog2e;
    const int page_shift = 31 - __clz(p.cache.page_size);
    // A group's weights' tiles are also where its values are turned from a thread a
    // key (or channel) to a warp a row: when no product reads them.
    const uint32_t p_mine = p_smem + grp * 2 * C::kP;
    float *const turn = reinterpret_cast<float *>(smem_raw + (p_mine - base));  // [row][128]
    float *const ref = sm.ref + first, *const neg = sm.neg + first, *const fac = sm.fac + first;
    uint32_t tile = 0, rn = 0;
    bool ok = true;
    if (p.debug_stall) ok = warp_wait(&sm.stall, 0, ctl);
    // What an item's first tile needs from memory: the words of the nodes that name this
    // key's page (lists), the mask words of nodes lane and lane + 32.
    struct Words {
      unsigned long long who, word[2];
    };
    auto lists_of = [&](const Item<MODE> &x) { return MODE == kSparse && (flags_of(x) & kLists); };
    auto names_of = [&](const Item<MODE> &x, int j, unsigned long long &who) {
      const int t = j * kKeys + key;
      if (lists_of(x) && j < x.nct && t < x.ctx) who = __ldg(p.plan.names + list_of(x) + (t >> page_shift));
    };
    auto words_of = [&](const Item<MODE> &x) {
      Words y = {};
      names_of(x, x.t0, y.who);
      if (x.t1 > x.nct) {
        if (lane < x.cnt[0]) y.word[0] = __ldg(p.mask + x.a0 + x.r0 + lane);
        if (NR > 32 && lane + 32 < x.cnt[0]) y.word[1] = __ldg(p.mask + x.a0 + x.r0 + lane + 32);
      }
      return y;
    };
    bool there = ok && next_item(0);
    Words ahead = {};
    if (there) ahead = words_of(it);
    for (int k = 0;; ++k) {
      if (any_of_four(grp, !there || !ok)) break;
      const int nt = it.t1 - it.t0, cnt = it.cnt[0], rows = min(max(cnt * G - first, 0), R);  // this group's rows
      const unsigned long long group = G >= 64 ? ~0ull : (1ull << G) - 1ull;
      const uint32_t mine = (1u << rows) - 1u;
      const bool lists = lists_of(it);
      unsigned long long who = ahead.who;  // (of the next tile)
      const unsigned long long word[2] = {ahead.word[0], ahead.word[1]};
      unsigned long long words = word[0] | word[1];  // of all the item's nodes
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) words |= __shfl_xor_sync(kFull, words, x);
      // The group's rows that see this key of tile j, and whether any row of the item
      // does: rows of nodes n0 ... are G bits each, the first of them cut off.
      const int n0 = first / G, cut = first - n0 * G, n1 = min((first + R - 1) / G + 1, cnt);
      auto rows_that_see = [&](int j, bool &some) {
        uint32_t r = 0;
        some = false;
        auto add = [&](int i, bool sees) {
          const int at = (i - n0) * G - cut;  // (a node has at most 64 rows, and the first may begin below)
          const unsigned long long bits = at >= 0 ? group << at : group >> -at;
          r |= sees ? (uint32_t)bits & 0xFFFFu : 0u;
        };
        if (j >= it.nct) {
          some = key < it.n && (words >> (key & 63) & 1ull);
          for (int i = n0; i < n1; ++i) {
            const unsigned long long w = __shfl_sync(kFull, i < 32 ? word[0] : word[1], i & 31);
            add(i, key < it.n && (w >> (key & 63) & 1ull));
          }
        } else if (j * kKeys + key < it.ctx) {
          some = true;
          if (!lists) return mine;
          const unsigned long long w = who >> it.r0;
          some = (w & (cnt >= 64 ? ~0ull : (1ull << cnt) - 1ull)) != 0ull;
          for (int i = n0; i < n1; ++i) add(i, w >> i & 1ull);
        }
        return r & mine;
      };
      float l[R];
#pragma unroll
      for (int r = 0; r < R; ++r) l[r] = 0.0f;
      if (key == 0) sm.bad[grp] = 0;
      uint32_t saw = 0;
      bool open = true;
      for (int i = 0; i < nt; ++i) {
        const int j = it.t0 + i;
        const uint32_t t = tile + i, sb = t & 1, ph = (t >> 1) & 1;
        bool some;
        const uint32_t see = rows_that_see(j, some);
        names_of(it, j + 1, who);
        saw |= see;
        if (!warp_wait(&sm.s_full[sb], ph, ctl)) ok = false;
        tc_fence_after();
        uint32_t s[R];
        tmem_ld_rows(tmem + lanes + sb * 64 + first, s);
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (!(see >> r & 1u)) s[r] = 0xFF800000u;
        bool past = false;
        // a row without a reference yet has an infinite `neg` (rows past the last one: 0)
        const auto open_rows = [&]() {
          bool x = false;
#pragma unroll
          for (int r = 0; r < R; ++r) x |= neg[r] == INFINITY;
          return x;
        };
        if (i == 0) {
          if (!lists && it.nct > it.t0) {
            // all rows see the tile's first key
            if (key == 0) {
#pragma unroll
              for (int r = 0; r < R; ++r)
                ref[r] = __uint_as_float(s[r]), neg[r] = r < rows ? -__uint_as_float(s[r]) * c : 0.0f;
            }
            sync_four(grp);
            open = open_rows();
          } else {
            past = true;
          }
        }
        uint32_t w[R / 2];  // weights, rounded to bf16, of two rows each
        const auto weigh = [&]() {
          float most = 0.0f;
          if (!open) {
#pragma unroll
            for (int r = 0; r < R; r += 2) {
              const float x = ex2(fmaf(__uint_as_float(s[r]), c, neg[r]));
              const float y = ex2(fmaf(__uint_as_float(s[r + 1]), c, neg[r + 1]));
              most = fmaxf(most, fmaxf(x, y));
              w[r / 2] = pack_bf16x2(x, y);
            }
          } else {
#pragma unroll
            for (int r = 0; r < R; r += 2) {
              float x[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float n = neg[r + e];
                x[e] = ex2(fmaf(__uint_as_float(s[r + e]), c, n == INFINITY ? 0.0f : n));
                most = fmaxf(most, n == INFINITY && s[r + e] != 0xFF800000u ? INFINITY : x[e]);
              }
              w[r / 2] = pack_bf16x2(x[0], x[1]);
            }
          }
          return most > kFewPast;
        };
        if (!past) past = any_of_four(grp, weigh());
        if (past) {
          const uint32_t prev = t - 1;
          if (i > 0 && !warp_wait(&sm.pv_done[prev & 1], (prev >> 1) & 1, ctl)) ok = false;
          // the rows' maxima: a first one is the reference, a later one moves it
          float x[R];
#pragma unroll
          for (int r = 0; r < R; ++r) x[r] = __uint_as_float(s[r]);
          const float top = over_lanes(x, lane, [](float a, float b) { return fmaxf(a, b); });
          if (!(lane & 1)) sm.part[grp][wi][lane >> 1] = top;
          sync_four(grp);
          if (key < R) {
            const float(&m4)[4][R] = sm.part[grp];
            const float old = i > 0 ? ref[key] : -INFINITY;
            const float m = fmaxf(fmaxf(old, fmaxf(m4[0][key], m4[1][key])), fmaxf(m4[2][key], m4[3][key]));
            fac[key] = m == old ? 1.0f : old == -INFINITY ? 0.0f : ex2((old - m) * c);
            ref[key] = m;
            neg[key] = key < rows ? -m * c : 0.0f;
          }
          sync_four(grp);
          open = open_rows();
          if (i > 0) {
            tc_fence_after();
            const uint32_t at = tmem + lanes + 128 + (k & 1) * 64 + first;
            uint32_t o[R];
            tmem_ld_rows(at, o);
#pragma unroll
            for (int r = 0; r < R; ++r) {
              const float f = fac[r];
              l[r] *= f;
              o[r] = __float_as_uint(__uint_as_float(o[r]) * f);
            }
            tmem_st16(at, o);
            tmem_st_wait();
            tc_fence_before();
          }
          weigh();
        }
        // For the product and as sums.  (The tile that had these two buffers before has
        // been multiplied: the scores came after it.)
        const uint32_t to = p_mine + sb * C::kP + (key >> 6) * (R * 128) + (key & 7) * 2, unit = (key >> 3) & 7;
#pragma unroll
        for (int r = 0; r < R; r += 2) {
          const uint32_t x = w[r / 2];
          l[r] += __uint_as_float(x << 16);
          l[r + 1] += __uint_as_float(x & 0xFFFF0000u);
          st_shared_u16(to + r * 128 + ((unit ^ (r & 7)) << 4), x);
          st_shared_u16(to + (r + 1) * 128 + ((unit ^ ((r + 1) & 7)) << 4), x >> 16);
        }
        if (grp == 0 && !some) {
          // no row sees this key: its v is made zero
          const uint32_t v_at = rn + (nt > 1 ? 2 : 1) + i + min(i, max(nt - 2, 0));  // the v tile's place in the ring
          if (!mbar_wait_quick(smem_addr(&sm.kv_full[v_at % S]), (v_at / S) & 1, ctl)) ok = false;
          const uint32_t v = kv_smem + (v_at % S) * C::kTile + key * 128;
#pragma unroll
          for (int h = 0; h < C::kHalves; ++h)
#pragma unroll
            for (int x = 0; x < 8; ++x) st_shared_v4(v + h * 16384 + ((x + lane) & 7) * 16, 0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        warp_arrive(&sm.p_ready[sb], lane);
      }
      ok = __all_sync(kFull, ok);
      // while the last product runs: the next item and its words, the rows' sums over the keys
      const Item<MODE> &cur = sm.items[k & 1];  // (this one: its place is not free yet)
      there = ok && next_item(k + 1);
      if (there) ahead = words_of(it);
      const float sum = over_lanes(l, lane, [](float a, float b) { return a + b; });
      if (!(lane & 1)) sm.part[grp][wi][lane >> 1] = sum;
      saw = __reduce_or_sync(kFull, saw);
      if (lane == 0) sm.seen[grp][wi] = saw;
      const uint32_t lastt = tile + nt - 1;
      if (!warp_wait(&sm.pv_done[lastt & 1], (lastt >> 1) & 1, ctl)) ok = false;
      tc_fence_after();
      // results turned to a warp a row
      uint32_t o[R];
      tmem_ld_rows(tmem + lanes + 128 + (k & 1) * 64 + first, o);
      tc_fence_before();
      warp_arrive(&sm.o_free[k & 1], lane);
      uint32_t bad = 0;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        turn[r * 128 + key] = __uint_as_float(o[r]);
        bad |= too_large(o[r]) ? 1u << r : 0u;
      }
      bad = key < D ? bad & mine : 0u;
      if (bad) atomicOr(&sm.bad[grp], bad);
      sync_four(grp);
      const uint32_t seen = sm.seen[grp][0] | sm.seen[grp][1] | sm.seen[grp][2] | sm.seen[grp][3];
      const float(&p4)[4][R] = sm.part[grp];
      bad = sm.bad[grp];
      if (bad) {  // what another row's NaN has spoilt, or a low reference, is summed again
        // (64 rows: a thread has 96 registers, and with more rows or keys at a time what the
        // call saves of them costs every tile: 8 trees of 8 nodes 37 to 44 us, so 36)
        constexpr int kAtOnce = NR == 64 ? 1 : 4, kLanes = 32 / kAtOnce;
#pragma unroll 1
        for (int r0 = wi; r0 < rows; r0 += 4 * kAtOnce) {
          const int r = r0 + 4 * (lane / kLanes);
          const bool is = r < rows && (bad >> r & 1u);
          if (!__any_sync(kFull, is)) continue;
          const float2 stat = sum_again<D, MODE, kAtOnce, NR == 64 ? 1 : 2>(p, cur, cur.r0, is ? first + r : -1,
                                                                            turn + r0 * 128, 4 * 128);
          if (is && lane % kLanes == 0) {
            ref[r] = stat.x;
            sm.part[grp][0][r] = stat.y;
            sm.part[grp][1][r] = sm.part[grp][2][r] = sm.part[grp][3][r] = 0.0f;
          }
          __syncwarp();
        }
        // (read again, so that the call does not have to save them)
        it = sm.items[(k + 1) & 1];
        ahead = {};
        if (there) ahead = words_of(it);
      }
      // Rows in memory, a warp a row: results, or parts in the CTA's slot or the rows' own
      // places.
      constexpr int V = D / 32;
      const int part = cur.part;
      float *const slot = p.ws + p.slots + ((long long)blockIdx.x * 2 + (part & 1)) * Cfg<D, MODE>::kSlotFloats;
      const long long kind = MODE == kShared ? (long long)(flags_of(cur) & kHasNodes) * p.T : 0;
#pragma unroll 1
      for (int r = wi; r < rows; r += 4) {
        const int row = first + r, nd = div_small(row, G);
        const int node = cur.a0 + cur.r0 + nd, hd = cur.hk * G + row - nd * G;
        const float m = ref[r], total = (p4[0][r] + p4[1][r]) + (p4[2][r] + p4[3][r]);
        const bool any = seen >> r & 1u;
        const float *y = turn + r * 128 + lane * V;
        if (part < 0) {
          const float inv = 1.0f / total;
          uint16_t *out = p.out.ptr + (long long)node * p.out.tok + hd * p.out.head + lane * V;
#pragma unroll
          for (int e = 0; e < V; e += 2)
            reinterpret_cast<uint32_t *>(out)[e / 2] = any ? pack_bf16x2(y[e] * inv, y[e + 1] * inv) : 0u;
        } else {
          const long long own = (kind + node) * p.Hq + hd;
          float *to = (part == 2 ? p.plan.rows + own * D : slot + row * D) + lane * V;
          if constexpr (V == 4) *reinterpret_cast<float4 *>(to) = *reinterpret_cast<const float4 *>(y);
          else *reinterpret_cast<float2 *>(to) = *reinterpret_cast<const float2 *>(y);
          if (lane == 0) {
            // (a sum of 0 says that the row sees nothing of the part)
            float *stat = part == 2 ? p.plan.stats + own * 2 : slot + D * kRowsT + row;
            stat[0] = m;
            stat[part == 2 ? 1 : kRowsT] = !any ? 0.0f : m == -INFINITY ? 1.0f : total;
          }
        }
      }
      tile += nt;
      rn += 2 * nt;
      done_item(k);
    }
  }

  if (late) pdl_wait();
  tc_fence_before();
  __syncthreads();
  if (warp == kSoft) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

template <int D, int NR, int MODE>
cudaError_t launch_few(const AttnParams &p, int sm_count, cudaStream_t stream) {
  using C = FewCfg<D, NR>;
  auto kern = attn_few_kernel<D, NR, MODE>;
  static DeviceOnce once;
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!once.done(dev)) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem)) != cudaSuccess) return e;
    once.set(dev);
  }
  const int G = p.Hq / p.Hkv, TQ = NR / G;
  CUtensorMap q, k, v, kc, vc;
  if (!heads_map(&q, p.q, p.Hq, p.T, D, G, TQ) || !heads_map(&k, p.k, p.Hkv, p.T, D, 1, kAttnMaxNodes) ||
      !heads_map(&v, p.v, p.Hkv, p.T, D, 1, kAttnMaxNodes) || !cache_maps(&kc, &vc, p))
    return cudaErrorInvalidValue;
  const int ctas = sm_count < kMaxCtas ? sm_count : kMaxCtas;
  cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)ctas), dim3(C::kThreads), C::kSmem, stream);
  cudaLaunchAttribute attr[1];
  attach_pdl(cfg, attr);
  return cudaLaunchKernelEx(&cfg, kern, q, k, v, kc, vc, p);
}

}  // namespace
}  // namespace mxg
