// index.cu -- bounds of the keys of full cache pages (kv_index) and the choice
// of pages by them (attn_select).
//
// A page's bounds of a kv head: with 2^e the least power of two, e >= -100, for
// which max |k| <= 127 * 2^e over the page's keys, upper[d] = ceil(max k[d] / 2^e)
// and lower[d] = floor(min k[d] / 2^e), whole numbers of 8 bits.  For every key of
// the page then q . k <= sum_d q[d] (q[d] > 0 ? upper[d] : lower[d]) 2^e, and with q
// in whole numbers too that sum is a whole number below 2^21: every step is exact,
// so the choice does not depend on an order of summation.
//
// What bounds them, and what was measured (GB300; a copy runs at 6.8 TB/s):
// - kv_index reads each key once: 4 documents of 16384 tokens, 5 layers of 8 heads of
//   128 (671 MB) 101 us, 6.7 TB/s.  A step's few pages 4.8 us: a launch, then sequences,
//   table, keys, one after another.
// - attn_select is a chain of dependent steps: offsets, q, page numbers, codes,
//   scores, two barriers and the choice's rounds: 11 us for one node of 64 / 8 heads
//   over 2048 pages and for 8 trees of 8 nodes over 128 to 256, 22 and 41 for 8 trees of
//   16 and 32 nodes (passes of eight).  A batch of 64 x 1024
//   pages reads 130 MB in 34 us, 3.9 TB/s: its blocks score, then choose, with nothing
//   to load meanwhile, and only others on the SM cover that.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <climits>
#include <cstdint>
#include <type_traits>

#include "attn.h"
#include "attn_ptx.cuh"
#include "kernels.h"

namespace mxg {
namespace {

constexpr int kBadIndex = 0x2;  // MXG_DEV_BAD_INDEX
constexpr int kLeastExp = -100;
constexpr unsigned kFull = 0xFFFFFFFFu;

// The least e >= -100 with amax <= 127 * 2^e, for a finite amax >= 0: amax = m 2^E
// with 1 <= m < 2 is 64 m in units of 2^(E - 6), and 64 m > 127 only for m > 127/64.
__device__ __forceinline__ int exponent_of(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127 - 6 + ((b & 0x7FFFFFu) > 0x7E0000u);
  return max(e, kLeastExp);
}
// 2^-e for e in [-100, 122]
__device__ __forceinline__ float scale_down(int e) { return __uint_as_float((uint32_t)(127 - e) << 23); }

// -------------------------------------------------------------- kv_index
constexpr int kIndexThreads = 256;

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}

// One page and kv head of a layer, a warp: a lane holds 8 channels of every R-th
// token.
template <int D>
__device__ __forceinline__ void bound_page(const IndexParams &p, int layer, int page, int head, int lane) {
  constexpr int L = D / 8, R = 32 / L;  // lanes of a token, tokens of a load
  const int sub = lane / L, c = lane % L;
  const uint16_t *k = p.cache.k + layer * p.cache.layer + page * p.cache.page + head * p.cache.head + c * 8;
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) hi[i] = 0xFF80FF80u, lo[i] = 0x7F807F80u;  // -inf, +inf
  // kAhead loads of a lane in flight (a step's few pages are a chain of them: with
  // four, 6.4 us)
  auto take = [&](auto ahead, int t) {
    constexpr int kAhead = decltype(ahead)::value;
    uint4 x[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      x[u] = __ldg(reinterpret_cast<const uint4 *>(k + (long long)((t + u) * R + sub) * p.cache.slot));
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      hi[0] = max2(hi[0], x[u].x), lo[0] = min2(lo[0], x[u].x);
      hi[1] = max2(hi[1], x[u].y), lo[1] = min2(lo[1], x[u].y);
      hi[2] = max2(hi[2], x[u].z), lo[2] = min2(lo[2], x[u].z);
      hi[3] = max2(hi[3], x[u].w), lo[3] = min2(lo[3], x[u].w);
    }
  };
  const int steps = p.cache.page_size / R;  // (a power of two, at least 4)
  if (steps >= 16) {
    for (int t = 0; t < steps; t += 16) take(std::integral_constant<int, 16>(), t);
  } else {
    for (int t = 0; t < steps; t += 4) take(std::integral_constant<int, 4>(), t);
  }
#pragma unroll
  for (int o = 16; o >= L; o >>= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hi[i] = max2(hi[i], __shfl_xor_sync(kFull, hi[i], o));
      lo[i] = min2(lo[i], __shfl_xor_sync(kFull, lo[i], o));
    }
  // the largest magnitude, as bits (NaN is above infinity)
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    top = max(top, max(max(hi[i] & 0x7FFFu, hi[i] >> 16 & 0x7FFFu), max(lo[i] & 0x7FFFu, lo[i] >> 16 & 0x7FFFu)));
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
  const bool finite = top < 0x7F80u;
  const int e = finite ? exponent_of(__uint_as_float(top << 16)) : 0;
  const float down = scale_down(e);
  if (sub > 1) return;
  uint32_t out[2] = {0, 0};
  if (finite) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w = sub == 0 ? hi[i / 2] : lo[i / 2];
      const float x = __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16), y = x * down;
      // (a quotient below fp32's least number still counts as one step)
      const float z = sub == 0 ? (x > 0.0f ? fmaxf(ceilf(y), 1.0f) : ceilf(y)) : (x < 0.0f ? fminf(floorf(y), -1.0f) : floorf(y));
      out[i / 4] |= ((uint32_t)(int)z & 0xFFu) << (i % 4 * 8);
    }
  }
  int8_t *codes = p.index.codes + layer * p.index.codes_layer + page * p.index.codes_page + head * p.index.codes_head;
  *reinterpret_cast<uint2 *>(codes + sub * D + c * 8) = make_uint2(out[0], out[1]);
  if (lane == 0)
    p.index.exps[layer * p.index.exps_layer + page * p.index.exps_page + head] = finite ? (uint8_t)(e + 127) : 255;
}

// Every block adds up the sequences' new full pages for itself, then the warps of
// the grid take pages, a kv head each: the heads of a page next to one another, so
// that a block reads whole tokens.
template <int D>
__global__ void __launch_bounds__(kIndexThreads, 2) index_kernel(const IndexParams p) {
  __shared__ int s_end[kAttnMaxSeqs], s_warp[kIndexThreads / 32];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int limit = p.table_cols * p.cache.page_size;
  const int per = (p.B + kIndexThreads - 1) / kIndexThreads, b0 = min((int)threadIdx.x * per, p.B), b1 = min(b0 + per, p.B);
  auto full = [&](int b, int &j0) {  // the new full pages of a sequence, the first of them
    const int old = p.old ? __ldg(p.old + b) : 0, now = __ldg(p.now + b);
    const int o = min(max(old, 0), limit), n = min(max(now, 0), limit);
    if (blockIdx.x == 0 && (o != old || n != now) && p.status) atomicOr(p.status, kBadIndex);
    j0 = o / p.cache.page_size;
    return max(n / p.cache.page_size - j0, 0);
  };
  int sum = 0, j0;
  for (int b = b0; b < b1; ++b) sum += full(b, j0);
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int at = incl - sum;
  for (int w = 0; w < warp; ++w) at += s_warp[w];
  for (int b = b0; b < b1; ++b) s_end[b] = at += full(b, j0);
  __syncthreads();
  const long long pages = s_end[p.B - 1], tasks = pages * p.Hkv * p.cache.layers;
  const long long stride = (long long)gridDim.x * (kIndexThreads / 32);
  for (long long t = (long long)blockIdx.x * (kIndexThreads / 32) + warp; t < tasks; t += stride) {
    const long long lp = t / p.Hkv;
    const int head = (int)(t - lp * p.Hkv), layer = (int)(lp / pages), x = (int)(lp - layer * pages);
    int lo = 0, hi = p.B - 1;  // the first sequence whose pages end after x
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (s_end[mid] > x) hi = mid;
      else lo = mid + 1;
    }
    const int n = full(lo, j0), j = j0 + x - (s_end[lo] - n);
    const int page = __ldg(p.table + (long long)lo * p.ld_table + j);
    if ((uint32_t)page >= (uint32_t)p.cache.pages) {
      if (p.status && lane == 0) atomicOr(p.status, kBadIndex);
      continue;
    }
    bound_page<D>(p, layer, page, head, lane);
  }
}

// ----------------------------------------------------------- attn_select
// A cluster of blocks a sequence and kv head.  Its warps score 16 pages at a time
// for the query heads of up to eight groups of eight columns, by
//   sum_d x (x > 0 ? u : l) = [max(x, 0) | min(x, 0)] . [u | l],
// a product of 2 D whole numbers below 2^7 that m16n8k16 in fp16 with fp32 sums has
// exactly (the 8-bit form of the instruction, without the codes' conversion, is far
// slower on this part: a batch of 64 x 1024 pages 102 us where this one took 72).  A
// page's codes are kept in the order in which the product wants them: which 16 of the
// 2 D positions a step takes does not matter as long as both operands agree.  A tile's
// registers are filled again for the next one as they are used.  A score goes, as a 32-bit key of the
// same order, to the shared memory of the block that chooses for its node; there the
// warps of a node find the key of the last page that is taken, bit by bit from the top,
// and write the pages out in order.
constexpr int kSelectWarps = 8;  // most warps of a block
template <bool MANY>
constexpr int kWarps = MANY ? 8 : 4;
constexpr int kSelectGroups = 8;            // groups of eight columns (query heads) that are multiplied at once
constexpr int kSelectMost = 16;             // in a pass: one node's most
constexpr int kSelectKeys = 12 * 1024;      // most keys of a block in shared memory, where one node's are no more
constexpr int kSelectMostCluster = 8;

struct SelectPlan {
  int cluster;  // blocks of a sequence and kv head, a power of two
  int shift;    // its logarithm
  int cols;     // keys of a node: the table's columns, rounded up to blocks (key_at)
  int slots;    // nodes that a block chooses for in a pass
  int gp;       // columns of a node: Hq / Hkv rounded up to 1, 2, 4 or a multiple of 8
  int gp_inv;   // 2^16 / gp, rounded up: c / gp = c * gp_inv >> 16 for the columns of a pass (a division took 25 instructions)
  int groups;   // of eight columns in a pass
  int shares;   // clusters of a sequence and kv head, which take its passes in turn
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
// Four signed bytes as fp16: 0x6400 + (x + 128) is 1152 + x.
__device__ __forceinline__ void bytes_to_half(uint32_t w, uint32_t &h01, uint32_t &h23) {
  const uint32_t u = w ^ 0x80808080u, lo = __byte_perm(u, 0x64646464u, 0x4140), hi = __byte_perm(u, 0x64646464u, 0x4342);
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(h01) : "r"(lo), "r"(0x64806480u));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(h23) : "r"(hi), "r"(0x64806480u));
}
// Unsigned numbers in the order of the floats; 0 is below all of them.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ void st_cluster(uint32_t saddr, uint32_t rank, uint32_t v) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\tst.shared::cluster.u32 [a], %2;\n\t}" ::"r"(saddr),
      "r"(rank), "r"(v)
      : "memory");
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Keys are kept in blocks of 32 lanes x 2^lg: a lane's are consecutive pages, four
// of them side by side, so that it reads its own ones 16 bytes at a time.
__host__ __device__ __forceinline__ int lane_shift(int pages) { return pages <= 256 ? 3 : 4; }
__device__ __forceinline__ int key_at(int j, int lg) {
  const int in = j & ((1 << lg) - 1), lane = (j >> lg) & 31;
  return (j & ~((32 << lg) - 1)) + (in >> 2) * 128 + lane * 4 + (in & 3);
}

// The choice for one node by `warps` warps (this one is the w-th) of a named
// barrier: candidates are the pages with a key above 0.
struct Choice {
  uint32_t (*box)[kSelectWarps][2];  // two of them, in turn
  int w, warps, bar, turn;
  // this warp's two numbers to all warps; lane i gets the i-th warp's
  __device__ __forceinline__ uint2 pass_round(uint32_t a, uint32_t b) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) box[turn][w][0] = a, box[turn][w][1] = b;
    named_sync(bar, warps * 32);
    const uint2 x = lane < warps ? make_uint2(box[turn][lane][0], box[turn][lane][1]) : make_uint2(0, 0);
    turn ^= 1;
    return x;
  }
};
template <int LG>
__device__ __forceinline__ void choose(const uint32_t *keys, int P, int first, int last, int n_sel, int *sel, Choice ch) {
  constexpr int kOwn = 1 << LG, kBlock = 32 * kOwn;  // keys that a lane, a warp holds in registers
  const int lane = threadIdx.x & 31, need = n_sel - first - last;
  const int blocks = (P + kBlock - 1) / kBlock, per = (blocks + ch.warps - 1) / ch.warps;
  const int c0 = min(ch.w * per, blocks), c1 = min(c0 + per, blocks);
  for (int i = ch.w * 32 + lane; i < first + last; i += ch.warps * 32) {
    const int x = i < first ? i : n_sel - last + i - first;
    sel[x] = i < first ? i : P - last + i - first;
  }
  if (need == 0) return;
  uint32_t k[kOwn];
  auto load = [&](int c) {
#pragma unroll
    for (int i = 0; i < kOwn / 4; ++i) {
      const uint4 x = c < c1 ? *reinterpret_cast<const uint4 *>(keys + (long long)c * kBlock + i * 128 + lane * 4)
                             : make_uint4(0, 0, 0, 0);
      k[4 * i] = x.x, k[4 * i + 1] = x.y, k[4 * i + 2] = x.z, k[4 * i + 3] = x.w;
    }
  };
  const bool held = c1 - c0 <= 1;
  // f over all of this warp's keys, a block at a time
  auto each = [&](auto f) {
    if (held) {
      f(c0);
    } else {
      for (int c = c0; c < c1; ++c) {
        load(c);
        f(c);
      }
    }
  };
  if (held) load(c0);
  // bits that all candidates have in common need no search
  uint32_t any = 0, all = ~0u;
  each([&](int) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      any |= k[i];
      all &= k[i] ? k[i] : ~0u;
    }
  });
  any = __reduce_or_sync(kFull, any);
  all = __reduce_and_sync(kFull, all);
  if (ch.warps > 1) {
    const uint2 x = ch.pass_round(any, ~all);
    any = __reduce_or_sync(kFull, x.x);
    all = ~__reduce_or_sync(kFull, x.y);
  }
  int bit = 31 - __clz(any ^ all);  // (-1: all the same)
  uint32_t cut = bit < 0 ? all : all & ~((2u << bit) - 1u);
  for (; bit >= 0; --bit) {
    const uint32_t next = cut | 1u << bit;
    uint32_t part[4] = {0, 0, 0, 0};
    each([&](int) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i) part[i & 3] += k[i] >= next;
    });
    uint32_t n = __reduce_add_sync(kFull, (part[0] + part[1]) + (part[2] + part[3]));
    if (ch.warps > 1) n = __reduce_add_sync(kFull, ch.pass_round(n, 0).x);
    if ((int)n >= need) cut = next;
    if ((int)n == need) break;
  }
  // those above the cut, and of those at it the first ones
  uint32_t above = 0, equal = 0;
  each([&](int) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) above += k[i] > cut, equal += k[i] == cut;
  });
  uint32_t before = 0, tied = 0, all_above = __reduce_add_sync(kFull, above);
  if (ch.warps > 1) {
    const uint2 x = ch.pass_round(all_above, __reduce_add_sync(kFull, equal));
    all_above = __reduce_add_sync(kFull, x.x);
    before = __reduce_add_sync(kFull, lane < ch.w ? x.x : 0);
    tied = __reduce_add_sync(kFull, lane < ch.w ? x.y : 0);
  }
  const int ties = need - (int)all_above;
  each([&](int c) {
    if (!held) {
      above = equal = 0;
#pragma unroll
      for (int i = 0; i < kOwn; ++i) above += k[i] > cut, equal += k[i] == cut;
    }
    uint32_t a = above, e = equal;  // up to and with this lane
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(kFull, a, o), y = __shfl_up_sync(kFull, e, o);
      if (lane >= o) a += x, e += y;
    }
    const uint32_t sum_a = __shfl_sync(kFull, a, 31), sum_e = __shfl_sync(kFull, e, 31);
    int eq = (int)(tied + e - equal), out = first + (int)(before + a - above) + min(eq, ties);
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const bool is = k[i] == cut;
      if (k[i] > cut || (is && eq < ties)) sel[out++] = c * kBlock + lane * kOwn + i;
      eq += is;
    }
    before += sum_a;
    tied += sum_e;
  });
}

// The product's second operand of a pass: the nodes' q in whole numbers, as fp16
// pairs of max(x, 0) and of min(x, 0).
template <int D, int WARPS>
__device__ __forceinline__ void prepare_q(const uint16_t *q, long long tok, long long head, int nodes, int G, int gp, uint2 *s_q) {
  constexpr int kSteps = D / 8;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // A node's columns are some warps', which all look for its largest value.  (x in
  // units of 2^e is exact; + 1.5 2^23 rounds it to a whole number, ties to even.)
  int team = 1;
  while (team < WARPS && nodes * team * 2 <= WARPS) team <<= 1;
  const int part = warp & (team - 1);
  constexpr int kAtOnce = WARPS == 8 ? 8 : 4;  // columns in flight (8 of them made the one-group kernel spill)
  for (int node = warp / team; node < nodes; node += WARPS / team) {
    const uint16_t *row = q + node * tok + lane * 4;
    auto load_q = [&](int g) {  // four channels of a head; the first one's in place of those past the last
      return lane * 4 < D ? __ldg(reinterpret_cast<const uint2 *>(row + (g < G ? g : 0) * head)) : make_uint2(0, 0);
    };
    uint32_t m = 0;
    uint2 x[kAtOnce];
    for (int g = 0; g < gp; g += kAtOnce) {
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) x[i] = load_q(g + i);
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        m = max(m, max(max(x[i].x & 0x7FFFu, x[i].x >> 16 & 0x7FFFu), max(x[i].y & 0x7FFFu, x[i].y >> 16 & 0x7FFFu)));
    }
    m = __reduce_max_sync(kFull, m);
    const bool fine = m < 0x7F80u;
    const float down = fine ? scale_down(exponent_of(__uint_as_float(m << 16))) : 0.0f;
    for (int g = 0; g < gp; g += kAtOnce) {
      if (gp > kAtOnce) {
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) x[i] = load_q(g + i);
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        if (g + i >= gp || (i & (team - 1)) != part) continue;
        const int c = node * gp + g + i;
        uint2 v = fine ? x[i] : make_uint2(0, 0);
        const uint32_t e[4] = {v.x << 16, v.x & 0xFFFF0000u, v.y << 16, v.y & 0xFFFF0000u};
        float f[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = __fmaf_rn(__uint_as_float(e[k]), down, 12582912.0f) - 12582912.0f;
        uint32_t w[2], up[2], lo[2];  // fp16 pairs of x, max(x, 0), min(x, 0)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[k]) : "f"(f[2 * k + 1]), "f"(f[2 * k]));
          asm("max.f16x2 %0, %1, %2;" : "=r"(up[k]) : "r"(w[k]), "r"(0u));
          asm("min.f16x2 %0, %1, %2;" : "=r"(lo[k]) : "r"(w[k]), "r"(0u));
        }
        if (lane * 4 < D) {
          // code positions byte .. byte + 3: word byte % 16 / 4 of what a lane reads of a chunk
          auto put = [&](int byte, const uint32_t(&y)[2]) {
            const int step = byte / 64 * 4 + byte % 16 / 4, to = (c & 7) * 4 + byte % 64 / 16;
            s_q[((c >> 3) * (kSteps / 2) + step / 2) * 64 + to * 2 + step % 2] = make_uint2(y[0], y[1]);
          };
          put(lane * 4, up);
          put(D + lane * 4, lo);
        }
      }
    }
  }
}

template <int D, bool MANY>
__global__ void __launch_bounds__(32 * kWarps<MANY>, MANY ? 1 : 4) select_kernel(const SelectParams p, const SelectPlan plan) {
  constexpr int kThreads = 32 * kWarps<MANY>;
  constexpr int kChunks = D / 32, kSteps = D / 8;  // 64-byte chunks of a page's 2 D codes, steps of 16 of them
  extern __shared__ __align__(16) uint32_t s_dyn[];
  __shared__ uint32_t s_box[kSelectWarps][2][kSelectWarps][2];
  __shared__ int s_max[kWarps<MANY>];
  // the product's second operand [group][pair of steps][lane][step], keys
  uint2 *s_q = reinterpret_cast<uint2 *>(s_dyn);
  uint32_t *s_keys = reinterpret_cast<uint32_t *>(s_q + plan.groups * kSteps * 32);
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quad = lane & 3, r0 = lane >> 2;
  const int cs = plan.cluster, rank = (int)cluster_rank(), h = blockIdx.x >> plan.shift, b = blockIdx.y;
  const int G = p.Hq / p.Hkv, gp = plan.gp;
  pdl_wait();
  // the sequence, its offsets within their bounds
  const int c0 = __ldg(p.cu + b), c1 = __ldg(p.cu + b + 1), raw = __ldg(p.ctx + b);
  int top = 0;
  for (int i = threadIdx.x; i <= b; i += kThreads) top = max(top, min(max(__ldg(p.cu + i), 0), p.N));
  top = __reduce_max_sync(kFull, top);
  if (lane == 0) s_max[warp] = top;
  __syncthreads();
  int a0 = 0;
#pragma unroll
  for (int w = 0; w < kWarps<MANY>; ++w) a0 = max(a0, s_max[w]);
  const int a1 = max(min(max(c1, 0), p.N), a0);
  const int n = min(a1 - a0, kAttnMaxNodes), ctx = min(max(raw, 0), p.table_cols * p.page_size);
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.status && (c0 != a0 || c1 != a1 || a1 - a0 > kAttnMaxNodes || raw != ctx))
    atomicOr(p.status, kBadIndex);
  const int P = (ctx + p.page_size - 1) / p.page_size;
  auto row_of = [&](int node) { return p.sel + ((long long)(a0 + node) * p.Hkv + h) * p.n_sel; };
  if (n == 0) return;
  if (P <= p.n_sel) {  // (the whole cluster)
    for (int node = rank + cs * blockIdx.z; node < n; node += cs * gridDim.z)
      for (int i = threadIdx.x; i < p.n_sel; i += kThreads) row_of(node)[i] = i < P ? i : -1;
    return;
  }
  const int lg = lane_shift(P), tiles = (P + 15) / 16, stride = cs * kWarps<MANY>;
  // nodes of a pass: as many as have a slot and columns
  auto node_of = [&](int c) { return c * plan.gp_inv >> 16; };
  const int pass = min(plan.slots * cs, node_of(plan.groups * 8));
  if (pass * (int)blockIdx.z >= n) return;  // (the whole cluster)
  cluster_begun();
  for (int n0 = pass * blockIdx.z; n0 < n; n0 += pass * gridDim.z) {
    const int nodes = min(pass, n - n0), groups = (nodes * gp + 7) / 8;
    int tile = rank * kWarps<MANY> + warp;
    if (tile < tiles) {  // the first pages come into L2 while q is made ready
      constexpr int kLines = 2 * D / 128;
      const int j = tile * 16 + lane / 2, line = lane % 2;
      if (j >= p.first && j < P - p.last && line < kLines) {
        const uint32_t id = (uint32_t)__ldg(p.table + (long long)b * p.ld_table + j);
        if (id < (uint32_t)p.index.pages)
          prefetch_l2(p.index.codes + h * p.index.codes_head + id * p.index.codes_page + line * 128);
      }
    }
    // q in whole numbers
    const int mine = (nodes - rank + cs - 1) >> plan.shift;  // nodes that this block chooses for
    const int block = 32 << lg, end = (P + block - 1) / block * block;
    for (int i = 0; i < mine; ++i)  // (keys past the last page)
      for (int j = tiles * 16 + threadIdx.x; j < end; j += kThreads) s_keys[i * plan.cols + key_at(j, lg)] = 0;
    prepare_q<D, kWarps<MANY>>(p.q.ptr + (long long)(a0 + n0) * p.q.tok + (long long)(h * G) * p.q.head, p.q.tok, p.q.head,
                               nodes, G, gp, s_q);
    __syncthreads();
    if (n0 == pass * (int)blockIdx.z) cluster_all_begun();
    // scores
    // (what follows is worked out anew in each pass: held through the other phases, it
    // made this one spill: a batch of 64 x 1024 pages 45 us instead of 33)
    int anew = 0;
    asm volatile("" : "+r"(anew));
    const int *table = p.table + (long long)(b + anew) * p.ld_table;
    const int8_t *codes = p.index.codes + (h + anew) * p.index.codes_head + quad * 16;
    const uint8_t *exps = p.index.exps + (h + anew);
    // This lane's two pages of a tile: their numbers (0 in place of one outside the
    // index), and for each whether it is a candidate (1) in the index (2).
    const uint32_t codes_page = (uint32_t)p.index.codes_page + anew, exps_page = (uint32_t)p.index.exps_page + anew;
    struct Pages {
      uint32_t id[2], kind[2];
    };
    bool outside = false;
    auto pages_of = [&](int t) {
      Pages x;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int j = t * 16 + r0 + 8 * i;
        const bool cand = j >= p.first && j < P - p.last;
        x.id[i] = cand ? (uint32_t)__ldg(table + j) : 0u;
        x.kind[i] = cand;
      }
      return x;
    };
    auto within = [&](Pages &x) {  // (once the numbers are there)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool in = x.id[i] < (uint32_t)p.index.pages;
        outside |= !in;
        x.id[i] = in ? x.id[i] : 0u;
        x.kind[i] |= in ? 2u : 0u;
      }
    };
    // where the codes of a page begin for this lane
    auto codes_at = [&](uint32_t id) {
      return reinterpret_cast<const uint4 *>(codes + (unsigned long long)id * codes_page);
    };
    auto code_of = [&](uint32_t id) { return (int)__ldg(exps + (unsigned long long)id * exps_page); };
    int code[2] = {0, 0};
    Pages now = {}, next = {};
    uint4 w[2][kChunks];
    if (tile < tiles) {
      now = pages_of(tile);
      if (tile + stride < tiles) next = pages_of(tile + stride);
      within(now);
      const uint4 *from[2] = {codes_at(now.id[0]), codes_at(now.id[1])};
#pragma unroll
      for (int k = 0; k < kChunks; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) w[i][k] = __ldg(from[i] + k * 4);
      code[0] = code_of(now.id[0]);
      code[1] = code_of(now.id[1]);
    }
    const uint4 *s_b = reinterpret_cast<const uint4 *>(s_q) + lane;  // two steps
    for (; tile < tiles; tile += stride) {
      const int code_now[2] = {code[0], code[1]};
      const uint32_t kind_now[2] = {now.kind[0], now.kind[1]};
      // a score, as its key, to the block that chooses for the node
      const uint32_t at = key_at(tile * 16 + r0, lg), at8 = lg == 3 ? 4 : 256;  // (eight pages on)
      auto put = [&](int node, bool second, float sum) {
        if (node >= nodes) return;
        const int code = second ? code_now[1] : code_now[0];
        const uint32_t kind = second ? kind_now[1] : kind_now[0], j = at + (second ? at8 : 0u);
        // 2^(code - 127 - 20): no score overflows, and 2^-147 is still a number of fp32, as are
        // its multiples; (+ 0: no zero below another one)
        float score = fmaf(sum, __uint_as_float(code > 20 ? (uint32_t)(code - 20) << 23 : 4u << code), 0.0f);
        if (code == 255) score = INFINITY;
        if (kind < 2) score = 0.0f;
        const uint32_t key = kind & 1 ? order_key(score) : 0u;
        st_cluster(smem_addr(s_keys + (node >> plan.shift) * plan.cols + j), node & (cs - 1), key);
      };
      // the largest of a node's columns, then its score
      float run[2];
      int node = 0, in_node = 0;  // of the next group of columns
      auto finish = [&](const float (&s)[4]) {
        if (gp == 1) {
#pragma unroll
          for (int i = 0; i < 4; ++i) put(node + quad * 2 + (i & 1), i >> 1, s[i]);
          node += 8;
          return;
        }
        float m[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          m[i] = fmaxf(s[2 * i], s[2 * i + 1]);
          if (gp >= 4) m[i] = fmaxf(m[i], __shfl_xor_sync(kFull, m[i], 1));
          if (gp >= 8) m[i] = fmaxf(m[i], __shfl_xor_sync(kFull, m[i], 2));
        }
        if (gp == 2) {
          put(node + quad, false, m[0]);
          put(node + quad, true, m[1]);
          node += 4;
          return;
        }
        // (a quad's lanes hold the same: one writes the first page's, one the second's)
        if (gp == 4) {
          put(node + (quad >> 1), quad & 1, quad & 1 ? m[1] : m[0]);
          node += 2;
          return;
        }
        if (MANY) {
#pragma unroll
          for (int i = 0; i < 2; ++i) run[i] = in_node == 0 ? m[i] : fmaxf(run[i], m[i]);
          in_node += 8;
          if (in_node < gp) return;
          in_node = 0;
          m[0] = run[0], m[1] = run[1];
        }
        if (quad < 2) put(node, quad, quad ? m[1] : m[0]);
        ++node;
      };
      const bool more = tile + stride < tiles;
      within(next);
      const uint4 *from[2] = {codes_at(next.id[0]), codes_at(next.id[1])};
      // codes converted as they are multiplied, the next tile's in their place: with
      // one group of columns in four sums, else for up to eight groups at once
      if constexpr (!MANY) {
        float v[4][4];
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
          const uint32_t w0[4] = {w[0][k].x, w[0][k].y, w[0][k].z, w[0][k].w};
          const uint32_t w1[4] = {w[1][k].x, w[1][k].y, w[1][k].z, w[1][k].w};
          const uint4 q[2] = {s_b[k * 64], s_b[k * 64 + 32]};
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            uint32_t a[4];
            bytes_to_half(w0[s], a[0], a[2]);
            bytes_to_half(w1[s], a[1], a[3]);
            const uint32_t b0 = s & 1 ? q[s / 2].z : q[s / 2].x, b1 = s & 1 ? q[s / 2].w : q[s / 2].y;
            if (k == 0) mma_f16_first(v[s], a[0], a[1], a[2], a[3], b0, b1);
            else mma_f16(v[s], a[0], a[1], a[2], a[3], b0, b1);
          }
          if (more) {
#pragma unroll
            for (int i = 0; i < 2; ++i) w[i][k] = __ldg(from[i] + k * 4);
          }
        }
        float sum[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = (v[0][i] + v[1][i]) + (v[2][i] + v[3][i]);
        finish(sum);
      } else {
        for (int g0 = 0; g0 < groups; g0 += kSelectGroups) {
          float v[kSelectGroups][4];
#pragma unroll
          for (int k = 0; k < kChunks; ++k) {
            const uint32_t w0[4] = {w[0][k].x, w[0][k].y, w[0][k].z, w[0][k].w};
            const uint32_t w1[4] = {w[1][k].x, w[1][k].y, w[1][k].z, w[1][k].w};
            uint32_t a[4][4];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              bytes_to_half(w0[s], a[s][0], a[s][2]);
              bytes_to_half(w1[s], a[s][1], a[s][3]);
            }
            if (more && g0 + kSelectGroups >= groups) {
#pragma unroll
              for (int i = 0; i < 2; ++i) w[i][k] = __ldg(from[i] + k * 4);
            }
#pragma unroll
            for (int g = 0; g < kSelectGroups; ++g) {
              if (g0 + g >= groups) break;
#pragma unroll
              for (int s = 0; s < 4; s += 2) {
                const uint4 q = s_b[((g0 + g) * (kSteps / 2) + k * 2 + s / 2) * 32];
                if (k == 0 && s == 0) mma_f16_first(v[g], a[s][0], a[s][1], a[s][2], a[s][3], q.x, q.y);
                else mma_f16(v[g], a[s][0], a[s][1], a[s][2], a[s][3], q.x, q.y);
                mma_f16(v[g], a[s + 1][0], a[s + 1][1], a[s + 1][2], a[s + 1][3], q.z, q.w);
              }
            }
            asm volatile("" ::: "memory");  // (one chunk's operands at a time in registers)
          }
#pragma unroll
          for (int g = 0; g < kSelectGroups; ++g) {
            if (g0 + g >= groups) break;
            finish(v[g]);
          }
        }
      }
      if (more) code[0] = code_of(next.id[0]), code[1] = code_of(next.id[1]);
      now = next;
      if (tile + 2 * stride < tiles) next = pages_of(tile + 2 * stride);
    }
    if (outside && p.status) atomicOr(p.status, kBadIndex);
    cluster_sync();
    // The choice: this block's nodes, some warps each -- as few as hold the keys in
    // registers, since their exchanges cost more than the counting.
    int wpn = 1;
    while (wpn < kWarps<MANY> && wpn * (32 << lg) < P) wpn <<= 1;
    while (wpn > 1 && mine * wpn > kWarps<MANY>) wpn >>= 1;
    const int crew = warp / wpn;
    Choice ch = {s_box[crew], warp - crew * wpn, wpn, 1 + crew, 0};
    for (int slot = crew; slot < mine; slot += kWarps<MANY> / wpn) {
      const int node = slot * cs + rank;
      const uint32_t *keys = s_keys + slot * plan.cols;
      if (lg == 3) choose<3>(keys, P, p.first, p.last, p.n_sel, row_of(n0 + node), ch);
      else choose<4>(keys, P, p.first, p.last, p.n_sel, row_of(n0 + node), ch);
    }
    if (n0 + pass * (int)gridDim.z < n) cluster_sync();  // (before the keys are written again)
  }
}

int select_cols(int table_cols) {
  const int block = 32 << lane_shift(table_cols);
  return (table_cols + block - 1) / block * block;
}

SelectPlan plan_select(const SelectParams &p, int sm_count) {
  SelectPlan s;
  const int G = p.Hq / p.Hkv;
  s.gp = G <= 2 ? G : G <= 4 ? 4 : (G + 7) / 8 * 8;
  // A group where an average sequence's nodes fit in it (a batch of 64 x 1024 pages 34
  // us, with the kernel of several groups 73), else eight.
  const long long columns = ((long long)p.N + p.B - 1) / p.B * s.gp;
  s.gp_inv = (65536 + s.gp - 1) / s.gp;
  s.groups = columns <= 8 ? 1 : kSelectGroups;
  if (s.groups < s.gp / 8) s.groups = s.gp / 8;
  s.cols = select_cols(p.table_cols);
  // blocks enough for every SM, as far as there are pages for their warps
  s.cluster = 1;
  s.shift = 0;
  while (s.cluster < kSelectMostCluster && (long long)p.B * p.Hkv * s.cluster < 2LL * sm_count &&
         s.cluster * 16 * (s.groups > 1 ? kWarps<true> : kWarps<false>) < p.table_cols)
    s.cluster *= 2, ++s.shift;
  // A sequence's passes beside one another, as far as there are SMs (to four times as
  // many blocks, of which those past a sequence's nodes end at once: 8 trees of 1 to 64
  // nodes 31.5 us, with twice as many 40.6, one after another 63); without room for two
  // the most columns in a pass instead (those that a sequence does not fill cost nothing,
  // another pass 4 us).
  const long long room = 4LL * sm_count / ((long long)p.B * p.Hkv * s.cluster);
  const int nodes = p.N < kAttnMaxNodes ? p.N : kAttnMaxNodes, pass = s.groups * 8 / s.gp, passes = (nodes + pass - 1) / pass;
  s.shares = room < 2 ? 1 : room < passes ? (int)room : passes;
  if (s.shares == 1 && s.groups > 1) {
    s.groups = (nodes * s.gp + 7) / 8;
    if (s.groups > kSelectMost) s.groups = kSelectMost;
    if (s.groups < 2) s.groups = 2;  // (the kernel of several)
  }
  const int most = (s.groups * 8 / s.gp + s.cluster - 1) / s.cluster;  // as many nodes as have columns
  s.slots = s.cols == 0 ? most : kSelectKeys / s.cols;
  s.slots = s.slots < 1 ? 1 : s.slots > most ? most : s.slots;
  return s;
}

template <int D, bool MANY>
cudaError_t launch_select(const SelectParams &p, const SelectPlan &plan, cudaStream_t stream) {
  auto kern = select_kernel<D, MANY>;
  constexpr int kMost = kSelectMost * (D / 8) * 256 + kAttnMaxScored * 4;  // with the most keys
  static_assert(kMost <= 225 * 1024, "shared memory");
  const size_t smem = (size_t)plan.groups * (D / 8) * 256 + (size_t)plan.slots * plan.cols * 4;
  static DeviceOnce once;
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!once.done(dev)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
    once.set(dev);
  }
  cudaLaunchConfig_t cfg =
      pdl_config(dim3((unsigned)(plan.cluster * p.Hkv), (unsigned)p.B, (unsigned)plan.shares), dim3(32 * kWarps<MANY>), smem, stream);
  cudaLaunchAttribute attr[2];
  attach_pdl(cfg, attr);
  attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
  attr[cfg.numAttrs].val.clusterDim = {(unsigned)plan.cluster, 1, 1};
  cfg.attrs = attr;
  ++cfg.numAttrs;
  return cudaLaunchKernelEx(&cfg, kern, p, plan);
}

}  // namespace

cudaError_t launch_kv_index(const IndexParams &p, int sm_count, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)(2 * sm_count)), dim3(kIndexThreads), 0, stream);
  cudaLaunchAttribute attr[1];
  attach_pdl(cfg, attr);
  return p.D == 64 ? cudaLaunchKernelEx(&cfg, index_kernel<64>, p) : cudaLaunchKernelEx(&cfg, index_kernel<128>, p);
}

cudaError_t launch_attn_select(const SelectParams &p, int sm_count, cudaStream_t stream) {
  const SelectPlan plan = plan_select(p, sm_count);
  if (plan.groups > 1)
    return p.D == 64 ? launch_select<64, true>(p, plan, stream) : launch_select<128, true>(p, plan, stream);
  return p.D == 64 ? launch_select<64, false>(p, plan, stream) : launch_select<128, false>(p, plan, stream);
}

}  // namespace mxg
