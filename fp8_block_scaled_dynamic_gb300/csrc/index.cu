// index.cu -- bounds of the keys of full cache pages (kv_index) and the choice
// of pages by them (attn_select).
//
// A page's bounds of a kv head: with 2^e the least power of two, e >= -100, for
// which max |k| <= 127 * 2^e over the page's keys, upper[d] = ceil(max k[d] / 2^e)
// and lower[d] = floor(min k[d] / 2^e), whole numbers of 8 bits.  For every key of
// the page then q . k <= sum_d q[d] (q[d] > 0 ? upper[d] : lower[d]) 2^e, and with q
// in whole numbers too that sum is a whole number below 2^21: every step is exact,
// so the choice does not depend on an order of summation.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <climits>
#include <cstdint>

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
  const int steps = p.cache.page_size / R;  // (a multiple of 4)
  for (int t = 0; t < steps; t += 4) {
    uint4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      x[u] = __ldg(reinterpret_cast<const uint4 *>(k + (long long)((t + u) * R + sub) * p.cache.slot));
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      hi[0] = max2(hi[0], x[u].x), lo[0] = min2(lo[0], x[u].x);
      hi[1] = max2(hi[1], x[u].y), lo[1] = min2(lo[1], x[u].y);
      hi[2] = max2(hi[2], x[u].z), lo[2] = min2(lo[2], x[u].z);
      hi[3] = max2(hi[3], x[u].w), lo[3] = min2(lo[3], x[u].w);
    }
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
__global__ void __launch_bounds__(kIndexThreads) index_kernel(const IndexParams p) {
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
// exactly.  (A page's codes are read straight into the order in which the product
// wants them: which 16 of the 2 D positions a step takes does not matter as long as
// both operands agree.)  A score goes, as a 32-bit key of the same order, to the
// shared memory of the block that chooses for its node; then the warps of a node
// find the key of the last page that is taken, bit by bit from the top, and write
// the pages out in order.
constexpr int kSelectThreads = 256, kSelectWarps = kSelectThreads / 32;
constexpr int kSelectGroups = 8;       // of eight columns (query heads) in a pass, or one node's
constexpr int kSelectKeys = 16 * 1024; // keys of a block in shared memory, where one node's are no more
constexpr int kSelectMostKeys = 38 * 1024;  // beyond that they are in the workspace
constexpr int kSelectMostCluster = 8;

struct SelectPlan {
  int cluster;   // blocks of a sequence and kv head
  int cols;      // keys of a node: the table's columns, rounded up to 128
  int slots;     // nodes that a block chooses for in a pass
  int gp;        // columns of a node: Hq / Hkv rounded up to 1, 2, 4 or a multiple of 8
  int groups;    // of eight columns in a pass
  bool spill;    // keys in the workspace
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
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

// The choice for one node by `warps` warps (this one is the w-th) of a named
// barrier: candidates are the pages with a key above 0.
struct Choice {
  uint32_t (*box)[kSelectWarps][2];  // two of them, in turn
  int w, warps, bar, turn;
  // both sums over the warps, and over those before this one
  __device__ __forceinline__ void sums(int &a, int &b, int &a_before, int &b_before) {
    a = __reduce_add_sync(kFull, a);
    b = __reduce_add_sync(kFull, b);
    a_before = b_before = 0;
    if (warps == 1) return;
    if ((threadIdx.x & 31) == 0) box[turn][w][0] = a, box[turn][w][1] = b;
    named_sync(bar, warps * 32);
    int x = 0, y = 0;
    for (int i = 0; i < warps; ++i) {
      if (i == w) a_before = x, b_before = y;
      x += box[turn][i][0];
      y += box[turn][i][1];
    }
    a = x;
    b = y;
    turn ^= 1;
  }
};
__device__ __forceinline__ void choose(const uint32_t *keys, int P, int first, int last, int n_sel, int *sel, Choice &ch) {
  const int lane = threadIdx.x & 31, need = n_sel - first - last;
  const int chunks = (P + 127) / 128, per = (chunks + ch.warps - 1) / ch.warps;
  const int c0 = min(ch.w * per, chunks), c1 = min(c0 + per, chunks);
  auto at = [&](int c) { return *reinterpret_cast<const uint4 *>(keys + c * 128 + lane * 4); };
  for (int i = ch.w * 32 + lane; i < first + last; i += ch.warps * 32) {
    const int x = i < first ? i : n_sel - last + i - first;
    sel[x] = i < first ? i : P - last + i - first;
  }
  uint32_t cut = 1;
  int dummy = 0, b0, b1;
  if (need > 0) {
    // bits that all candidates have in common need no search
    uint32_t any = 0, all = ~0u;
    for (int c = c0; c < c1; ++c) {
      const uint4 k = at(c);
      for (const uint32_t x : {k.x, k.y, k.z, k.w})
        if (x) any |= x, all &= x;
    }
    any = __reduce_or_sync(kFull, any);
    all = __reduce_and_sync(kFull, all);
    if (ch.warps > 1) {
      if (lane == 0) ch.box[ch.turn][ch.w][0] = any, ch.box[ch.turn][ch.w][1] = all;
      named_sync(ch.bar, ch.warps * 32);
      for (int i = 0; i < ch.warps; ++i) any |= ch.box[ch.turn][i][0], all &= ch.box[ch.turn][i][1];
      ch.turn ^= 1;
    }
    const uint32_t differ = any ^ all;
    int bit = 31 - __clz(differ);  // (-1: all the same)
    cut = bit < 0 ? all : all & ~((2u << bit) - 1u);
    for (; bit >= 0; --bit) {
      const uint32_t next = cut | 1u << bit;
      int n = 0;
      for (int c = c0; c < c1; ++c) {
        const uint4 k = at(c);
        n += (k.x >= next) + (k.y >= next) + (k.z >= next) + (k.w >= next);
      }
      dummy = 0;
      ch.sums(n, dummy, b0, b1);
      if (n >= need) cut = next;
      if (n == need) break;
    }
  }
  // those above the cut, and of those at it the first ones
  int above = 0, equal = 0, above_before, equal_before;
  for (int c = c0; c < c1; ++c) {
    const uint4 k = at(c);
    above += (k.x > cut) + (k.y > cut) + (k.z > cut) + (k.w > cut);
    equal += (k.x == cut) + (k.y == cut) + (k.z == cut) + (k.w == cut);
  }
  ch.sums(above, equal, above_before, equal_before);
  if (need <= 0) return;
  const int ties = need - above;
  const uint32_t below = (1u << lane) - 1u;
  int out = first + above_before + min(equal_before, ties), tied = equal_before;
  for (int c = c0; c < c1; ++c) {
    const uint4 k4 = at(c);
    const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
    uint32_t eq[4], take[4];
    int eq_mine = tied, eq_all = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      eq[e] = __ballot_sync(kFull, k[e] == cut);
      eq_mine += __popc(eq[e] & below);
      eq_all += __popc(eq[e]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool is = k[e] == cut;
      take[e] = __ballot_sync(kFull, k[e] > cut || (is && eq_mine < ties));
      eq_mine += is;
    }
    int to = out;
#pragma unroll
    for (int e = 0; e < 4; ++e) to += __popc(take[e] & below);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (take[e] >> lane & 1u) sel[to++] = c * 128 + lane * 4 + e;
      out += __popc(take[e]);
    }
    tied += eq_all;
  }
}

template <int D>
__global__ void __launch_bounds__(kSelectThreads, 2) select_kernel(const SelectParams p, const SelectPlan plan) {
  constexpr int kChunks = D / 32, kSteps = D / 8;  // 64-byte chunks of a page's 2 D codes, steps of 16 of them
  extern __shared__ __align__(16) uint32_t s_dyn[];
  __shared__ uint32_t s_top[kSelectGroups * 8];
  __shared__ uint32_t s_box[kSelectWarps][2][kSelectWarps][2];
  __shared__ int s_max[kSelectWarps];
  uint2 *s_q = reinterpret_cast<uint2 *>(s_dyn);  // [group][step][lane]: the product's second operand
  uint32_t *s_keys = s_dyn + plan.groups * kSteps * 64;  // [slot][page]
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quad = lane & 3;
  const int cs = plan.cluster, rank = (int)cluster_rank(), h = blockIdx.x / cs, b = blockIdx.y;
  const int G = p.Hq / p.Hkv, gp = plan.gp;
  pdl_wait();
  // the sequence, its offsets within their bounds
  int top = 0;
  for (int i = threadIdx.x; i <= b; i += kSelectThreads) top = max(top, min(max(__ldg(p.cu + i), 0), p.N));
  top = __reduce_max_sync(kFull, top);
  if (lane == 0) s_max[warp] = top;
  __syncthreads();
  int a0 = 0;
#pragma unroll
  for (int w = 0; w < kSelectWarps; ++w) a0 = max(a0, s_max[w]);
  const int c0 = __ldg(p.cu + b), c1 = __ldg(p.cu + b + 1), a1 = max(min(max(c1, 0), p.N), a0);
  const int n = min(a1 - a0, kAttnMaxNodes), raw = __ldg(p.ctx + b), ctx = min(max(raw, 0), p.table_cols * p.page_size);
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.status && (c0 != a0 || c1 != a1 || a1 - a0 > kAttnMaxNodes || raw != ctx))
    atomicOr(p.status, kBadIndex);
  const int P = (ctx + p.page_size - 1) / p.page_size;
  auto row_of = [&](int node) { return p.sel + ((long long)(a0 + node) * p.Hkv + h) * p.n_sel; };
  if (n == 0) return;
  if (P <= p.n_sel) {  // (the whole cluster)
    for (int node = rank; node < n; node += cs)
      for (int i = threadIdx.x; i < p.n_sel; i += kSelectThreads) row_of(node)[i] = i < P ? i : -1;
    return;
  }
  const int *table = p.table + (long long)b * p.ld_table;
  const int8_t *codes = p.index.codes + h * p.index.codes_head;
  const uint8_t *exps = p.index.exps + h;
  const int tiles = (P + 127) / 128 * 8, stride = cs * kSelectWarps;
  // nodes of a pass: as many as have a slot and columns
  const int pass = min(plan.slots * cs, plan.groups * 8 / gp);
  for (int n0 = 0; n0 < n; n0 += pass) {
    const int nodes = min(pass, n - n0), columns = nodes * gp, groups = (columns + 7) / 8;
    // q in whole numbers
    for (int i = threadIdx.x; i < nodes; i += kSelectThreads) s_top[i] = 0;
    __syncthreads();
    auto load_q = [&](int c, int &node) {  // four channels of a column
      node = c / gp;
      const int g = c - node * gp, head = h * G + (g < G ? g : 0);
      uint2 x = make_uint2(0, 0);
      if (lane * 4 < D && node < nodes)
        x = *reinterpret_cast<const uint2 *>(p.q.ptr + (long long)(a0 + n0 + node) * p.q.tok + head * p.q.head + lane * 4);
      return x;
    };
    for (int c = warp; c < columns; c += kSelectWarps) {
      int node;
      const uint2 x = load_q(c, node);
      uint32_t m = max(max(x.x & 0x7FFFu, x.x >> 16 & 0x7FFFu), max(x.y & 0x7FFFu, x.y >> 16 & 0x7FFFu));
      m = __reduce_max_sync(kFull, m);
      if (lane == 0) atomicMax(&s_top[node], m);
    }
    __syncthreads();
    for (int c = warp; c < groups * 8; c += kSelectWarps) {
      int node;
      const uint2 x = load_q(c, node);
      const uint32_t m = node < nodes ? s_top[node] : 0;
      const float down = m < 0x7F80u ? scale_down(exponent_of(__uint_as_float(m << 16))) : 0.0f;
      const uint32_t w[4] = {x.x << 16, x.x & 0xFFFF0000u, x.y << 16, x.y & 0xFFFF0000u};
      uint32_t up[2] = {0, 0}, lo[2] = {0, 0};  // fp16 pairs of max(x, 0), min(x, 0)
      if (m < 0x7F80u) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = rintf(__uint_as_float(w[i]) * down);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(up[i]) : "f"(fmaxf(v[2 * i + 1], 0.0f)), "f"(fmaxf(v[2 * i], 0.0f)));
          asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(lo[i]) : "f"(fminf(v[2 * i + 1], 0.0f)), "f"(fminf(v[2 * i], 0.0f)));
        }
      }
      if (lane * 4 < D) {
        auto put = [&](int byte, uint32_t h01, uint32_t h23) {  // code positions byte .. byte + 3
          const int step = byte / 64 * 4 + byte % 16 / 4, to = (c & 7) * 4 + byte % 64 / 16;
          s_q[((c >> 3) * kSteps + step) * 32 + to] = make_uint2(h01, h23);
        };
        put(lane * 4, up[0], up[1]);
        put(D + lane * 4, lo[0], lo[1]);
      }
    }
    __syncthreads();
    // scores
    auto page_at = [&](int tile, int r) {  // -2: no candidate, -1: outside the index
      const int j = tile * 16 + r;
      if (tile >= tiles || j < p.first || j >= P - p.last) return -2;
      const int pg = __ldg(table + j);
      return (uint32_t)pg < (uint32_t)p.index.pages ? pg : -1;
    };
    const int r0 = lane >> 2;
    int tile = rank * kSelectWarps + warp;
    int pg[2] = {page_at(tile, r0), page_at(tile, r0 + 8)};
    for (; tile < tiles; tile += stride) {
      uint4 x[2][kChunks];
      int code[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        code[i] = 0;
        if (pg[i] >= 0) code[i] = __ldg(exps + pg[i] * p.index.exps_page);
#pragma unroll
        for (int k = 0; k < kChunks; ++k)
          x[i][k] = pg[i] >= 0 ? __ldg(reinterpret_cast<const uint4 *>(codes + pg[i] * p.index.codes_page + k * 64 + quad * 16))
                               : make_uint4(0, 0, 0, 0);
      }
      if (p.status && (pg[0] == -1 || pg[1] == -1)) atomicOr(p.status, kBadIndex);
      const bool cand[2] = {pg[0] != -2, pg[1] != -2}, in[2] = {pg[0] >= 0, pg[1] >= 0};
      pg[0] = page_at(tile + stride, r0);
      pg[1] = page_at(tile + stride, r0 + 8);
      uint32_t a[kSteps][4];
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        const uint32_t w0[4] = {x[0][k].x, x[0][k].y, x[0][k].z, x[0][k].w};
        const uint32_t w1[4] = {x[1][k].x, x[1][k].y, x[1][k].z, x[1][k].w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          bytes_to_half(w0[w], a[k * 4 + w][0], a[k * 4 + w][2]);
          bytes_to_half(w1[w], a[k * 4 + w][1], a[k * 4 + w][3]);
        }
      }
      // 2^(code - 127 - 20): no score overflows
      const float up[2] = {__uint_as_float((uint32_t)max(code[0] - 20, 1) << 23),
                           __uint_as_float((uint32_t)max(code[1] - 20, 1) << 23)};
      auto put = [&](int node, int i, float s) {
        if (node >= nodes) return;
        const uint32_t key = !cand[i] ? 0u
                             : !in[i] ? order_key(0.0f)
                             : code[i] == 255 ? order_key(INFINITY)
                                              : order_key(s * up[i] + 0.0f);  // (no zero below another one)
        const int j = tile * 16 + r0 + 8 * i;
        if (plan.spill)
          reinterpret_cast<uint32_t *>(p.ws)[((long long)(a0 + n0 + node) * p.Hkv + h) * plan.cols + j] = key;
        else
          st_cluster(smem_addr(s_keys + (node / cs) * plan.cols + j), node % cs, key);
      };
      float run[2] = {-INFINITY, -INFINITY};
      for (int g = 0; g < groups; ++g) {
        float c[2][4] = {};
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          const uint2 q = s_q[(g * kSteps + s) * 32 + lane];
          mma_f16(c[s & 1], a[s], q.x, q.y);
        }
        const float v[4] = {c[0][0] + c[1][0], c[0][1] + c[1][1], c[0][2] + c[1][2], c[0][3] + c[1][3]};
        if (gp == 1) {
#pragma unroll
          for (int i = 0; i < 4; ++i) put(g * 8 + quad * 2 + (i & 1), i >> 1, v[i]);
          continue;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float m = fmaxf(v[2 * i], v[2 * i + 1]);
          if (gp >= 4) m = fmaxf(m, __shfl_xor_sync(kFull, m, 1));
          if (gp >= 8) m = fmaxf(m, __shfl_xor_sync(kFull, m, 2));
          if (gp <= 4) {
            if (quad % (gp / 2) == 0) put((g * 8 + quad * 2) / gp, i, m);
          } else {
            run[i] = fmaxf(run[i], m);
            if ((g + 1) * 8 % gp == 0) {
              if (quad == 0) put(g * 8 / gp, i, run[i]);
              run[i] = -INFINITY;
            }
          }
        }
      }
    }
    cluster_sync();
    // the choice: this block's nodes, some warps each
    const int mine = (nodes - rank + cs - 1) / cs;
    int wpn = kSelectWarps;
    while (wpn > 1 && mine * wpn > kSelectWarps) wpn >>= 1;
    const int team = warp / wpn;
    Choice ch = {s_box[team], warp - team * wpn, wpn, 1 + team, 0};
    for (int slot = team; slot < mine; slot += kSelectWarps / wpn) {
      const int node = slot * cs + rank;
      const uint32_t *keys = plan.spill ? reinterpret_cast<const uint32_t *>(p.ws) +
                                              ((long long)(a0 + n0 + node) * p.Hkv + h) * plan.cols
                                        : s_keys + slot * plan.cols;
      choose(keys, P, p.first, p.last, p.n_sel, row_of(n0 + node), ch);
    }
    if (n0 + pass < n) cluster_sync();  // (before the keys are written again)
  }
}

SelectPlan plan_select(const SelectParams &p, int sm_count) {
  SelectPlan s;
  const int G = p.Hq / p.Hkv;
  s.gp = G <= 2 ? G : G <= 4 ? 4 : (G + 7) / 8 * 8;
  s.groups = s.gp / 8 > kSelectGroups ? s.gp / 8 : kSelectGroups;
  s.cols = (p.table_cols + 127) / 128 * 128;
  s.spill = s.cols > kSelectMostKeys;
  // blocks enough for every SM, as far as there are pages for their warps
  s.cluster = 1;
  while (s.cluster < kSelectMostCluster && (long long)p.B * p.Hkv * s.cluster < 2LL * sm_count &&
         s.cluster * 16 * kSelectWarps < s.cols)
    s.cluster *= 2;
  s.slots = s.spill || s.cols == 0 ? kSelectWarps : kSelectKeys / s.cols;
  s.slots = s.slots < 1 ? 1 : s.slots > kSelectWarps ? kSelectWarps : s.slots;
  // (as many nodes as have columns)
  const int most = (s.groups * 8 / s.gp + s.cluster - 1) / s.cluster;
  if (s.slots > most) s.slots = most;
  return s;
}

template <int D>
cudaError_t launch_select(const SelectParams &p, int sm_count, cudaStream_t stream) {
  auto kern = select_kernel<D>;
  constexpr int kMost = 16 * (D / 8) * 256 + kSelectMostKeys * 4;  // 128 heads of a kv head, and the most keys
  static_assert(kMost <= 220 * 1024, "shared memory");
  const SelectPlan plan = plan_select(p, sm_count);
  const size_t smem = (size_t)plan.groups * (D / 8) * 256 + (plan.spill ? 0 : (size_t)plan.slots * plan.cols * 4);
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
      pdl_config(dim3((unsigned)(plan.cluster * p.Hkv), (unsigned)p.B), dim3(kSelectThreads), smem, stream);
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
  cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)(4 * sm_count)), dim3(kIndexThreads), 0, stream);
  cudaLaunchAttribute attr[1];
  attach_pdl(cfg, attr);
  return p.D == 64 ? cudaLaunchKernelEx(&cfg, index_kernel<64>, p) : cudaLaunchKernelEx(&cfg, index_kernel<128>, p);
}

cudaError_t launch_attn_select(const SelectParams &p, int sm_count, cudaStream_t stream) {
  return p.D == 64 ? launch_select<64>(p, sm_count, stream) : launch_select<128>(p, sm_count, stream);
}

size_t attn_select_ws_bytes(long long N, int Hkv, int table_cols) {
  const long long cols = ((long long)table_cols + 127) / 128 * 128;
  return cols > kSelectMostKeys ? (size_t)(N * Hkv * cols * 4) : 256;
}

}  // namespace mxg
