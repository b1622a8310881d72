// attn_long.cu -- attention of drafted trees whose sequences share a prefix by
// groups (attn_shared) and over selected pages (attn_sparse).
#include <cuda_runtime.h>
#include <cstdint>

#include "attn.h"
#include "attn_ptx.cuh"
#include "kernels.h"

namespace mxg {
namespace {

constexpr int kBadIndex = 0x2;  // MXG_DEV_BAD_INDEX
constexpr unsigned kFull = 0xFFFFFFFFu;

// One warp a node and query head, keys one after another with a running maximum.
template <int D>
__global__ void __launch_bounds__(32) simple_kernel(const AttnParams p, const int *groups, const int *prefix, int n_groups,
                                                    const int *sel, int n_sel) {
  constexpr int V = D / 32;
  const int node = blockIdx.x, head = blockIdx.y, hk = head / (p.Hq / p.Hkv), lane = threadIdx.x, page = p.cache.page_size;
  const int limit = p.table_cols * page;
  int running = 0, b = -1, a0 = 0, n = 0;
  bool bad = false;
  for (int i = 0; i < p.B; ++i) {
    const int c0 = p.cu[i], c1 = p.cu[i + 1], x0 = max(min(max(c0, 0), p.T), running);
    int x1 = max(min(max(c1, 0), p.T), x0);
    bad |= c0 != x0 || c1 != x1 || x1 - x0 > kAttnMaxNodes || p.ctx[i] < 0 || p.ctx[i] > limit;
    x1 = min(x1, x0 + kAttnMaxNodes);
    running = x0;
    if (node >= x0 && node < x1) b = i, a0 = x0, n = x1 - x0;
  }
  int shared = 0, first = b;
  running = 0;
  for (int g = 0; g < n_groups; ++g) {
    const int c0 = groups[g], c1 = groups[g + 1], g0 = max(min(max(c0, 0), p.B), running);
    const int g1 = max(min(max(c1, 0), p.B), g0);
    bad |= c0 != g0 || c1 != g1;
    running = g0;
    int least = limit;
    for (int i = g0; i < g1; ++i) least = min(least, min(max(p.ctx[i], 0), limit));
    const int len = min(max(prefix[g], 0), least) / page * page;
    bad |= len != prefix[g];
    if (b >= g0 && b < g1) shared = len, first = g0;
  }
  if (bad && p.status && lane == 0) atomicOr(p.status, kBadIndex);
  if (b < 0) return;
  const int ctx = min(max(p.ctx[b], 0), limit);
  float q[V], o[V] = {}, m = -INFINITY, l = 0.0f;
  bool any = false;
  auto value = [](uint16_t x) { return __uint_as_float((uint32_t)x << 16); };
  for (int i = 0; i < V; ++i) q[i] = value(p.q.ptr[node * p.q.tok + head * p.q.head + lane * V + i]);
  auto take = [&](const uint16_t *k, const uint16_t *v) {
    float s = 0.0f;
    for (int i = 0; i < V; ++i) s += q[i] * (k ? value(k[lane * V + i]) : 0.0f);
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(kFull, s, x);
    s *= p.scale * 1.4426950408889634f;
    any = true;
    const float mn = fmaxf(m, s), f = m == mn ? 1.0f : ex2(m - mn), w = ex2(s - mn);
    l = l * f + w;
    for (int i = 0; i < V; ++i) o[i] = o[i] * f + w * (v ? value(v[lane * V + i]) : 0.0f);
    m = mn;
  };
  auto take_page = [&](int row, int j, int n_tok) {
    const int pg = p.table[(long long)row * p.ld_table + j];
    const bool in = (uint32_t)pg < (uint32_t)p.cache.pages;
    if (!in && p.status && lane == 0) atomicOr(p.status, kBadIndex);
    for (int t = 0; t < n_tok; ++t) {
      const long long at = pg * p.cache.page + t * p.cache.slot + hk * p.cache.head;
      take(in ? p.cache.k + at : nullptr, in ? p.cache.v + at : nullptr);
    }
  };
  if (sel) {
    const int *mine = sel + ((long long)node * p.Hkv + hk) * n_sel;
    for (int i = 0; i < n_sel; ++i)
      if (mine[i] >= 0 && (long long)mine[i] * page >= ctx && p.status && lane == 0) atomicOr(p.status, kBadIndex);
    for (int j = 0; j * page < ctx; ++j) {
      bool named = false;
      for (int i = lane; i < n_sel; i += 32) named |= mine[i] == j;
      if (__any_sync(kFull, named)) take_page(b, j, min(page, ctx - j * page));
    }
  } else {
    for (int j = 0; j * page < ctx; ++j) take_page(j * page < shared ? first : b, j, min(page, ctx - j * page));
  }
  for (int i = 0; i < n; ++i)
    if (p.mask[node] >> i & 1ull)
      take(p.k.ptr + (a0 + i) * p.k.tok + hk * p.k.head, p.v.ptr + (a0 + i) * p.v.tok + hk * p.v.head);
  uint16_t *out = p.out.ptr + node * p.out.tok + head * p.out.head;
  for (int i = 0; i < V; ++i) out[lane * V + i] = any ? (uint16_t)pack_bf16x2(o[i] / l, 0.0f) : 0;
}

cudaError_t launch(const AttnParams &p, const int *groups, const int *prefix, int n_groups, const int *sel, int n_sel,
                   cudaStream_t stream) {
  const dim3 grid((unsigned)p.T, (unsigned)p.Hq);
  if (p.D == 64) simple_kernel<64><<<grid, 32, 0, stream>>>(p, groups, prefix, n_groups, sel, n_sel);
  else simple_kernel<128><<<grid, 32, 0, stream>>>(p, groups, prefix, n_groups, sel, n_sel);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_shared(const SharedParams &p, int, cudaStream_t stream) {
  return launch(p.a, p.groups, p.prefix, p.n_groups, nullptr, 0, stream);
}
size_t attn_shared_ws_bytes(long long, int, int, int) { return 256; }
cudaError_t launch_attn_sparse(const SparseParams &p, int, cudaStream_t stream) {
  return launch(p.a, nullptr, nullptr, 0, p.sel, p.n_sel, stream);
}
size_t attn_sparse_ws_bytes(long long, int, int, int, int) { return 256; }

}  // namespace mxg
