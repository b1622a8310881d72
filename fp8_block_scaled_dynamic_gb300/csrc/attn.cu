// attn.cu -- attention of packed prompts and of drafted token trees.
#include <cstdint>
#include <cuda_runtime.h>

#include "attn.h"
#include "kernels.h"
#include "ptx.cuh"

namespace mxg {
namespace {

constexpr int kBadIndex = 0x2;  // MXG_DEV_BAD_INDEX

// One warp per (token, query head): the plainest right form.  The lanes hold
// D / 32 channels each; a key costs one warp sum.
template <int D, bool TREE>
__global__ void __launch_bounds__(128) attn_rows_kernel(const AttnParams p) {
  constexpr int E = D / 32;
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= (long long)p.T * p.Hq) return;
  const int t = (int)(row / p.Hq), h = (int)(row % p.Hq), hk = h / (p.Hq / p.Hkv);
  int b = -1, a0 = 0, a1 = 0;  // the sequence whose clamped range holds t
  for (int s = 0, prev = 0; s < p.B && b < 0; ++s) {
    const int x0 = max(min(max(p.cu[s], 0), p.T), prev), x1 = max(min(max(p.cu[s + 1], 0), p.T), x0);
    if (t >= x0 && t < x1) b = s, a0 = x0, a1 = x1;
    prev = x0;
  }
  if (b < 0) return;
  float q[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __uint_as_float((uint32_t)p.q.ptr[t * p.q.tok + h * p.q.head + lane * E + e] << 16) * p.scale;
    o[e] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  auto key = [&](const uint16_t *k, const uint16_t *v) {
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], k ? __uint_as_float((uint32_t)k[lane * E + e] << 16) : 0.0f, s);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
    const float mn = fmaxf(m, s);
    const float f = m == mn ? 1.0f : __expf(m - mn), w = __expf(s - mn);
    l = l * f + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + w * (v ? __uint_as_float((uint32_t)v[lane * E + e] << 16) : 0.0f);
    m = mn;
  };
  bool any = true;
  if (!TREE) {
    for (int j = a0; j <= t; ++j) key(p.k.ptr + j * p.k.tok + hk * p.k.head, p.v.ptr + j * p.v.tok + hk * p.v.head);
  } else {
    if (t - a0 >= kAttnMaxNodes) {
      if (p.status && lane == 0) atomicOr(p.status, kBadIndex);
      return;
    }
    const long long room = (long long)p.table_cols * p.cache.page_size;
    int ctx = p.ctx[b];
    if ((ctx < 0 || ctx > room) && p.status && lane == 0) atomicOr(p.status, kBadIndex);
    ctx = (int)min((long long)max(ctx, 0), room);
    for (int j = 0; j < ctx; ++j) {
      const int pg = p.table[(long long)b * p.ld_table + j / p.cache.page_size];
      const bool ok = pg >= 0 && pg < p.cache.pages;
      if (!ok && p.status && lane == 0) atomicOr(p.status, kBadIndex);
      const long long at = pg * p.cache.page + (j % p.cache.page_size) * p.cache.slot + hk * p.cache.head;
      key(ok ? p.cache.k + at : nullptr, ok ? p.cache.v + at : nullptr);
    }
    const int n = min(a1 - a0, kAttnMaxNodes);
    const unsigned long long word = p.mask[t] & (n >= 64 ? ~0ull : (1ull << n) - 1ull);
    for (int j = 0; j < n; ++j)
      if (word >> j & 1ull)
        key(p.k.ptr + (a0 + j) * p.k.tok + hk * p.k.head, p.v.ptr + (a0 + j) * p.v.tok + hk * p.v.head);
    any = ctx > 0 || word != 0ull;
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    p.out.ptr[t * p.out.tok + h * p.out.head + lane * E + e] =
        (uint16_t)(pack_bf16x2(any ? o[e] / l : 0.0f, 0.0f) & 0xFFFFu);
}

template <bool TREE>
cudaError_t launch_rows(const AttnParams &p, cudaStream_t stream) {
  const long long rows = (long long)p.T * p.Hq;
  cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, stream);
  cudaLaunchAttribute attr[1];
  attach_pdl(cfg, attr);
  return p.D == 64 ? cudaLaunchKernelEx(&cfg, attn_rows_kernel<64, TREE>, p)
                   : cudaLaunchKernelEx(&cfg, attn_rows_kernel<128, TREE>, p);
}

}  // namespace

cudaError_t launch_attn_prompt(const AttnParams &p, int, cudaStream_t stream) { return launch_rows<false>(p, stream); }
cudaError_t launch_attn_tree(const AttnParams &p, int, cudaStream_t stream) { return launch_rows<true>(p, stream); }
size_t attn_tree_ws_bytes(int, int) { return 256; }

}  // namespace mxg
