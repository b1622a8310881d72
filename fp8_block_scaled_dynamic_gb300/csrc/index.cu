// index.cu -- bounds of the keys of full cache pages (kv_index) and the choice
// of pages by them (attn_select).
//
// A page's bounds of a kv head: with 2^e the least power of two, e >= -100, for
// which max |k| <= 127 * 2^e over the page's keys, upper[d] = ceil(max k[d] / 2^e)
// and lower[d] = floor(min k[d] / 2^e), whole numbers of 8 bits.  For every key of
// the page then q . k <= sum_d max(q[d] upper[d], q[d] lower[d]) 2^e, and with q
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
constexpr int kSelectThreads = 256;

template <int D>
__global__ void __launch_bounds__(kSelectThreads) select_kernel(const SelectParams p) {
  __shared__ int s_seq[3];  // sequence's node count, logical pages, table row
  __shared__ int8_t s_q[128 * D];
  __shared__ float s_best[kSelectThreads / 32];
  __shared__ int s_at[kSelectThreads / 32];
  __shared__ int s_sel[kAttnMaxSelect];
  pdl_trigger();
  pdl_wait();
  const int node = blockIdx.x, h = blockIdx.y, G = p.Hq / p.Hkv, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    int running = 0, found = -1;
    bool bad = false;
    for (int b = 0; b < p.B; ++b) {
      const int c0 = p.cu[b], c1 = p.cu[b + 1], a0 = max(min(max(c0, 0), p.N), running);
      int a1 = max(min(max(c1, 0), p.N), a0);
      bad |= c0 != a0 || c1 != a1 || a1 - a0 > kAttnMaxNodes;
      a1 = min(a1, a0 + kAttnMaxNodes);
      running = a0;
      const int c = min(max(p.ctx[b], 0), p.table_cols * p.page_size);
      bad |= c != p.ctx[b];
      if (node >= a0 && node < a1) found = b;
    }
    if (bad && p.status) atomicOr(p.status, kBadIndex);
    s_seq[0] = found;
    s_seq[1] = found < 0 ? 0 : (min(max(p.ctx[found], 0), p.table_cols * p.page_size) + p.page_size - 1) / p.page_size;
    // whole numbers of q
    uint32_t top = 0;
    for (int g = 0; g < G; ++g)
      for (int d = 0; d < D; ++d)
        top = max(top, p.q.ptr[node * p.q.tok + (h * G + g) * p.q.head + d] & 0x7FFFu);
    const float down = top < 0x7F80u ? scale_down(exponent_of(__uint_as_float(top << 16))) : 0.0f;
    for (int g = 0; g < G; ++g)
      for (int d = 0; d < D; ++d) {
        const float x = __uint_as_float((uint32_t)p.q.ptr[node * p.q.tok + (h * G + g) * p.q.head + d] << 16);
        s_q[g * D + d] = top < 0x7F80u ? (int8_t)(int)rintf(x * down) : 0;
      }
  }
  __syncthreads();
  const int b = s_seq[0], P = s_seq[1];
  if (b < 0) return;
  int *sel = p.sel + ((long long)node * p.Hkv + h) * p.n_sel;
  float *score = p.ws + ((long long)node * p.Hkv + h) * p.table_cols;
  if (P <= p.n_sel) {
    for (int i = threadIdx.x; i < p.n_sel; i += kSelectThreads) sel[i] = i < P ? i : -1;
    return;
  }
  for (int j = threadIdx.x; j < P; j += kSelectThreads) {
    float s = INFINITY;
    if (j >= p.first && j < P - p.last) {
      const int page = p.table[(long long)b * p.ld_table + j];
      if ((uint32_t)page >= (uint32_t)p.index.pages) {
        if (p.status) atomicOr(p.status, kBadIndex);
        s = 0.0f;
      } else {
        const int8_t *c = p.index.codes + page * p.index.codes_page + h * p.index.codes_head;
        const int code = p.index.exps[page * p.index.exps_page + h];
        if (code < 255) {
          int best = INT_MIN;
          for (int g = 0; g < G; ++g) {
            int sum = 0;
            for (int d = 0; d < D; ++d) sum += max((int)s_q[g * D + d] * c[d], (int)s_q[g * D + d] * c[D + d]);
            best = max(best, sum);
          }
          s = (float)best * __uint_as_float((uint32_t)max(code - 20, 1) << 23);
        }
      }
    }
    score[j] = s;
  }
  __syncthreads();
  for (int n = 0; n < p.n_sel; ++n) {
    // the forced pages first, then the best of the others, the lowest among equals
    int at = INT_MAX;
    float best = -INFINITY;
    if (n < p.first) at = n;
    else if (n < p.first + p.last) at = P - p.last + n - p.first;
    else {
      for (int j = p.first + threadIdx.x; j < P - p.last; j += kSelectThreads)
        if (score[j] > best) best = score[j], at = j;
      for (int o = 16; o > 0; o >>= 1) {
        const float x = __shfl_xor_sync(kFull, best, o);
        const int y = __shfl_xor_sync(kFull, at, o);
        if (x > best || (x == best && y < at)) best = x, at = y;
      }
      if (lane == 0) s_best[warp] = best, s_at[warp] = at;
      __syncthreads();
      for (int w = 0; w < kSelectThreads / 32; ++w)
        if (s_best[w] > best || (s_best[w] == best && s_at[w] < at)) best = s_best[w], at = s_at[w];
      __syncthreads();
      if (threadIdx.x == 0) score[at] = -INFINITY;
    }
    if (threadIdx.x == 0) s_sel[n] = at;
    __syncthreads();
  }
  for (int i = threadIdx.x; i < p.n_sel; i += kSelectThreads) {
    int rank = 0;
    for (int n = 0; n < p.n_sel; ++n) rank += s_sel[n] < s_sel[i];
    sel[rank] = s_sel[i];
  }
}

}  // namespace

cudaError_t launch_kv_index(const IndexParams &p, int sm_count, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)(4 * sm_count)), dim3(kIndexThreads), 0, stream);
  cudaLaunchAttribute attr[1];
  attach_pdl(cfg, attr);
  return p.D == 64 ? cudaLaunchKernelEx(&cfg, index_kernel<64>, p) : cudaLaunchKernelEx(&cfg, index_kernel<128>, p);
}

cudaError_t launch_attn_select(const SelectParams &p, int, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)p.N, (unsigned)p.Hkv), dim3(kSelectThreads), 0, stream);
  cudaLaunchAttribute attr[1];
  attach_pdl(cfg, attr);
  return p.D == 64 ? cudaLaunchKernelEx(&cfg, select_kernel<64>, p) : cudaLaunchKernelEx(&cfg, select_kernel<128>, p);
}

size_t attn_select_ws_bytes(long long N, int Hkv, int table_cols) {
  const long long n = N * Hkv * (long long)table_cols * 4;
  return (size_t)(n < 256 ? 256 : n);
}

}  // namespace mxg
