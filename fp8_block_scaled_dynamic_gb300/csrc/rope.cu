// rope.cu -- what happens to q, k and v around the cache: the norm and
// rotation of query and key heads (qk_norm_rope) and the copy of accepted
// tokens into the cache pages (kv_append).
#include <cstdint>
#include <cuda_runtime.h>

#include "attn.h"
#include "kernels.h"
#include "ptx.cuh"

namespace mxg {
namespace {

constexpr int kBadIndex = 0x2;  // MXG_DEV_BAD_INDEX

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ void unpack8(const uint4 &w, float (&x)[8]) {
  x[0] = lo_f(w.x), x[1] = hi_f(w.x), x[2] = lo_f(w.y), x[3] = hi_f(w.y);
  x[4] = lo_f(w.z), x[5] = hi_f(w.z), x[6] = lo_f(w.w), x[7] = hi_f(w.w);
}

// ------------------------------------------------------------ qk_norm_rope
// y = x * rsqrt(mean x^2 + eps) * w, then the rotation of the first rot
// channels: every value is read once and written once, so HBM bounds a long
// prompt and latency a decode step.  A head takes L lanes of 8 channels (one
// 16-byte load each): the mean is a butterfly over them, the rotation partner
// of a half-split pair is a shuffle away.  A CTA works on one token, so each
// thread loads its 16 cosines and sines once and reuses them for every head it
// takes; the loads of kU heads go out before the first is used.
constexpr int kRopeThreads = 256;
constexpr int kU = 3;

template <int L, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
  constexpr unsigned kFull = 0xFFFFFFFFu;
  constexpr int kGroups = kRopeThreads / L;
  pdl_trigger();
  const int t = blockIdx.x;
  const int c = threadIdx.x % L, g = threadIdx.x / L;
  const bool in = c * 8 < p.D;
  const int heads = p.Hq + p.Hkv + (p.v.ptr ? p.Hkv : 0);
  const int step = gridDim.y * kGroups;
  pdl_wait();

  // the cache place of this token; an out-of-range slot is not written
  uint16_t *kc = nullptr, *vc = nullptr;
  if (p.cache.k) {
    const long long s = p.slots[t];
    if (s >= 0) {
      const long long pg = s / p.cache.page_size;
      if (pg < p.cache.pages) {
        const long long at = pg * p.cache.page + (s - pg * p.cache.page_size) * p.cache.slot;
        kc = p.cache.k + at;
        vc = p.cache.v + at;
      } else if (p.status && threadIdx.x == 0) {
        atomicOr(p.status, kBadIndex);
      }
    }
  }
  // this lane's cosines and sines (8 of each, or the 4 of its own pairs)
  constexpr int kA = INTER ? 4 : 8;
  float cs[kA], sn[kA];
  bool bad = false;
  const int half = p.rot >> 1;
  const int hc = p.rot >> 4;  // 8-channel chunks in a half
  const bool turned = c * 8 < p.rot;
  if (p.rot > 0) {
    const int pos = p.pos[t];
    bad = pos < 0 || pos >= p.max_pos;
    if (bad && p.status && threadIdx.x == 0) atomicOr(p.status, kBadIndex);
    if (turned && !bad) {
      const float *row = p.cos_sin + (size_t)pos * p.rot;
      const int a = INTER ? c * 4 : (c < hc ? c : c - hc) * 8;
#pragma unroll
      for (int j = 0; j < kA; j += 4) {
        const float4 x = __ldg(reinterpret_cast<const float4 *>(row + a + j));
        const float4 y = __ldg(reinterpret_cast<const float4 *>(row + half + a + j));
        cs[j] = x.x, cs[j + 1] = x.y, cs[j + 2] = x.z, cs[j + 3] = x.w;
        sn[j] = y.x, sn[j + 1] = y.y, sn[j + 2] = y.z, sn[j + 3] = y.w;
      }
      if (!INTER && c < hc) {
#pragma unroll
        for (int j = 0; j < kA; ++j) sn[j] = -sn[j];  // the lower half subtracts
      }
    }
  }
  const int partner = !turned ? c : c < hc ? c + hc : c - hc;
  const uint4 one = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
  uint4 wq = one, wk = one;
  if (in && p.wq) wq = __ldg(reinterpret_cast<const uint4 *>(p.wq) + c);
  if (in && p.wk) wk = __ldg(reinterpret_cast<const uint4 *>(p.wk) + c);

  // every lane of a warp takes the same number of turns (the shuffles need it)
  for (int h0 = blockIdx.y * kGroups; h0 < heads; h0 += kU * step) {
    uint4 x[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int h = h0 + u * step + g;
      x[u] = make_uint4(0, 0, 0, 0);
      if (in && h < heads) {
        const uint16_t *src = h < p.Hq          ? p.q.ptr + t * p.q.tok + h * p.q.head
                              : h < p.Hq + p.Hkv ? p.k.ptr + t * p.k.tok + (h - p.Hq) * p.k.head
                                                 : p.v.ptr + t * p.v.tok + (h - p.Hq - p.Hkv) * p.v.head;
        x[u] = *reinterpret_cast<const uint4 *>(src + c * 8);
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (h0 + u * step >= heads) break;  // uniform over the CTA
      const int h = h0 + u * step + g;
      const bool is_q = h < p.Hq;
      float y[8], w[8];
      unpack8(x[u], y);
      if (is_q ? p.wq != nullptr : p.wk != nullptr) unpack8(is_q ? wq : wk, w);
      else
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = 1.0f;
      float ss = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(y[j], y[j], ss);
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o, L);
      const bool norm = is_q ? p.wq != nullptr : p.wk != nullptr;
      const float r = norm ? rsqrtf(ss / (float)p.D + p.eps) : 1.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = y[j] * r * w[j];
      float z[8];
      if (INTER) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          z[2 * j] = turned ? y[2 * j] * cs[j] - y[2 * j + 1] * sn[j] : y[2 * j];
          z[2 * j + 1] = turned ? y[2 * j + 1] * cs[j] + y[2 * j] * sn[j] : y[2 * j + 1];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float o = __shfl_sync(kFull, y[j], partner, L);
          z[j] = turned ? fmaf(y[j], cs[j % kA], o * sn[j % kA]) : y[j];
        }
      }
      uint4 out = make_uint4(pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3]), pack_bf16x2(z[4], z[5]),
                             pack_bf16x2(z[6], z[7]));
      if (bad) out = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
      if (!in || h >= heads) continue;
      if (is_q) {
        *reinterpret_cast<uint4 *>(p.q_out.ptr + t * p.q_out.tok + h * p.q_out.head + c * 8) = out;
      } else if (h < p.Hq + p.Hkv) {
        const int hk = h - p.Hq;
        if (p.k_out.ptr)
          *reinterpret_cast<uint4 *>(p.k_out.ptr + t * p.k_out.tok + hk * p.k_out.head + c * 8) = out;
        if (kc) *reinterpret_cast<uint4 *>(kc + hk * p.cache.head + c * 8) = out;
      } else if (vc) {
        *reinterpret_cast<uint4 *>(vc + (h - p.Hq - p.Hkv) * p.cache.head + c * 8) = x[u];
      }
    }
  }
}

template <int L>
cudaError_t rope_launch(const RopeParams &p, bool inter, int sm_count, cudaStream_t stream) {
  // few tokens: a token's heads go to several CTAs, so that about two CTAs per
  // SM share the work of a decode step
  const int groups = kRopeThreads / L;
  const int heads = p.Hq + p.Hkv + (p.v.ptr ? p.Hkv : 0);
  const int most = (heads + groups - 1) / groups;
  int split = (2 * sm_count + p.T - 1) / p.T;
  split = split < 1 ? 1 : split > most ? most : split;
  cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)p.T, (unsigned)split), dim3(kRopeThreads), 0, stream);
  cudaLaunchAttribute attr[1];
  attach_pdl(cfg, attr);
  return inter ? cudaLaunchKernelEx(&cfg, rope_kernel<L, true>, p)
               : cudaLaunchKernelEx(&cfg, rope_kernel<L, false>, p);
}

// --------------------------------------------------------------- kv_append
// A copy of (accepted rows) x (heads) x (k, v) in each layer: HBM bounds a
// large batch, latency a step.  One CTA per (sequence, layer): its threads
// work out where up to kRows accepted rows come from and go to, then copy them
// as 16-byte units.
constexpr int kAppendThreads = 256;
constexpr int kRows = 64;

__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams p) {
  __shared__ long long s_dst[kRows];
  __shared__ int s_src[kRows], s_end[2];
  pdl_trigger();
  const int b = blockIdx.x, layer = blockIdx.y;
  pdl_wait();
  const int ctx = p.ctx[b];
  // the sequence's rows, clamped to the tensor
  int n0 = p.cu[b], n1 = p.cu[b + 1];
  n0 = min(max(n0, 0), p.N);
  n1 = min(max(n1, n0), p.N);
  const int *acc = p.accept + (size_t)b * p.ld_accept;
  const int unit = p.D / 8, per_row = p.Hkv * unit;
  int done = 0;
  bool more = true;
  while (more && done < p.max_accept) {
    const int n = min(kRows, p.max_accept - done);
    bool bad = false;
    if (threadIdx.x < kRows) {
      const int i = threadIdx.x;
      const int a = i < n ? acc[done + i] : -1;
      const unsigned neg = __ballot_sync(0xFFFFFFFFu, a < 0);
      if ((i & 31) == 0) s_end[i >> 5] = neg ? __ffs(neg) - 1 : 32;
      long long dst = -1;
      if (a >= 0) {
        const long long at = (long long)ctx + done + i;
        const long long col = at / p.cache.page_size;
        bad = a >= n1 - n0 || ctx < 0 || col >= p.table_cols;
        if (!bad) {
          const int pg = p.table[(size_t)b * p.ld_table + col];
          bad = pg < 0 || pg >= p.cache.pages;
          if (!bad) dst = pg * p.cache.page + (at - col * p.cache.page_size) * p.cache.slot;
        }
      }
      s_src[i] = n0 + a;
      s_dst[i] = dst;
    }
    __syncthreads();
    const int rows = s_end[0] < 32 ? s_end[0] : 32 + s_end[1];
    more = rows == kRows;
    // (a bad entry past the end of the list is nobody's)
    if (bad && (int)threadIdx.x < rows && p.status && layer == 0) atomicOr(p.status, kBadIndex);
    const int units = rows * per_row;
    for (int u = threadIdx.x; u < units; u += kAppendThreads) {
      const int i = u / per_row, r = u - i * per_row;
      const int h = r / unit, c = r - h * unit;
      if (s_dst[i] < 0) continue;
      const long long at = layer * p.cache.layer + s_dst[i] + h * p.cache.head + c * 8;
      const uint4 kv = *reinterpret_cast<const uint4 *>(p.k.ptr + layer * p.k_layer + s_src[i] * p.k.tok +
                                                        h * p.k.head + c * 8);
      const uint4 vv = *reinterpret_cast<const uint4 *>(p.v.ptr + layer * p.v_layer + s_src[i] * p.v.tok +
                                                        h * p.v.head + c * 8);
      *reinterpret_cast<uint4 *>(p.cache.k + at) = kv;
      *reinterpret_cast<uint4 *>(p.cache.v + at) = vv;
    }
    done += rows;
    __syncthreads();
  }
  if (layer == 0 && threadIdx.x == 0 && p.ctx_out) p.ctx_out[b] = ctx + done;
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeParams &p, bool interleaved, int sm_count, cudaStream_t stream) {
  const int chunks = p.D / 8;
  if (chunks <= 2) return rope_launch<2>(p, interleaved, sm_count, stream);
  if (chunks <= 4) return rope_launch<4>(p, interleaved, sm_count, stream);
  if (chunks <= 8) return rope_launch<8>(p, interleaved, sm_count, stream);
  if (chunks <= 16) return rope_launch<16>(p, interleaved, sm_count, stream);
  return rope_launch<32>(p, interleaved, sm_count, stream);
}

cudaError_t launch_kv_append(const AppendParams &p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg =
      pdl_config(dim3((unsigned)p.B, (unsigned)p.cache.layers), dim3(kAppendThreads), 0, stream);
  cudaLaunchAttribute attr[1];
  attach_pdl(cfg, attr);
  return cudaLaunchKernelEx(&cfg, append_kernel, p);
}

}  // namespace mxg
