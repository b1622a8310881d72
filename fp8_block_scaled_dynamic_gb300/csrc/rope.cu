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
// prompt and latency a decode step.  A head takes L lanes of two 16-byte units
// each, and a lane's two units are each other's rotation partners (half-split:
// units c and c + rot/16; neighbouring pairs: two units in a row), so the
// rotation needs no exchange between lanes and the mean log2 L shuffles.  A
// CTA works on one token: each thread loads its 8 cosines and sines once for
// all the heads it takes, behind the loads of the first kU heads.
// 8192 tokens of 64 + 8 heads of 128, with the cache (353 MB): 57.4 us, 6.1
// TB/s of 6.8 measured for a copy.  Issue slots count beside the loads in
// flight: two-value arithmetic, and no bounds of a head's units where it fills
// its lanes (FULL), took 63.5 us to 59.3.  Threads of a CTA, heads in flight and
// CTAs per SM were swept: 64, 2, 14; 3 heads and 12 CTAs take 59.3 us, 1 and 18
// 60.8, 2 and 16 (fewer registers) 58.1; 32 threads 62.1, 128 threads 61.5.
constexpr int kRopeThreads = 64;
constexpr int kU = 2;

// Two fp32 operations in one instruction: s += a * b, a *= b, a -= b.
__device__ __forceinline__ void fma2(float &s0, float &s1, float a0, float a1, float b0, float b1) {
  asm("{\n\t.reg .b64 a, b, s;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 s, {%0, %1};\n\t"
      "fma.rn.f32x2 s, a, b, s;\n\tmov.b64 {%0, %1}, s;\n\t}"
      : "+f"(s0), "+f"(s1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void mul2(float &a0, float &a1, float b0, float b1) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
      "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1));
}
__device__ __forceinline__ void sub2(float &a0, float &a1, float b0, float b1) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
      "sub.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1));
}

template <int L, bool INTER, bool FULL>
__global__ void __launch_bounds__(kRopeThreads, 14) rope_kernel(const RopeParams p) {
  constexpr unsigned kFull = 0xFFFFFFFFu;
  constexpr int kGroups = kRopeThreads / L;
  pdl_trigger();
  const int t = blockIdx.x;
  const int c = threadIdx.x % L, g = threadIdx.x / L;
  const int units = p.D >> 3, hc = p.rot >> 4;
  // this lane's units of a head; past hc (half-split) they are not rotated
  const bool turned = INTER ? 16 * c < p.rot : c < hc;
  const int ua = INTER ? 2 * c : turned ? c : 2 * c, ub = INTER || !turned ? ua + 1 : c + hc;
  const bool ina = FULL || ua < units, inb = FULL || ub < units;
  const int heads_qk = p.Hq + p.Hkv, heads = heads_qk + (p.v.ptr ? p.Hkv : 0);
  const int step = gridDim.y * kGroups;
  pdl_wait();

  const int pos = p.rot > 0 ? __ldg(p.pos + t) : 0;
  const long long slot = p.cache.k ? __ldg(p.slots + t) : -1;
  const uint16_t *q = p.q.ptr + t * p.q.tok, *k = p.k.ptr + t * p.k.tok, *v = p.v.ptr + t * p.v.tok;
  uint4 xa[kU], xb[kU];
  auto load = [&](int h0) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int h = h0 + u * step + g;
      if (!FULL) xa[u] = xb[u] = make_uint4(0, 0, 0, 0);
      if (h < heads) {
        const uint16_t *src = h < p.Hq       ? q + h * p.q.head
                              : h < heads_qk ? k + (h - p.Hq) * p.k.head
                                             : v + (h - heads_qk) * p.v.head;
        if (ina) xa[u] = *reinterpret_cast<const uint4 *>(src + ua * 8);
        if (inb) xb[u] = *reinterpret_cast<const uint4 *>(src + ub * 8);
      }
    }
  };
  load(blockIdx.y * kGroups);

  // a position outside the table makes the token NaN
  const bool bad = p.rot > 0 && (pos < 0 || pos >= p.max_pos);
  float cs[8], sn[8];
  if (turned && !bad) {
    const float4 *row = reinterpret_cast<const float4 *>(p.cos_sin + (size_t)pos * p.rot) + c * 2;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 x = __ldg(row + i), y = __ldg(row + (p.rot >> 3) + i);
      cs[4 * i] = x.x, cs[4 * i + 1] = x.y, cs[4 * i + 2] = x.z, cs[4 * i + 3] = x.w;
      sn[4 * i] = y.x, sn[4 * i + 1] = y.y, sn[4 * i + 2] = y.z, sn[4 * i + 3] = y.w;
    }
  }
  // the cache place of this token; an out-of-range slot is not written
  long long at = -1;
  if (slot >= 0) {
    const long long pg = slot / p.cache.page_size;
    if (pg < p.cache.pages) at = pg * p.cache.page + (slot - pg * p.cache.page_size) * p.cache.slot;
  }
  if (threadIdx.x == 0 && p.status && (bad || (slot >= 0 && at < 0))) atomicOr(p.status, kBadIndex);
  const float inv_d = 1.0f / (float)p.D;

  // every lane of a warp takes the same number of turns (the shuffles need it)
  for (int h0 = blockIdx.y * kGroups; h0 < heads; h0 += kU * step) {
    if (h0 != blockIdx.y * kGroups) load(h0);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (h0 + u * step >= heads) break;  // uniform over the CTA
      const int h = h0 + u * step + g;
      const bool is_q = h < p.Hq;
      const uint16_t *gain = is_q ? p.wq : p.wk;  // (read again for each head: it is in L1, registers are short)
      uint4 wa = {}, wb = {};
      if (gain && ina) wa = __ldg(reinterpret_cast<const uint4 *>(gain) + ua);
      if (gain && inb) wb = __ldg(reinterpret_cast<const uint4 *>(gain) + ub);
      float a[8], b[8], w[8], ss = 0.0f;
      unpack8(xa[u], a);
      unpack8(xb[u], b);
      float s2 = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        fma2(ss, s2, a[j], a[j + 1], a[j], a[j + 1]);
        fma2(ss, s2, b[j], b[j + 1], b[j], b[j + 1]);
      }
      ss += s2;
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o, L);
      if (gain) {
        const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
        unpack8(wa, w);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          mul2(a[j], a[j + 1], r, r);
          mul2(a[j], a[j + 1], w[j], w[j + 1]);
        }
        unpack8(wb, w);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          mul2(b[j], b[j + 1], r, r);
          mul2(b[j], b[j + 1], w[j], w[j + 1]);
        }
      }
      if (turned) {
        if (INTER) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float x0 = a[2 * j], x1 = a[2 * j + 1], y0 = b[2 * j], y1 = b[2 * j + 1];
            a[2 * j] = x0 * cs[j] - x1 * sn[j];
            a[2 * j + 1] = x1 * cs[j] + x0 * sn[j];
            b[2 * j] = y0 * cs[4 + j] - y1 * sn[4 + j];
            b[2 * j + 1] = y1 * cs[4 + j] + y0 * sn[4 + j];
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            float x0 = a[j], x1 = a[j + 1], y0 = b[j], y1 = b[j + 1];
            mul2(a[j], a[j + 1], cs[j], cs[j + 1]);
            mul2(y0, y1, sn[j], sn[j + 1]);
            sub2(a[j], a[j + 1], y0, y1);
            mul2(b[j], b[j + 1], cs[j], cs[j + 1]);
            fma2(b[j], b[j + 1], x0, x1, sn[j], sn[j + 1]);
          }
        }
      }
      if (h >= heads) continue;
      uint4 ra = make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(a[4], a[5]),
                            pack_bf16x2(a[6], a[7]));
      uint4 rb = make_uint4(pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3]), pack_bf16x2(b[4], b[5]),
                            pack_bf16x2(b[6], b[7]));
      if (bad) ra = rb = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
      auto put = [&](uint16_t *dst, const uint4 &x, const uint4 &y) {
        if (ina) *reinterpret_cast<uint4 *>(dst + ua * 8) = x;
        if (inb) *reinterpret_cast<uint4 *>(dst + ub * 8) = y;
      };
      if (is_q) {
        put(p.q_out.ptr + t * p.q_out.tok + h * p.q_out.head, ra, rb);
      } else if (h < heads_qk) {
        const int hk = h - p.Hq;
        if (p.k_out.ptr) put(p.k_out.ptr + t * p.k_out.tok + hk * p.k_out.head, ra, rb);
        if (at >= 0) put(p.cache.k + at + hk * p.cache.head, ra, rb);
      } else if (at >= 0) {
        put(p.cache.v + at + (h - heads_qk) * p.cache.head, xa[u], xb[u]);
      }
    }
  }
}

template <int L>
cudaError_t rope_launch(const RopeParams &p, bool inter, int sm_count, cudaStream_t stream) {
  // few tokens: a token's heads go to several CTAs, so that about two CTAs per
  // SM share the work of a decode step (64 tokens of 64 + 8 heads: 3.2 us; one
  // CTA a token 6.2, one or four an SM 3.2)
  const int groups = kRopeThreads / L;
  const int heads = p.Hq + p.Hkv + (p.v.ptr ? p.Hkv : 0);
  const int most = (heads + groups - 1) / groups;
  int split = (2 * sm_count + p.T - 1) / p.T;
  split = split < 1 ? 1 : split > most ? most : split;
  cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)p.T, (unsigned)split), dim3(kRopeThreads), 0, stream);
  cudaLaunchAttribute attr[1];
  attach_pdl(cfg, attr);
  if (p.D == 16 * L)
    return inter ? cudaLaunchKernelEx(&cfg, rope_kernel<L, true, true>, p)
                 : cudaLaunchKernelEx(&cfg, rope_kernel<L, false, true>, p);
  return inter ? cudaLaunchKernelEx(&cfg, rope_kernel<L, true, false>, p)
               : cudaLaunchKernelEx(&cfg, rope_kernel<L, false, false>, p);
}

// --------------------------------------------------------------- kv_append
// A copy of (accepted rows) x (heads) x (k, v) in each layer: HBM bounds a
// large batch, latency a step.  One CTA per (sequence, layer): its threads
// work out where up to kRows accepted rows come from and go to, then copy them
// as 16-byte units, a thread the same place of every row it takes.
// 64 sequences of up to 8 rows x 32 layers (87 MB): 17.1 us, 5.1 TB/s (list,
// page and row are read one after another before the first row moves); a
// step's 5 layers 3.0 us, of which 2.5 are a launch (128 threads 3.6).
constexpr int kAppendThreads = 256;
constexpr int kRows = 64;

__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams p) {
  __shared__ long long s_dst[kRows];
  __shared__ int s_src[kRows], s_end[2];
  pdl_trigger();
  const int b = blockIdx.x, layer = blockIdx.y;
  const int unit = p.D / 8, per_row = p.Hkv * unit;
  // rows that are copied side by side, and this thread's place: row lane, head, 16-byte unit
  const int side = per_row < kAppendThreads ? kAppendThreads / per_row : 1;
  const int rl = per_row < kAppendThreads ? (int)threadIdx.x / per_row : 0, u0 = (int)threadIdx.x - rl * per_row;
  pdl_wait();
  const int ctx = __ldg(p.ctx + b), c0 = __ldg(p.cu + b), c1 = __ldg(p.cu + b + 1);
  // the sequence's rows, clamped to the tensor
  const int n0 = min(max(c0, 0), p.N), n1 = min(max(c1, n0), p.N);
  const int *acc = p.accept + (size_t)b * p.ld_accept;
  int done = 0;
  bool more = true;
  while (more && done < p.max_accept) {
    const int n = min(kRows, p.max_accept - done);
    bool refused = false;
    if (threadIdx.x < kRows) {
      const int i = threadIdx.x;
      const int a = i < n ? __ldg(acc + done + i) : -1;
      // (the page is read whatever the entry turns out to be)
      const long long at = (long long)ctx + done + i;
      const long long col = at / p.cache.page_size;
      const bool in = i < n && ctx >= 0 && col < p.table_cols;
      const int pg = in ? __ldg(p.table + (size_t)b * p.ld_table + col) : -1;
      refused = a >= 0 && (a >= n1 - n0 || pg < 0 || pg >= p.cache.pages);
      const unsigned stop = __ballot_sync(0xFFFFFFFFu, a < 0 || refused);
      if ((i & 31) == 0) s_end[i >> 5] = stop ? __ffs(stop) - 1 : 32;
      s_src[i] = n0 + a;
      s_dst[i] = pg * p.cache.page + (at - col * p.cache.page_size) * p.cache.slot;  // (used before the end alone)
    }
    __syncthreads();
    // The list ends at its first negative entry and at the first one that
    // cannot be written: a sequence never counts a token that is not there.
    const int rows = s_end[0] < 32 ? s_end[0] : 32 + s_end[1];
    more = rows == kRows;
    // (a bad entry past the end of the list is nobody's)
    if (refused && (int)threadIdx.x == rows && p.status && layer == 0) atomicOr(p.status, kBadIndex);
    for (int u = u0; u < per_row && rl < side; u += kAppendThreads) {
      const int h = u / unit, c = u - h * unit;
      const uint16_t *k = p.k.ptr + layer * p.k_layer + h * p.k.head + c * 8;
      const uint16_t *v = p.v.ptr + layer * p.v_layer + h * p.v.head + c * 8;
      const long long to = layer * p.cache.layer + h * p.cache.head + c * 8;
#pragma unroll 1  // (two rows at a time 18.3 us for the large batch)
      for (int i = rl; i < rows; i += side) {
        const long long dst = s_dst[i], src = s_src[i];
        const uint4 kv = *reinterpret_cast<const uint4 *>(k + src * p.k.tok);
        const uint4 vv = *reinterpret_cast<const uint4 *>(v + src * p.v.tok);
        *reinterpret_cast<uint4 *>(p.cache.k + dst + to) = kv;
        *reinterpret_cast<uint4 *>(p.cache.v + dst + to) = vv;
      }
    }
    done += rows;
    __syncthreads();
  }
  if (layer == 0 && threadIdx.x == 0 && p.ctx_out) p.ctx_out[b] = ctx + done;
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeParams &p, bool interleaved, int sm_count, cudaStream_t stream) {
  // lanes of a head: two units each; a half-split rotation pairs them first
  const int units = p.D / 8, pairs = p.rot / 16;
  const int lanes = pairs + (units - 2 * pairs + 1) / 2;
  if (lanes <= 1) return rope_launch<1>(p, interleaved, sm_count, stream);
  if (lanes <= 2) return rope_launch<2>(p, interleaved, sm_count, stream);
  if (lanes <= 4) return rope_launch<4>(p, interleaved, sm_count, stream);
  if (lanes <= 8) return rope_launch<8>(p, interleaved, sm_count, stream);
  return rope_launch<16>(p, interleaved, sm_count, stream);
}

cudaError_t launch_kv_append(const AppendParams &p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg =
      pdl_config(dim3((unsigned)p.B, (unsigned)p.cache.layers), dim3(kAppendThreads), 0, stream);
  cudaLaunchAttribute attr[1];
  attach_pdl(cfg, attr);
  return cudaLaunchKernelEx(&cfg, append_kernel, p);
}

}  // namespace mxg
