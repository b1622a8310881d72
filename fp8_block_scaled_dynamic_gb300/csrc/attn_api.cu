// attn_api.cu -- the C ABI declared in include/mxattn.h: argument and device
// checks and launches.  Every host-detectable error is returned before
// anything is launched.
#include <algorithm>
#include <array>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <utility>
#include <cuda.h>
#include <cuda_runtime.h>

#include "attn.h"
#include "mxattn.h"

static_assert(mxg::kAttnMaxSeqs == MXG_ATTN_MAX_SEQS && mxg::kAttnMaxNodes == MXG_ATTN_MAX_NODES &&
                  mxg::kAttnMaxSelect == MXG_ATTN_MAX_SELECT,
              "limits");

namespace {

// Current device must be compute capability 10.3; returns its SM count.
mxg_status device_sms(int *sm_count) {
  int dev = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sm_count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MXG_ERR_CUDA;
  return major == 10 && minor == 3 ? MXG_OK : MXG_ERR_UNSUPPORTED_DEVICE;
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool stride_ok(int64_t s) { return s >= 0 && s % 8 == 0 && s < (1LL << 38); }

mxg_status check_heads(const mxg_heads *h) {
  if (!h || !h->ptr || h->tok_stride < 0 || h->head_stride < 0) return MXG_ERR_INVALID_ARG;
  if (!aligned(h->ptr, 16) || !stride_ok(h->tok_stride) || !stride_ok(h->head_stride)) return MXG_ERR_MISALIGNED;
  return MXG_OK;
}

mxg_status check_cache(const mxg_kv_cache *c) {
  if (!c || !c->k || !c->v || c->layers < 1 || c->pages < 1 || c->layer_stride < 0 || c->page_stride < 0 ||
      c->slot_stride < 0 || c->head_stride < 0)
    return MXG_ERR_INVALID_ARG;
  const int s = c->page_size;
  if (s != 16 && s != 32 && s != 64 && s != 128 && s != 256) return MXG_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !stride_ok(c->layer_stride) || !stride_ok(c->page_stride) ||
      !stride_ok(c->slot_stride) || !stride_ok(c->head_stride))
    return MXG_ERR_MISALIGNED;
  return MXG_OK;
}

mxg::Heads heads(const mxg_heads *h) {
  mxg::Heads r = {};
  if (h) r = {static_cast<uint16_t *>(h->ptr), h->tok_stride, h->head_stride};
  return r;
}

mxg::Cache cache_of(const mxg_kv_cache *c) {
  mxg::Cache r = {};
  if (c)
    r = {static_cast<uint16_t *>(c->k), static_cast<uint16_t *>(c->v), c->layer_stride, c->page_stride,
         c->slot_stride, c->head_stride, c->layers, c->pages, c->page_size};
  return r;
}

// What attn_prompt and attn_tree check alike.
mxg_status check_attn(const mxg_heads *q, const mxg_heads *k, const mxg_heads *v, const int *cu, int B, int T,
                      int Hq, int Hkv, int D, float scale, const mxg_heads *out, const mxg_attn_opts *opts) {
  if (!cu || B < 1 || T < 0 || Hq < 1 || Hkv < 1 || !std::isfinite(scale) || !(scale > 0.0f)) return MXG_ERR_INVALID_ARG;
  if ((D != 64 && D != 128) || Hq % Hkv != 0 || Hq / Hkv > 128 || B > mxg::kAttnMaxSeqs)
    return MXG_ERR_UNSUPPORTED_SHAPE;
  if (opts && (opts->debug_stall < 0 || opts->debug_stall > 1)) return MXG_ERR_INVALID_ARG;
  if (!aligned(cu, 4) || (opts && opts->dev_status && !aligned(opts->dev_status, 4))) return MXG_ERR_MISALIGNED;
  if (T == 0) return MXG_OK;  // nothing to read: the tensors may be empty
  mxg_status st;
  for (const mxg_heads *h : {q, k, v, out})
    if ((st = check_heads(h)) != MXG_OK) return st;
  // (a tensor map has no stride of zero)
  if ((T > 1 && (!q->tok_stride || !k->tok_stride || !v->tok_stride || !out->tok_stride)) ||
      (Hq > 1 && (!q->head_stride || !out->head_stride)) || (Hkv > 1 && (!k->head_stride || !v->head_stride)))
    return MXG_ERR_UNSUPPORTED_SHAPE;
  return MXG_OK;
}

// What attn_tree, attn_shared and attn_sparse check alike of the cache side.
mxg_status check_paged(int N, const uint64_t *mask, const mxg_kv_cache *cache, const int *block_table, int ld_table,
                       int table_cols, const int *ctx_len, int Hkv) {
  if ((N > 0 && !mask) || !ctx_len || table_cols < 0 || ld_table < table_cols || (table_cols > 0 && !block_table))
    return MXG_ERR_INVALID_ARG;
  mxg_status st;
  if ((st = check_cache(cache)) != MXG_OK) return st;
  if (!cache->slot_stride || (cache->pages > 1 && !cache->page_stride) || (Hkv > 1 && !cache->head_stride))
    return MXG_ERR_UNSUPPORTED_SHAPE;
  if ((long long)table_cols * cache->page_size > 0x7fffff00LL) return MXG_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(mask, 8) || !aligned(ctx_len, 4) || !aligned(block_table, 4)) return MXG_ERR_MISALIGNED;
  return MXG_OK;
}

// Row groups x kv heads x key tiles, numbered in 32 bits; starts: row groups that
// begin anew, besides the full ones.  (Two a sequence for attn_shared and
// attn_sparse: a prefix's, or the smaller row groups of few rows, which hold an
// average sequence's nodes: full ones are then no more than the sequences.)
mxg_status check_units(int N, int Hq, int Hkv, long long starts, int table_cols, int page_size) {
  const int tq = 128 / (Hq / Hkv);
  const long long groups = N / (2 * tq) + starts;
  return groups * Hkv * ((long long)table_cols * page_size / 128 + 2) > 0x3fffffffLL || Hkv >= (1 << 16)
             ? MXG_ERR_UNSUPPORTED_SHAPE
             : MXG_OK;
}

mxg_status check_ws(const mxg_attn_opts *opts, size_t need) {
  if (!opts || !opts->workspace || need == 0 || opts->ws_bytes < need) return MXG_ERR_WORKSPACE;
  return aligned(opts->workspace, 256) ? MXG_OK : MXG_ERR_MISALIGNED;
}

// Bytes, a multiple of 16 of them, that no reachable entry's offset overflows.
bool bytes_ok(int64_t s) { return s >= 0 && s % 16 == 0 && s < (1LL << 38); }

mxg_status check_index(const mxg_page_index *x) {
  if (!x || !x->codes || !x->exps || x->layers < 1 || x->pages < 1 || x->codes_layer < 0 || x->codes_page < 0 ||
      x->codes_head < 0 || x->exps_layer < 0 || x->exps_page < 0)
    return MXG_ERR_INVALID_ARG;
  if (!aligned(x->codes, 16) || !bytes_ok(x->codes_layer) || !bytes_ok(x->codes_page) || !bytes_ok(x->codes_head) ||
      x->codes_page > INT32_MAX || x->exps_page > INT32_MAX ||
      x->exps_layer >= (1LL << 38) || x->exps_page >= (1LL << 38))
    return MXG_ERR_MISALIGNED;
  return MXG_OK;
}

// Entries of `bytes` in three dimensions of (stride, number), apart from one another: each
// dimension's stride spans the entries of those with smaller strides.
bool apart(std::array<std::pair<int64_t, int>, 3> dims, int64_t bytes) {
  std::sort(dims.begin(), dims.end());
  __int128 span = bytes;
  for (const auto &[stride, n] : dims) {
    if (n < 2) continue;
    if (stride < span) return false;
    span += (__int128)stride * (n - 1);
  }
  return true;
}

mxg::PageIndex index_of(const mxg_page_index *x) {
  return {x->codes,      x->exps,      x->codes_layer, x->codes_page, x->codes_head,
          x->exps_layer, x->exps_page, x->layers,      x->pages};
}

mxg::AttnParams attn_params(const mxg_heads *q, const mxg_heads *k, const mxg_heads *v, const int *cu, int B, int T,
                            int Hq, int Hkv, int D, float scale, const mxg_heads *out, const mxg_attn_opts *opts) {
  mxg::AttnParams p = {};
  p.q = heads(q);
  p.k = heads(k);
  p.v = heads(v);
  p.out = heads(out);
  p.cu = cu;
  p.B = B;
  p.T = T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.D = D;
  p.scale = scale;
  p.status = opts ? opts->dev_status : nullptr;
  p.timeout_ns = (unsigned long long)(opts && opts->timeout_ms ? opts->timeout_ms : 1000u) * 1000000ull;
  p.debug_stall = opts ? opts->debug_stall : 0;
  return p;
}

void paged(mxg::AttnParams &p, const uint64_t *mask, const mxg_kv_cache *cache, const int *block_table, int ld_table,
           int table_cols, const int *ctx_len, const mxg_attn_opts *opts) {
  p.cache = cache_of(cache);
  p.mask = reinterpret_cast<const unsigned long long *>(mask);
  p.table = block_table;
  p.ctx = ctx_len;
  p.ld_table = table_cols > 0 ? ld_table : 0;  // (no columns: the table may be null, and nothing of it is touched)
  p.table_cols = table_cols;
  p.ws = static_cast<float *>(opts->workspace);
}

}  // namespace

extern "C" {

mxg_status qk_norm_rope(const mxg_heads *q, const mxg_heads *k, int T, int Hq, int Hkv, int D, const void *wq_bf16,
                        const void *wk_bf16, float eps, const int *pos, const float *cos_sin, int max_pos, int rot,
                        int interleaved, const mxg_heads *q_out, const mxg_heads *k_out, const mxg_heads *v,
                        const mxg_kv_cache *cache, const int64_t *slots, int *dev_status, mxg_stream_t stream) {
  if (T < 0 || Hq < 1 || Hkv < 1 || D < 1 || rot < 0 || rot > D || !(eps >= 0.0f) ||
      (interleaved != 0 && interleaved != 1))
    return MXG_ERR_INVALID_ARG;
  if (D % 8 != 0 || D < 16 || D > 256 || rot % 16 != 0) return MXG_ERR_UNSUPPORTED_SHAPE;
  if (rot > 0 && (!cos_sin || max_pos < 1)) return MXG_ERR_INVALID_ARG;
  mxg_status st;
  if (cache && (st = check_cache(cache)) != MXG_OK) return st;
  if (T > 0) {
    if ((rot > 0 && !pos) || (cache && !slots) || (!k_out && !cache)) return MXG_ERR_INVALID_ARG;
    if ((st = check_heads(q)) != MXG_OK || (st = check_heads(k)) != MXG_OK || (st = check_heads(q_out)) != MXG_OK)
      return st;
    if (k_out && (st = check_heads(k_out)) != MXG_OK) return st;
    if (cache && (st = check_heads(v)) != MXG_OK) return st;
  }
  if (!aligned(wq_bf16, 16) || !aligned(wk_bf16, 16) || !aligned(cos_sin, 16) || !aligned(pos, 4) ||
      !aligned(slots, 8) || !aligned(dev_status, 4))
    return MXG_ERR_MISALIGNED;
  int sm = 0;
  if ((st = device_sms(&sm)) != MXG_OK) return st;
  if (T == 0) return MXG_OK;
  mxg::RopeParams p = {};
  p.q = heads(q);
  p.k = heads(k);
  p.q_out = heads(q_out);
  p.k_out = heads(k_out);
  if (cache) {
    p.v = heads(v);
    p.cache = cache_of(cache);
    p.slots = reinterpret_cast<const long long *>(slots);
  }
  p.T = T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.D = D;
  p.rot = rot;
  p.max_pos = max_pos;
  p.eps = eps;
  p.wq = static_cast<const uint16_t *>(wq_bf16);
  p.wk = static_cast<const uint16_t *>(wk_bf16);
  p.pos = pos;
  p.cos_sin = cos_sin;
  p.status = dev_status;
  const cudaError_t e = mxg::launch_qk_norm_rope(p, interleaved != 0, sm, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MXG_OK : MXG_ERR_CUDA;
}

mxg_status attn_prompt(const mxg_heads *q, const mxg_heads *k, const mxg_heads *v, const int *cu_seqlens, int B,
                       int T, int Hq, int Hkv, int D, float scale, const mxg_heads *out, const mxg_attn_opts *opts,
                       mxg_stream_t stream) {
  mxg_status st = check_attn(q, k, v, cu_seqlens, B, T, Hq, Hkv, D, scale, out, opts);
  if (st != MXG_OK) return st;
  int sm = 0;
  if ((st = device_sms(&sm)) != MXG_OK) return st;
  if (T == 0) return MXG_OK;
  // row groups x kv heads, numbered in 32 bits
  const int tq = 128 / (Hq / Hkv);
  if (((long long)T / (2 * tq) + B) * Hkv > 0x3fffffffLL || T / (2 * tq) >= (1 << 22) || Hkv >= (1 << 16))
    return MXG_ERR_UNSUPPORTED_SHAPE;
  const mxg::AttnParams p = attn_params(q, k, v, cu_seqlens, B, T, Hq, Hkv, D, scale, out, opts);
  const cudaError_t e = mxg::launch_attn_prompt(p, sm, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MXG_OK : MXG_ERR_CUDA;
}

size_t mxg_attn_tree_workspace_bytes(int D) {
  int sm = 0;
  if ((D != 64 && D != 128) || device_sms(&sm) != MXG_OK) return 0;
  return mxg::attn_tree_ws_bytes(D, sm);
}

mxg_status attn_tree(const mxg_heads *q, const mxg_heads *k, const mxg_heads *v, const int *cu_nodes,
                     const uint64_t *mask, int B, int N, const mxg_kv_cache *cache, const int *block_table,
                     int ld_table, int table_cols, const int *ctx_len, int Hq, int Hkv, int D, float scale,
                     const mxg_heads *out, const mxg_attn_opts *opts, mxg_stream_t stream) {
  mxg_status st = check_attn(q, k, v, cu_nodes, B, N, Hq, Hkv, D, scale, out, opts);
  if (st != MXG_OK) return st;
  if ((st = check_paged(N, mask, cache, block_table, ld_table, table_cols, ctx_len, Hkv)) != MXG_OK) return st;
  int sm = 0;
  if ((st = device_sms(&sm)) != MXG_OK) return st;
  if ((st = check_ws(opts, mxg::attn_tree_ws_bytes(D, sm))) != MXG_OK) return st;
  if ((st = check_units(N, Hq, Hkv, N < B ? N : B, table_cols, cache->page_size)) != MXG_OK) return st;
  if (N == 0) return MXG_OK;
  mxg::AttnParams p = attn_params(q, k, v, cu_nodes, B, N, Hq, Hkv, D, scale, out, opts);
  paged(p, mask, cache, block_table, ld_table, table_cols, ctx_len, opts);
  const cudaError_t e = mxg::launch_attn_tree(p, sm, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MXG_OK : MXG_ERR_CUDA;
}

mxg_status kv_append(const mxg_heads *k, int64_t k_layer_stride, const mxg_heads *v, int64_t v_layer_stride,
                     const int *cu_nodes, int B, int N, const int *accept, int ld_accept, int max_accept,
                     const mxg_kv_cache *cache, const int *block_table, int ld_table, int table_cols,
                     const int *ctx_len, int Hkv, int D, int *ctx_out, int *dev_status, mxg_stream_t stream) {
  if (!cu_nodes || B < 1 || N < 0 || Hkv < 1 || D < 1 || max_accept < 0 || ld_accept < max_accept ||
      (max_accept > 0 && !accept) || !ctx_len || ctx_out == ctx_len || table_cols < 0 || ld_table < table_cols ||
      (table_cols > 0 && !block_table) || k_layer_stride < 0 || v_layer_stride < 0)
    return MXG_ERR_INVALID_ARG;
  if (D % 8 != 0 || D > 1024 || B > mxg::kAttnMaxSeqs || (long long)Hkv * D > (1 << 20))
    return MXG_ERR_UNSUPPORTED_SHAPE;
  mxg_status st;
  if ((st = check_cache(cache)) != MXG_OK) return st;
  if (cache->layers > 65535) return MXG_ERR_UNSUPPORTED_SHAPE;
  if (N > 0 && ((st = check_heads(k)) != MXG_OK || (st = check_heads(v)) != MXG_OK)) return st;
  if (!stride_ok(k_layer_stride) || !stride_ok(v_layer_stride) || !aligned(cu_nodes, 4) || !aligned(accept, 4) ||
      !aligned(block_table, 4) || !aligned(ctx_len, 4) || !aligned(ctx_out, 4) || !aligned(dev_status, 4))
    return MXG_ERR_MISALIGNED;
  int sm = 0;
  if ((st = device_sms(&sm)) != MXG_OK) return st;
  mxg::AppendParams p = {};
  p.k = heads(k);
  p.v = heads(v);
  p.k_layer = k_layer_stride;
  p.v_layer = v_layer_stride;
  p.cache = cache_of(cache);
  p.cu = cu_nodes;
  p.accept = accept;
  p.table = block_table;
  p.ctx = ctx_len;
  p.ctx_out = ctx_out;
  p.status = dev_status;
  p.B = B;
  p.N = N;
  p.Hkv = Hkv;
  p.D = D;
  p.ld_accept = ld_accept;
  p.max_accept = max_accept;
  p.ld_table = ld_table;
  p.table_cols = table_cols;
  const cudaError_t e = mxg::launch_kv_append(p, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MXG_OK : MXG_ERR_CUDA;
}

size_t mxg_attn_shared_workspace_bytes(int N, int Hq, int D) {
  int sm = 0;
  if ((D != 64 && D != 128) || N < 0 || Hq < 1 || device_sms(&sm) != MXG_OK) return 0;
  return mxg::attn_shared_ws_bytes(N, Hq, D, sm);
}

mxg_status attn_shared(const mxg_heads *q, const mxg_heads *k, const mxg_heads *v, const int *cu_nodes,
                       const uint64_t *mask, int B, int N, const mxg_kv_cache *cache, const int *block_table,
                       int ld_table, int table_cols, const int *ctx_len, const int *cu_groups, const int *prefix_len,
                       int n_groups, int Hq, int Hkv, int D, float scale, const mxg_heads *out,
                       const mxg_attn_opts *opts, mxg_stream_t stream) {
  mxg_status st = check_attn(q, k, v, cu_nodes, B, N, Hq, Hkv, D, scale, out, opts);
  if (st != MXG_OK) return st;
  if (n_groups < 0 || n_groups > B || (n_groups > 0 && (!cu_groups || !prefix_len))) return MXG_ERR_INVALID_ARG;
  const int span = 2 * (128 / (Hq / Hkv));  // nodes of a row group
  if (N / span >= (1 << 22)) return MXG_ERR_UNSUPPORTED_SHAPE;  // (a group's row groups)
  if ((st = check_paged(N, mask, cache, block_table, ld_table, table_cols, ctx_len, Hkv)) != MXG_OK) return st;
  if (!aligned(cu_groups, 4) || !aligned(prefix_len, 4)) return MXG_ERR_MISALIGNED;
  int sm = 0;
  if ((st = device_sms(&sm)) != MXG_OK) return st;
  if ((st = check_ws(opts, mxg::attn_shared_ws_bytes(N, Hq, D, sm))) != MXG_OK) return st;
  // (prefixes' full row groups besides the sequences')
  const long long starts = 2LL * (N < B ? N : B) + N / span;
  if ((st = check_units(N, Hq, Hkv, starts, table_cols, cache->page_size)) != MXG_OK) return st;
  if (N == 0) return MXG_OK;
  mxg::SharedParams p = {};
  p.a = attn_params(q, k, v, cu_nodes, B, N, Hq, Hkv, D, scale, out, opts);
  paged(p.a, mask, cache, block_table, ld_table, table_cols, ctx_len, opts);
  p.groups = cu_groups;
  p.prefix = prefix_len;
  p.n_groups = n_groups;
  const cudaError_t e = mxg::launch_attn_shared(p, sm, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MXG_OK : MXG_ERR_CUDA;
}

mxg_status kv_index(const mxg_kv_cache *cache, int Hkv, int D, const mxg_page_index *index, const int *block_table,
                    int B, int ld_table, int table_cols, const int *ctx_old, const int *ctx_new, int *dev_status,
                    mxg_stream_t stream) {
  if (B < 1 || Hkv < 1 || D < 1 || !ctx_new || table_cols < 0 || ld_table < table_cols ||
      (table_cols > 0 && !block_table))
    return MXG_ERR_INVALID_ARG;
  if ((D != 64 && D != 128) || B > mxg::kAttnMaxSeqs || Hkv > 65535) return MXG_ERR_UNSUPPORTED_SHAPE;
  mxg_status st;
  if ((st = check_cache(cache)) != MXG_OK || (st = check_index(index)) != MXG_OK) return st;
  if (index->layers < cache->layers || index->pages < cache->pages) return MXG_ERR_INVALID_ARG;
  // (entries are written: none over another)
  if (!apart({{{index->codes_layer, index->layers}, {index->codes_page, index->pages}, {index->codes_head, Hkv}}}, 2 * D) ||
      !apart({{{index->exps_layer, index->layers}, {index->exps_page, index->pages}, {0, 1}}}, Hkv))
    return MXG_ERR_UNSUPPORTED_SHAPE;
  // (pages of all sequences, numbered in 32 bits)
  if ((long long)table_cols * cache->page_size > 0x7fffff00LL || (long long)table_cols * B > 0x7fffffffLL)
    return MXG_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(block_table, 4) || !aligned(ctx_old, 4) || !aligned(ctx_new, 4) || !aligned(dev_status, 4))
    return MXG_ERR_MISALIGNED;
  int sm = 0;
  if ((st = device_sms(&sm)) != MXG_OK) return st;
  if (table_cols == 0) return MXG_OK;
  mxg::IndexParams p = {};
  p.cache = cache_of(cache);
  p.index = index_of(index);
  p.table = block_table;
  p.old = ctx_old;
  p.now = ctx_new;
  p.status = dev_status;
  p.B = B;
  p.Hkv = Hkv;
  p.D = D;
  p.ld_table = ld_table;
  p.table_cols = table_cols;
  const cudaError_t e = mxg::launch_kv_index(p, sm, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MXG_OK : MXG_ERR_CUDA;
}

mxg_status attn_select(const mxg_heads *q, const int *cu_nodes, int B, int N, const mxg_page_index *index,
                       int page_size, const int *block_table, int ld_table, int table_cols, const int *ctx_len, int Hq,
                       int Hkv, int D, int n_sel, int first, int last, int *sel, int *dev_status,
                       mxg_stream_t stream) {
  if (!cu_nodes || B < 1 || N < 0 || Hq < 1 || Hkv < 1 || !ctx_len || table_cols < 0 || ld_table < table_cols ||
      (table_cols > 0 && !block_table) || (N > 0 && !sel) || first < 0 || last < 1 || n_sel < 1 || first > n_sel ||
      last > n_sel - first || page_size < 1)
    return MXG_ERR_INVALID_ARG;
  if ((D != 64 && D != 128) || Hq % Hkv != 0 || Hq / Hkv > 128 || B > mxg::kAttnMaxSeqs ||
      n_sel > mxg::kAttnMaxSelect || table_cols > mxg::kAttnMaxScored || (long long)Hkv * 8 > 0x7fffffffLL ||
      (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128 && page_size != 256) ||
      (long long)table_cols * page_size > 0x7fffff00LL || (long long)N * Hkv > 0x7fffffffLL)
    return MXG_ERR_UNSUPPORTED_SHAPE;
  mxg_status st;
  if ((st = check_index(index)) != MXG_OK) return st;
  if (N > 0 && (st = check_heads(q)) != MXG_OK) return st;
  if (!aligned(cu_nodes, 4) || !aligned(block_table, 4) || !aligned(ctx_len, 4) || !aligned(sel, 4) ||
      !aligned(dev_status, 4))
    return MXG_ERR_MISALIGNED;
  int sm = 0;
  if ((st = device_sms(&sm)) != MXG_OK) return st;
  if (N == 0) return MXG_OK;
  mxg::SelectParams p = {};
  p.q = heads(q);
  p.index = index_of(index);
  p.cu = cu_nodes;
  p.table = block_table;
  p.ctx = ctx_len;
  p.sel = sel;
  p.status = dev_status;
  p.B = B;
  p.N = N;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.D = D;
  p.page_size = page_size;
  p.ld_table = table_cols > 0 ? ld_table : 0;
  p.table_cols = table_cols;
  p.n_sel = n_sel;
  p.first = first;
  p.last = last;
  const cudaError_t e = mxg::launch_attn_select(p, sm, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MXG_OK : MXG_ERR_CUDA;
}

size_t mxg_attn_sparse_workspace_bytes(int N, int Hkv, int n_sel, int D) {
  int sm = 0;
  if ((D != 64 && D != 128) || N < 0 || Hkv < 1 || n_sel < 1 || device_sms(&sm) != MXG_OK) return 0;
  return mxg::attn_sparse_ws_bytes(N, Hkv, n_sel, D, sm);
}

mxg_status attn_sparse(const mxg_heads *q, const mxg_heads *k, const mxg_heads *v, const int *cu_nodes,
                       const uint64_t *mask, int B, int N, const mxg_kv_cache *cache, const int *block_table,
                       int ld_table, int table_cols, const int *ctx_len, const int *sel, int n_sel, int Hq, int Hkv,
                       int D, float scale, const mxg_heads *out, const mxg_attn_opts *opts, mxg_stream_t stream) {
  mxg_status st = check_attn(q, k, v, cu_nodes, B, N, Hq, Hkv, D, scale, out, opts);
  if (st != MXG_OK) return st;
  if (n_sel < 1 || (N > 0 && !sel)) return MXG_ERR_INVALID_ARG;
  if (n_sel > mxg::kAttnMaxSelect || table_cols > mxg::kAttnMaxListed)
    return MXG_ERR_UNSUPPORTED_SHAPE;
  if ((st = check_paged(N, mask, cache, block_table, ld_table, table_cols, ctx_len, Hkv)) != MXG_OK) return st;
  if (!aligned(sel, 4)) return MXG_ERR_MISALIGNED;
  int sm = 0;
  if ((st = device_sms(&sm)) != MXG_OK) return st;
  if ((st = check_ws(opts, mxg::attn_sparse_ws_bytes(N, Hkv, n_sel, D, sm))) != MXG_OK) return st;
  // (a sequence's nodes name no more pages than there are, nor than all their lists hold)
  const long long named = (long long)mxg::kAttnMaxNodes * n_sel;
  const int cols = named < table_cols ? (int)named : table_cols;
  if ((st = check_units(N, Hq, Hkv, 2LL * (N < B ? N : B), cols, cache->page_size)) != MXG_OK) return st;
  if (N == 0) return MXG_OK;
  mxg::SparseParams p = {};
  p.a = attn_params(q, k, v, cu_nodes, B, N, Hq, Hkv, D, scale, out, opts);
  paged(p.a, mask, cache, block_table, ld_table, table_cols, ctx_len, opts);
  p.sel = sel;
  p.n_sel = n_sel;
  const cudaError_t e = mxg::launch_attn_sparse(p, sm, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MXG_OK : MXG_ERR_CUDA;
}

}  // extern "C"
