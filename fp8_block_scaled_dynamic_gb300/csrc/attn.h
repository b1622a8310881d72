// attn.h -- launchers of the attention operators (not part of the public C ABI).
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace mxg {

struct Heads {  // bf16, strides in elements
  uint16_t *ptr;
  long long tok, head;
};

struct Cache {  // bf16, strides in elements
  uint16_t *k, *v;
  long long layer, page, slot, head;
  int layers, pages, page_size;
};

struct RopeParams {
  Heads q, k, v, q_out, k_out;  // v.ptr null: no cache; k_out.ptr null: cache only
  Cache cache;                  // cache.k null: none
  int T, Hq, Hkv, D, rot, max_pos;
  float eps;
  const uint16_t *wq, *wk;  // null: no norm
  const int *pos;
  const float *cos_sin;
  const long long *slots;
  int *status;
};

struct AppendParams {
  Heads k, v;
  long long k_layer, v_layer;
  Cache cache;
  const int *cu, *accept, *table, *ctx;
  int *ctx_out, *status;
  int B, N, Hkv, D, ld_accept, max_accept, ld_table, table_cols;
};

struct AttnParams {
  Heads q, k, v, out;
  Cache cache;              // tree only
  const int *cu;            // B + 1 token (node) offsets
  const unsigned long long *mask;
  const int *table, *ctx;
  int B, T, Hq, Hkv, D, ld_table, table_cols;
  float scale;
  float *ws;
  int *status;
  unsigned long long timeout_ns;
  int debug_stall;
};

constexpr int kAttnMaxSeqs = 4096;
constexpr int kAttnMaxNodes = 64;

cudaError_t launch_qk_norm_rope(const RopeParams &p, bool interleaved, int sm_count, cudaStream_t stream);
cudaError_t launch_kv_append(const AppendParams &p, cudaStream_t stream);
cudaError_t launch_attn_prompt(const AttnParams &p, int sm_count, cudaStream_t stream);
cudaError_t launch_attn_tree(const AttnParams &p, int sm_count, cudaStream_t stream);
size_t attn_tree_ws_bytes(int D, int sm_count);

}  // namespace mxg
