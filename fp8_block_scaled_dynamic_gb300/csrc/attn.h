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

// A sequence as the kernels see it where a plan kernel has worked it out: its
// nodes as queries (rows), the keys in a list of pages, and perhaps its nodes.
struct PlanRec {
  int a0, n, ctx, hk;  // first node, nodes, cached tokens in the list, kv head or -1 (all)
  long long list;      // where its page numbers begin
  int flags, pad;
};
static_assert(sizeof(PlanRec) == 32, "read as two 16-byte words");

struct Plan {
  const PlanRec *rec;
  int n;                            // records
  const int *units;                 // of each record, zeros behind the last one (PlanUnits)
  const int *list;                  // sparse: page numbers
  const unsigned long long *names;  // sparse: the nodes that name a page, a bit each
  const int *info;                  // shared: of each node, how its parts are joined
  float *rows, *stats;              // shared: parts of whole rows (prefix, own): sums, references and weights
  float *part_ws[2];                // shared: the two launches' items and slots
  bool beside;                      // shared: the launch may run beside the one before it
  const int *ctas;                  // shared: the launch's CTAs that have a share of its work
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
  long long slots;  // floats before the CTAs' parts
  int *status;
  unsigned long long timeout_ns;
  int debug_stall;
  Plan plan;
};

struct SharedParams {  // attn_shared
  AttnParams a;
  const int *groups, *prefix;  // n_groups + 1 sequence offsets, n_groups lengths
  int n_groups;
};

struct SparseParams {  // attn_sparse
  AttnParams a;
  const int *sel;  // (T, Hkv, n_sel)
  int n_sel;
};

struct PageIndex {  // strides in bytes
  int8_t *codes;
  uint8_t *exps;
  long long codes_layer, codes_page, codes_head, exps_layer, exps_page;
  int layers, pages;
};

struct IndexParams {
  Cache cache;
  PageIndex index;
  const int *table, *old, *now;  // old null: zeros
  int *status;
  int B, Hkv, D, ld_table, table_cols;
};

struct SelectParams {
  Heads q;
  PageIndex index;
  const int *cu, *table, *ctx;
  int *sel, *status;
  int B, N, Hq, Hkv, D, page_size, ld_table, table_cols, n_sel, first, last;
};

constexpr int kAttnMaxSeqs = 4096;
constexpr int kAttnMaxNodes = 64;
constexpr int kAttnMaxSelect = 512;
constexpr int kAttnMaxScored = 1 << 15;  // columns of attn_select's block table (a node's keys in shared memory)
constexpr int kAttnMaxListed = 1 << 19;  // columns of attn_sparse's block table (a bit each in shared memory)

cudaError_t launch_qk_norm_rope(const RopeParams &p, bool interleaved, int sm_count, cudaStream_t stream);
cudaError_t launch_kv_append(const AppendParams &p, cudaStream_t stream);
cudaError_t launch_attn_prompt(const AttnParams &p, int sm_count, cudaStream_t stream);
cudaError_t launch_attn_tree(const AttnParams &p, int sm_count, cudaStream_t stream);
size_t attn_tree_ws_bytes(int D, int sm_count);
cudaError_t launch_attn_shared(const SharedParams &p, int sm_count, cudaStream_t stream);
size_t attn_shared_ws_bytes(long long N, int Hq, int D, int sm_count);
cudaError_t launch_attn_sparse(const SparseParams &p, int sm_count, cudaStream_t stream);
size_t attn_sparse_ws_bytes(long long N, int Hkv, int n_sel, int D, int sm_count);
cudaError_t launch_kv_index(const IndexParams &p, int sm_count, cudaStream_t stream);
cudaError_t launch_attn_select(const SelectParams &p, int sm_count, cudaStream_t stream);

}  // namespace mxg
