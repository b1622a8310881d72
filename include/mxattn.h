/*
 * mxattn.h -- C ABI of the attention operators between the qkv projection and
 * o_proj: the work of a layer that the GEMMs of mxgemm.h do not cover.
 *
 *   qk_norm_rope   RMS norm of every query and key head and the position
 *                  rotation in one pass, with k and v into cache pages
 *   attn_prompt    causal attention of packed prompts
 *   attn_tree      attention of drafted token trees (or of single decoded
 *                  tokens) over a paged cache
 *   kv_append      accepted tokens' keys and values into the cache
 *
 * A prompt pass is qk_norm_rope (which also fills the cache), attn_prompt,
 * o_proj.  A verify step is qk_norm_rope, attn_tree, o_proj per layer, then
 * -- once the accepted path is known -- one kv_append for all layers: the
 * drafted tokens' keys and values stay out of the cache until they count.
 *
 * Conventions are those of mxgemm.h: DEVICE pointers owned by the caller,
 * 16-byte aligned (index arrays: aligned to their element); calls asynchronous
 * on `stream`, launched with programmatic stream serialization, capturable in
 * a CUDA graph; host-detectable errors returned before anything is launched;
 * device waits bounded (mxg_attn_opts.timeout_ms); no memory allocated and no
 * pointer kept.  All tensors are bf16; norms, rotations, scores, softmax
 * statistics and accumulators are fp32, rounded to bf16 once at the end (the
 * softmax weights are rounded to bf16 before their product with v).
 * These are inference operators: there are no gradients.
 *
 * What the host cannot see -- lengths, positions, page numbers, node indices
 * -- the kernels check: an entry out of its range touches no memory outside
 * the tensors, ORs MXG_DEV_BAD_INDEX into the status word (if given;
 * mxg_query_status then returns MXG_ERR_CUDA) and has the effect its
 * entry point states.
 */
#ifndef MXATTN_H
#define MXATTN_H

#include "mxgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Heads of tokens: element (token t, head h, channel d) at
 * ptr[t * tok_stride + h * head_stride + d], strides in elements, multiples
 * of 8 (attn_prompt and attn_tree: not 0 where there is more than one token or
 * head).  A slice of a packed qkv projection, or a tensor of its own. */
typedef struct {
    void *ptr;
    int64_t tok_stride;
    int64_t head_stride;
} mxg_heads;

/* A paged cache of `pages` pages of `page_size` tokens, page_size in {16, 32,
 * 64, 128, 256}: element (layer l, page p, slot s, head h, channel d) of k and
 * of v at l * layer_stride + p * page_stride + s * slot_stride +
 * h * head_stride + d, strides in elements, multiples of 8.  layers > 1 only
 * matters to kv_append; the other entry points use layer 0. */
typedef struct {
    void *k, *v;
    int64_t layer_stride, page_stride, slot_stride, head_stride;
    int layers, pages, page_size;
} mxg_kv_cache;

typedef struct {
    void *workspace;     /* attn_tree: device scratch of >= mxg_attn_tree_workspace_bytes(),
                            256-byte aligned; its contents on entry do not matter.  Calls that
                            overlap on the GPU need separate workspaces. */
    size_t ws_bytes;
    int *dev_status;     /* optional device int; kernels OR MXG_DEV_* bits into it */
    uint32_t timeout_ms; /* limit of every device-side wait; 0 = 1000 ms.  The longest legitimate
                            one lasts as long as a CTA's keys: about 2 us for 128 of them */
    int debug_stall;     /* test hook: 1 makes the first wait of every CTA one that nothing
                            satisfies, so that the timeout path runs (no fault, no hang) */
} mxg_attn_opts;

/* Most sequences of one attn_prompt, attn_tree or kv_append call, and most
 * nodes of one sequence's tree (the bits of a mask word). */
#define MXG_ATTN_MAX_SEQS 4096
#define MXG_ATTN_MAX_NODES 64

/* For every token t < T and every head of q (Hq heads) and k (Hkv heads):
 *   y = x * rsqrt(mean(x^2) + eps) * w     (w: wq or wk, D bf16 gains;
 *                                           NULL = y = x, no norm)
 *   the first `rot` channels rotated by the angles of position pos[t]: pair i
 *   (i < rot/2) is (y[i], y[i + rot/2]), or (y[2i], y[2i + 1]) when
 *   `interleaved`;  (a, b) -> (a cos - b sin, b cos + a sin)
 *   rounded to bf16.
 * cos_sin: (max_pos, rot) floats, a row [cos (rot/2) | sin (rot/2)]; NULL with
 * rot == 0 (no rotation; pos may then be NULL).
 * Results: q to q_out, k to k_out (may be NULL when cache is given); q_out may
 * be q itself and k_out k itself (in place), other overlaps are not allowed.
 * cache (nullable): k also to slot slots[t] of layer 0 -- slot number page *
 * page_size + place -- and v (Hkv heads; required then) as it is.  A negative
 * slot is not written (padding tokens).  Two tokens of one call must not share
 * a slot.
 * D % 8 == 0, 16 <= D <= 256; rot % 16 == 0, rot <= D; T >= 0.
 * Out of range: pos[t] outside [0, max_pos) makes token t's q and k NaN; a slot
 * >= pages * page_size is not written. */
mxg_status qk_norm_rope(const mxg_heads *q, const mxg_heads *k, int T, int Hq, int Hkv, int D,
                        const void *wq_bf16, const void *wk_bf16, float eps, const int *pos,
                        const float *cos_sin, int max_pos, int rot, int interleaved,
                        const mxg_heads *q_out, const mxg_heads *k_out, const mxg_heads *v,
                        const mxg_kv_cache *cache, const int64_t *slots, int *dev_status,
                        mxg_stream_t stream);

/* Causal attention of B packed prompts: sequence b is tokens cu_seqlens[b] ..
 * cu_seqlens[b+1] - 1 of q (T tokens, Hq heads), k and v (Hkv heads; Hq % Hkv
 * == 0, query head h reads kv head h / (Hq / Hkv)); token i of a sequence sees
 * its tokens j <= i:
 *   out_i = sum_j p_ij v_j,  p_i = softmax_j(scale * q_i . k_j).
 * cu_seqlens: B + 1 ints, cu_seqlens[0] = 0, non-decreasing (empty sequences
 * allowed), cu_seqlens[B] <= T; tokens past cu_seqlens[B] are not written.
 * D in {64, 128}, Hq / Hkv <= 128, 1 <= B <= MXG_ATTN_MAX_SEQS, T >= 0,
 * scale > 0.
 * out may be q itself; it must not overlap k or v, nor q in any other way.
 * v of a token that a query does not see has no influence on it, NaN and
 * infinities included.  opts may be NULL; no workspace is needed.
 * Out of range: offsets are clamped to [0, T] and to the offsets before. */
mxg_status attn_prompt(const mxg_heads *q, const mxg_heads *k, const mxg_heads *v,
                       const int *cu_seqlens, int B, int T, int Hq, int Hkv, int D, float scale,
                       const mxg_heads *out, const mxg_attn_opts *opts, mxg_stream_t stream);

/* Attention of drafted token trees over a paged cache.  Sequence b has
 * ctx_len[b] tokens in the cache -- token j in slot j % page_size of page
 * block_table[b * ld_table + j / page_size] -- and the nodes cu_nodes[b] ..
 * cu_nodes[b+1] - 1 (at most MXG_ATTN_MAX_NODES) of q (N nodes in all, Hq
 * heads), k and v (Hkv heads, not in the cache).  Node i sees all of the
 * sequence's cached tokens and the nodes j whose bit j is set in mask[i] (i
 * global, j counted from the sequence's first node; bits at or past the
 * sequence's node count are ignored).  A node that sees nothing gets 0.
 * One node a sequence with mask 1 is plain decoding.
 * table_cols: columns of block_table that may be read.  D, Hq, Hkv, B, scale
 * and out as for attn_prompt (nor may out overlap the cache); N >= 0.  v of
 * what a node does not see has no influence on it.
 * opts with a workspace is required.  Results do not depend on timing: the
 * parts of a long context are joined in a fixed order.
 * Out of range: offsets are clamped as for attn_prompt, a tree's nodes past
 * the 64th are not written and not seen, ctx_len is clamped to [0, table_cols
 * * page_size], a page outside [0, pages) reads as zeros. */
size_t mxg_attn_tree_workspace_bytes(int D);
mxg_status attn_tree(const mxg_heads *q, const mxg_heads *k, const mxg_heads *v,
                     const int *cu_nodes, const uint64_t *mask, int B, int N,
                     const mxg_kv_cache *cache, const int *block_table, int ld_table,
                     int table_cols, const int *ctx_len, int Hq, int Hkv, int D, float scale,
                     const mxg_heads *out, const mxg_attn_opts *opts, mxg_stream_t stream);

/* The accepted nodes of each sequence into the cache, in every layer: entry i
 * of accept[b * ld_accept ...] (max_accept entries; the first negative one
 * ends the list) names the node that becomes token ctx_len[b] + i of the
 * sequence (counted from cu_nodes[b]); its k and v (layer l at
 * l * k_layer_stride / v_layer_stride elements) are copied to that token's
 * slot, and ctx_out[b] = ctx_len[b] + (tokens written).  The page of every slot
 * written must be in the block table, and no two sequences may write the same
 * page.  ctx_out (nullable) must not be ctx_len.
 * D % 8 == 0, 8 <= D <= 1024; cache->layers layers; max_accept >= 0.
 * Out of range: a node index at or past the sequence's nodes, or a token whose
 * page is not in the table or not in the cache, ends the list as a negative
 * entry does: neither it nor what follows is written or counted. */
mxg_status kv_append(const mxg_heads *k, int64_t k_layer_stride, const mxg_heads *v,
                     int64_t v_layer_stride, const int *cu_nodes, int B, int N, const int *accept,
                     int ld_accept, int max_accept, const mxg_kv_cache *cache,
                     const int *block_table, int ld_table, int table_cols, const int *ctx_len,
                     int Hkv, int D, int *ctx_out, int *dev_status, mxg_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MXATTN_H */
