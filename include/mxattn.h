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
 * and, for long contexts over the same cache:
 *
 *   attn_shared    attn_tree for sequences that share a prefix by groups
 *   kv_index       8-bit bounds of the keys of each full page
 *   attn_select    the pages whose bounds promise the largest scores
 *   attn_sparse    attn_tree over selected pages
 *
 * A prompt pass is qk_norm_rope (which also fills the cache), attn_prompt,
 * o_proj.  A verify step is qk_norm_rope, attn_tree, o_proj per layer, then
 * -- once the accepted path is known -- one kv_append for all layers: the
 * drafted tokens' keys and values stay out of the cache until they count.  Over
 * selected pages a step is qk_norm_rope, attn_select, attn_sparse, o_proj per
 * layer, then one kv_append and one kv_index for all layers.
 *
 * Conventions are those of mxgemm.h: DEVICE pointers owned by the caller,
 * 16-byte aligned (index arrays: aligned to their element); calls asynchronous
 * on `stream`, launched with programmatic stream serialization, capturable in
 * a CUDA graph; host-detectable errors returned before anything is launched;
 * device waits bounded (mxg_attn_opts.timeout_ms); no memory allocated and no
 * pointer kept.  All tensors are bf16; norms, rotations, scores, softmax
 * statistics and accumulators are fp32, rounded to bf16 once at the end (the
 * softmax weights are rounded to bf16 before their product with v).  A row's
 * sums hold |v| times the number of keys that it sees below 2^119.  The bounds
 * and scores of kv_index and attn_select are whole numbers times powers of two,
 * computed without rounding: what is selected is the same on any machine.
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

/* Bounds of the keys of a paged cache's full pages, by physical page: of (layer
 * l, page p, head h) two rows of D codes -- the upper bounds, then the lower --
 * at codes + l * codes_layer + p * codes_page + h * codes_head (strides in
 * bytes, multiples of 16; those of pages below 2^31) and the power of two that
 * they count, as an E8M0 code, at exps + l * exps_layer + p * exps_page + h. */
typedef struct {
    int8_t *codes;
    uint8_t *exps;
    int64_t codes_layer, codes_page, codes_head, exps_layer, exps_page;
    int layers, pages;
} mxg_page_index;

typedef struct {
    void *workspace;     /* attn_tree, attn_shared, attn_sparse: device scratch of >=
                            mxg_<name>_workspace_bytes(), 256-byte aligned; its contents on
                            entry do not matter.  Calls that overlap on the GPU need separate
                            workspaces. */
    size_t ws_bytes;
    int *dev_status;     /* optional device int; kernels OR MXG_DEV_* bits into it */
    uint32_t timeout_ms; /* limit of every device-side wait; 0 = 1000 ms.  The longest legitimate
                            one lasts as long as a CTA's keys: about 2 us for 128 of them.  Where
                            attn_shared and attn_sparse meet a v that is not finite, rows are
                            summed again, for up to 2 us a key (0.25 s for the 131072 keys of 512
                            pages of 256) */
    int debug_stall;     /* test hook: 1 makes the first wait of every CTA one that nothing
                            satisfies, so that the timeout path runs (no fault, no hang) */
} mxg_attn_opts;

/* Most sequences of one attn_prompt, attn_tree or kv_append call, and most
 * nodes of one sequence's tree (the bits of a mask word). */
#define MXG_ATTN_MAX_SEQS 4096
#define MXG_ATTN_MAX_NODES 64
/* Most pages that attn_select selects and attn_sparse takes. */
#define MXG_ATTN_MAX_SELECT 512

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

/* attn_tree for sequences that share the beginning of their contexts by groups,
 * which is then read once for the group: faster than attn_tree where many share
 * much (64 sequences of a node: 68 us against 90 behind 1024 tokens, 93 against
 * 388 behind 16384; 8 of them 26 against 37 behind 8192), slower where few share
 * little (8 trees of 8 nodes behind 1024 tokens 31 against 20).  Group g is
 * sequences cu_groups[g] .. cu_groups[g+1] - 1 (n_groups + 1 ints, cu_groups[0] =
 * 0, non-decreasing, cu_groups[n_groups] <= B; sequences past it share nothing);
 * the first prefix_len[g] cached tokens of each of them, a multiple of page_size,
 * are read from the pages in the block table's row of the group's first sequence
 * (where the others name the same pages, the result is attn_tree's).  ctx_len counts
 * them: it is at least prefix_len[g] throughout the group.  Everything else is as
 * for attn_tree.
 * n_groups <= B; n_groups 0: cu_groups and prefix_len may be NULL.
 * Out of range, besides attn_tree's: cu_groups is clamped as offsets are,
 * prefix_len to [0, the group's smallest ctx_len] and then to whole pages. */
size_t mxg_attn_shared_workspace_bytes(int N, int Hq, int D);
mxg_status attn_shared(const mxg_heads *q, const mxg_heads *k, const mxg_heads *v,
                       const int *cu_nodes, const uint64_t *mask, int B, int N,
                       const mxg_kv_cache *cache, const int *block_table, int ld_table,
                       int table_cols, const int *ctx_len, const int *cu_groups,
                       const int *prefix_len, int n_groups, int Hq, int Hkv, int D, float scale,
                       const mxg_heads *out, const mxg_attn_opts *opts, mxg_stream_t stream);

/* Bounds of the pages that became full, in every layer: of each sequence b, the
 * pages j with floor(ctx_old[b] / page_size) <= j < floor(ctx_new[b] / page_size)
 * (ctx_old NULL: all zero), after their keys were written.  Of the page's keys of
 * a layer and kv head:
 *   e = the least whole number >= -100 with max |k| <= 127 * 2^e
 *   upper[d] = ceil(max k[d] / 2^e), lower[d] = floor(min k[d] / 2^e)
 *   E8M0 code e + 127;  255 and all bounds zero where a key is NaN or infinite.
 * Sequences may share pages.  Other pages' entries are left as they were; v is
 * not read (cache->v must be given all the same).  index: as many layers as the
 * cache, entries for at least its pages.
 * D in {64, 128}, B <= MXG_ATTN_MAX_SEQS; entries of index (2 D codes; Hkv exponents)
 * apart from one another: of layers, pages and heads, in any order, each stride at
 * least as long as all entries of those with smaller strides.
 * Out of range: ctx_old and ctx_new are clamped to [0, table_cols * page_size], a
 * page outside [0, pages) is skipped. */
mxg_status kv_index(const mxg_kv_cache *cache, int Hkv, int D, const mxg_page_index *index,
                    const int *block_table, int B, int ld_table, int table_cols,
                    const int *ctx_old, const int *ctx_new, int *dev_status, mxg_stream_t stream);

/* The pages that each node attends to, for each kv head h: of the sequence's
 * P = ceil(ctx_len / page_size) logical pages the first `first` and the last
 * `last`, and of the others those with the highest scores, lower pages first
 * among equals, until there are n_sel (all, if P <= n_sel).  With the bounds of
 * the page (layer 0 of index) and the query heads g of kv head h:
 *   e = the least whole number >= -100 with max |q| <= 127 * 2^e over g and d
 *   x[g][d] = q[g][d] / 2^e rounded to the nearest whole number, ties to even
 *   score = 2^(code - 127) * max_g sum_d x[g][d] * (x[g][d] > 0 ? upper[d] : lower[d])
 * which is an upper bound of q . k over the page's keys, up to the rounding of q
 * and a factor that the node's scores have in common.  A page of code 255 comes
 * before all others; a q that holds a NaN or an infinity counts as zero.
 * sel: (N, Hkv, n_sel) ints: logical page numbers, ascending, then -1; rows of
 * nodes past cu_nodes[B] are not written.  The last page, which may not be full, is
 * always selected and needs no bounds: 1 <= last, 0 <= first, first + last <= n_sel
 * <= MXG_ATTN_MAX_SELECT.
 * D in {64, 128}, Hq % Hkv == 0, Hq / Hkv <= 128, B <= MXG_ATTN_MAX_SEQS,
 * table_cols <= 32768.
 * Out of range: offsets, nodes and ctx_len are clamped as for attn_tree; a page
 * whose number is outside [0, index->pages) has the score zero. */
mxg_status attn_select(const mxg_heads *q, const int *cu_nodes, int B, int N,
                       const mxg_page_index *index, int page_size, const int *block_table,
                       int ld_table, int table_cols, const int *ctx_len, int Hq, int Hkv, int D,
                       int n_sel, int first, int last, int *sel, int *dev_status,
                       mxg_stream_t stream);

/* attn_tree where node i and the query heads of kv head h see, of the sequence's
 * cached tokens, those in the logical pages sel[(i * Hkv + h) * n_sel ...]
 * (negative entries name none; any order; a page named twice is seen once).  A
 * page is read once for all nodes of its sequence that name it.  Everything else
 * is as for attn_tree.
 * 1 <= n_sel <= MXG_ATTN_MAX_SELECT, table_cols <= 524288.
 * Out of range, besides attn_tree's: a logical page past the sequence's last one
 * (ceil(ctx_len / page_size) or more) names none. */
size_t mxg_attn_sparse_workspace_bytes(int N, int Hkv, int n_sel, int D);
mxg_status attn_sparse(const mxg_heads *q, const mxg_heads *k, const mxg_heads *v,
                       const int *cu_nodes, const uint64_t *mask, int B, int N,
                       const mxg_kv_cache *cache, const int *block_table, int ld_table,
                       int table_cols, const int *ctx_len, const int *sel, int n_sel, int Hq,
                       int Hkv, int D, float scale, const mxg_heads *out,
                       const mxg_attn_opts *opts, mxg_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MXATTN_H */
