/*
 * lora_attention.h -- C ABI of the operators that follow the adapters' q/k/v
 * projection in a serving step: rotary positions (with or without a norm of
 * each head), a paged key/value cache, attention for a tree of drafted tokens
 * over that cache, and keeping the accepted path of a tree.
 *
 * A step with the rows y = [q | k | v] that lora_shrink_expand updated:
 *
 *     lora_build_tree      masks, positions and cache rows of the step, once
 *     per layer:
 *       lora_rotary or lora_qk_norm_rotary   q in place, k and v into the cache
 *       lora_tree_attention                  over context and drafted tokens
 *     lora_keep_path       after verification, every layer's cache in one call
 *
 * One node per sequence is an ordinary decode step; a NULL mask makes the
 * tokens of a sequence a chain (several drafted tokens, or a piece of a
 * prompt).
 *
 * The conventions of lora.h hold: device pointers unless marked [host], the
 * caller owns every buffer, calls are asynchronous and ordered on `stream`,
 * arguments are checked on the host before anything is enqueued, and
 * lora_last_error() describes a refusal.  Nothing here allocates,
 * synchronises or keeps state between calls, so every call can be captured in
 * a HIP graph.  Forward only: the library serves adapters and has no
 * gradients.
 *
 * Head shapes: head_dim d is a multiple of 8 from 8 to LORA_MAX_HEAD_DIM;
 * q_heads is a multiple of kv_heads, query head h reads key/value head
 * h / (q_heads / kv_heads).  Rows and cache tensors have unit inner stride;
 * the other strides are free multiples of 16 bytes (a page and a row of a cache
 * within 4 GiB for the attention), and base pointers are 16-byte aligned
 * (LORA_ERR_UNSUPPORTED otherwise).
 */
#ifndef LORA_ATTENTION_MI355X_H
#define LORA_ATTENTION_MI355X_H

#include "lora.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LORA_MAX_HEAD_DIM 256
#define LORA_MAX_HEADS 1024
/* Most nodes of a sequence's tree with a mask (a chain has no limit). */
#define LORA_MAX_TREE_NODES 1024
/* Most layers lora_keep_path takes at once, and nodes of an accepted path. */
#define LORA_MAX_KEEP_LAYERS 128
#define LORA_MAX_KEEP_PATH 1024

/* ------------------------------------------------------------------------ */
/* Rotary positions                                                         */
/* ------------------------------------------------------------------------ */

/* Which elements of a head form the pair that angle i turns (i < rot_dim / 2):
 * HALF (i, i + rot_dim / 2), INTERLEAVED (2 i, 2 i + 1). */
typedef LORA_ENUM { LORA_ROPE_HALF = 0, LORA_ROPE_INTERLEAVED = 1 } lora_rope_layout;

/* How the frequencies f_i = base^(-2 i / rot_dim) are changed for contexts
 * longer than the model was trained on (s = factor, L = original_context):
 *   NONE     f_i
 *   LINEAR   f_i / s
 *   NTK      f_i with the base raised to base * s^(rot_dim / (rot_dim - 2))
 *   LLAMA3   by the turns n_i = L f_i / (2 pi) a pair makes in L positions:
 *            f_i where n_i >= high, f_i / s where n_i <= low, between them
 *            (1 - m) f_i / s + m f_i with m = (n_i - low) / (high - low)
 *   YARN     f_i / s (1 - k_i) + f_i k_i, k_i falling from 1 to 0 in even steps
 *            over the pairs from floor(c(high)) to ceil(c(low)),
 *            c(n) = rot_dim ln(L / (2 pi n)) / (2 ln base) (both within
 *            [0, rot_dim - 1]); cos and sin are multiplied by
 *            0.1 ln(s) + 1, or by `magnitude` where that is not 0
 * low and high: turns; 0 takes 1 and 4 (LLAMA3) or 1 and 32 (YARN). */
typedef LORA_ENUM {
  LORA_ROPE_NONE = 0,
  LORA_ROPE_LINEAR = 1,
  LORA_ROPE_NTK = 2,
  LORA_ROPE_LLAMA3 = 3,
  LORA_ROPE_YARN = 4
} lora_rope_scaling;

typedef struct {
  int32_t scaling; /* a lora_rope_scaling */
  double factor;   /* s > 0 */
  double original_context;
  double low, high;
  double magnitude;
} lora_rope_config;

/*
 * The frequencies of a rotation, on the host; no GPU call.
 *   rot_dim    even, 2 .. LORA_MAX_HEAD_DIM
 *   config     [host] nullable (= LORA_ROPE_NONE)
 *   inv_freq   [host] rot_dim / 2 doubles, written
 *   magnitude  [host] one double, written: the factor of cos and sin
 * A caller with frequencies of its own (one factor for each pair) skips this.
 */
lora_status lora_rope_frequencies(int32_t rot_dim, double base, const lora_rope_config *config, double *inv_freq,
                                  double *magnitude);

/*
 * The table of positions first .. first + n - 1:
 *     table[p][i]               = magnitude * cos((first + p) * inv_freq[i])
 *     table[p][rot_dim / 2 + i] = magnitude * sin((first + p) * inv_freq[i])
 * The angle, its cosine and sine are computed in 64 bits and rounded once.
 *   inv_freq   [host] rot_dim / 2 doubles
 *   first, n   >= 0; first + n <= 2^31
 *   table      [n][rot_dim] fp32 device, 16-byte aligned
 */
lora_status lora_rope_table(const double *inv_freq, int32_t rot_dim, double magnitude, int64_t first, int64_t n,
                            float *table, hipStream_t stream);

/* A paged cache of one layer: position p of a sequence lies in row
 * p % page_size of page page_table[p / page_size].  Element [page][head][row]
 * [0 .. d) of k starts at k + page * k_page + head * k_head + row * k_row
 * elements; v the same with its own strides. */
typedef struct {
  void *k, *v;
  int64_t k_page, k_head, k_row;
  int64_t v_page, v_head, v_row;
  int64_t n_pages;
  int32_t page_size;
} lora_kv_cache;

/*
 * Rotate the first rot_dim elements of every head of q and k by the row
 * table[positions[t]], copy the rest of the head, and optionally place the
 * rotated k and the v rows into a cache, in one pass.  With (a, b) a pair and
 * (c, s) its cosine and sine: a' = a c - b s, b' = b c + a s, in fp32, rounded
 * once.
 *   q, k, v      [T][ld] rows of q_heads * d (k, v: kv_heads * d) elements;
 *                v only with a cache; q_heads or kv_heads may be 0 (no q, no k)
 *   layout       a lora_rope_layout
 *   rot_dim      even, 2 .. d
 *   table        [n_positions][rot_dim] fp32
 *   positions    [T] int32; a token whose position is outside the table is
 *                padding: nothing of it is written
 *   q_out, k_out [T][ld]; may be q and k themselves (same pointer and stride)
 *                but not overlap them otherwise; k_out nullable with a cache
 *   cache        [host] nullable; its heads are kv_heads
 *   cache_rows   [T] int32, with a cache: page * page_size + row of each token;
 *                a token with a value outside the cache is not placed in it.
 *                Values of tokens that are placed must differ.
 */
lora_status lora_rotary(lora_dtype dt, const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v,
                        int64_t ldv, int32_t T, int32_t q_heads, int32_t kv_heads, int32_t d, int32_t layout,
                        int32_t rot_dim, const float *table, int64_t n_positions, const int32_t *positions,
                        void *q_out, int64_t ldqo, void *k_out, int64_t ldko, const lora_kv_cache *cache,
                        const int32_t *cache_rows, hipStream_t stream);

/*
 * The same with every head of q and k normed first, over its d elements:
 *     x[i] <- x[i] * w[i] / sqrt(mean(x^2) + eps)
 *   q_weight, k_weight   [d] of type dt, 16-byte aligned; nullable (= 1)
 *   eps                  >= 0
 */
lora_status lora_qk_norm_rotary(lora_dtype dt, const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v,
                                int64_t ldv, int32_t T, int32_t q_heads, int32_t kv_heads, int32_t d, int32_t layout,
                                int32_t rot_dim, const void *q_weight, const void *k_weight, float eps,
                                const float *table, int64_t n_positions, const int32_t *positions, void *q_out,
                                int64_t ldqo, void *k_out, int64_t ldko, const lora_kv_cache *cache,
                                const int32_t *cache_rows, hipStream_t stream);

/* ------------------------------------------------------------------------ */
/* Trees of drafted tokens                                                  */
/* ------------------------------------------------------------------------ */
/*
 * A step has B sequences; sequence b has context[b] tokens in the cache and
 * n_b = q_start[b + 1] - q_start[b] new tokens, its nodes: rows
 * q_start[b] .. of the step's T rows.  Node j of sequence b has the cache
 * position context[b] + j, whatever its depth in the tree.
 *
 * Device values are taken as far as they are sound: n_b is cut to
 * [0, max_nodes] and to the T rows, context[b] to [0, max_context], and
 * a key whose page is missing from the table or whose entry lies outside
 * [0, n_pages) (-1, say) is not read and counts as masked.
 */

/*
 * What a step's layers share, from the trees:
 *   parents     [T] int32 nullable: the node (within the sequence, smaller than
 *               the token's own) that a token follows, or -1 where it follows
 *               the context; other values count as -1.  NULL: a chain.
 *   mask        [T][mask_words] uint64, nullable: bit j of a row says that the
 *               token sees node j: itself and its ancestors
 *   mask_words  >= ceil(max_nodes / 64)
 *   positions   [T] int32, nullable: context[b] + the token's depth
 *   cache_rows  [T] int32, nullable: page * page_size + row of position
 *               context[b] + j; -1 where the table has no page for it
 *   page_table  [B][ld_table] int32, n_table columns (for cache_rows)
 * Rows of no sequence are not written.  max_nodes <= LORA_MAX_TREE_NODES
 * where parents are given.
 */
lora_status lora_build_tree(const int32_t *parents, int32_t T, int32_t B, const int32_t *q_start,
                            const int32_t *context, int32_t max_nodes, const int32_t *page_table, int64_t ld_table,
                            int32_t n_table, int64_t n_pages, int32_t page_size, uint64_t *mask, int32_t mask_words,
                            int32_t *positions, int32_t *cache_rows, hipStream_t stream);

/*
 * Attention of the step's T rows over the cache: with s_p = scale * q . k_p,
 *     out = sum_p softmax(s)_p v_p
 * over the keys p < context[b] and the nodes p = context[b] + j that the
 * token's mask row has (chain: j up to its own).  Scores, softmax statistics
 * and sums are fp32; the weights of a product with 16-bit v are rounded to
 * v's type, out is rounded once.  A row that sees no key gives 0 (lse
 * -infinity).  Masked keys and values may hold anything, NaN too.
 *   q, out      [T][ld] rows of q_heads * d; out may be q itself.  Rows of no
 *               sequence (a padded batch, nodes past max_nodes) are not written
 *   lse         nullable [T][q_heads] fp32: ln sum_p exp(s_p)
 *   max_nodes, max_context   [host] bounds of n_b and context[b]; the closer,
 *               the better the work is spread
 *   workspace   256-byte aligned, of lora_tree_attention_workspace_bytes for
 *               the same heads and sizes B, T, max_nodes and max_context that
 *               are not smaller than the call's; nullable where that is 0.  It
 *               needs no clearing and holds nothing between calls; calls that
 *               may overlap need distinct ones.
 */
size_t lora_tree_attention_workspace_bytes(int32_t B, int32_t T, int32_t max_nodes, int32_t max_context,
                                           int32_t q_heads, int32_t kv_heads, int32_t d);

lora_status lora_tree_attention(lora_dtype dt, const void *q, int64_t ldq, int32_t T, int32_t B, int32_t q_heads,
                                int32_t kv_heads, int32_t d, const lora_kv_cache *cache, const int32_t *page_table,
                                int64_t ld_table, int32_t n_table, const int32_t *context, const int32_t *q_start,
                                int32_t max_nodes, int32_t max_context, const uint64_t *mask, int32_t mask_words,
                                float scale, void *out, int64_t ldo, float *lse, void *workspace,
                                size_t workspace_bytes, hipStream_t stream);

/*
 * Keep the accepted path of every sequence's tree: for j < n_kept[b] the cache
 * row of position context[b] + path[b][j] moves to position context[b] + j, in
 * K and V of every layer.  A path's entries must ascend; it ends before the
 * first that does not (or is negative), and a row whose page is missing at
 * either end stays.
 *   cache       [host] the layers' strides and sizes, which they share; its k
 *               and v are not read
 *   k, v        [host] n_layers pointers each
 *   path        [B][ld_path] int32, n_path columns
 *   n_kept      [B] int32
 */
lora_status lora_keep_path(lora_dtype dt, const lora_kv_cache *cache, void *const *k, void *const *v,
                           int32_t n_layers, int32_t kv_heads, int32_t d, int32_t B, const int32_t *page_table, int64_t ld_table, int32_t n_table,
                           const int32_t *context, const int32_t *path, int64_t ld_path, int32_t n_path,
                           const int32_t *n_kept, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_ATTENTION_MI355X_H */
