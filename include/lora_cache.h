/*
 * lora_cache.h -- C ABI of a paged key/value cache held in 8 bits (the store
 * that fills it, the attention that reads it, the move of an accepted path in
 * it) and of the pages of a cache of any type: which sequences hold them, and
 * copying, forking, releasing and compacting them.
 *
 * A step over a quantized cache:
 *
 *     lora_reserve_pages   pages for the step's tokens
 *     lora_build_tree      masks, positions and cache rows, once
 *     per layer:
 *       lora_rotary or lora_qk_norm_rotary   q and k in place, no cache
 *       lora_store_quantized                 k and v into the cache
 *       lora_tree_attention_quantized        over context and drafted tokens
 *     lora_keep_path_quantized   after verification, every layer in one call
 *
 * The conventions of lora.h and lora_attention.h hold: device pointers unless
 * marked [host], caller-owned buffers, asynchronous calls ordered on `stream`,
 * checks on the host before anything is enqueued, no allocation, no
 * synchronisation and no state between calls, so every call can be captured in
 * a HIP graph.
 */
#ifndef LORA_CACHE_MI355X_H
#define LORA_CACHE_MI355X_H

#include "lora_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------ */
/* A cache in 8 bits                                                        */
/* ------------------------------------------------------------------------ */

/* What a byte holds: E4M3 a float of 4 exponent and 3 mantissa bits (largest
 * 448, NaN but no infinity), INT8 a whole number from -127 to 127 (a stored
 * -128 is read as -128). */
typedef LORA_ENUM { LORA_CACHE_E4M3 = 0, LORA_CACHE_INT8 = 1 } lora_cache_format;

/* One layer of a quantized cache.  A page's rows are cut into blocks of `block`
 * rows (a divisor of page_size); a block of a head has one exponent e, keys and
 * values each their own, and a byte's value is its number times 2^e.  Exponents
 * lie from -126 to 119 (E4M3) or 121 (INT8), where every value is finite in
 * fp32; others are read as the nearest of these.  Powers of two: raising a
 * block's exponent is then exact but for numbers that fall below the format's
 * grid, and so is the conversion to the 16-bit operands of the products.
 *   k, v           as in lora_kv_cache, one byte an element; strides in bytes,
 *                  multiples of 16 (as head_dim then is)
 *   k_exp, v_exp   [page][head][block] int8, unit stride over the blocks of a page
 * With n_pages = 0 none of the pointers is read: nothing is placed or moved, and no
 * sequence has keys. */
typedef struct {
  void *k, *v;
  int8_t *k_exp, *v_exp;
  int64_t k_page, k_head, k_row;
  int64_t v_page, v_head, v_row;
  int64_t k_exp_page, k_exp_head, v_exp_page, v_exp_head;
  int64_t n_pages;
  int32_t page_size, block;
  int32_t format; /* a lora_cache_format */
} lora_quantized_cache;

/*
 * Put the rows of k and v into the cache: token t's at cache_rows[t] = page *
 * page_size + row (from lora_build_tree; one outside the cache is not placed).
 * The tokens of one block have to be neighbours in k and v, in ascending and
 * consecutive rows, as the tokens of a sequence are.  Rows of a block before
 * its first new one are taken to hold the sequence's earlier tokens, those
 * behind its last new one to hold nothing.  With a the largest finite magnitude
 * of a block's new rows in a head, M the format's largest number:
 *     e' = the least exponent with a <= M 2^e'
 *     e  = max(e', the block's exponent) where it has earlier rows, else e'
 * Earlier rows change from q to q 2^(old - e) where the exponent grows, new
 * rows are x 2^-e, both rounded to the nearest number (ties to even).
 * Infinities become the largest number; a NaN stays one in E4M3 and becomes 0
 * in INT8; neither has a part in a.
 *   dt     of k and v: [T][ld] rows of kv_heads * d elements
 *   d      a multiple of 16, up to LORA_MAX_HEAD_DIM
 *   cache  [host]
 */
lora_status lora_store_quantized(lora_dtype dt, const void *k, int64_t ldk, const void *v, int64_t ldv, int32_t T,
                                 int32_t kv_heads, int32_t d, const lora_quantized_cache *cache,
                                 const int32_t *cache_rows, hipStream_t stream);

/*
 * lora_tree_attention over a quantized cache: the same rows, masks, bounds and
 * workspace rules (the bytes from lora_quantized_workspace_bytes).
 *   dt   of q and out.  Keys and values enter the products as they are held,
 *        exactly.  q is exact too; the softmax weights, times the power of two
 *        of their value's block, are rounded to 8 bits for bf16, 11 at least
 *        for fp16 and 24 for fp32.  fp16 calls of more than 32 rows a key head
 *        (max_nodes times the q_heads / kv_heads heads that share it) round such
 *        a product to 11 bits down to 2^-26 of the row's largest one, to steps of
 *        2^-36 of that below.  Sums hold every value: an output is infinite only
 *        where it is beyond its type.
 */
size_t lora_quantized_workspace_bytes(int32_t B, int32_t T, int32_t max_nodes, int32_t max_context, int32_t q_heads,
                                      int32_t kv_heads, int32_t d);

lora_status lora_tree_attention_quantized(lora_dtype dt, const void *q, int64_t ldq, int32_t T, int32_t B,
                                          int32_t q_heads, int32_t kv_heads, int32_t d,
                                          const lora_quantized_cache *cache, const int32_t *page_table,
                                          int64_t ld_table, int32_t n_table, const int32_t *context,
                                          const int32_t *q_start, int32_t max_nodes, int32_t max_context,
                                          const uint64_t *mask, int32_t mask_words, float scale, void *out,
                                          int64_t ldo, float *lse, void *workspace, size_t workspace_bytes,
                                          hipStream_t stream);

/*
 * lora_keep_path over quantized caches.  A block that takes kept rows gets the
 * largest exponent of the blocks that they come from, and of its own where it
 * has rows of the context; rows are rounded again (to the nearest, ties to
 * even) where their exponent grows.  Rows behind the kept ones hold nothing
 * afterwards.  An exponent that a token raised which is not kept stays where its
 * block has rows of the context: they have been rounded for it.
 *   cache                  [host] strides and sizes of every layer; its pointers
 *                          are not read
 *   k, v, k_exp, v_exp     [host] n_layers pointers each, no address twice in all (checked)
 */
lora_status lora_keep_path_quantized(const lora_quantized_cache *cache, void *const *k, void *const *v,
                                     int8_t *const *k_exp, int8_t *const *v_exp, int32_t n_layers, int32_t kv_heads,
                                     int32_t d, int32_t B, const int32_t *page_table, int64_t ld_table,
                                     int32_t n_table, const int32_t *context, const int32_t *path, int64_t ld_path,
                                     int32_t n_path, const int32_t *n_kept, hipStream_t stream);

/* ------------------------------------------------------------------------ */
/* Pages                                                                    */
/* ------------------------------------------------------------------------ */
/*
 * A pool of n_pages pages: refs [n_pages] int32 says how many entries of page
 * tables name a page; 0 (or less): it is free.  A page table [B][ld_table] int32,
 * n_table columns, has -1 where a sequence holds no page.  Every layer's cache
 * has the same pages, so one table and one refs serve all of them.
 *
 * Entries outside [0, n_pages) count as -1.  Free pages are taken from the
 * lowest number on, so the same calls give the same pages.  The calls that take
 * or move pages need a workspace of lora_pages_workspace_bytes (4-byte aligned,
 * no clearing, nothing kept in it; calls that may overlap need distinct ones).
 * Calls on one pool have to follow one another.
 *
 * A page that several sequences hold is not to be written.  Forks see to that:
 * what follows a sequence's tokens lies on a page of its own.  A sequence that
 * goes back to a length inside a page that it shares is forked at that length.
 */
#define LORA_MAX_POOL_PAGES (1 << 28)
size_t lora_pages_workspace_bytes(int64_t n_pages, int32_t n_seqs);

/* A tensor with pages: page p is n_outer x n_inner runs of `run` bytes, the
 * strides between them in bytes. */
typedef struct {
  void *data;
  int64_t page, outer, inner;
  int32_t n_outer, n_inner, run;
} lora_paged_tensor;

/*
 * Pages for sequences to grow into: of each sequence b, the entries of the
 * columns below ceil(lengths[b] / page_size) that are -1 get a free page each
 * (refs becomes 1), in the order of sequences and columns.  Where free pages run
 * out the rest stays -1.
 *   lengths   [B] int32
 *   missing   nullable, one int32, written: entries that got no page
 */
lora_status lora_reserve_pages(int32_t *refs, int64_t n_pages, int32_t *page_table, int64_t ld_table, int32_t n_table,
                               int32_t B, const int32_t *lengths, int32_t page_size, int32_t *missing, void *workspace,
                               size_t workspace_bytes, hipStream_t stream);

/*
 * Fork f makes row children[f] of to_table a sequence with the first lengths[f]
 * tokens of row parents[f] of from_table: it shares the pages that are full
 * (refs + 1) and gets a free page (refs = 1) for one that is filled in part;
 * its other entries become -1.  The free pages go to the forks in their order.
 * What the partly filled pages hold is copied in every tensor.
 *   from_table, to_table   [B][..], n_table columns each; may be the same where
 *                          no child is a parent of the call.  What a child's row
 *                          held before is overwritten, not released.
 *   parents, children, lengths   [n_forks] int32; children must differ.  A fork
 *                          with a child outside [0, B_to) does nothing, with a
 *                          parent outside [0, B_from) it makes an empty sequence
 *   source, target         [n_forks] int32, written: the page that was copied and
 *                          where to, -1 where there is none
 *   missing                nullable, one int32, written: forks whose partly
 *                          filled page got no free one (their entry is -1)
 *   tensors                [host] n_tensors of them, maybe none
 */
lora_status lora_fork_sequences(int32_t *refs, int64_t n_pages, const int32_t *from_table, int64_t ld_from, int32_t B_from,
                                int32_t *to_table, int64_t ld_to, int32_t B_to, int32_t n_table,
                                const int32_t *parents, const int32_t *children, const int32_t *lengths,
                                int32_t n_forks, int32_t page_size, int32_t *source, int32_t *target, int32_t *missing,
                                const lora_paged_tensor *tensors, int32_t n_tensors, void *workspace,
                                size_t workspace_bytes, hipStream_t stream);

/*
 * Give pages back: of each row listed, the entries from column
 * ceil(keep / page_size) on become -1, and the pages that they named have one
 * reference less.
 *   rows   [n] int32, rows of the table (one outside [0, B) is passed over; one
 *          listed twice is released once); NULL: all of them, n = B
 *   keep   [n] int32 tokens, nullable (= 0)
 */
lora_status lora_release_pages(int32_t *refs, int64_t n_pages, int32_t *page_table, int64_t ld_table, int32_t n_table,
                               int32_t B, const int32_t *rows, const int32_t *keep, int32_t n, int32_t page_size,
                               hipStream_t stream);

/*
 * Make the pages in use the lowest ones: with n_live of them, each page in use
 * whose number is n_live or more moves to a free one below it, both in ascending
 * order.  refs and page_table follow, and what the pages hold is copied in every
 * tensor.  Every entry that names a page of the pool has to be in this table.
 *   source, target     [n_pages / 2] int32, written as far as there are moves
 *   n_live, n_moves    one int32 each, written
 *   tensors            [host] n_tensors of them, maybe none
 */
lora_status lora_compact_pages(int32_t *refs, int64_t n_pages, int32_t *page_table, int64_t ld_table, int32_t n_table,
                               int32_t B, int32_t *source, int32_t *target, int32_t *n_live, int32_t *n_moves,
                               const lora_paged_tensor *tensors, int32_t n_tensors, void *workspace,
                               size_t workspace_bytes, hipStream_t stream);

/*
 * Copy page source[i] to page target[i] in every tensor, i < n (or *count, if
 * that is less).  Pairs with a number outside [0, n_pages) are passed over.  No
 * target may be the source or target of another pair.
 *   tensors          [host]
 *   source, target   [n] int32
 *   count            nullable, one int32
 */
lora_status lora_copy_pages(const lora_paged_tensor *tensors, int32_t n_tensors, int64_t n_pages,
                            const int32_t *source, const int32_t *target, int32_t n, const int32_t *count,
                            hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_CACHE_MI355X_H */
