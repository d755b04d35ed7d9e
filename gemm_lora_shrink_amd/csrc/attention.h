// Internal definitions of the operators after the q/k/v projection (rotary
// positions, paged cache, tree attention): the parameter blocks passed to
// their kernels and the host launchers.
#pragma once

#include "../../include/lora_attention.h"
#include "common.h"

namespace lora {

// Division of 0 <= n < 2^31 by a fixed d >= 1 with one high product: for
// 2^l >= d > 2^(l - 1) and m = floor(2^32 (2^l - d) / d) + 1 the quotient is
// (mulhi(n, m) + n) >> l (the method of invariant multiplication of Granlund
// and Montgomery); the sum stays below 2^32 as mulhi(n, m) <= n.
struct FastDiv {
  uint32_t d, mul, shift;
  __device__ inline uint32_t div(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
};
inline FastDiv fast_div(uint32_t d) {
  uint32_t l = 0;
  while (((uint64_t)1 << l) < d) ++l;
  const uint64_t m = ((((uint64_t)1 << l) - d) << 32) / d + 1;
  return FastDiv{d, (uint32_t)m, l};
}

// A paged cache of one layer as the kernels see it (strides in elements).
struct CacheView {
  void *k, *v;
  int64_t k_page, k_head, k_row, v_page, v_head, v_row;
  int64_t n_pages;
  FastDiv page;  // by the page size
};

struct RotaryParams {
  const void *q, *k, *v;
  void *q_out, *k_out;  // k_out nullable
  int64_t ldq, ldk, ldv, ldqo, ldko;
  const void *qw, *kw;  // nullable
  const float* table;
  const int32_t* positions;
  const int32_t* cache_rows;  // with a cache
  CacheView cache;            // cache.k null: none
  int64_t n_positions;
  int64_t n_rows;  // n_pages * page_size
  int32_t T, hq, hk, d, rot, layout;
  int32_t norm;
  float eps;
  // filled by the launcher: heads walked by one lane group, groups of a token
  int32_t lane_shift, units;
  FastDiv groups;
};

struct BuildTreeParams {
  const int32_t *parents, *q_start, *context, *page_table;
  int64_t ld_table, n_pages;
  uint64_t* mask;
  int32_t *positions, *cache_rows;
  int32_t T, B, max_nodes, n_table, mask_words;
  FastDiv page;
};

struct KeepParams {
  const int32_t *page_table, *context, *path, *n_kept;
  int64_t ld_table, ld_path, n_pages;
  int64_t k_page, k_head, k_row, v_page, v_head, v_row;  // bytes
  int32_t n_table, n_path, row_bytes;
  FastDiv page;
  void* k[LORA_MAX_KEEP_LAYERS];
  void* v[LORA_MAX_KEEP_LAYERS];
};

struct AttendParams {
  const void* q;
  void* out;
  int64_t ldq, ldo;
  float* lse;  // nullable
  CacheView cache;
  const int32_t *page_table, *context, *q_start;
  const uint64_t* mask;  // nullable: a chain
  int64_t ld_table;
  float scale;
  int32_t T, B, hq, hk, d, n_table, max_nodes, max_context, mask_words;
  FastDiv group;  // by q_heads / kv_heads
  float* part;    // workspace
  // filled by the launcher (AttendPlan)
  int32_t chunk, splits, row_tiles, part_rows;
  FastDiv by_tiles, by_splits, by_sequences, by_heads, by_chunk;
};

hipError_t launch_rope_table(const double* inv_freq, int32_t rot, double magnitude, int64_t first, int64_t n,
                             float* table, hipStream_t stream);
// Whether launch_rotary's grid holds T tokens of `heads` heads (q, k and cached v).
bool rotary_fits(int32_t T, int heads, int32_t d, int32_t rot);
hipError_t launch_rotary(lora_dtype dt, RotaryParams p, hipStream_t stream);
hipError_t launch_build_tree(const BuildTreeParams& p, hipStream_t stream);
hipError_t launch_keep_path(const KeepParams& p, int32_t n_layers, int32_t kv_heads, int32_t B, hipStream_t stream);
hipError_t launch_attend(lora_dtype dt, const AttendParams& p, hipStream_t stream);
// Whether launch_attend's grids hold the work of these sizes.
bool attend_fits(lora_dtype dt, int32_t B, int32_t max_nodes, int32_t max_context, int32_t hq, int32_t hk, int32_t d);
// Bytes of workspace launch_attend needs for these sizes (0: none), and the most it
// needs for any type and any sizes up to these.
int64_t attend_need_bytes(lora_dtype dt, int32_t B, int32_t T, int32_t max_nodes, int32_t max_context, int32_t hq,
                          int32_t hk, int32_t d);
int64_t attend_most_bytes(int32_t B, int32_t T, int32_t max_nodes, int32_t max_context, int32_t hq, int32_t hk,
                          int32_t d);

}  // namespace lora
