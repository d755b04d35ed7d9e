// C ABI entry points of the quantized cache and the pages of a cache
// (include/lora_cache.h): host-side argument checks and dispatch.  Every check
// runs before anything is enqueued.
#include <math.h>

#include <algorithm>

#include "cache.h"

#define LORA_EXPORT extern "C" __attribute__((visibility("default")))

namespace lora {
namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 31;

lora_status check_quantized_heads(int32_t q_heads, int32_t kv_heads, int32_t d) {
  if (d < 1) return fail(LORA_ERR_INVALID_ARG, "head_dim = %d must be >= 1", d);
  if (d % 16 || d > LORA_MAX_HEAD_DIM)
    return fail(LORA_ERR_UNSUPPORTED, "head_dim = %d of a quantized cache must be a multiple of 16 up to %d", d,
                LORA_MAX_HEAD_DIM);
  if (q_heads < 1 || kv_heads < 1) return fail(LORA_ERR_INVALID_ARG, "the numbers of heads must be >= 1");
  if (q_heads > LORA_MAX_HEADS || kv_heads > LORA_MAX_HEADS)
    return fail(LORA_ERR_UNSUPPORTED, "more than %d heads", LORA_MAX_HEADS);
  return LORA_OK;
}

lora_status check_rows(lora_dtype dt, const char* name, const void* p, int64_t ld, int64_t width) {
  if (!p) return fail(LORA_ERR_INVALID_ARG, "%s is null", name);
  if (!aligned16(p)) return fail(LORA_ERR_UNSUPPORTED, "%s must be 16-byte aligned", name);
  if (ld < width) return fail(LORA_ERR_INVALID_ARG, "the row stride of %s, %lld, is smaller than its %lld elements", name,
                              (long long)ld, (long long)width);
  if (ld % vec_of(dt))
    return fail(LORA_ERR_UNSUPPORTED, "the row stride of %s must be a multiple of %d elements", name, vec_of(dt));
  return LORA_OK;
}

lora_status check_format(const lora_quantized_cache& c) {
  if (c.format != LORA_CACHE_E4M3 && c.format != LORA_CACHE_INT8)
    return fail(LORA_ERR_INVALID_ARG, "unknown cache format %d", (int)c.format);
  if (c.page_size < 1) return fail(LORA_ERR_INVALID_ARG, "page_size = %d must be >= 1", c.page_size);
  if (c.block < 1 || c.page_size % c.block)
    return fail(LORA_ERR_INVALID_ARG, "block = %d must divide page_size = %d", c.block, c.page_size);
  if (c.n_pages < 0) return fail(LORA_ERR_INVALID_ARG, "n_pages is negative");
  const int64_t strides[6] = {c.k_page, c.k_head, c.k_row, c.v_page, c.v_head, c.v_row};
  for (int64_t s : strides) {
    if (s < 0) return fail(LORA_ERR_INVALID_ARG, "a cache stride is negative");
    if (s % 16) return fail(LORA_ERR_UNSUPPORTED, "cache strides must be multiples of 16 bytes");
  }
  const int64_t of_exps[4] = {c.k_exp_page, c.k_exp_head, c.v_exp_page, c.v_exp_head};
  for (int64_t s : of_exps)
    if (s < 0) return fail(LORA_ERR_INVALID_ARG, "a stride of the exponents is negative");
  return LORA_OK;
}

lora_status check_pointers(const void* k, const void* v, const int8_t* k_exp, const int8_t* v_exp) {
  if (!k || !v || !k_exp || !v_exp) return fail(LORA_ERR_INVALID_ARG, "the cache's k, v, k_exp or v_exp is null");
  if (!aligned16(k) || !aligned16(v)) return fail(LORA_ERR_UNSUPPORTED, "the cache must be 16-byte aligned");
  return LORA_OK;
}

// Whether some address comes twice among n of each list (n <= LORA_MAX_KEEP_LAYERS).
bool any_twice(const void* const* const (&lists)[4], int n) {
  const void* seen[8 * LORA_MAX_KEEP_LAYERS];
  uint32_t slots = 8;  // a power of two of which half stay empty
  while (slots < 8 * (uint32_t)n) slots *= 2;
  static_assert((LORA_MAX_KEEP_LAYERS & (LORA_MAX_KEEP_LAYERS - 1)) == 0, "");
  std::fill_n(seen, slots, nullptr);
  for (const void* const* list : lists)
    for (int i = 0; i < n; ++i) {
      uint32_t at = (uint32_t)((reinterpret_cast<uintptr_t>(list[i]) * 0x9e3779b97f4a7c15ull) >> 40);
      for (; seen[at % slots]; ++at)
        if (seen[at % slots] == list[i]) return true;
      seen[at % slots] = list[i];
    }
  return false;
}

QuantizedView view_of(const lora_quantized_cache& c) {
  return QuantizedView{c.k,      c.v,          c.k_exp,      c.v_exp,      c.k_page,
                       c.k_head, c.k_row,      c.v_page,     c.v_head,     c.v_row,
                       c.k_exp_page, c.k_exp_head, c.v_exp_page, c.v_exp_head, c.n_pages,
                       fast_div((uint32_t)c.page_size), fast_div((uint32_t)c.block)};
}

lora_status check_table(const int32_t* page_table, int64_t ld_table, int32_t n_table, int32_t B) {
  if (n_table < 0) return fail(LORA_ERR_INVALID_ARG, "n_table = %d is negative", n_table);
  if (B > 0 && n_table > 0 && !page_table) return fail(LORA_ERR_INVALID_ARG, "page_table is null");
  if (ld_table < n_table) return fail(LORA_ERR_INVALID_ARG, "ld_table is smaller than n_table");
  return LORA_OK;
}

lora_status check_sequences(int32_t B) {
  if (B < 0) return fail(LORA_ERR_INVALID_ARG, "B = %d is negative", B);
  if (B > 65535) return fail(LORA_ERR_UNSUPPORTED, "B = %d exceeds 65535", B);
  return LORA_OK;
}

lora_status check_attend_sizes(int32_t B, int32_t T, int32_t max_nodes, int32_t max_context, int32_t q_heads,
                               int32_t kv_heads, int32_t d) {
  if (T < 0) return fail(LORA_ERR_INVALID_ARG, "T = %d is negative", T);
  lora_status st = check_sequences(B);
  if (st != LORA_OK) return st;
  if (max_nodes < 1) return fail(LORA_ERR_INVALID_ARG, "max_nodes = %d must be >= 1", max_nodes);
  if (max_context < 0) return fail(LORA_ERR_INVALID_ARG, "max_context = %d is negative", max_context);
  if ((st = check_quantized_heads(q_heads, kv_heads, d)) != LORA_OK) return st;
  if (q_heads % kv_heads)
    return fail(LORA_ERR_INVALID_ARG, "q_heads = %d must be a multiple of kv_heads = %d", q_heads, kv_heads);
  if ((int64_t)max_context + max_nodes >= kMaxRows)
    return fail(LORA_ERR_UNSUPPORTED, "max_context + max_nodes reaches 2^31");
  if ((int64_t)max_nodes * (q_heads / kv_heads) >= (int64_t)1 << 27)
    return fail(LORA_ERR_UNSUPPORTED, "max_nodes times the heads of a group reaches 2^27");
  return LORA_OK;
}

lora_status check_pool(const int32_t* refs, int64_t n_pages, const int32_t* table, int64_t ld_table, int32_t n_table,
                       int32_t B) {
  if (n_pages < 0) return fail(LORA_ERR_INVALID_ARG, "n_pages is negative");
  if (n_pages > LORA_MAX_POOL_PAGES)
    return fail(LORA_ERR_UNSUPPORTED, "n_pages = %lld exceeds %d", (long long)n_pages, LORA_MAX_POOL_PAGES);
  if (n_pages > 0 && !refs) return fail(LORA_ERR_INVALID_ARG, "refs is null");
  lora_status st = check_sequences(B);
  if (st != LORA_OK) return st;
  return B > 0 ? check_table(table, ld_table, n_table, B) : LORA_OK;
}

lora_status check_workspace(const void* workspace, size_t bytes, int64_t n_pages, int32_t n_seqs) {
  const int64_t need = pages_scratch_bytes(n_pages, n_seqs);
  if (!workspace) return fail(LORA_ERR_INVALID_ARG, "workspace is null");
  if (reinterpret_cast<uintptr_t>(workspace) & 3u)
    return fail(LORA_ERR_INVALID_ARG, "workspace must be 4-byte aligned");
  if (bytes < (size_t)need)
    return fail(LORA_ERR_INVALID_ARG, "workspace has %zu bytes, the call needs %lld", bytes, (long long)need);
  return LORA_OK;
}

lora_status check_tensors(const lora_paged_tensor* tensors, int32_t n_tensors, int64_t n_pages) {
  if (n_tensors < 0) return fail(LORA_ERR_INVALID_ARG, "n_tensors = %d is negative", n_tensors);
  if (n_tensors > 0 && !tensors) return fail(LORA_ERR_INVALID_ARG, "tensors is null");
  for (int i = 0; i < n_tensors; ++i) {
    const lora_paged_tensor& t = tensors[i];
    if (!t.data && n_pages > 0) return fail(LORA_ERR_INVALID_ARG, "tensor %d has no data", i);
    if (t.n_outer < 1 || t.n_inner < 1 || t.run < 1)
      return fail(LORA_ERR_INVALID_ARG, "the pages of tensor %d hold nothing", i);
    if (t.page < 0 || t.outer < 0 || t.inner < 0) return fail(LORA_ERR_INVALID_ARG, "a stride of tensor %d is negative", i);
    if ((double)t.n_outer * t.n_inner * t.run >= 2147483648.0)
      return fail(LORA_ERR_UNSUPPORTED, "a page of tensor %d has 2 GiB or more", i);
  }
  return LORA_OK;
}

// The widest access that the tensor's addresses and runs allow.
PagedTensor tensor_of(const lora_paged_tensor& t) {
  const uint64_t all = reinterpret_cast<uintptr_t>(t.data) | (uint64_t)t.page | (uint64_t)t.run |
                       (t.n_outer > 1 ? (uint64_t)t.outer : 0) | (t.n_inner > 1 ? (uint64_t)t.inner : 0);
  const uint32_t unit = all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : 1, run = (uint32_t)t.run / unit;
  return PagedTensor{static_cast<char*>(t.data), t.page, t.outer, t.inner, run * t.n_outer * t.n_inner, run,
                     (uint32_t)t.n_inner, (uint16_t)unit, (uint16_t)(t.n_outer == 1 && t.n_inner == 1)};
}

// The tensors' copies, kCopyTensors a launch, p.task beside the first of them.
hipError_t move_all(MoveParams& p, const lora_paged_tensor* tensors, int32_t n_tensors, hipStream_t stream) {
  int i = 0;
  do {
    for (p.n_tensors = 0; p.n_tensors < kCopyTensors && i < n_tensors; ++i) p.t[p.n_tensors++] = tensor_of(tensors[i]);
    const hipError_t e = launch_move(p, stream);
    if (e != hipSuccess) return e;
    p.task = MoveParams::kNone;
  } while (i < n_tensors);
  return hipSuccess;
}

PoolParams pool_of(int32_t* refs, int64_t n_pages, int32_t* table, int64_t ld_table, int32_t n_table, int32_t B,
                   int32_t page_size, void* workspace) {
  return PoolParams{refs, n_pages, table, ld_table, n_table, B, fast_div((uint32_t)page_size),
                    static_cast<int32_t*>(workspace)};
}

}  // namespace
}  // namespace lora

using namespace lora;

LORA_EXPORT lora_status lora_store_quantized(lora_dtype dt, const void* k, int64_t ldk, const void* v, int64_t ldv,
                                             int32_t T, int32_t kv_heads, int32_t d, const lora_quantized_cache* cache,
                                             const int32_t* cache_rows, hipStream_t stream) {
  clear_error();
  if (!valid_dtype(dt)) return fail(LORA_ERR_INVALID_ARG, "unknown dtype %d", dt);
  if (T < 0) return fail(LORA_ERR_INVALID_ARG, "T = %d is negative", T);
  lora_status st = check_quantized_heads(1, kv_heads, d);
  if (st != LORA_OK) return st;
  if (!cache) return fail(LORA_ERR_INVALID_ARG, "cache is null");
  if ((st = check_format(*cache)) != LORA_OK) return st;
  if (cache->n_pages > kMaxRows / cache->page_size)
    return fail(LORA_ERR_UNSUPPORTED, "the cache has more rows than cache_rows can name");
  if (!store_quantized_fits(T)) return fail(LORA_ERR_UNSUPPORTED, "T = %d tokens are more than a launch holds", T);
  if (T == 0) return LORA_OK;
  if (cache->n_pages > 0 && (st = check_pointers(cache->k, cache->v, cache->k_exp, cache->v_exp)) != LORA_OK) return st;
  const int64_t width = (int64_t)kv_heads * d;
  if ((st = check_rows(dt, "k", k, ldk, width)) != LORA_OK) return st;
  if ((st = check_rows(dt, "v", v, ldv, width)) != LORA_OK) return st;
  if (!cache_rows) return fail(LORA_ERR_INVALID_ARG, "cache_rows is null");
  if (cache->n_pages == 0) return LORA_OK;
  StoreParams p{};
  p.k = k;
  p.v = v;
  p.ldk = ldk;
  p.ldv = ldv;
  p.cache = view_of(*cache);
  p.rows = cache_rows;
  p.n_rows = cache->n_pages * cache->page_size;
  p.T = T;
  p.hk = kv_heads;
  p.d = d;
  const hipError_t e = launch_store_quantized(dt, cache->format, p, stream);
  if (e != hipSuccess) return hip_fail(e, "quantized store launch");
  return LORA_OK;
}

LORA_EXPORT size_t lora_quantized_workspace_bytes(int32_t B, int32_t T, int32_t max_nodes, int32_t max_context,
                                                  int32_t q_heads, int32_t kv_heads, int32_t d) {
  if (check_attend_sizes(B, T, max_nodes, max_context, q_heads, kv_heads, d) != LORA_OK) return 0;
  return (size_t)attend_quantized_most_bytes(B, T, max_nodes, max_context, q_heads, kv_heads, d);
}

LORA_EXPORT lora_status lora_tree_attention_quantized(lora_dtype dt, const void* q, int64_t ldq, int32_t T, int32_t B,
                                                      int32_t q_heads, int32_t kv_heads, int32_t d,
                                                      const lora_quantized_cache* cache, const int32_t* page_table,
                                                      int64_t ld_table, int32_t n_table, const int32_t* context,
                                                      const int32_t* q_start, int32_t max_nodes, int32_t max_context,
                                                      const uint64_t* mask, int32_t mask_words, float scale, void* out,
                                                      int64_t ldo, float* lse, void* workspace, size_t workspace_bytes,
                                                      hipStream_t stream) {
  clear_error();
  if (!valid_dtype(dt)) return fail(LORA_ERR_INVALID_ARG, "unknown dtype %d", dt);
  lora_status st = check_attend_sizes(B, T, max_nodes, max_context, q_heads, kv_heads, d);
  if (st != LORA_OK) return st;
  if (!isfinite(scale)) return fail(LORA_ERR_INVALID_ARG, "scale is not finite");
  if (mask) {
    if (max_nodes > LORA_MAX_TREE_NODES)
      return fail(LORA_ERR_UNSUPPORTED, "max_nodes = %d exceeds %d with a mask", max_nodes, LORA_MAX_TREE_NODES);
    if (mask_words < (max_nodes + 63) / 64)
      return fail(LORA_ERR_INVALID_ARG, "mask_words = %d is too small for %d nodes", mask_words, max_nodes);
    if (reinterpret_cast<uintptr_t>(mask) & 7u) return fail(LORA_ERR_UNSUPPORTED, "mask must be 8-byte aligned");
  }
  if ((st = check_table(page_table, ld_table, n_table, B)) != LORA_OK) return st;
  if (!cache) return fail(LORA_ERR_INVALID_ARG, "cache is null");
  if ((st = check_format(*cache)) != LORA_OK) return st;
  if (T == 0 || B == 0) return LORA_OK;
  if (!context || !q_start) return fail(LORA_ERR_INVALID_ARG, "context or q_start is null");
  if (cache->n_pages > 0 && (st = check_pointers(cache->k, cache->v, cache->k_exp, cache->v_exp)) != LORA_OK) return st;
  const int64_t most = ((int64_t)1 << 32) - 1;
  if (cache->k_page > most || cache->v_page > most || cache->k_row > most || cache->v_row > most ||
      cache->k_exp_page > most || cache->v_exp_page > most)
    return fail(LORA_ERR_UNSUPPORTED, "a page or row of the cache spans 4 GiB");
  if (!attend_quantized_fits(dt, B, max_nodes, max_context, q_heads, kv_heads, d))
    return fail(LORA_ERR_UNSUPPORTED, "B = %d sequences of up to %d nodes are more than a launch holds", B, max_nodes);
  const int64_t need = attend_quantized_need_bytes(dt, B, T, max_nodes, max_context, q_heads, kv_heads, d);
  if (need > 0) {
    if (!workspace) return fail(LORA_ERR_INVALID_ARG, "workspace is null");
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
      return fail(LORA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    if (workspace_bytes < (size_t)need)
      return fail(LORA_ERR_INVALID_ARG, "workspace has %zu bytes, the call needs %lld", workspace_bytes,
                  (long long)need);
  }
  const int64_t width = (int64_t)q_heads * d;
  if ((st = check_rows(dt, "q", q, ldq, width)) != LORA_OK) return st;
  if ((st = check_rows(dt, "out", out, ldo, width)) != LORA_OK) return st;
  if (out == q && ldo != ldq) return fail(LORA_ERR_INVALID_ARG, "out is q with another row stride");
  AttendQuantizedParams p{};
  p.q = q;
  p.out = out;
  p.ldq = ldq;
  p.ldo = ldo;
  p.lse = lse;
  p.cache = CacheView{cache->k,      cache->v,     cache->k_page, cache->k_head, cache->k_row,
                      cache->v_page, cache->v_head, cache->v_row, cache->n_pages, fast_div((uint32_t)cache->page_size)};
  p.k_exp = cache->k_exp;
  p.v_exp = cache->v_exp;
  p.k_exp_page = cache->k_exp_page;
  p.k_exp_head = cache->k_exp_head;
  p.v_exp_page = cache->v_exp_page;
  p.v_exp_head = cache->v_exp_head;
  p.block = fast_div((uint32_t)cache->block);
  p.page_table = page_table;
  p.context = context;
  p.q_start = q_start;
  p.mask = mask;
  p.ld_table = ld_table;
  p.scale = scale;
  p.T = T;
  p.B = B;
  p.hq = q_heads;
  p.hk = kv_heads;
  p.d = d;
  p.n_table = n_table;
  p.max_nodes = max_nodes;
  p.max_context = max_context;
  p.mask_words = mask_words;
  p.group = fast_div((uint32_t)(q_heads / kv_heads));
  p.part = static_cast<float*>(workspace);
  const hipError_t e = launch_attend_quantized(dt, cache->format, p, stream);
  if (e != hipSuccess) return hip_fail(e, "quantized tree attention launch");
  return LORA_OK;
}

LORA_EXPORT lora_status lora_keep_path_quantized(const lora_quantized_cache* cache, void* const* k, void* const* v,
                                                 int8_t* const* k_exp, int8_t* const* v_exp, int32_t n_layers,
                                                 int32_t kv_heads, int32_t d, int32_t B, const int32_t* page_table,
                                                 int64_t ld_table, int32_t n_table, const int32_t* context,
                                                 const int32_t* path, int64_t ld_path, int32_t n_path,
                                                 const int32_t* n_kept, hipStream_t stream) {
  clear_error();
  lora_status st = check_sequences(B);
  if (st != LORA_OK) return st;
  if ((st = check_quantized_heads(1, kv_heads, d)) != LORA_OK) return st;
  if (n_layers < 0) return fail(LORA_ERR_INVALID_ARG, "n_layers = %d is negative", n_layers);
  if (n_layers > LORA_MAX_KEEP_LAYERS)
    return fail(LORA_ERR_UNSUPPORTED, "n_layers = %d exceeds %d", n_layers, LORA_MAX_KEEP_LAYERS);
  if (n_path < 0) return fail(LORA_ERR_INVALID_ARG, "n_path = %d is negative", n_path);
  if (n_path > LORA_MAX_KEEP_PATH)
    return fail(LORA_ERR_UNSUPPORTED, "n_path = %d exceeds %d", n_path, LORA_MAX_KEEP_PATH);
  if (ld_path < n_path) return fail(LORA_ERR_INVALID_ARG, "ld_path is smaller than n_path");
  if ((st = check_table(page_table, ld_table, n_table, B)) != LORA_OK) return st;
  if (!cache) return fail(LORA_ERR_INVALID_ARG, "cache is null");
  if ((st = check_format(*cache)) != LORA_OK) return st;
  if (B == 0 || n_layers == 0 || n_path == 0) return LORA_OK;
  if (!k || !v || !k_exp || !v_exp || !context || !path || !n_kept)
    return fail(LORA_ERR_INVALID_ARG, "k, v, k_exp, v_exp, context, path or n_kept is null");
  if (cache->n_pages == 0) return LORA_OK;
  for (int i = 0; i < n_layers; ++i)
    if ((st = check_pointers(k[i], v[i], k_exp[i], v_exp[i])) != LORA_OK) return st;
  if (any_twice({k, v, reinterpret_cast<const void* const*>(k_exp), reinterpret_cast<const void* const*>(v_exp)}, n_layers))
    return fail(LORA_ERR_INVALID_ARG, "an address is listed twice: its rows would move twice at once");
  KeepQuantizedParams p{};
  p.page_table = page_table;
  p.context = context;
  p.path = path;
  p.n_kept = n_kept;
  p.ld_table = ld_table;
  p.ld_path = ld_path;
  p.cache = view_of(*cache);
  p.n_table = n_table;
  p.n_path = n_path;
  p.kv_heads = kv_heads;
  p.d = d;
  for (int i = 0; i < n_layers; i += kKeepLayers) {
    const int n = n_layers - i < kKeepLayers ? n_layers - i : kKeepLayers;
    for (int j = 0; j < n; ++j) {
      p.k[j] = k[i + j];
      p.v[j] = v[i + j];
      p.k_exp[j] = k_exp[i + j];
      p.v_exp[j] = v_exp[i + j];
    }
    const hipError_t e = launch_keep_quantized(cache->format, p, n, B, stream);
    if (e != hipSuccess) return hip_fail(e, "quantized keep path launch");
  }
  return LORA_OK;
}

LORA_EXPORT size_t lora_pages_workspace_bytes(int64_t n_pages, int32_t n_seqs) {
  if (n_pages < 0 || n_pages > LORA_MAX_POOL_PAGES || n_seqs < 0) return 0;
  return (size_t)pages_scratch_bytes(n_pages, n_seqs);
}

LORA_EXPORT lora_status lora_reserve_pages(int32_t* refs, int64_t n_pages, int32_t* page_table, int64_t ld_table,
                                           int32_t n_table, int32_t B, const int32_t* lengths, int32_t page_size,
                                           int32_t* missing, void* workspace, size_t workspace_bytes,
                                           hipStream_t stream) {
  clear_error();
  lora_status st = check_pool(refs, n_pages, page_table, ld_table, n_table, B);
  if (st != LORA_OK) return st;
  if (page_size < 1) return fail(LORA_ERR_INVALID_ARG, "page_size = %d must be >= 1", page_size);
  if ((int64_t)B * n_table >= kMaxRows) return fail(LORA_ERR_UNSUPPORTED, "the page table has 2^31 entries or more");
  if (B > 0 && !lengths) return fail(LORA_ERR_INVALID_ARG, "lengths is null");
  if (B == 0 && !missing) return LORA_OK;
  if ((st = check_workspace(workspace, workspace_bytes, n_pages, B)) != LORA_OK) return st;
  const PoolParams p = pool_of(refs, n_pages, page_table, ld_table, n_table, B, page_size, workspace);
  const hipError_t e = launch_reserve(p, lengths, missing, stream);
  if (e != hipSuccess) return hip_fail(e, "page reservation launch");
  return LORA_OK;
}

LORA_EXPORT lora_status lora_fork_sequences(int32_t* refs, int64_t n_pages, const int32_t* from_table, int64_t ld_from,
                                            int32_t B_from, int32_t* to_table, int64_t ld_to, int32_t B_to,
                                            int32_t n_table, const int32_t* parents, const int32_t* children,
                                            const int32_t* lengths, int32_t n_forks, int32_t page_size, int32_t* source,
                                            int32_t* target, int32_t* missing, const lora_paged_tensor* tensors,
                                            int32_t n_tensors, void* workspace, size_t workspace_bytes,
                                            hipStream_t stream) {
  clear_error();
  lora_status st = check_pool(refs, n_pages, to_table, ld_to, n_table, B_to);
  if (st != LORA_OK) return st;
  if ((st = check_sequences(B_from)) != LORA_OK) return st;
  if (B_from > 0 && (st = check_table(from_table, ld_from, n_table, B_from)) != LORA_OK) return st;
  if (n_forks < 0) return fail(LORA_ERR_INVALID_ARG, "n_forks = %d is negative", n_forks);
  if (n_forks > 65535) return fail(LORA_ERR_UNSUPPORTED, "n_forks = %d exceeds 65535", n_forks);
  if (page_size < 1) return fail(LORA_ERR_INVALID_ARG, "page_size = %d must be >= 1", page_size);
  if (n_forks > 0 && (!parents || !children || !lengths || !source || !target))
    return fail(LORA_ERR_INVALID_ARG, "parents, children, lengths, source or target is null");
  if ((st = check_tensors(tensors, n_tensors, n_pages)) != LORA_OK) return st;
  if (n_forks == 0 && !missing) return LORA_OK;
  if ((st = check_workspace(workspace, workspace_bytes, n_pages, n_forks)) != LORA_OK) return st;
  const PoolParams p = pool_of(refs, n_pages, to_table, ld_to, n_table, B_to, page_size, workspace);
  const ForkParams f{from_table, ld_from, B_from, n_forks, parents, children, lengths, source, target, missing};
  hipError_t e = launch_fork(p, f, stream);
  if (e == hipSuccess && n_forks > 0) {
    MoveParams m{};
    m.n_pages = n_pages;
    m.source = source;
    m.target = target;
    m.n = n_forks;
    m.task = MoveParams::kFork;
    m.pool = p;
    m.fork = f;
    e = move_all(m, tensors, n_tensors, stream);
  }
  if (e != hipSuccess) return hip_fail(e, "fork launch");
  return LORA_OK;
}

LORA_EXPORT lora_status lora_release_pages(int32_t* refs, int64_t n_pages, int32_t* page_table, int64_t ld_table,
                                           int32_t n_table, int32_t B, const int32_t* rows, const int32_t* keep,
                                           int32_t n, int32_t page_size, hipStream_t stream) {
  clear_error();
  lora_status st = check_pool(refs, n_pages, page_table, ld_table, n_table, B);
  if (st != LORA_OK) return st;
  if (page_size < 1) return fail(LORA_ERR_INVALID_ARG, "page_size = %d must be >= 1", page_size);
  if (n < 0) return fail(LORA_ERR_INVALID_ARG, "n = %d is negative", n);
  if (n > 65535) return fail(LORA_ERR_UNSUPPORTED, "n = %d exceeds 65535", n);
  if (!rows && n != 0 && n != B) return fail(LORA_ERR_INVALID_ARG, "n = %d must be B = %d where no rows are listed", n, B);
  if (n == 0 || n_table == 0) return LORA_OK;
  const PoolParams p = pool_of(refs, n_pages, page_table, ld_table, n_table, B, page_size, nullptr);
  const hipError_t e = launch_release(p, rows, keep, n, stream);
  if (e != hipSuccess) return hip_fail(e, "page release launch");
  return LORA_OK;
}

LORA_EXPORT lora_status lora_compact_pages(int32_t* refs, int64_t n_pages, int32_t* page_table, int64_t ld_table,
                                           int32_t n_table, int32_t B, int32_t* source, int32_t* target,
                                           int32_t* n_live, int32_t* n_moves, const lora_paged_tensor* tensors,
                                           int32_t n_tensors, void* workspace, size_t workspace_bytes,
                                           hipStream_t stream) {
  clear_error();
  lora_status st = check_pool(refs, n_pages, page_table, ld_table, n_table, B);
  if (st != LORA_OK) return st;
  if (!n_live || !n_moves) return fail(LORA_ERR_INVALID_ARG, "n_live or n_moves is null");
  if (n_pages > 1 && (!source || !target)) return fail(LORA_ERR_INVALID_ARG, "source or target is null");
  if ((st = check_tensors(tensors, n_tensors, n_pages)) != LORA_OK) return st;
  if ((st = check_workspace(workspace, workspace_bytes, n_pages, 0)) != LORA_OK) return st;
  const PoolParams p = pool_of(refs, n_pages, page_table, ld_table, n_table, B, 1, workspace);
  hipError_t e = launch_compact(p, source, target, n_live, n_moves, stream);
  if (e == hipSuccess) {
    MoveParams m{};
    m.n_pages = n_pages;
    m.source = source;
    m.target = target;
    m.count = n_moves;
    m.n = (int32_t)(n_pages / 2);
    m.task = B > 0 ? MoveParams::kRename : MoveParams::kNone;
    m.pool = p;
    m.n_live = n_live;
    e = move_all(m, tensors, n_tensors, stream);
  }
  if (e != hipSuccess) return hip_fail(e, "page compaction launch");
  return LORA_OK;
}

LORA_EXPORT lora_status lora_copy_pages(const lora_paged_tensor* tensors, int32_t n_tensors, int64_t n_pages,
                                        const int32_t* source, const int32_t* target, int32_t n, const int32_t* count,
                                        hipStream_t stream) {
  clear_error();
  if (n < 0) return fail(LORA_ERR_INVALID_ARG, "n = %d is negative", n);
  if (n_pages < 0 || n_pages > LORA_MAX_POOL_PAGES)
    return fail(LORA_ERR_INVALID_ARG, "n_pages = %lld is not within 0 and %d", (long long)n_pages, LORA_MAX_POOL_PAGES);
  const lora_status st = check_tensors(tensors, n_tensors, n_pages);
  if (st != LORA_OK) return st;
  if (n_tensors == 0 || n == 0 || n_pages == 0) return LORA_OK;
  if (!source || !target) return fail(LORA_ERR_INVALID_ARG, "source or target is null");
  MoveParams m{};
  m.n_pages = n_pages;
  m.source = source;
  m.target = target;
  m.count = count;
  m.n = n;
  const hipError_t e = move_all(m, tensors, n_tensors, stream);
  if (e != hipSuccess) return hip_fail(e, "page copy launch");
  return LORA_OK;
}
