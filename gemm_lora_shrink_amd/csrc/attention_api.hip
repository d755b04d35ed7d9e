// C ABI entry points of the operators after the q/k/v projection
// (include/lora_attention.h): host-side argument checks and dispatch.  Every
// check runs before anything is enqueued.
#include <math.h>

#include "attention.h"

#define LORA_EXPORT extern "C" __attribute__((visibility("default")))

namespace lora {
namespace {

constexpr int64_t kMaxPositions = (int64_t)1 << 31;

int elem_bytes(lora_dtype dt) { return dt == LORA_F32 ? 4 : 2; }

lora_status check_heads(int32_t q_heads, int32_t kv_heads, int32_t d) {
  if (d < 1) return fail(LORA_ERR_INVALID_ARG, "head_dim = %d must be >= 1", d);
  if (d % 8 || d > LORA_MAX_HEAD_DIM)
    return fail(LORA_ERR_UNSUPPORTED, "head_dim = %d must be a multiple of 8 up to %d", d, LORA_MAX_HEAD_DIM);
  if (q_heads < 0 || kv_heads < 0) return fail(LORA_ERR_INVALID_ARG, "a number of heads is negative");
  if (q_heads > LORA_MAX_HEADS || kv_heads > LORA_MAX_HEADS)
    return fail(LORA_ERR_UNSUPPORTED, "more than %d heads", LORA_MAX_HEADS);
  return LORA_OK;
}

// Rows of `width` elements with stride ld.
lora_status check_rows(lora_dtype dt, const char* name, const void* p, int64_t ld, int64_t width) {
  if (!p) return fail(LORA_ERR_INVALID_ARG, "%s is null", name);
  if (!aligned16(p)) return fail(LORA_ERR_UNSUPPORTED, "%s must be 16-byte aligned", name);
  if (ld < width) return fail(LORA_ERR_INVALID_ARG, "the row stride of %s, %lld, is smaller than its %lld elements", name,
                              (long long)ld, (long long)width);
  if (ld % vec_of(dt))
    return fail(LORA_ERR_UNSUPPORTED, "the row stride of %s must be a multiple of %d elements", name, vec_of(dt));
  return LORA_OK;
}

lora_status check_cache(lora_dtype dt, const lora_kv_cache& c) {
  if (!c.k || !c.v) return fail(LORA_ERR_INVALID_ARG, "the cache's k or v is null");
  if (!aligned16(c.k) || !aligned16(c.v)) return fail(LORA_ERR_UNSUPPORTED, "the cache must be 16-byte aligned");
  if (c.page_size < 1) return fail(LORA_ERR_INVALID_ARG, "page_size = %d must be >= 1", c.page_size);
  if (c.n_pages < 0) return fail(LORA_ERR_INVALID_ARG, "n_pages is negative");
  const int64_t strides[6] = {c.k_page, c.k_head, c.k_row, c.v_page, c.v_head, c.v_row};
  for (int64_t s : strides) {
    if (s < 0) return fail(LORA_ERR_INVALID_ARG, "a cache stride is negative");
    if (s % vec_of(dt))
      return fail(LORA_ERR_UNSUPPORTED, "cache strides must be multiples of %d elements", vec_of(dt));
  }
  return LORA_OK;
}

CacheView view_of(const lora_kv_cache& c) {
  return CacheView{c.k,      c.v,      c.k_page,  c.k_head,  c.k_row, c.v_page,
                   c.v_head, c.v_row,  c.n_pages, fast_div((uint32_t)c.page_size)};
}

lora_status check_table(const int32_t* page_table, int64_t ld_table, int32_t n_table) {
  if (n_table < 0) return fail(LORA_ERR_INVALID_ARG, "n_table = %d is negative", n_table);
  if (n_table > 0 && !page_table) return fail(LORA_ERR_INVALID_ARG, "page_table is null");
  if (ld_table < n_table) return fail(LORA_ERR_INVALID_ARG, "ld_table is smaller than n_table");
  return LORA_OK;
}

lora_status rotary_impl(bool norm, lora_dtype dt, const void* q, int64_t ldq, const void* k, int64_t ldk,
                        const void* v, int64_t ldv, int32_t T, int32_t q_heads, int32_t kv_heads, int32_t d,
                        int32_t layout, int32_t rot_dim, const void* q_weight, const void* k_weight, float eps,
                        const float* table, int64_t n_positions, const int32_t* positions, void* q_out, int64_t ldqo,
                        void* k_out, int64_t ldko, const lora_kv_cache* cache, const int32_t* cache_rows,
                        hipStream_t stream) {
  clear_error();
  if (!valid_dtype(dt)) return fail(LORA_ERR_INVALID_ARG, "unknown dtype %d", dt);
  if (T < 0) return fail(LORA_ERR_INVALID_ARG, "T = %d is negative", T);
  lora_status st = check_heads(q_heads, kv_heads, d);
  if (st != LORA_OK) return st;
  if (q_heads + kv_heads < 1) return fail(LORA_ERR_INVALID_ARG, "no heads");
  if (layout != LORA_ROPE_HALF && layout != LORA_ROPE_INTERLEAVED)
    return fail(LORA_ERR_INVALID_ARG, "unknown rotary layout %d", layout);
  if (rot_dim < 2 || rot_dim % 2 || rot_dim > d)
    return fail(LORA_ERR_INVALID_ARG, "rot_dim = %d must be even, from 2 to head_dim = %d", rot_dim, d);
  if (n_positions < 1) return fail(LORA_ERR_INVALID_ARG, "n_positions = %lld must be >= 1", (long long)n_positions);
  if (norm && !(eps >= 0.f && eps <= 3.0e38f)) return fail(LORA_ERR_INVALID_ARG, "eps must be >= 0 and finite");
  if (cache && kv_heads < 1) return fail(LORA_ERR_INVALID_ARG, "a cache needs kv_heads >= 1");
  if (T == 0) return LORA_OK;
  if (!table || !positions) return fail(LORA_ERR_INVALID_ARG, "table or positions is null");
  if (!aligned16(table)) return fail(LORA_ERR_UNSUPPORTED, "table must be 16-byte aligned");
  const int64_t qw = (int64_t)q_heads * d, kw = (int64_t)kv_heads * d;
  if (q_heads > 0) {
    if ((st = check_rows(dt, "q", q, ldq, qw)) != LORA_OK) return st;
    if ((st = check_rows(dt, "q_out", q_out, ldqo, qw)) != LORA_OK) return st;
    if (q_out == q && ldqo != ldq) return fail(LORA_ERR_INVALID_ARG, "q_out is q with another row stride");
  }
  if (kv_heads > 0) {
    if ((st = check_rows(dt, "k", k, ldk, kw)) != LORA_OK) return st;
    if (!k_out && !cache) return fail(LORA_ERR_INVALID_ARG, "k_out is null and there is no cache");
    if (k_out && (st = check_rows(dt, "k_out", k_out, ldko, kw)) != LORA_OK) return st;
    if (k_out == k && ldko != ldk) return fail(LORA_ERR_INVALID_ARG, "k_out is k with another row stride");
  }
  if (!aligned16(q_weight) || !aligned16(k_weight))
    return fail(LORA_ERR_UNSUPPORTED, "q_weight and k_weight must be 16-byte aligned");
  if ((int64_t)T * (q_heads + 2 * (int64_t)kv_heads) >= kMaxPositions)
    return fail(LORA_ERR_UNSUPPORTED, "T times the heads reaches 2^31");
  if (!rotary_fits(T, q_heads + (cache ? 2 : 1) * kv_heads, d, rot_dim))
    return fail(LORA_ERR_UNSUPPORTED, "T = %d tokens of these heads are more than a launch holds", T);
  RotaryParams p{};
  if (cache) {
    if ((st = check_cache(dt, *cache)) != LORA_OK) return st;
    if ((st = check_rows(dt, "v", v, ldv, kw)) != LORA_OK) return st;
    if (!cache_rows) return fail(LORA_ERR_INVALID_ARG, "cache_rows is null");
    if (cache->n_pages > kMaxPositions / cache->page_size)
      return fail(LORA_ERR_UNSUPPORTED, "the cache has more rows than cache_rows can name");
    p.cache = view_of(*cache);
    p.n_rows = cache->n_pages * cache->page_size;
  }
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_out = q_out;
  p.k_out = k_out;
  p.ldq = ldq;
  p.ldk = ldk;
  p.ldv = ldv;
  p.ldqo = ldqo;
  p.ldko = ldko;
  p.qw = q_weight;
  p.kw = k_weight;
  p.table = table;
  p.positions = positions;
  p.cache_rows = cache_rows;
  p.n_positions = n_positions;
  p.T = T;
  p.hq = q_heads;
  p.hk = kv_heads;
  p.d = d;
  p.rot = rot_dim;
  p.layout = layout;
  p.norm = norm;
  p.eps = eps;
  const hipError_t e = launch_rotary(dt, p, stream);
  if (e != hipSuccess) return hip_fail(e, "rotary launch");
  return LORA_OK;
}

lora_status check_tree(int32_t T, int32_t B, int32_t max_nodes) {
  if (T < 0) return fail(LORA_ERR_INVALID_ARG, "T = %d is negative", T);
  if (B < 0) return fail(LORA_ERR_INVALID_ARG, "B = %d is negative", B);
  if (B > 65535) return fail(LORA_ERR_UNSUPPORTED, "B = %d exceeds 65535", B);
  if (max_nodes < 1) return fail(LORA_ERR_INVALID_ARG, "max_nodes = %d must be >= 1", max_nodes);
  return LORA_OK;
}

lora_status check_mask(const uint64_t* mask, int32_t mask_words, int32_t max_nodes) {
  if (!mask) return LORA_OK;
  if (max_nodes > LORA_MAX_TREE_NODES)
    return fail(LORA_ERR_UNSUPPORTED, "max_nodes = %d exceeds %d with a mask", max_nodes, LORA_MAX_TREE_NODES);
  if (mask_words < (max_nodes + 63) / 64)
    return fail(LORA_ERR_INVALID_ARG, "mask_words = %d is too small for %d nodes", mask_words, max_nodes);
  if (reinterpret_cast<uintptr_t>(mask) & 7u) return fail(LORA_ERR_UNSUPPORTED, "mask must be 8-byte aligned");
  return LORA_OK;
}

}  // namespace
}  // namespace lora

using namespace lora;

LORA_EXPORT lora_status lora_rope_frequencies(int32_t rot_dim, double base, const lora_rope_config* config,
                                              double* inv_freq, double* magnitude) {
  clear_error();
  if (rot_dim < 2 || rot_dim % 2 || rot_dim > LORA_MAX_HEAD_DIM)
    return fail(LORA_ERR_INVALID_ARG, "rot_dim = %d must be even, from 2 to %d", rot_dim, LORA_MAX_HEAD_DIM);
  if (!(base > 0.0) || !isfinite(base)) return fail(LORA_ERR_INVALID_ARG, "base must be positive and finite");
  if (!inv_freq || !magnitude) return fail(LORA_ERR_INVALID_ARG, "inv_freq or magnitude is null");
  const lora_rope_config c = config ? *config : lora_rope_config{};
  const int kind = c.scaling;
  if (kind < LORA_ROPE_NONE || kind > LORA_ROPE_YARN)
    return fail(LORA_ERR_INVALID_ARG, "unknown rotary scaling %d", kind);
  const double s = c.factor, L = c.original_context;
  if (kind != LORA_ROPE_NONE && (!(s > 0.0) || !isfinite(s)))
    return fail(LORA_ERR_INVALID_ARG, "factor must be positive and finite");
  const bool by_turns = kind == LORA_ROPE_LLAMA3 || kind == LORA_ROPE_YARN;
  if (by_turns && (!(L > 0.0) || !isfinite(L)))
    return fail(LORA_ERR_INVALID_ARG, "original_context must be positive and finite");
  const double low = c.low != 0.0 ? c.low : 1.0;
  const double high = c.high != 0.0 ? c.high : (kind == LORA_ROPE_LLAMA3 ? 4.0 : 32.0);
  if (by_turns && !(low > 0.0 && high > low && isfinite(high)))
    return fail(LORA_ERR_INVALID_ARG, "need 0 < low < high");
  if (kind == LORA_ROPE_NTK && rot_dim < 4) return fail(LORA_ERR_UNSUPPORTED, "NTK scaling needs rot_dim >= 4");
  if (kind == LORA_ROPE_YARN && !(base > 1.0)) return fail(LORA_ERR_INVALID_ARG, "YARN scaling needs base > 1");
  if (!(c.magnitude >= 0.0) || !isfinite(c.magnitude))
    return fail(LORA_ERR_INVALID_ARG, "magnitude must be >= 0 and finite");
  const double two_pi = 6.283185307179586476925286766559;
  const double b = kind == LORA_ROPE_NTK ? base * pow(s, rot_dim / (rot_dim - 2.0)) : base;
  double first = 0.0, last = 0.0;
  if (kind == LORA_ROPE_YARN) {
    const auto pair = [&](double turns) { return rot_dim * log(L / (two_pi * turns)) / (2.0 * log(base)); };
    first = fmax(floor(pair(high)), 0.0);
    last = fmin(ceil(pair(low)), rot_dim - 1.0);
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double f = pow(b, -2.0 * i / rot_dim);
    double got = f;
    if (kind == LORA_ROPE_LINEAR) {
      got = f / s;
    } else if (kind == LORA_ROPE_LLAMA3) {
      const double m = fmin(1.0, fmax(0.0, (L * f / two_pi - low) / (high - low)));
      got = (1.0 - m) * f / s + m * f;
    } else if (kind == LORA_ROPE_YARN) {
      const double k = 1.0 - fmin(1.0, fmax(0.0, (i - first) / fmax(last - first, 1e-3)));
      got = f / s * (1.0 - k) + f * k;
    }
    inv_freq[i] = got;
  }
  *magnitude = c.magnitude != 0.0 ? c.magnitude : (kind == LORA_ROPE_YARN && s > 1.0 ? 0.1 * log(s) + 1.0 : 1.0);
  return LORA_OK;
}

LORA_EXPORT lora_status lora_rope_table(const double* inv_freq, int32_t rot_dim, double magnitude, int64_t first,
                                        int64_t n, float* table, hipStream_t stream) {
  clear_error();
  if (rot_dim < 2 || rot_dim % 2 || rot_dim > LORA_MAX_HEAD_DIM)
    return fail(LORA_ERR_INVALID_ARG, "rot_dim = %d must be even, from 2 to %d", rot_dim, LORA_MAX_HEAD_DIM);
  if (!inv_freq) return fail(LORA_ERR_INVALID_ARG, "inv_freq is null");
  if (first < 0 || n < 0 || first > kMaxPositions || n > kMaxPositions - first)
    return fail(LORA_ERR_INVALID_ARG, "positions must lie in [0, 2^31)");
  if (n == 0) return LORA_OK;
  if (!table) return fail(LORA_ERR_INVALID_ARG, "table is null");
  if (!aligned16(table)) return fail(LORA_ERR_UNSUPPORTED, "table must be 16-byte aligned");
  const hipError_t e = launch_rope_table(inv_freq, rot_dim, magnitude, first, n, table, stream);
  if (e != hipSuccess) return hip_fail(e, "rope table launch");
  return LORA_OK;
}

LORA_EXPORT lora_status lora_rotary(lora_dtype dt, const void* q, int64_t ldq, const void* k, int64_t ldk,
                                    const void* v, int64_t ldv, int32_t T, int32_t q_heads, int32_t kv_heads,
                                    int32_t d, int32_t layout, int32_t rot_dim, const float* table,
                                    int64_t n_positions, const int32_t* positions, void* q_out, int64_t ldqo,
                                    void* k_out, int64_t ldko, const lora_kv_cache* cache, const int32_t* cache_rows,
                                    hipStream_t stream) {
  return rotary_impl(false, dt, q, ldq, k, ldk, v, ldv, T, q_heads, kv_heads, d, layout, rot_dim, nullptr, nullptr,
                     0.f, table, n_positions, positions, q_out, ldqo, k_out, ldko, cache, cache_rows, stream);
}

LORA_EXPORT lora_status lora_qk_norm_rotary(lora_dtype dt, const void* q, int64_t ldq, const void* k, int64_t ldk,
                                            const void* v, int64_t ldv, int32_t T, int32_t q_heads, int32_t kv_heads,
                                            int32_t d, int32_t layout, int32_t rot_dim, const void* q_weight,
                                            const void* k_weight, float eps, const float* table, int64_t n_positions,
                                            const int32_t* positions, void* q_out, int64_t ldqo, void* k_out,
                                            int64_t ldko, const lora_kv_cache* cache, const int32_t* cache_rows,
                                            hipStream_t stream) {
  return rotary_impl(true, dt, q, ldq, k, ldk, v, ldv, T, q_heads, kv_heads, d, layout, rot_dim, q_weight, k_weight,
                     eps, table, n_positions, positions, q_out, ldqo, k_out, ldko, cache, cache_rows, stream);
}

LORA_EXPORT lora_status lora_build_tree(const int32_t* parents, int32_t T, int32_t B, const int32_t* q_start,
                                        const int32_t* context, int32_t max_nodes, const int32_t* page_table,
                                        int64_t ld_table, int32_t n_table, int64_t n_pages, int32_t page_size,
                                        uint64_t* mask, int32_t mask_words, int32_t* positions, int32_t* cache_rows,
                                        hipStream_t stream) {
  clear_error();
  lora_status st = check_tree(T, B, max_nodes);
  if (st != LORA_OK) return st;
  if (parents && max_nodes > LORA_MAX_TREE_NODES)
    return fail(LORA_ERR_UNSUPPORTED, "max_nodes = %d exceeds %d", max_nodes, LORA_MAX_TREE_NODES);
  if ((st = check_mask(mask, mask_words, max_nodes)) != LORA_OK) return st;
  if (cache_rows) {
    if ((st = check_table(page_table, ld_table, n_table)) != LORA_OK) return st;
    if (page_size < 1 || n_pages < 0) return fail(LORA_ERR_INVALID_ARG, "bad page_size or n_pages");
    if (n_pages > kMaxPositions / page_size)
      return fail(LORA_ERR_UNSUPPORTED, "the cache has more rows than cache_rows can name");
  }
  if (T == 0 || B == 0) return LORA_OK;
  if (!q_start || !context) return fail(LORA_ERR_INVALID_ARG, "q_start or context is null");
  if (!mask && !positions && !cache_rows) return LORA_OK;
  BuildTreeParams p{};
  p.parents = parents;
  p.q_start = q_start;
  p.context = context;
  p.page_table = page_table;
  p.ld_table = ld_table;
  p.n_pages = n_pages;
  p.mask = mask;
  p.positions = positions;
  p.cache_rows = cache_rows;
  p.T = T;
  p.B = B;
  p.max_nodes = max_nodes;
  p.n_table = n_table;
  p.mask_words = mask_words;
  p.page = fast_div((uint32_t)(cache_rows ? page_size : 1));
  const hipError_t e = launch_build_tree(p, stream);
  if (e != hipSuccess) return hip_fail(e, "tree build launch");
  return LORA_OK;
}

namespace lora {
namespace {

lora_status check_attend_sizes(int32_t B, int32_t T, int32_t max_nodes, int32_t max_context, int32_t q_heads,
                               int32_t kv_heads, int32_t d) {
  lora_status st = check_tree(T, B, max_nodes);
  if (st != LORA_OK) return st;
  if (max_context < 0) return fail(LORA_ERR_INVALID_ARG, "max_context = %d is negative", max_context);
  if ((st = check_heads(q_heads, kv_heads, d)) != LORA_OK) return st;
  if (q_heads < 1 || kv_heads < 1 || q_heads % kv_heads)
    return fail(LORA_ERR_INVALID_ARG, "q_heads = %d must be a multiple of kv_heads = %d, both >= 1", q_heads, kv_heads);
  if ((int64_t)max_context + max_nodes >= kMaxPositions)
    return fail(LORA_ERR_UNSUPPORTED, "max_context + max_nodes reaches 2^31");
  if ((int64_t)max_nodes * (q_heads / kv_heads) >= (int64_t)1 << 27)
    return fail(LORA_ERR_UNSUPPORTED, "max_nodes times the heads of a group reaches 2^27");
  return LORA_OK;
}

}  // namespace
}  // namespace lora

LORA_EXPORT size_t lora_tree_attention_workspace_bytes(int32_t B, int32_t T, int32_t max_nodes, int32_t max_context,
                                                       int32_t q_heads, int32_t kv_heads, int32_t d) {
  if (check_attend_sizes(B, T, max_nodes, max_context, q_heads, kv_heads, d) != LORA_OK) return 0;
  return (size_t)attend_most_bytes(B, T, max_nodes, max_context, q_heads, kv_heads, d);
}

LORA_EXPORT lora_status lora_tree_attention(lora_dtype dt, const void* q, int64_t ldq, int32_t T, int32_t B,
                                            int32_t q_heads, int32_t kv_heads, int32_t d, const lora_kv_cache* cache,
                                            const int32_t* page_table, int64_t ld_table, int32_t n_table,
                                            const int32_t* context, const int32_t* q_start, int32_t max_nodes,
                                            int32_t max_context, const uint64_t* mask, int32_t mask_words, float scale,
                                            void* out, int64_t ldo, float* lse, void* workspace,
                                            size_t workspace_bytes, hipStream_t stream) {
  clear_error();
  if (!valid_dtype(dt)) return fail(LORA_ERR_INVALID_ARG, "unknown dtype %d", dt);
  lora_status st = check_attend_sizes(B, T, max_nodes, max_context, q_heads, kv_heads, d);
  if (st != LORA_OK) return st;
  if (!isfinite(scale)) return fail(LORA_ERR_INVALID_ARG, "scale is not finite");
  if ((st = check_mask(mask, mask_words, max_nodes)) != LORA_OK) return st;
  if ((st = check_table(page_table, ld_table, n_table)) != LORA_OK) return st;
  if (T == 0 || B == 0) return LORA_OK;
  if (!context || !q_start) return fail(LORA_ERR_INVALID_ARG, "context or q_start is null");
  if (!cache) return fail(LORA_ERR_INVALID_ARG, "cache is null");
  if ((st = check_cache(dt, *cache)) != LORA_OK) return st;
  const int64_t most = (((int64_t)1 << 32) - 1) / elem_bytes(dt);
  if (cache->k_page > most || cache->v_page > most || cache->k_row > most || cache->v_row > most)
    return fail(LORA_ERR_UNSUPPORTED, "a page or row of the cache spans 4 GiB");
  if (!attend_fits(dt, B, max_nodes, max_context, q_heads, kv_heads, d))
    return fail(LORA_ERR_UNSUPPORTED, "B = %d sequences of up to %d nodes are more than a launch holds", B, max_nodes);
  const int64_t need = attend_need_bytes(dt, B, T, max_nodes, max_context, q_heads, kv_heads, d);
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
  AttendParams p{};
  p.q = q;
  p.out = out;
  p.ldq = ldq;
  p.ldo = ldo;
  p.lse = lse;
  p.cache = view_of(*cache);
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
  const hipError_t e = launch_attend(dt, p, stream);
  if (e != hipSuccess) return hip_fail(e, "tree attention launch");
  return LORA_OK;
}

LORA_EXPORT lora_status lora_keep_path(lora_dtype dt, const lora_kv_cache* cache, void* const* k, void* const* v,
                                       int32_t n_layers, int32_t kv_heads, int32_t d, int32_t B, const int32_t* page_table, int64_t ld_table,
                                       int32_t n_table, const int32_t* context, const int32_t* path, int64_t ld_path,
                                       int32_t n_path, const int32_t* n_kept, hipStream_t stream) {
  clear_error();
  if (!valid_dtype(dt)) return fail(LORA_ERR_INVALID_ARG, "unknown dtype %d", dt);
  lora_status st = check_tree(0, B, 1);
  if (st != LORA_OK) return st;
  if ((st = check_heads(0, kv_heads, d)) != LORA_OK) return st;
  if (kv_heads < 1) return fail(LORA_ERR_INVALID_ARG, "kv_heads = %d must be >= 1", kv_heads);
  if (n_layers < 0) return fail(LORA_ERR_INVALID_ARG, "n_layers = %d is negative", n_layers);
  if (n_layers > LORA_MAX_KEEP_LAYERS)
    return fail(LORA_ERR_UNSUPPORTED, "n_layers = %d exceeds %d", n_layers, LORA_MAX_KEEP_LAYERS);
  if (n_path < 0) return fail(LORA_ERR_INVALID_ARG, "n_path = %d is negative", n_path);
  if (n_path > LORA_MAX_KEEP_PATH)
    return fail(LORA_ERR_UNSUPPORTED, "n_path = %d exceeds %d", n_path, LORA_MAX_KEEP_PATH);
  if (ld_path < n_path) return fail(LORA_ERR_INVALID_ARG, "ld_path is smaller than n_path");
  if ((st = check_table(page_table, ld_table, n_table)) != LORA_OK) return st;
  if (B == 0 || n_layers == 0 || n_path == 0) return LORA_OK;
  if (!cache || !k || !v || !context || !path || !n_kept)
    return fail(LORA_ERR_INVALID_ARG, "cache, k, v, context, path or n_kept is null");
  KeepParams p{};
  lora_kv_cache c = *cache;
  for (int i = 0; i < n_layers; ++i) {
    c.k = k[i];
    c.v = v[i];
    if ((st = check_cache(dt, c)) != LORA_OK) return st;
    p.k[i] = k[i];
    p.v[i] = v[i];
  }
  const int64_t e = elem_bytes(dt);
  p.page_table = page_table;
  p.context = context;
  p.path = path;
  p.n_kept = n_kept;
  p.ld_table = ld_table;
  p.ld_path = ld_path;
  p.n_pages = c.n_pages;
  p.k_page = c.k_page * e;
  p.k_head = c.k_head * e;
  p.k_row = c.k_row * e;
  p.v_page = c.v_page * e;
  p.v_head = c.v_head * e;
  p.v_row = c.v_row * e;
  p.n_table = n_table;
  p.n_path = n_path;
  p.row_bytes = (int32_t)(d * e);
  p.page = fast_div((uint32_t)c.page_size);
  const hipError_t err = launch_keep_path(p, n_layers, kv_heads, B, stream);
  if (err != hipSuccess) return hip_fail(err, "keep path launch");
  return LORA_OK;
}
