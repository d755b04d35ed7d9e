// Internal definitions of the quantized cache and the pages of a cache
// (include/lora_cache.h): what a byte holds, the parameter blocks passed to the
// kernels and the host launchers.
#pragma once

#include "../../include/lora_cache.h"
#include "attention.h"

namespace lora {

constexpr int kExpLow = -126;  // the smallest exponent of a block

// What a byte holds.
struct E4m3 {
  static constexpr bool kHasNan = true;
  static constexpr int kTop = 119;          // the largest exponent
  static constexpr float kLargest = 448.f;  // the largest number, 1.75 * 2^8
  static constexpr int kLargestExp = 8;
  static constexpr uint32_t kLargestMantissa = 0x600000u;
  __device__ static inline void numbers(uint32_t w, float* x) {  // of a word's four bytes
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    x[0] = a[0];
    x[1] = a[1];
    x[2] = b[0];
    x[3] = b[1];
  }
  // The nearest numbers, ties to even; |x| beyond the largest becomes it.
  __device__ static inline uint32_t bytes(const float* x) {
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)  // (the median drops a NaN)
      y[i] = x[i] != x[i] ? x[i] : __builtin_amdgcn_fmed3f(x[i], -kLargest, kLargest);
    return bytes_within(y, 1.0f);
  }
  // The same of x times a power of two where no |x| passes the largest.
  __device__ static inline uint32_t bytes_within(const float* x, float by) {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * by, x[1] * by, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[2] * by, x[3] * by, lo, true);
  }
};
struct Int8 {
  static constexpr bool kHasNan = false;
  static constexpr int kTop = 121;
  static constexpr float kLargest = 127.f;  // 1.984375 * 2^6
  static constexpr int kLargestExp = 6;
  static constexpr uint32_t kLargestMantissa = 0x7e0000u;
  __device__ static inline void numbers(uint32_t w, float* x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = (float)(int8_t)(w >> (8 * i));
  }
  __device__ static inline uint32_t bytes(const float* x) {
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = x[i] != x[i] ? 0.f : __builtin_amdgcn_fmed3f(x[i], -kLargest, kLargest);
    return bytes_within(y, 1.0f);
  }
  // In 1.5 * 2^23 + x the sum's rounding (to the nearest, ties to even) leaves the
  // whole number x in the low byte.
  __device__ static inline uint32_t bytes_within(const float* x, float by) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(__builtin_fmaf(x[i], by, 12582912.0f));
    // (bytes 0 .. 3 of the second operand are 0 .. 3, of the first 4 .. 7)
    const uint32_t lo = __builtin_amdgcn_perm(w[1], w[0], 0x0c0c0400u), hi = __builtin_amdgcn_perm(w[3], w[2], 0x04000c0cu);
    return lo | hi;
  }
};

// 2^e, for e from -126 to 127.
__device__ inline float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
template <typename F> __device__ inline int exponent_of(int8_t stored) {
  return stored < kExpLow ? kExpLow : (stored > F::kTop ? F::kTop : stored);
}

// A layer's quantized cache as the kernels see it (strides in bytes).
struct QuantizedView {
  void *k, *v;
  int8_t *k_exp, *v_exp;
  int64_t k_page, k_head, k_row, v_page, v_head, v_row;
  int64_t k_exp_page, k_exp_head, v_exp_page, v_exp_head;
  int64_t n_pages;
  FastDiv page, block;  // by the page size, by the rows of a block
};

struct StoreParams {
  const void *k, *v;
  int64_t ldk, ldv;
  QuantizedView cache;
  const int32_t* rows;
  int64_t n_rows;  // n_pages * page_size
  int32_t T, hk, d;
  int32_t chunk, lane_shift;  // filled by the launcher: tokens of a workgroup, log2 of the lanes of a row
};

constexpr int kKeepLayers = 64;  // layers of one launch
struct KeepQuantizedParams {
  const int32_t *page_table, *context, *path, *n_kept;
  int64_t ld_table, ld_path;
  QuantizedView cache;  // its pointers: unused
  int32_t n_table, n_path, kv_heads, d;
  void *k[kKeepLayers], *v[kKeepLayers];
  int8_t *k_exp[kKeepLayers], *v_exp[kKeepLayers];
};

// The attention's parameters, with the cache's strides in bytes.
struct AttendQuantizedParams : AttendParams {
  const int8_t *k_exp, *v_exp;
  int64_t k_exp_page, k_exp_head, v_exp_page, v_exp_head;
  FastDiv block;  // by the rows of a block
  int cuts;       // chunks to be had where they are cut by the sequences' lengths, else 0
};

struct PoolParams {
  int32_t* refs;
  int64_t n_pages;
  int32_t* table;
  int64_t ld_table;
  int32_t n_table, B;
  FastDiv page;      // by the page size
  int32_t* scratch;  // the workspace
};
struct ForkParams {
  const int32_t* from;
  int64_t ld_from;
  int32_t B_from, n;
  const int32_t *parents, *children, *lengths;
  int32_t *source, *target, *missing;  // missing nullable
};

// A tensor with pages, counted in accesses of `unit` bytes (strides in bytes).
struct PagedTensor {
  char* data;
  int64_t page, outer, inner;
  uint32_t units, run, n_inner;  // of a page, of a run; runs of the inner dimension
  uint16_t unit, whole;          // whole: a page is one run
};
constexpr int kCopyTensors = 64;
struct MoveParams {
  enum Task : int32_t { kNone = 0, kFork = 1, kRename = 2 };
  PagedTensor t[kCopyTensors];
  int64_t n_pages;
  const int32_t *source, *target, *count;  // count nullable
  int32_t n, n_tensors;
  Task task;
  PoolParams pool;
  ForkParams fork;        // kFork
  const int32_t* n_live;  // kRename
};
static_assert(sizeof(MoveParams) <= 4096, "a kernel's arguments");

// Whether launch_store_quantized's grid holds T tokens.
bool store_quantized_fits(int32_t T);
hipError_t launch_store_quantized(lora_dtype dt, int format, StoreParams p, hipStream_t stream);
hipError_t launch_keep_quantized(int format, const KeepQuantizedParams& p, int32_t n_layers, int32_t B,
                                 hipStream_t stream);
hipError_t launch_attend_quantized(lora_dtype dt, int format, AttendQuantizedParams p, hipStream_t stream);
bool attend_quantized_fits(lora_dtype dt, int32_t B, int32_t max_nodes, int32_t max_context, int32_t hq, int32_t hk,
                           int32_t d);
int64_t attend_quantized_need_bytes(lora_dtype dt, int32_t B, int32_t T, int32_t max_nodes, int32_t max_context,
                                    int32_t hq, int32_t hk, int32_t d);
int64_t attend_quantized_most_bytes(int32_t B, int32_t T, int32_t max_nodes, int32_t max_context, int32_t hq,
                                    int32_t hk, int32_t d);

int64_t pages_scratch_bytes(int64_t n_pages, int32_t n_seqs);
hipError_t launch_reserve(const PoolParams& p, const int32_t* lengths, int32_t* missing, hipStream_t stream);
hipError_t launch_fork(const PoolParams& p, const ForkParams& f, hipStream_t stream);
hipError_t launch_release(const PoolParams& p, const int32_t* rows, const int32_t* keep, int32_t n, hipStream_t stream);
hipError_t launch_compact(const PoolParams& p, int32_t* source, int32_t* target, int32_t* n_live, int32_t* n_moves,
                          hipStream_t stream);
// The copies and, beside them, the rows of p.task.
hipError_t launch_move(const MoveParams& p, hipStream_t stream);

}  // namespace lora
