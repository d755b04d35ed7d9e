// Attention of a step's tokens over the paged cache.
//
// For one sequence and one key/value head the rows are its nodes times the
// query heads of the group; all of them read the same keys, so a workgroup
// takes up to 256 rows of one (sequence, key/value head) over one chunk of the
// keys, and a second launch joins the chunks where there are several.  With m
// the running maximum and l the running sum of a row, a tile of scores s
// changes them by
//     m' = max(m, max s),  l' = l e^(m - m') + sum e^(s - m'),
//     o' = o e^(m - m') + sum e^(s - m') v,
// all in fp32 and in powers of two (scores are multiplied by scale * log2 e).  m need
// not be the maximum itself: any m near it that a row's l and o agree on will do.
//
// Products run on the matrix cores as 32 x 32 blocks, transposed: S^T = K Q^T
// leaves a lane with 16 scores of ONE row (row = lane % 32; lanes l and l + 32
// share it), so maximum, sum and rescaling are per-lane scalars and one half
// swap, and the scores are already the operand of O^T = V^T P^T: the contraction
// index may run over the keys in any order as long as both operands agree, and
// taking it in the order in which S^T lies in registers needs no exchange.
// V^T comes from row-major V in LDS by transposing reads (16-bit) or single
// element reads (fp32).
//
// K and V rows go from global memory to LDS by direct loads, whole rows of
// contiguous bytes; the 16-byte pieces of a row lie XOR-swizzled by row so that
// reading 16 rows at one piece, and 4 rows at 64 contiguous bytes, are both
// free of bank conflicts.  A row that is no key (past the end, no page) is
// loaded from a row of zeros.
#include <algorithm>

#include "attention.h"

namespace lora {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) const u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) const float lds_float;
typedef __attribute__((address_space(3))) char lds_byte;

constexpr int kThreads = 256;
constexpr int kBlock = 32;  // rows and keys of a matrix block
constexpr float kLn2 = 0.69314718055994530942f, kLog2e = 1.44269504088896340736f;

__device__ const u32x4 g_zero_row[64] = {};  // 1 KB of zeros: the longest row

// kBelow, kMost: the range of the weights.  A row's weights are 2^(s - m); where the
// largest would pass 2^kMost, m is moved to that score less kBelow.
template <typename Elem> struct Mma32;
template <> struct Mma32<bf16_t> {
  __device__ static inline f32x16 mma(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  }
  __device__ static inline uint32_t pack2(float a, float b) { return pack2_bf16(a, b); }
  static constexpr uint32_t kExp = 0x7f80u;  // all ones: no finite number
  static constexpr float kBelow = 0.f, kMost = 8.f;
};
template <> struct Mma32<half_t> {
  __device__ static inline f32x16 mma(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
  }
  __device__ static inline uint32_t pack2(float a, float b) { return pack2_f16(a, b); }
  static constexpr uint32_t kExp = 0x7c00u;
  // fp16 has 14 powers of two below 1 before it loses bits, and 15 above: with the
  // largest weight at 1 the keys 2^-14 below a high one (a sink at the context's
  // start) enter with few bits and those 2^-25 below not at all, however many
  // they are.  Measured from 2^12 up, a weight keeps all bits down to 2^-26 of the
  // largest; 2^15.9 is 61147 of 65504.  The narrower range moves m more often: 133 us
  // for 130.5 with weights from 1 to 2^8 on 16 ragged sequences of up to 45 nodes and
  // 8192 keys, and 137 from 2^13 to 2^15.
  static constexpr float kBelow = 12.f, kMost = 15.9f;
};
template <> struct Mma32<float> {
  __device__ static inline f32x16 mma1(float a, float b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x2f32(a, b, c, 0, 0, 0);
  }
  // element e of every lane's four is one product of 32 x 32 x 2
  __device__ static inline f32x16 mma(u32x4 a, u32x4 b, f32x16 c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t ae = a[e], be = b[e];
      c = mma1(__uint_as_float(ae), __uint_as_float(be), c);
    }
    return c;
  }
  static constexpr uint32_t kExp = 0x7f800000u;
  static constexpr float kBelow = 0.f, kMost = 8.f;
};

// Rows of DP elements (the head, padded) in LDS.
template <typename Elem, int DP> struct Rows {
  static constexpr bool k16 = sizeof(Elem) == 2;
  static constexpr int kBytes = DP * (int)sizeof(Elem);  // of a row
  static constexpr int kPieces = kBytes / 16;
  static constexpr int kSteps = kBytes / 32;       // 16-byte operands of a lane and half
  static constexpr int kDB = DP / kBlock;          // blocks of the output
  static constexpr int kPerLoad = 1024 / kBytes;   // rows of one 64-lane load
  // waves of a SIMD that the narrow kernel is compiled for
  static constexpr int kNarrowWaves = DP <= 64 ? 2 : 1;
  static_assert(kBytes >= 128 && kBytes <= 1024, "");
  // position of piece c of row r: c ^ swz(r)
  __device__ static inline int swz(int r) {
    if (kBytes == 128) return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
    if (k16) return ((r & 3) << 2) | ((r >> 2) & 3);
    return (((r >> 2) & 1) << 3) | ((r & 3) << 1) | ((r >> 3) & 1);
  }
};

// Global-to-LDS loads with 64-bit addresses: lane l's 16 (or 4) bytes land at
// LDS byte lds + 16 l (4 l); load i of a call 1 KB further.  Issued by hand for
// the reason given at the shrink's: the compiler would wait for every load in
// flight before each LDS read.  lds is wave-uniform.  ONCE: a non-temporal hint,
// for rows that no other workgroup reads.
#define LORA_LOAD_ROWS(NT)                                                                                      \
  asm volatile(                                                                                                 \
      "s_mov_b32 %0, m0\n\t"                                                                                    \
      "s_mov_b32 m0, %1\n\t"                                                                                    \
      "s_nop 0\n\t"                                                                                             \
      "global_load_lds_dwordx4 %2, off" NT "\n\t"                                                               \
      "s_add_u32 m0, m0, 0x400\n\t"                                                                             \
      "s_nop 0\n\t"                                                                                             \
      "global_load_lds_dwordx4 %3, off" NT "\n\t"                                                               \
      "s_mov_b32 m0, %0"                                                                                        \
      : "=&s"(saved)                                                                                            \
      : "s"(lds), "v"(a), "v"(b)                                                                                \
      : "memory", "scc")
__device__ inline void row_to_lds(const char* a, uint32_t lds) {
  lds = __builtin_amdgcn_readfirstlane(lds);
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %1\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %2, off\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "s"(lds), "v"(a)
      : "memory");
}
template <bool ONCE> __device__ inline void two_rows_to_lds(const char* a, const char* b, uint32_t lds) {
  lds = __builtin_amdgcn_readfirstlane(lds);
  uint32_t saved;
  if constexpr (ONCE) LORA_LOAD_ROWS(" nt");
  else LORA_LOAD_ROWS("");
}
#undef LORA_LOAD_ROWS
__device__ inline void word_to_lds(const char* g, uint32_t lds) {
  lds = __builtin_amdgcn_readfirstlane(lds);
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %1\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dword %2, off\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "s"(lds), "v"(g)
      : "memory");
}
template <int n> __device__ inline void wait_loads() {
  static_assert(n <= 63, "the wait counter's range");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(n) : "memory");
}
__device__ inline void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// The two lanes of a row.
__device__ inline float half_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ inline float half_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// What a workgroup works on.
struct Work {
  int64_t start;       // first row of the sequence
  int b, h, n, ctx;    // sequence, key/value head, nodes, context
  int row0, rows;      // this workgroup's first row (node * group + head) and the sequence's rows
  int k0, k1, split;   // keys [k0, k1)
  bool whole;          // the sequence's keys are one chunk
  bool none;           // nothing to do
};

__device__ inline void sequence_of(const AttendParams& p, int b, int64_t& start, int& n, int& ctx) {
  start = p.q_start[b];
  int64_t c = (int64_t)p.q_start[b + 1] - start;
  if (start < 0 || start > p.T) {
    start = 0;
    c = 0;
  }
  if (c > p.T - start) c = p.T - start;
  n = (int)(c < 0 ? 0 : (c > p.max_nodes ? p.max_nodes : c));
  const int x = p.context[b];
  ctx = x < 0 ? 0 : (x > p.max_context ? p.max_context : x);
}
__device__ inline int splits_of(const AttendParams& p, int n, int ctx) {
  const int last = ctx + n - 1;
  return last < 0 ? 1 : (int)p.by_chunk.div((uint32_t)last) + 1;
}

// Units of work are (chunk, sequence, head), in that order.
// SPREAD: they go to the XCDs (b % 8) in turn.  The first chunks, the long ones
// where contexts differ, are on all XCDs from the start: 25.5 us for 33.5 with the
// order below for 8 fp32 sequences of 46 to 1500 keys, 351 for 359 for 256 bf16
// ones of 128 to 4096.
// Else an XCD takes a contiguous range of the order sequence, head, chunk: heads
// side by side in memory are read through one L2, which is worth more where the
// matrix cores bound the time: 132.8 us for 134.6 for 16 sequences of 256 to 8192
// keys and 23 to 45 nodes (one of 32768 keys and 64 nodes: 65 either way).
// Either way the row tiles of a unit follow one another on one XCD.
template <int ROWS, bool SPREAD>
__device__ inline Work work_of(const AttendParams& p) {
  Work w;
  const uint32_t xcd = blockIdx.x % kXcds, j = blockIdx.x / kXcds, of_xcd = p.by_tiles.div(j);
  const int rt = (int)(j - of_xcd * p.by_tiles.d);
  uint32_t u = SPREAD ? of_xcd * kXcds + xcd : xcd * p.by_tiles.div(gridDim.x / kXcds) + of_xcd, v;
  if constexpr (!SPREAD) {
    v = p.by_splits.div(u);
    w.split = (int)(u - v * p.by_splits.d);
    u = v;
  }
  v = p.by_heads.div(u);
  w.h = (int)(u - v * p.by_heads.d);
  if constexpr (SPREAD) {
    u = v;
    v = p.by_sequences.div(u);
    w.b = (int)(u - v * p.by_sequences.d);
    w.split = (int)v;
  } else {
    w.b = (int)v;
  }
  w.none = SPREAD ? w.split >= p.splits : w.b >= p.B;
  if (w.none) return w;
  sequence_of(p, w.b, w.start, w.n, w.ctx);
  const int group = (int)p.group.d;
  w.row0 = rt * ROWS;
  w.rows = w.n * group;
  const int splits = splits_of(p, w.n, w.ctx);
  w.whole = splits == 1;
  w.none = w.row0 >= w.rows || w.split >= splits;
  const int last = min(w.row0 + ROWS, w.rows) - 1;
  const int end = w.ctx + (p.mask ? w.n : min(w.n, (int)p.group.div((uint32_t)max(last, 0)) + 1));
  const int64_t k0 = (int64_t)w.split * p.chunk;
  w.k0 = (int)k0;
  w.k1 = (int)min(k0 + p.chunk, (int64_t)end);
  return w;
}

// One row block of 32 rows: the query operand, the running softmax and the
// output, held by one wave.
template <typename Elem, int DP> struct RowBlock {
  using R = Rows<Elem, DP>;
  u32x4 q[R::kSteps];
  f32x16 o[R::kDB];
  float m, l;
  int lane, r32, hi;   // row in the block, half
  int node;            // of this lane's row
  int64_t row;         // of q and out, -1: none
  int head;
  uint64_t bits0;      // first word of the mask row
  // LDS addresses of this lane's operands in a tile: piece 2 st + hi of key row
  // r32 for the scores; for the values the rows and pieces described at
  // add_values.  What differs from these by a constant is an offset of the read.
  // Rows past 256 bytes leave no registers for them: their pieces are found by an
  // XOR from the first one's at each read.
  static constexpr bool kHeld = R::kBytes <= 256;
  static constexpr int kAhead = R::kSteps < 8 ? R::kSteps : 8, kKeyAt = kHeld ? kAhead : 1;
  static constexpr int kValueAt = !R::k16 || !kHeld ? 1 : R::kDB < 4 ? R::kDB : 4;
  uint32_t key_at[kKeyAt];
  uint32_t value_a[kValueAt], value_b[kValueAt];
  __device__ __forceinline__ static uint32_t value_piece(const uint32_t (&at)[kValueAt], int db) {
    return kHeld ? at[kHeld ? db : 0] : at[0] ^ (64 * db);
  }

  // Tiles of keys and values start at these LDS addresses.
  __device__ __forceinline__ void place(uint32_t keys, uint32_t values) {
#pragma unroll
    for (int st = 0; st < kKeyAt; ++st) key_at[st] = keys + r32 * R::kBytes + (((2 * st) ^ R::swz(r32) ^ hi) << 4);
    if constexpr (R::k16) {
      const int j = lane & 15, g1 = (lane >> 4) & 1;
      const int ra = 4 * hi + (j >> 2), rb = ra + 8;
      const int c = 2 * g1 + ((j & 3) >> 1), tail = (j & 1) * 8;
#pragma unroll
      for (int db = 0; db < kValueAt; ++db) {
        value_a[db] = values + ra * R::kBytes + tail + ((c ^ R::swz(ra) ^ (4 * db)) << 4);
        value_b[db] = values + rb * R::kBytes + tail + ((c ^ R::swz(rb) ^ (4 * db)) << 4);
      }
    } else {
      value_a[0] = values;
    }
  }
  // On to another tile, whose address differs in the bits of `by`.
  __device__ __forceinline__ void move_keys(uint32_t by) {
#pragma unroll
    for (int st = 0; st < kKeyAt; ++st) key_at[st] ^= by;
  }
  __device__ __forceinline__ void move_values(uint32_t by) {
#pragma unroll
    for (int db = 0; db < kValueAt; ++db) {
      value_a[db] ^= by;
      if (R::k16) value_b[db] ^= by;
    }
  }

  __device__ __forceinline__ void init(const AttendParams& p, const Work& w, int row_first) {
    lane = threadIdx.x & 63;
    r32 = lane & 31;
    hi = lane >> 5;
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int db = 0; db < R::kDB; ++db)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[db][i] = 0.f;
    const int r = row_first + r32;
    const bool ok = r < w.rows;
    node = (int)p.group.div((uint32_t)(ok ? r : 0));
    head = w.h * (int)p.group.d + (ok ? r - node * (int)p.group.d : 0);
    row = ok ? w.start + node : -1;
    const Elem* qr = static_cast<const Elem*>(p.q) + (ok ? row : 0) * p.ldq + (int64_t)head * p.d;
    constexpr int kVec = Traits<Elem>::kVec;
    // the softmax takes a positive factor: a negative scale turns q's signs
    // instead, and a scale of 0 is a q of zeros
    const uint32_t flip = p.scale < 0.f ? (R::k16 ? 0x80008000u : 0x80000000u) : 0u;
#pragma unroll
    for (int s = 0; s < R::kSteps; ++s) {
      const int c = (2 * s + hi) * kVec;
      q[s] = ld16_or0(qr + c, ok && c < p.d && p.scale != 0.f);
#pragma unroll
      for (int e = 0; e < 4; ++e) q[s][e] ^= flip;
    }
    bits0 = 0;
    if (p.mask && ok) bits0 = p.mask[row * p.mask_words];
    // here, so that no wait for it lands among the loads of the loop
    asm volatile("" ::"v"((uint32_t)bits0), "v"((uint32_t)(bits0 >> 32)));
  }

  // Bit j: this lane's row sees key first + j (j < 32) as far as the mask goes.
  __device__ __forceinline__ uint32_t sees(const AttendParams& p, const Work& w, int first) const {
    const int rel = first - w.ctx;  // of node 0
    if (row < 0 || rel <= -32) return ~0u;
    if (!p.mask) {
      const int c = node + 1 - rel;  // keys up to its own
      return c >= 32 ? ~0u : (c <= 0 ? 0u : (1u << c) - 1u);
    }
    if (rel < 0) return ((uint32_t)bits0 << -rel) | ((1u << -rel) - 1u);
    const int word = rel >> 6, sh = rel & 63;
    if (word >= p.mask_words) return 0u;
    const uint64_t* mr = p.mask + row * p.mask_words;
    uint64_t x = (word ? mr[word] : bits0) >> sh;
    if (sh > 32 && word + 1 < p.mask_words) x |= mr[word + 1] << (64 - sh);
    return (uint32_t)x;
  }

  // Scores of the 32 keys from row kFirst of the tile on.  The keys' operands
  // are requested eight at a time ahead of their products.
  template <int kFirst> __device__ __forceinline__ f32x16 scores() const {
    f32x16 s;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = 0.f;
#pragma unroll
    for (int s0 = 0; s0 < R::kSteps; s0 += kAhead) {
      u32x4 a[kAhead];
#pragma unroll
      for (int st = 0; st < kAhead; ++st)
        a[st] = *((lds_u32x4*)(lds_byte*)(uintptr_t)(kHeld ? key_at[kHeld ? st : 0] : key_at[0] ^ (32 * st)) +
                  (kFirst * R::kBytes + 32 * s0) / 16);
#pragma unroll
      for (int st = 0; st < kAhead; ++st) s = Mma32<Elem>::mma(a[st], q[s0 + st], s);
    }
    return s;
  }

  // Running softmax over NS blocks of scores (-inf where masked): scores become
  // weights.  c > 0 turns scores into powers of two.  m is moved only where a weight
  // would pass 2^kMost, and then below the score by kBelow: most tiles leave the
  // output as it is, and sums and weights stay clear of overflow.
  template <int NS> __device__ __forceinline__ void weigh(f32x16 (&s)[NS], float c) {
    constexpr float kBelow = Mma32<Elem>::kBelow, kMost = Mma32<Elem>::kMost;
    // four chains each for the maximum and the sum: an operation waits twice its
    // own time for the one before it
    float mx4[4] = {s[0][0], s[0][1], s[0][2], s[0][3]};
#pragma unroll
    for (int b = 0; b < NS; ++b)
#pragma unroll
      for (int i = b ? 0 : 4; i < 16; ++i) mx4[i & 3] = fmaxf(mx4[i & 3], s[b][i]);
    float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
    mx = __fmul_rn(half_max(mx), c);
    if (__any(mx - m > kMost)) {
      float mn = mx - kBelow;
      if (kBelow > 0.f && mx - mn > kMost) mn = mx;  // a score that has no units left
      if (!(mx - m > kMost)) mn = m;
      const float f = __builtin_amdgcn_exp2f(m - (mn == -INFINITY ? 0.f : mn));
      l *= f;
#pragma unroll
      for (int db = 0; db < R::kDB; ++db)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[db][i] *= f;
      m = mn;
    }
    const float ms = m == -INFINITY ? 0.f : m;
    // s c - m is taken without rounding s c, as m's product was: by up to half a step of
    // m the difference may pass kMost, or leave no weight at all.  Where that is more
    // than a sixteenth of a power of two, s c is rounded too.
    if (__builtin_expect(__any(fabsf(ms) >= 0x1p20f), 0)) {
#pragma unroll
      for (int b = 0; b < NS; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[b][i] = __fmul_rn(s[b][i], c);
      c = 1.0f;
    }
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int b = 0; b < NS; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[b][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][i], c, -ms));
        sum[i & 3] += s[b][i];
      }
    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
  }

  // -inf for the keys that this lane's row does not see.
  __device__ __forceinline__ void mask_scores(f32x16& s, uint32_t seen) const {
    const uint32_t sb = seen >> (4 * hi);
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = (sb >> (8 * (i >> 2) + (i & 3))) & 1 ? s[i] : -INFINITY;
  }

  // A block's weights as the operand of its product with the values, which takes
  // both in one type: with 16-bit values each weight is rounded to theirs, off by half
  // a step of itself (l sums them unrounded).  Outputs then lie 0.0019 to 0.0023 from
  // 64 bits relative to their rows in bf16 and 0.00028 in fp16, where rounding them
  // alone gives 0.0017 and 0.00021; a second product with what the rounding took
  // off would double the matrix work on the values.
  struct Weights {
    u32x4 w[R::k16 ? 2 : 4];
  };
  __device__ __forceinline__ static Weights pack(const f32x16& s) {
    Weights r;
#pragma unroll
    for (int i = 0; i < (R::k16 ? 2 : 4); ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (R::k16) r.w[i][e] = Mma32<Elem>::pack2(s[8 * i + 2 * e], s[8 * i + 2 * e + 1]);
        else r.w[i][e] = __float_as_uint(s[4 * i + e]);
      }
    return r;
  }

  // o += V^T P^T over the 32 keys from row kFirst of the tile on.  ODD: what is no
  // finite number enters as 0 (see add_odd).
  // 16-bit: for step u the contraction runs over keys 16 u + 4 hi + (0..3) and
  // 16 u + 8 + 4 hi + (0..3), as the weights lie in registers; a transposing read
  // gives a lane 4 keys of one element, its 16 lanes reading 4 rows of 32 bytes.
  template <bool ODD, int kFirst> __device__ __forceinline__ void add_values(const Weights& p) {
    if constexpr (R::k16) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        s16x4 va[R::kDB], vc[R::kDB];
#pragma unroll
        for (int db = 0; db < R::kDB; ++db) {
          // blocks past the fourth lie 256 bytes (the swizzle's range) further
          const int off = ((kFirst + 16 * u) * R::kBytes + (db / 4) * 256) / 8;
          va[db] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (lds_s16x4*)(lds_byte*)(uintptr_t)value_piece(value_a, db % 4) + off);
          vc[db] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (lds_s16x4*)(lds_byte*)(uintptr_t)value_piece(value_b, db % 4) + off);
        }
#pragma unroll
        for (int db = 0; db < R::kDB; ++db) {
          const u32x2 a2 = __builtin_bit_cast(u32x2, va[db]), b2 = __builtin_bit_cast(u32x2, vc[db]);
          u32x4 v = u32x4{a2[0], a2[1], b2[0], b2[1]};
          if constexpr (ODD)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t x = v[e], e1 = Mma32<Elem>::kExp, e2 = e1 << 16;
              v[e] = ((x & e1) == e1 ? 0u : x & 0xffffu) | ((x & e2) == e2 ? 0u : x & 0xffff0000u);
            }
          o[db] = Mma32<Elem>::mma(v, p.w[u], o[db]);
        }
      }
    } else {
      const int c = (r32 >> 2) ^ (hi << 3);
      const lds_byte* pr = (lds_byte*)(uintptr_t)(value_a[0] + 4 * hi * R::kBytes + (r32 & 3) * 4);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int key = 8 * (i >> 2) + (i & 3);  // + 4 hi
        const int x = ((i & 3) << 1) | ((i >> 2) & 1);
        float v[R::kDB];
#pragma unroll
        for (int db = 0; db < R::kDB; ++db) {
          v[db] = *(lds_float*)(pr + ((((8 * db) & 8) ^ c ^ x) << 4) + (kFirst + key) * R::kBytes + (db / 2) * 256);
          if (ODD && (__float_as_uint(v[db]) & Mma32<Elem>::kExp) == Mma32<Elem>::kExp) v[db] = 0.f;
        }
        const uint32_t wi = p.w[i / 4][i % 4];
#pragma unroll
        for (int db = 0; db < R::kDB; ++db) o[db] = Mma32<Elem>::mma1(v[db], __uint_as_float(wi), o[db]);
      }
    }
  }

  // The values that add_values<true> left out: infinities and NaN reach the rows
  // that see their key.  In the product a masked weight of 0 would have turned
  // them into NaN for every row.
  __device__ __forceinline__ void add_odd(const char* vb, uint32_t seen) {
#pragma unroll 1
    for (int k = 0; k < kBlock; ++k) {
      if (!any_odd(vb + k * R::kBytes, 1)) continue;
      const bool mine = (seen >> k) & 1;
#pragma unroll
      for (int db = 0; db < R::kDB; ++db)
#pragma unroll
        for (int qd = 0; qd < 4; ++qd) {
          const int at = element(db, qd) * (int)sizeof(Elem);
          const char* px = vb + k * R::kBytes + (((at >> 4) ^ R::swz(k)) << 4) + (at & 15);
          uint32_t x[4];
          if constexpr (R::k16) {
            const u32x2 h = *reinterpret_cast<const u32x2*>(px);
            const uint32_t h0 = h[0], h1 = h[1];
            x[0] = h0 & 0xffffu;
            x[1] = h0 >> 16;
            x[2] = h1 & 0xffffu;
            x[3] = h1 >> 16;
          } else {
            const u32x4 h = *reinterpret_cast<const u32x4*>(px);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = h[e];
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (mine && (x[e] & Mma32<Elem>::kExp) == Mma32<Elem>::kExp)
              o[db][4 * qd + e] += Traits<Elem>::elem_to_float(x[e]);
        }
    }
  }

  // Whether the value rows [0, keys) at vb hold something that is no finite
  // number; the wave looks at all of them.
  __device__ __forceinline__ bool any_odd(const char* vb, int keys) const {
    bool odd = false;
    for (int e = lane; e < keys * R::kPieces; e += 64) {
      const u32x4 x = *reinterpret_cast<const u32x4*>(vb + 16 * e);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = x[i], e1 = Mma32<Elem>::kExp;
        if constexpr (R::k16) odd |= (w & e1) == e1 || ((w >> 16) & e1) == e1;
        else odd |= (w & e1) == e1;
      }
    }
    return __any(odd);
  }

  // Store four consecutive elements of the row's output.
  __device__ __forceinline__ static void store4(const AttendParams& p, int64_t row, int head, int at, f32x4 x) {
    Elem* out = static_cast<Elem*>(p.out) + row * p.ldo + (int64_t)head * p.d + at;
    if constexpr (R::k16) {
      *reinterpret_cast<u32x2*>(out) =
          u32x2{Mma32<Elem>::pack2(x[0], x[1]), Mma32<Elem>::pack2(x[2], x[3])};
    } else {
      *reinterpret_cast<f32x4*>(out) = x;
    }
  }
  // Element of the row that register quad qd of block db holds first.
  __device__ __forceinline__ int element(int db, int qd) const { return 32 * db + 8 * qd + 4 * hi; }
};

struct No {
  static constexpr bool value = false;
};
struct Yes {
  static constexpr bool value = true;
};

__device__ inline float inverse(float l) { return l == 0.f ? 0.f : 1.0f / l; }

// The workspace: for each chunk and row the unnormalised output and (m, l).  It has
// part_rows rows a chunk: the call's T, or where T is more than the sequences can
// have (a padded batch) max_nodes of each sequence.
__device__ inline int64_t part_row(const AttendParams& p, int b, int64_t start, int node) {
  return (p.part_rows < p.T ? (int64_t)b * p.max_nodes : start) + node;
}
__device__ inline float* part_o(const AttendParams& p, int split, int64_t row, int head) {
  return p.part + (((int64_t)split * p.part_rows + row) * p.hq + head) * p.d;
}
__device__ inline float* part_ml(const AttendParams& p, int split, int64_t row, int head) {
  return p.part + (int64_t)p.splits * p.part_rows * p.hq * p.d + (((int64_t)split * p.part_rows + row) * p.hq + head) * 2;
}

// Store the rows of a block whose keys are all done: the output where the sequence's
// keys are one chunk, else the chunk's part.  A lane holds 4 elements here and there
// of one row; they pass through `lds` (kBlock rows of DP floats, this wave's own),
// so that a store of the wave covers whole rows, up to 128 elements at a time.
// The 16-byte pieces of a row lie XOR-swizzled by row there, without which the 32
// rows of a write would meet in the same banks.
template <int DP> constexpr int kStoreBytes = kBlock * (DP < 128 ? DP : 128) * 4;
template <typename Elem, int DP>
__device__ __forceinline__ void store_rows(const AttendParams& p, const Work& w, const RowBlock<Elem, DP>& rb, float l,
                                           int row_first, char* lds) {
  constexpr int kCols = DP < 128 ? DP : 128, kPieces = kCols / 4, kRowsAtOnce = 64 / kPieces;
  const bool whole = w.whole;
  const float inv = whole ? inverse(l) : 1.0f;
  f32x4* at = reinterpret_cast<f32x4*>(lds);
  const int lane = rb.lane, piece = lane % kPieces;
#pragma unroll
  for (int c0 = 0; c0 < DP; c0 += kCols) {
#pragma unroll
    for (int db = 0; db < kCols / kBlock; ++db)
#pragma unroll
      for (int qd = 0; qd < 4; ++qd) {
        const f32x16& o = rb.o[c0 / kBlock + db];
        const f32x4 x = f32x4{o[4 * qd] * inv, o[4 * qd + 1] * inv, o[4 * qd + 2] * inv, o[4 * qd + 3] * inv};
        at[rb.r32 * kPieces + ((8 * db + 2 * qd + rb.hi) ^ (rb.r32 & 15))] = x;
      }
    wait_lds();
    const int col = c0 + 4 * piece;
    // (a loop: code that runs once is fetched at a miss of the instruction cache a line)
#pragma unroll 2
    for (int r0 = 0; r0 < kBlock; r0 += kRowsAtOnce) {
      const int r = r0 + lane / kPieces, row = row_first + r;
      const f32x4 x = at[r * kPieces + (piece ^ (r & 15))];
      if (row >= w.rows || col >= p.d) continue;
      const int node = (int)p.group.div((uint32_t)row), head = w.h * (int)p.group.d + row - node * (int)p.group.d;
      if (whole) rb.store4(p, w.start + node, head, col, x);
      else *reinterpret_cast<f32x4*>(part_o(p, w.split, part_row(p, w.b, w.start, node), head) + col) = x;
    }
    wait_lds();
  }
  if (rb.row < 0 || rb.hi) return;
  if (!whole) {
    float* ml = part_ml(p, w.split, part_row(p, w.b, w.start, rb.node), rb.head);
    ml[0] = rb.m;
    ml[1] = l;
  } else if (p.lse) {
    p.lse[rb.row * p.hq + rb.head] = (rb.m + __builtin_amdgcn_logf(l)) * kLn2;
  }
}

// Where a lane's key lies: its page's number comes from the table by way of LDS.
struct PageAt {
  int place;      // row in the page
  bool in_table;  // a key of the chunk whose page the table has
};
__device__ inline PageAt page_at(const AttendParams& p, int64_t pos, int end, int& col) {
  PageAt a;
  const uint32_t at = (uint32_t)min(pos, (int64_t)end);
  col = (int)p.cache.page.div(at);
  a.place = (int)(at - (uint32_t)col * p.cache.page.d);
  a.in_table = pos < end && col < p.n_table;
  return a;
}
__device__ inline const char* entry_of(const AttendParams& p, int b, const PageAt& a, int col) {
  return a.in_table ? reinterpret_cast<const char*>(p.page_table + b * p.ld_table + col)
                    : reinterpret_cast<const char*>(g_zero_row);
}
// One of the cache's two tensors, at the call's head; strides in bytes below
// 2^32 (the host checks), so a row's address is two 32 x 32 + 64-bit products.
struct HeadAt {
  uint64_t base;
  uint32_t page, row;
  __device__ __forceinline__ uint64_t row_at(uint32_t id, int place) const {
    return base + (uint64_t)id * page + (uint64_t)(uint32_t)place * row;
  }
};
template <typename Elem> __device__ inline HeadAt head_at(const AttendParams& p, int h, bool is_v) {
  const CacheView& c = p.cache;
  HeadAt a;
  a.base = reinterpret_cast<uint64_t>(is_v ? c.v : c.k) + (uint64_t)(h * (is_v ? c.v_head : c.k_head)) * sizeof(Elem);
  a.page = (uint32_t)((is_v ? c.v_page : c.k_page) * (int64_t)sizeof(Elem));
  a.row = (uint32_t)((is_v ? c.v_row : c.k_row) * (int64_t)sizeof(Elem));
  return a;
}

// The global addresses that this lane loads for a tile, found one tile ahead
// (NL loads of the keys and of the values), where the registers have room for
// them; else they are read from the rows' addresses in LDS for each load.
template <typename Elem, int DP, int NL, bool HELD> struct TileRows {
  using R = Rows<Elem, DP>;
  static constexpr bool kHeld = HELD;
  const char *k[kHeld ? NL : 1], *v[kHeld ? NL : 1];
  uint32_t valid;  // rows that are keys
};
// Address of the 16-byte piece that this lane brings in load i: the rows'
// addresses are in LDS at `rows`, row_0 is the tile's row of the first of them.
template <typename Elem, int DP>
__device__ __forceinline__ const char* piece_of(const AttendParams& p, const char* const* rows, int row_0, int i,
                                                int lane) {
  using R = Rows<Elem, DP>;
  const int r = i * R::kPerLoad + lane / R::kPieces;
  const int piece = (lane % R::kPieces) ^ R::swz(row_0 + r);
  const char* at = rows[r];
  if (p.d != DP && piece * 16 >= p.d * (int)sizeof(Elem)) at = reinterpret_cast<const char*>(g_zero_row);
  return at + 16 * piece;
}

// Up to 32 rows: the NW waves of the workgroup hold the same rows and take the
// chunk's blocks of 32 keys in turn, each through LDS of its own, so no wave
// waits for another until their outputs meet at the end.  The next block's
// keys are on their way during the weights and values of this one, its values
// during the next scores; page numbers come through LDS three blocks ahead,
// addresses are found two blocks ahead.
// Bound by memory: 256 sequences of 128 to 4096 keys, 32 + 8 bf16 heads of 128
// (2.2 GB): 350 us, 6.3 TB/s.  One workgroup a compute unit, 16 KB in flight a
// wave; two push each other's rows out of L2 (4.9 TB/s).  Loads are non-temporal,
// each row is read once.  fp32 heads of 64 have too little in flight in one
// workgroup and run two a compute unit: 25.5 us for 29.8 (8 sequences of 46 to 1500
// keys).  Heads of 256 elements spill some registers: 64 sequences of 4096 keys, 16
// + 4 bf16 heads (1.07 GB), 254 us.
template <typename Elem, int DP, int NW>
__global__ __launch_bounds__(NW * 64, (Rows<Elem, DP>::kNarrowWaves)) void attend_narrow_kernel(AttendParams p) {
  using R = Rows<Elem, DP>;
  constexpr int kTile = kBlock * R::kBytes;
  constexpr int NL = kTile / 1024;  // loads of a tile of keys or values
  __shared__ __attribute__((aligned(1024))) char s_kv[NW][2 * kTile];
  __shared__ __attribute__((aligned(16))) const char* s_row[NW][64];
  __shared__ int s_id[NW][2][64];
  __shared__ float s_ml[NW][2][kBlock];
  warm_args(p);
  const Work w = work_of<kBlock, true>(p);
  if (w.none) return;
  RowBlock<Elem, DP> rb;
  rb.init(p, w, w.row0);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = rb.lane;
  char* kbuf = s_kv[wave];
  char* vbuf = kbuf + kTile;
  const uint32_t k_lds = (uint32_t)(uintptr_t)kbuf, v_lds = (uint32_t)(uintptr_t)vbuf;
  const float c = p.scale == 0.f ? 1.0f : fabsf(p.scale) * kLog2e;
  // this wave's tiles, the first nf of them wholly inside the context
  const auto tiles = [&](int keys, bool whole) {
    const int blocks = keys <= 0 ? 0 : whole ? keys / kBlock : (keys + kBlock - 1) / kBlock;
    return blocks > wave ? (blocks - wave + NW - 1) / NW : 0;
  };
  const int nt = tiles(w.k1 - w.k0, false), nf = tiles(min(w.ctx, w.k1) - w.k0, true);

  auto first_key = [&](int t) { return (int64_t)w.k0 + ((int64_t)wave + (int64_t)NW * t) * kBlock; };
  const HeadAt hk = head_at<Elem>(p, w.h, false), hv = head_at<Elem>(p, w.h, true);
  PageAt ahead[2];
  auto fetch_ids = [&](int t, PageAt& a) {
    int col;
    a = page_at(p, first_key(t) + rb.r32, w.k1, col);
    word_to_lds(entry_of(p, w.b, a, col), (uint32_t)(uintptr_t)s_id[wave][t & 1]);
  };
  TileRows<Elem, DP, NL, (NL <= 8)> at;
  auto find_rows = [&](int t, const PageAt& a) {  // half of the lanes the keys' rows, half the values'
    const uint32_t id = (uint32_t)s_id[wave][t & 1][lane];
    const bool valid = a.in_table && id < (uint64_t)p.cache.n_pages && (int)id >= 0;
    const uint64_t row = (rb.hi ? hv : hk).row_at(id, a.place);
    s_row[wave][lane] = valid ? reinterpret_cast<const char*>(row) : reinterpret_cast<const char*>(g_zero_row);
    at.valid = (uint32_t)__ballot(valid);
    if constexpr (at.kHeld) {
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        at.k[i] = piece_of<Elem, DP>(p, s_row[wave], 0, i, lane);
        at.v[i] = piece_of<Elem, DP>(p, s_row[wave] + 32, 0, i, lane);
      }
    }
  };
  auto load = [&](const char* const* held, const char* const* rows, uint32_t lds) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NL; i += 2) {
      const char* a = at.kHeld ? held[at.kHeld ? i : 0] : piece_of<Elem, DP>(p, rows, 0, i, lane);
      const char* b = at.kHeld ? held[at.kHeld ? i + 1 : 0] : piece_of<Elem, DP>(p, rows, 0, i + 1, lane);
      two_rows_to_lds<true>(a, b, lds + 1024 * i);
    }
  };

  uint32_t valid = 0;
  if (nt > 0) {
    fetch_ids(0, ahead[0]);
    fetch_ids(1, ahead[1]);
    wait_loads<0>();
    find_rows(0, ahead[0]);
    valid = at.valid;
    load(at.k, s_row[wave], k_lds);
    fetch_ids(2, ahead[0]);
    load(at.v, s_row[wave] + 32, v_lds);
    find_rows(1, ahead[1]);
  }
  auto tile = [&](int t, auto tail) __attribute__((always_inline)) {
    constexpr bool kTail = decltype(tail)::value;
    const bool more = t + 1 < nt;
    wait_loads<NL>();  // keys of t and page numbers of t + 2 are there
    f32x16 s[1] = {rb.template scores<0>()};
    wait_lds();
    if (more) {
      load(at.k, s_row[wave], k_lds);
      fetch_ids(t + 3, ahead[1]);
    }
    uint32_t seen = valid;
    if constexpr (kTail) seen &= rb.sees(p, w, (int)first_key(t));
    if (__any(seen != ~0u)) rb.mask_scores(s[0], seen);
    rb.weigh(s, c);
    if (more) wait_loads<NL + 1>();
    else wait_loads<0>();
    if (kTail && __any(seen != valid) && rb.any_odd(vbuf, kBlock)) {
      rb.template add_values<kTail, 0>(rb.pack(s[0]));
      rb.add_odd(vbuf, seen);
    } else {
      rb.template add_values<false, 0>(rb.pack(s[0]));
    }
    wait_lds();
    valid = at.valid;
    if (more) {
      load(at.v, s_row[wave] + 32, v_lds);
      find_rows(t + 2, ahead[0]);
      ahead[0] = ahead[1];
    }
  };
  rb.place(k_lds, v_lds);
  int t = 0;
  for (; t < nf; ++t) tile(t, No{});
  for (; t < nt; ++t) tile(t, Yes{});

  // the waves' outputs meet: weights to their common maximum, then block db of
  // the output is summed and stored by wave db % NW
  const float l = half_sum(rb.l);
  if (rb.hi == 0) {
    s_ml[wave][0][rb.r32] = rb.m;
    s_ml[wave][1][rb.r32] = l;
  }
  f32x4* red = reinterpret_cast<f32x4*>(kbuf);
#pragma unroll
  for (int db = 0; db < R::kDB; ++db)
#pragma unroll
    for (int qd = 0; qd < 4; ++qd)
      red[(db * 4 + qd) * 64 + lane] =
          f32x4{rb.o[db][4 * qd], rb.o[db][4 * qd + 1], rb.o[db][4 * qd + 2], rb.o[db][4 * qd + 3]};
  __syncthreads();
  float M = -INFINITY, L = 0.f, f[NW];
#pragma unroll
  for (int i = 0; i < NW; ++i) M = fmaxf(M, s_ml[i][0][rb.r32]);
  const float ms = M == -INFINITY ? 0.f : M;
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    f[i] = __builtin_amdgcn_exp2f(s_ml[i][0][rb.r32] - ms);
    L += s_ml[i][1][rb.r32] * f[i];
  }
  if (rb.row < 0) return;
  const bool whole = w.whole;
  const float inv = whole ? inverse(L) : 1.0f;
  for (int db = wave; db < R::kDB; db += NW) {
#pragma unroll
    for (int qd = 0; qd < 4; ++qd) {
      const int at = rb.element(db, qd);
      if (at >= p.d) continue;
      f32x4 sum = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        const f32x4 x = reinterpret_cast<const f32x4*>(s_kv[i])[(db * 4 + qd) * 64 + lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] = __builtin_fmaf(x[e], f[i], sum[e]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] *= inv;
      if (whole) rb.store4(p, rb.row, rb.head, at, sum);
      else *reinterpret_cast<f32x4*>(part_o(p, w.split, part_row(p, w.b, w.start, rb.node), rb.head) + at) = sum;
    }
  }
  if (wave == 0 && rb.hi == 0) {
    if (!whole) {
      float* ml = part_ml(p, w.split, part_row(p, w.b, w.start, rb.node), rb.head);
      ml[0] = M;
      ml[1] = L;
    } else if (p.lse) {
      p.lse[rb.row * p.hq + rb.head] = (M + __builtin_amdgcn_logf(L)) * kLn2;
    }
  }
}

// More rows of more than 256 bytes (fp32 heads from 72 elements, 16-bit ones from
// 136), whose outputs leave no registers for the kernel below: four waves of 32
// rows share tiles of 32 keys, double buffered; a wave fetches a quarter of each
// tile's rows.  One workgroup a compute unit.  Bound by the matrix cores and the
// weights in turn, heads of 256 elements by spilled registers too (fp32 234 a lane,
// 16-bit 74): 3 sequences of 12 nodes over 1949 keys, 32 + 8 fp32 heads of 256, 228
// us; 4 of 32 nodes over 8224, 16 + 4 bf16 heads of 256 (135 MB, 17 GFLOP), 113 us.
template <typename Elem, int DP>
__global__ __launch_bounds__(kThreads, 1) void attend_wide_kernel(AttendParams p) {
  using R = Rows<Elem, DP>;
  constexpr int KT = kBlock;
  constexpr int kTile = KT * R::kBytes;
  constexpr int kMine = KT / 4;  // rows a wave fetches of K, and of V
  constexpr int NL = kMine * R::kBytes / 1024;
  static_assert(kMine % R::kPerLoad == 0 && NL >= 1, "");
  // (a multiple of its two tiles' distance, so that an XOR changes tiles)
  __shared__ __attribute__((aligned(4 * kTile))) char s_kv[2][2 * kTile];
  static_assert(4 * kStoreBytes<DP> <= 4 * kTile, "");
  __shared__ __attribute__((aligned(16))) const char* s_row[4][64];
  __shared__ int s_id[4][2][64];
  __shared__ uint32_t s_valid[4][4];
  warm_args(p);
  const Work w = work_of<4 * kBlock, true>(p);
  if (w.none) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  RowBlock<Elem, DP> rb;
  rb.init(p, w, w.row0 + wave * kBlock);
  const bool idle = w.row0 + wave * kBlock >= w.rows;  // a wave without rows only fetches
  const int lane = rb.lane;
  const float c = p.scale == 0.f ? 1.0f : fabsf(p.scale) * kLog2e;
  const int keys = w.k1 - w.k0, inside = min(w.ctx, w.k1) - w.k0;
  const int nt = keys > 0 ? (keys + KT - 1) / KT : 0, nf = inside > 0 ? inside / KT : 0;
  const int my = lane % kMine, my_v = (lane / kMine) & 1;

  const HeadAt hk = head_at<Elem>(p, w.h, false), hv = head_at<Elem>(p, w.h, true);
  PageAt ahead[2];
  auto fetch_ids = [&](int t, PageAt& a) {
    int col;
    a = page_at(p, (int64_t)w.k0 + (int64_t)t * KT + wave * kMine + my, w.k1, col);
    word_to_lds(entry_of(p, w.b, a, col), (uint32_t)(uintptr_t)s_id[wave][t & 1]);
  };
  auto find_rows = [&](int t, const PageAt& a) {
    const uint32_t id = (uint32_t)s_id[wave][t & 1][lane];
    const bool valid = a.in_table && id < (uint64_t)p.cache.n_pages && (int)id >= 0;
    const uint64_t row = (my_v ? hv : hk).row_at(id, a.place);
    s_row[wave][lane] = valid ? reinterpret_cast<const char*>(row) : reinterpret_cast<const char*>(g_zero_row);
    const uint32_t got = (uint32_t)__ballot(valid) & (uint32_t)((1ull << kMine) - 1);
    if (lane == 0) s_valid[t & 3][wave] = got;
  };
  auto load_tile = [&](int t) {
    const uint32_t to = (uint32_t)(uintptr_t)s_kv[t & 1] + wave * kMine * R::kBytes;
    const char* a[2 * NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      a[i] = piece_of<Elem, DP>(p, s_row[wave], wave * kMine, i, lane);
      a[NL + i] = piece_of<Elem, DP>(p, s_row[wave] + kMine, wave * kMine, i, lane);
    }
#pragma unroll
    for (int i = 0; i < NL; i += 2) two_rows_to_lds<false>(a[i], a[i + 1], to + 1024 * i);
#pragma unroll
    for (int i = 0; i < NL; i += 2) two_rows_to_lds<false>(a[NL + i], a[NL + i + 1], to + kTile + 1024 * i);
  };

  if (nt > 0) {
    fetch_ids(0, ahead[0]);
    fetch_ids(1, ahead[1]);
    wait_loads<0>();
    find_rows(0, ahead[0]);
    load_tile(0);
    fetch_ids(2, ahead[0]);
    find_rows(1, ahead[1]);
  }
  auto tile = [&](int t, auto tail) __attribute__((always_inline)) {
    constexpr bool kTail = decltype(tail)::value;
    wait_loads<0>();  // this wave's part of tile t, and its page numbers of t + 2
    lds_barrier();    // everyone's, and everyone is done with tile t - 1
    const bool more = t + 1 < nt;
    if (more) {
      load_tile(t + 1);
      fetch_ids(t + 3, ahead[1]);
    }
    if (!idle) {
      f32x16 s[1] = {rb.template scores<0>()};
      uint32_t valid = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) valid |= s_valid[t & 3][i] << (i * kMine);
      uint32_t seen = valid;
      bool uneven = false;
      if constexpr (kTail) {
        seen &= rb.sees(p, w, w.k0 + t * KT);
        uneven = __any(seen != valid);
      }
      if (__any(seen != ~0u)) rb.mask_scores(s[0], seen);
      rb.weigh(s, c);
      const char* vb = s_kv[t & 1] + kTile;
      if (kTail && uneven && rb.any_odd(vb, KT)) {
        rb.template add_values<kTail, 0>(rb.pack(s[0]));
        rb.add_odd(vb, seen);
      } else {
        rb.template add_values<false, 0>(rb.pack(s[0]));
      }
    }
    rb.move_keys(2 * kTile);
    rb.move_values(2 * kTile);
    if (more) {
      find_rows(t + 2, ahead[0]);
      ahead[0] = ahead[1];
    }
  };
  rb.place((uint32_t)(uintptr_t)s_kv[0], (uint32_t)(uintptr_t)s_kv[0] + kTile);
  int t = 0;
  for (; t < nf; ++t) tile(t, No{});
  for (; t < nt; ++t) tile(t, Yes{});

  __syncthreads();
  store_rows(p, w, rb, half_sum(rb.l), w.row0 + wave * kBlock, &s_kv[0][0] + wave * kStoreBytes<DP>);
}

// Rows of 16-bit heads up to 128 elements and fp32 heads up to 64: eight waves
// in two groups of four that take turns.  While one group multiplies (the
// values of its last tile and the scores of its next, on the matrix cores), the
// other computes weights (on the vector unit); a barrier ends each half step,
// and the second group runs one half step behind, so that each SIMD always has
// one wave of each kind.  KG = 1: the eight waves hold 256 rows and all take a
// stage's 64 keys.  KG = 2: the groups hold the same 128 rows and take 32 keys of
// a stage each; their outputs meet at the end.
// Stages are in a ring of four: before the weights of step t a wave fetches its
// eighth of stage t + 2 into the ring place that stage t - 2 left.  The row
// addresses of four stages are found together, one a lane, at the second step of
// the four before; their page numbers are requested two steps earlier.
// Bound by the issue of a stage's work, matrix products (0.5 us a group), weights
// (0.5), the loads' issue and addresses (0.4): 2.3 to 2.6 us a stage of 64 keys with
// every compute unit at work, of which keys in L2 save a fifth.  One sequence of 64
// nodes over 32768 keys, 32 + 8 bf16 heads of 128: 61 to 65 us (134 MB, 34 GFLOP; 8
// are the join); 32 fp16 sequences of 64 over 4032: 185 us, 730 TFLOP/s.  Measured and
// slower, each against the kernel as it was then:
// all eight waves in step (75 for 71 us on the first), the loads before the products
// (66 for 64; 143 for 132 on 16 ragged sequences), spread over the products (78) or
// over the weights (72), chunks for two workgroups a compute unit in turn (89), no
// priority for the products (132 for 130 on the ragged ones) or the weights' (155).
template <typename Elem, int DP, int KG>
__global__ __launch_bounds__(512, 2) void attend_turns_kernel(AttendParams p) {
  using R = Rows<Elem, DP>;
  using Block = RowBlock<Elem, DP>;
  constexpr int KT = 64, NS = 2 / KG, kRing = 4;
  constexpr int kTile = KT * R::kBytes, kStage = 2 * kTile;
  constexpr int kMine = KT / 8;  // rows a wave fetches of K, and of V
  constexpr int NL = kMine * R::kBytes / 1024;
  static_assert(NL >= 1, "");
  // (aligned to its size, so that an XOR changes stages)
  __shared__ __attribute__((aligned(kRing * kStage))) char s_kv[kRing][kStage];
  __shared__ __attribute__((aligned(16))) const char* s_row[8][64];
  __shared__ int s_id[8][2][64];
  __shared__ __attribute__((aligned(8))) uint8_t s_valid[8][8];
  warm_args(p);
  const Work w = work_of<32 * 8 / KG, false>(p);
  if (w.none) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int late = wave >> 2;                        // the group that runs behind
  const int block = KG == 1 ? wave : wave & 3, part = KG == 1 ? 0 : late;
  Block rb;
  rb.init(p, w, w.row0 + block * kBlock);
  const bool idle = w.row0 + block * kBlock >= w.rows;  // a wave without rows only fetches
  const int lane = rb.lane;
  const float c = p.scale == 0.f ? 1.0f : fabsf(p.scale) * kLog2e;
  const int keys = w.k1 - w.k0, inside = min(w.ctx, w.k1) - w.k0;
  const int nt = keys > 0 ? (keys + KT - 1) / KT : 0, nf = inside > 0 ? inside / KT : 0;

  // lane 16 i + 8 v + r finds row r of this wave's eighth of the i-th of four
  // stages, of the keys (v = 0) and of the values
  const int my_v = (lane >> 3) & 1;
  PageAt ahead;
  auto position = [&](int four) {
    return (int64_t)w.k0 + ((int64_t)four * 4 + (lane >> 4)) * KT + wave * kMine + (lane & 7);
  };
  auto fetch_ids = [&](int four) {
    int col;
    ahead = page_at(p, position(four), w.k1, col);
    word_to_lds(entry_of(p, w.b, ahead, col), (uint32_t)(uintptr_t)s_id[wave][four & 1]);
  };
  auto find_rows = [&](int four, const PageAt& a) {
    const HeadAt h = head_at<Elem>(p, w.h, my_v);
    const uint32_t id = (uint32_t)s_id[wave][four & 1][lane];
    const bool valid = a.in_table && id < (uint64_t)p.cache.n_pages && (int)id >= 0;
    s_row[wave][lane] =
        valid ? reinterpret_cast<const char*>(h.row_at(id, a.place)) : reinterpret_cast<const char*>(g_zero_row);
    const uint64_t all = __ballot(valid);
    if ((lane & 15) == 0) s_valid[(four * 4 + (lane >> 4)) & 7][wave] = (uint8_t)(all >> lane);
  };
  auto load_stage = [&](int t) {
    const uint32_t to = (uint32_t)(uintptr_t)s_kv[t % kRing] + wave * kMine * R::kBytes;
    const char* const* rows = s_row[wave] + 16 * (t & 3);
    const char* a[2 * NL];
#pragma unroll
    for (int i = 0; i < 2 * NL; ++i) a[i] = rows[(i / NL) * kMine + (i % NL) * R::kPerLoad + lane / R::kPieces];
#pragma unroll
    for (int i = 0; i < 2 * NL; ++i) {
      const int piece = (lane % R::kPieces) ^ R::swz(wave * kMine + (i % NL) * R::kPerLoad + lane / R::kPieces);
      if (p.d != DP && piece * 16 >= p.d * (int)sizeof(Elem)) a[i] = reinterpret_cast<const char*>(g_zero_row);
      row_to_lds(a[i] + 16 * piece, to + (i / NL) * kTile + 1024 * (i % NL));
    }
  };

  f32x16 s[NS];
  typename Block::Weights weights[NS];
  uint32_t seen[NS];
  bool odd = false;
  uint32_t keys_in = 0, values_in = 0;  // ring places that the operand addresses are at
  auto multiply = [&](int t, bool values, bool scores, auto tail) __attribute__((always_inline)) {
    if (idle) return;
    if (values) {
      const uint32_t at = (uint32_t)(t - 1) % kRing;
      rb.move_values((values_in ^ at) * kStage);
      values_in = at;
      if (decltype(tail)::value && odd) {
        const char* vb = s_kv[at] + kTile + part * kBlock * R::kBytes;
        rb.template add_values<decltype(tail)::value, 0>(weights[0]);
        rb.add_odd(vb, seen[0]);
        if constexpr (NS == 2) {
          rb.template add_values<decltype(tail)::value, kBlock>(weights[1]);
          rb.add_odd(vb + kBlock * R::kBytes, seen[1]);
        }
      } else {
        rb.template add_values<false, 0>(weights[0]);
        if constexpr (NS == 2) rb.template add_values<false, kBlock>(weights[1]);
      }
    }
    if (scores) {
      const uint32_t at = (uint32_t)t % kRing;
      rb.move_keys((keys_in ^ at) * kStage);
      keys_in = at;
      s[0] = rb.template scores<0>();
      if constexpr (NS == 2) s[1] = rb.template scores<kBlock>();
    }
  };
  auto soften = [&](int t, auto tail) __attribute__((always_inline)) {
    if (idle) return;
    const uint64_t at = *reinterpret_cast<const uint64_t*>(s_valid[t & 7]);
    const uint64_t all = ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(at >> 32)) << 32) |
                         (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)at);
    bool uneven = false;
#pragma unroll
    for (int b = 0; b < NS; ++b) {
      const uint32_t valid = (uint32_t)(all >> (32 * (part + b)));
      seen[b] = valid;
      if constexpr (decltype(tail)::value) {
        seen[b] &= rb.sees(p, w, w.k0 + t * KT + (part + b) * kBlock);
        uneven |= __any(seen[b] != valid);
        if (__any(seen[b] != ~0u)) rb.mask_scores(s[b], seen[b]);
      } else if (valid != ~0u) {
        rb.mask_scores(s[b], valid);
      }
    }
    rb.weigh(s, c);
#pragma unroll
    for (int b = 0; b < NS; ++b) weights[b] = rb.pack(s[b]);
    if constexpr (decltype(tail)::value)
      odd = uneven && rb.any_odd(s_kv[t % kRing] + kTile + part * kBlock * R::kBytes, NS * kBlock);
  };
  auto step = [&](int t, auto tail) __attribute__((always_inline)) {
    const bool more = t + 2 < nt, ask = more && (t & 3) == 3;
    if (ask) fetch_ids((t >> 2) + 2);
    __builtin_amdgcn_s_setprio(1);
    multiply(t, t > 0, true, tail);
    __builtin_amdgcn_s_setprio(0);
    // this wave's part of stage t + 1, and what was asked for before this step
    if (ask) wait_loads<1>();
    else wait_loads<0>();
    lds_barrier();
    if (more) load_stage(t + 2);
    soften(t, tail);
    if (more && (t & 3) == 1) find_rows((t >> 2) + 1, ahead);
    lds_barrier();
  };

  if (nt > 0) {
    fetch_ids(0);
    const PageAt first = ahead;
    fetch_ids(1);
    wait_loads<0>();
    find_rows(0, first);
    load_stage(0);
    load_stage(1);
    wait_loads<2 * NL>();  // all but stage 1
    rb.place((uint32_t)(uintptr_t)s_kv[0] + part * kBlock * R::kBytes,
             (uint32_t)(uintptr_t)s_kv[0] + kTile + part * kBlock * R::kBytes);
    lds_barrier();
    if (late) lds_barrier();
    int t = 0;
    for (; t < nf; ++t) step(t, No{});
    for (; t < nt; ++t) step(t, Yes{});
    multiply(nt, true, false, Yes{});
    if (!late) lds_barrier();
  }

  constexpr int kOut = (R::kDB * 4 + 1) * 1024;  // a block's outputs, maxima and sums in LDS
  static_assert((KG == 1 ? 8 * kStoreBytes<DP> : 4 * kOut) <= kRing * kStage && kStoreBytes<DP> <= kOut, "");
  float l = half_sum(rb.l);
  if constexpr (KG == 2) {
    // the second group's outputs pass through LDS; nothing is in flight any more
    __syncthreads();
    f32x4* red = reinterpret_cast<f32x4*>(&s_kv[0][0] + block * kOut);
    if (late) {
#pragma unroll
      for (int db = 0; db < R::kDB; ++db)
#pragma unroll
        for (int qd = 0; qd < 4; ++qd)
          red[(db * 4 + qd) * 64 + lane] =
              f32x4{rb.o[db][4 * qd], rb.o[db][4 * qd + 1], rb.o[db][4 * qd + 2], rb.o[db][4 * qd + 3]};
      red[R::kDB * 4 * 64 + lane] = f32x4{rb.m, l, 0.f, 0.f};
    }
    __syncthreads();
    if (late) return;
    const f32x4 ml = red[R::kDB * 4 * 64 + lane];
    const float M = fmaxf(rb.m, ml[0]), ms = M == -INFINITY ? 0.f : M;
    const float f = __builtin_amdgcn_exp2f(rb.m - ms), g = __builtin_amdgcn_exp2f(ml[0] - ms);
    l = l * f + ml[1] * g;
    rb.m = M;
#pragma unroll
    for (int db = 0; db < R::kDB; ++db)
#pragma unroll
      for (int qd = 0; qd < 4; ++qd) {
        const f32x4 x = red[(db * 4 + qd) * 64 + lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) rb.o[db][4 * qd + e] = rb.o[db][4 * qd + e] * f + x[e] * g;
      }
  }
  // (each wave's LDS lies where it read the other group's outputs, or where no one
  // reads any more)
  if constexpr (KG == 1) __syncthreads();
  store_rows(p, w, rb, l, w.row0 + block * kBlock, &s_kv[0][0] + block * (KG == 1 ? kStoreBytes<DP> : kOut));
}

// Join a row's chunks, in their order: one wave a row, 4 elements a lane, the
// lanes left over by a short head taking every second (fourth, ..) chunk.
template <typename Elem>
__global__ __launch_bounds__(kThreads) void attend_join_kernel(AttendParams p) {
  warm_args(p);
  // grid: (rows of the longest sequence * heads / 4, sequences)
  const int b = blockIdx.y;
  int64_t start;
  int n, ctx;
  sequence_of(p, b, start, n, ctx);
  const int r = (int)blockIdx.x * (kThreads / 64) + (int)(threadIdx.x >> 6);
  const int i = r / p.hq, h = r - i * p.hq;
  const int splits = splits_of(p, n, ctx);
  if (i >= n || splits == 1) return;  // one chunk: its workgroup wrote the output
  const int64_t row = start + i, of = part_row(p, b, start, i);
  const int lane = threadIdx.x & 63;
  int lanes = 1;  // lanes of one chunk: a power of two
  while (lanes * 4 < p.d) lanes *= 2;
  const int at = 4 * (lane % lanes);
  const bool ok = at < p.d;
  float M = -INFINITY;
  for (int s = lane; s < splits; s += 64) M = fmaxf(M, part_ml(p, s, of, h)[0]);
#pragma unroll
  for (int o = 32; o; o >>= 1) M = fmaxf(M, __shfl_xor(M, o));
  const float ms = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  f32x4 sum = f32x4{0.f, 0.f, 0.f, 0.f};
  // four chunks' loads at a time: one by one, each waited for the one before it
  // (13.3 -> 8.1 us for 2048 rows of 31 chunks, 33 MB)
  constexpr int kAhead = 4;
  const int step = 64 / lanes;
  for (int s = lane / lanes; s < splits; s += kAhead * step) {
    float m[kAhead], l[kAhead];
    f32x4 x[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const bool there = s + i * step < splits;
      const int si = there ? s + i * step : s;
      const float* ml = part_ml(p, si, of, h);
      m[i] = ml[0];
      l[i] = there ? ml[1] : 0.f;
      x[i] = ldf4_or0(part_o(p, si, of, h) + at, ok);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const bool any = l[i] != 0.f;  // the chunk has keys that the row sees
      const float f = any ? __builtin_amdgcn_exp2f(m[i] - ms) : 0.f;
      L = __builtin_fmaf(l[i], f, L);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] = __builtin_fmaf(any ? x[i][e] : 0.f, f, sum[e]);
    }
  }
  for (int o = lanes; o < 64; o <<= 1) {
    L += __shfl_xor(L, o);
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] += __shfl_xor(sum[e], o);
  }
  const float inv = inverse(L);
#pragma unroll
  for (int e = 0; e < 4; ++e) sum[e] *= inv;
  if (lane < lanes && ok) RowBlock<Elem, 64>::store4(p, row, h, at, sum);
  if (p.lse && lane == 0) p.lse[row * p.hq + h] = (M + __builtin_amdgcn_logf(L)) * kLn2;
}

// ---- host ------------------------------------------------------------------

// Which kernel takes a call, by the rows of a (sequence, key/value head) and the
// bytes of a padded head: up to 32 rows the narrow one, else the one whose waves
// take turns where its rows fit its registers, or the wide one.
enum class Kind { kNarrow, kTurns128, kTurns256, kWide };
struct AttendPlan {
  Kind kind;
  int32_t chunk, splits, row_tiles;
  int32_t block;   // threads of a workgroup
  int64_t groups;  // workgroups to be had from cutting the keys
  int64_t grid;
};
constexpr int narrow_waves(int row_bytes) { return row_bytes <= 512 ? 4 : 2; }
AttendPlan attend_kind(int elem, int32_t nodes, int32_t group, int32_t d) {
  AttendPlan a{};
  const int64_t rows = (int64_t)nodes * group;
  const int row_bytes = elem * (d <= 64 ? 64 : d <= 128 ? 128 : 256);
  int64_t tile = kBlock;
  a.groups = 1024;
  a.kind = Kind::kNarrow;
  a.block = 64 * narrow_waves(row_bytes);
  if (rows > kBlock) {
    a.kind = row_bytes > 256 ? Kind::kWide : rows > 4 * kBlock ? Kind::kTurns256 : Kind::kTurns128;
    tile = a.kind == Kind::kTurns256 ? 8 * kBlock : 4 * kBlock;
    a.groups = a.kind == Kind::kWide ? 512 : 256;
    a.block = a.kind == Kind::kWide ? kThreads : 512;
  }
  a.row_tiles = (int32_t)ceil_div(rows, tile);
  return a;
}

// How the keys are cut: even chunks, so long that about `groups` workgroups run
// in all where every sequence is as long as its bound, and no shorter than
// kMinChunk keys.  One workgroup a compute unit of the kernel with turns, whose
// prologue, parts and join cost some 24 us (one sequence of 32768 keys and 64 nodes:
// 65 us, with two 84); two of the wide one; four of the narrow one (64 sequences of
// 4096 keys, 32 + 8 bf16 heads of 128: 176 us, with eight 188; one of 32768: 43, with
// eight 54).
constexpr int64_t kMinChunk = 256;
constexpr int64_t kMaxChunk = (int64_t)1 << 30;

AttendPlan attend_plan(int elem, int32_t B, int32_t max_nodes, int32_t max_context, int32_t hq, int32_t hk,
                       int32_t d) {
  AttendPlan a = attend_kind(elem, max_nodes, hq / hk, d);
  const int64_t keys = (int64_t)max_context + max_nodes;
  const int64_t units = (int64_t)B * hk * a.row_tiles;
  int64_t chunk = units < a.groups ? ceil_div(keys * units, a.groups) : keys;
  if (chunk < kMinChunk) chunk = kMinChunk;
  // even chunks of whole stages (128 keys are one block of each narrow wave)
  const int64_t unit = a.kind == Kind::kNarrow ? 4 * kBlock : 2 * kBlock;
  chunk = ceil_div(ceil_div(keys, ceil_div(keys, chunk)), unit) * unit;
  if (chunk > kMaxChunk) chunk = kMaxChunk;
  a.chunk = (int32_t)chunk;
  a.splits = (int32_t)ceil_div(keys, chunk);
  a.grid = ceil_div((int64_t)B * hk * a.splits, kXcds) * kXcds * a.row_tiles;
  return a;
}

int64_t join_grid(int32_t max_nodes, int32_t hq) { return ceil_div((int64_t)max_nodes * hq, kThreads / 64); }

int32_t part_rows_of(int32_t B, int32_t T, int32_t max_nodes) {
  return (int32_t)std::min<int64_t>(T, (int64_t)B * max_nodes);
}
int64_t part_bytes(int64_t rows, int32_t hq, int32_t d) { return (rows * hq * (d + 2) * 4 + 255) & ~int64_t(255); }

template <typename Elem, int DP>
hipError_t launch_d(const AttendParams& p, const AttendPlan& a, hipStream_t stream) {
  constexpr int kRow = DP * (int)sizeof(Elem);
  const dim3 g((unsigned)a.grid), b((unsigned)a.block);
  if (a.kind == Kind::kNarrow) {
    hipLaunchKernelGGL((attend_narrow_kernel<Elem, DP, narrow_waves(kRow)>), g, b, 0, stream, p);
  } else if constexpr (kRow > 256) {
    hipLaunchKernelGGL((attend_wide_kernel<Elem, DP>), g, b, 0, stream, p);
  } else if (a.kind == Kind::kTurns256) {
    hipLaunchKernelGGL((attend_turns_kernel<Elem, DP, 1>), g, b, 0, stream, p);
  } else {
    hipLaunchKernelGGL((attend_turns_kernel<Elem, DP, 2>), g, b, 0, stream, p);
  }
  return hipGetLastError();
}

template <typename Elem>
hipError_t launch(AttendParams p, hipStream_t stream) {
  const AttendPlan a = attend_plan(sizeof(Elem), p.B, p.max_nodes, p.max_context, p.hq, p.hk, p.d);
  p.chunk = a.chunk;
  p.splits = a.splits;
  p.row_tiles = a.row_tiles;
  p.part_rows = part_rows_of(p.B, p.T, p.max_nodes);
  p.by_tiles = fast_div((uint32_t)a.row_tiles);
  p.by_splits = fast_div((uint32_t)a.splits);
  p.by_sequences = fast_div((uint32_t)p.B);
  p.by_heads = fast_div((uint32_t)p.hk);
  p.by_chunk = fast_div((uint32_t)a.chunk);
  hipError_t e = p.d <= 64    ? launch_d<Elem, 64>(p, a, stream)
                 : p.d <= 128 ? launch_d<Elem, 128>(p, a, stream)
                              : launch_d<Elem, 256>(p, a, stream);
  if (e != hipSuccess || p.splits == 1) return e;
  hipLaunchKernelGGL(attend_join_kernel<Elem>, dim3((unsigned)join_grid(p.max_nodes, p.hq), (unsigned)p.B),
                     dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

bool attend_fits(lora_dtype dt, int32_t B, int32_t max_nodes, int32_t max_context, int32_t hq, int32_t hk, int32_t d) {
  const AttendPlan a = attend_plan(dt == LORA_F32 ? 4 : 2, B, max_nodes, max_context, hq, hk, d);
  const int64_t most = ((int64_t)1 << 32) - 1;  // threads in a dimension of a grid
  return a.grid <= most / a.block && (a.splits == 1 || join_grid(max_nodes, hq) <= most / kThreads);
}

int64_t attend_need_bytes(lora_dtype dt, int32_t B, int32_t T, int32_t max_nodes, int32_t max_context, int32_t hq,
                          int32_t hk, int32_t d) {
  const int64_t splits = attend_plan(dt == LORA_F32 ? 4 : 2, B, max_nodes, max_context, hq, hk, d).splits;
  return splits == 1 ? 0 : part_bytes(splits * part_rows_of(B, T, max_nodes), hq, d);
}

// Fewer sequences or nodes are cut into more chunks, so the bytes of a call do not
// grow with its sizes; these are the most of any call up to them.  With G workgroups
// to be had and u = sequences * kv_heads * row tiles a call has at most ceil(keys /
// kMinChunk) and ceil(G / u) chunks (2^30 keys at most a chunk), both largest at the
// most keys; rows only grow.  What is left is to try the numbers of sequences and,
// of the nodes, those that fill their row tiles.
int64_t attend_most_bytes(int32_t B, int32_t T, int32_t max_nodes, int32_t max_context, int32_t hq, int32_t hk,
                          int32_t d) {
  const int32_t group = hq / hk;
  const int64_t keys = (int64_t)max_context + max_nodes, by_keys = ceil_div(keys, kMinChunk);
  const int64_t uncut = ceil_div(keys, kMaxChunk);
  int64_t most = uncut > 1 ? uncut * part_rows_of(B, T, max_nodes) : 0;
  const auto nodes_up_to = [&](int elem, int64_t nodes) {
    if (nodes < 1) return;
    nodes = std::min<int64_t>(nodes, max_nodes);
    const AttendPlan a = attend_kind(elem, (int32_t)nodes, group, d);
    const int64_t per = (int64_t)hk * a.row_tiles;
    for (int64_t b = 1; b <= B && b * per < a.groups; ++b) {
      const int64_t splits = std::max(std::min(by_keys, ceil_div(a.groups, b * per)), uncut);
      if (splits > 1) most = std::max(most, splits * part_rows_of((int32_t)b, T, (int32_t)nodes));
    }
  };
  for (int elem : {2, 4}) {
    nodes_up_to(elem, kBlock / group);
    for (int64_t tiles = 1; tiles * hk < 512; ++tiles) {
      nodes_up_to(elem, tiles * 4 * kBlock / group);
      nodes_up_to(elem, tiles * 8 * kBlock / group);
      if (tiles * 4 * kBlock / group >= max_nodes) break;
    }
    nodes_up_to(elem, max_nodes);
  }
  return part_bytes(most, hq, d);
}

hipError_t launch_attend(lora_dtype dt, const AttendParams& p, hipStream_t stream) {
  switch (dt) {
    case LORA_F32: return launch<float>(p, stream);
    case LORA_F16: return launch<half_t>(p, stream);
    case LORA_BF16: return launch<bf16_t>(p, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace lora
