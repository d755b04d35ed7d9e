// What the attention kernels share: the work of a workgroup, matrix blocks, a
// block of rows with its running softmax, global-to-LDS loads, parts and their
// join.  Included once by each source with attention kernels.
#pragma once

#include "attention.h"

namespace lora {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) const u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) const float lds_float;
typedef __attribute__((address_space(3))) const f32x4 lds_f32x4;
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
// Where a kernel that finds its chunks' length leaves it: kChunkBytes before the parts.
constexpr int64_t kChunkBytes = 256;
__device__ inline int* chunk_of_parts(const AttendParams& p) { return reinterpret_cast<int*>(p.part) - kChunkBytes / 4; }
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
// output, held by one wave.  Elem: what the tiles in LDS hold.  Out: the type of q
// and out where it is another one; q and the weights then enter the products as NT
// numbers of type Elem that add up to them.
template <typename Elem, int DP, typename Out = Elem, int NT = 1> struct RowBlock {
  using R = Rows<Elem, DP>;
  u32x4 q[NT][R::kSteps];
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

  // PAIRS: q's pieces of 8 elements in the order in which a lane half takes pieces
  // of 16 of the keys.
  template <bool PAIRS = false> __device__ __forceinline__ void init(const AttendParams& p, const Work& w, int row_first) {
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
    const Out* qr = static_cast<const Out*>(p.q) + (ok ? row : 0) * p.ldq + (int64_t)head * p.d;
    constexpr int kVec = Traits<Elem>::kVec;
    // the softmax takes a positive factor: a negative scale turns q's signs
    // instead, and a scale of 0 is a q of zeros
    if constexpr (sizeof(Out) == sizeof(Elem) && NT == 1) {
      const uint32_t flip = p.scale < 0.f ? (R::k16 ? 0x80008000u : 0x80000000u) : 0u;
#pragma unroll
      for (int s = 0; s < R::kSteps; ++s) {
        const int c = PAIRS ? 32 * (s / 2) + 16 * hi + 8 * (s % 2) : (2 * s + hi) * kVec;
        q[0][s] = ld16_or0(qr + c, ok && c < p.d && p.scale != 0.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) q[0][s][e] ^= flip;
      }
    } else {
      const float sign = p.scale < 0.f ? -1.f : 1.f;
#pragma unroll
      for (int s = 0; s < R::kSteps; ++s) {
        const int c = PAIRS ? 32 * (s / 2) + 16 * hi + 8 * (s % 2) : (2 * s + hi) * kVec;
        const bool there = ok && c < p.d && p.scale != 0.f;
        float x[kVec];
#pragma unroll
        for (int i = 0; i < kVec; i += Traits<Out>::kVec) Traits<Out>::to_float(ld16_or0(qr + c + i, there), x + i);
#pragma unroll
        for (int i = 0; i < kVec; ++i) x[i] *= sign;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t terms[NT];
          split(x[2 * e], x[2 * e + 1], terms);
#pragma unroll
          for (int n = 0; n < NT; ++n) q[n][s][e] = terms[n];
        }
      }
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
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int st = 0; st < kAhead; ++st) s = Mma32<Elem>::mma(a[st], q[n][s0 + st], s);
    }
    return s;
  }

  // Running softmax over NS blocks of scores (-inf where masked): scores become
  // weights.  c > 0 turns scores into powers of two.  m is moved only where a weight
  // would pass 2^kMost, and then below the score by kBelow: most tiles leave the
  // output as it is, and sums and weights stay clear of overflow.  RAISED: m stays
  // `above` these scores, so that the weights are at most 2^(kMost - above).
  template <bool RAISED = false, int NS>
  __device__ __forceinline__ void weigh(f32x16 (&s)[NS], float c, float above = 0.f) {
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
    if constexpr (RAISED) mx += above;
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

  // The same where keys and values lie in the tiles without their powers of two: key
  // i's score is s a[i], its value's factor 2^b[i].  The factor is part of the
  // weight, 2^(s a + b - m), so m follows what weights and values are together
  // and small factors cost a weight no bits; l sums the weights without it, times
  // c[i] = 2^-b[i].  a, b and c: LDS addresses of the 32 NS keys' numbers; seen:
  // which keys the row sees.
  template <int NS>
  __device__ __forceinline__ void weigh_scaled(f32x16 (&s)[NS], const uint32_t (&seen)[NS], uint32_t a, uint32_t b, uint32_t c) {
    constexpr float kBelow = Mma32<Elem>::kBelow, kMost = Mma32<Elem>::kMost;
    const auto four = [&](uint32_t at, int n, int g) {
      return *((lds_f32x4*)(lds_byte*)(uintptr_t)(at + 16 * hi) + (8 * n + 2 * g));
    };
#pragma unroll
    for (int n = 0; n < NS; ++n) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4 an = four(a, n, g), bn = four(b, n, g);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][4 * g + e] = __builtin_fmaf(s[n][4 * g + e], an[e], bn[e]);
      }
      if (__any(seen[n] != ~0u)) mask_scores(s[n], seen[n]);
    }
    float mx4[4] = {s[0][0], s[0][1], s[0][2], s[0][3]};
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
      for (int i = n ? 0 : 4; i < 16; ++i) mx4[i & 3] = fmaxf(mx4[i & 3], s[n][i]);
    const float mx = half_max(fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])));
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
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4 cn = four(c, n, g);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float w = __builtin_amdgcn_exp2f(s[n][4 * g + e] - ms);
          s[n][4 * g + e] = w;
          sum[e] = __builtin_fmaf(w, cn[e], sum[e]);
        }
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
    u32x4 w[NT][R::k16 ? 2 : 4];
  };
  // Two numbers as NT pairs of 16-bit ones: the nearest, the nearest to what is
  // left, and so on (8 bits of a bf16 term each).
  __device__ __forceinline__ static void split(float a, float b, uint32_t (&terms)[NT]) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      terms[n] = Mma32<Elem>::pack2(a, b);
      if (n + 1 < NT) {
        a -= Traits<Elem>::elem_to_float(terms[n] & 0xffffu);
        b -= Traits<Elem>::elem_to_float(terms[n] >> 16);
      }
    }
  }
  __device__ __forceinline__ static Weights pack(const f32x16& s) {
    Weights r;
#pragma unroll
    for (int i = 0; i < (R::k16 ? 2 : 4); ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (R::k16) {
          uint32_t terms[NT];
          split(s[8 * i + 2 * e], s[8 * i + 2 * e + 1], terms);
#pragma unroll
          for (int n = 0; n < NT; ++n) r.w[n][i][e] = terms[n];
        } else {
          r.w[0][i][e] = __float_as_uint(s[4 * i + e]);
        }
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
#pragma unroll
          for (int n = 0; n < NT; ++n) o[db] = Mma32<Elem>::mma(v, p.w[n][u], o[db]);
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
        const uint32_t wi = p.w[0][i / 4][i % 4];
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
    Out* out = static_cast<Out*>(p.out) + row * p.ldo + (int64_t)head * p.d + at;
    if constexpr (sizeof(Out) == 2) {
      *reinterpret_cast<u32x2*>(out) =
          u32x2{Mma32<Out>::pack2(x[0], x[1]), Mma32<Out>::pack2(x[2], x[3])};
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
template <int DP, typename Block>
__device__ __forceinline__ void store_rows(const AttendParams& p, const Work& w, const Block& rb, float l, int row_first,
                                           char* lds) {
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

// Join a row's chunks, in their order: one wave a row, 4 elements a lane, the
// lanes left over by a short head taking every second (fourth, ..) chunk.
// FOUND: the chunks' length is the device's (chunk_of_parts).
template <typename Elem, bool FOUND = false>
__global__ __launch_bounds__(kThreads) void attend_join_kernel(AttendParams p) {
  warm_args(p);
  // grid: (rows of the longest sequence * heads / 4, sequences)
  const int b = blockIdx.y;
  int64_t start;
  int n, ctx;
  sequence_of(p, b, start, n, ctx);
  const int r = (int)blockIdx.x * (kThreads / 64) + (int)(threadIdx.x >> 6);
  const int i = r / p.hq, h = r - i * p.hq;
  const int splits = FOUND ? (int)(((uint32_t)max(ctx + n, 1) - 1) / (uint32_t)*chunk_of_parts(p)) + 1 : splits_of(p, n, ctx);
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

}  // namespace

}  // namespace lora
