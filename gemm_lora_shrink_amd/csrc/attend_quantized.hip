// Attention of a step's tokens over a quantized cache: the work, the row blocks
// and the join of the other attention kernels, with keys and values that lie in
// memory as bytes with an exponent for each block of rows.
//
// A byte's number is a bf16 number, and so is that number times a power of two,
// so keys and values enter the products exactly, as bf16 (on this chip one
// instruction makes two of them from two e4m3 bytes and a scale).  q and the
// softmax weights do too where they are bf16; fp16 ones enter as the sum of two
// bf16 numbers, fp32 ones of three, each of which has 8 bits of them.
#include <algorithm>

#include "attend_unit.h"
#include "cache.h"
#include "stage_order.h"

namespace lora {

namespace {

typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i32x2 lds_i32x2;
typedef __attribute__((address_space(3))) const int lds_int;
typedef __attribute__((address_space(1))) const int8_t global_int8;
typedef __attribute__((address_space(1))) const int32_t global_int;

// Two words (eight bytes) as eight bf16 numbers, times `scale`.
template <typename F> __device__ __forceinline__ u32x4 to_bf16(uint32_t w0, uint32_t w1, float scale);
template <> __device__ __forceinline__ u32x4 to_bf16<E4m3>(uint32_t w0, uint32_t w1, float scale) {
  return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, scale, false)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, scale, true)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, scale, false)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, scale, true))};
}
template <> __device__ __forceinline__ u32x4 to_bf16<Int8>(uint32_t w0, uint32_t w1, float scale) {
  float x[8];
  Int8::numbers(w0, x);
  Int8::numbers(w1, x + 4);
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = pack2_bf16(x[2 * i] * scale, x[2 * i + 1] * scale);
  return r;
}
// Eight bytes' numbers as fp16 ones.
template <typename F> __device__ __forceinline__ u32x4 to_f16(uint32_t w0, uint32_t w1) {
  float x[8];
  F::numbers(w0, x);
  F::numbers(w1, x + 4);
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = pack2_f16(x[2 * i], x[2 * i + 1]);
  return r;
}
// Bit 7 of each byte that is a NaN.
template <typename F> __device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return F::kHasNan ? ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u : 0u;
}

// How many bf16 numbers a number of the call's type enters as.
template <typename Out> constexpr int kTerms = sizeof(Out) == 4 ? 3 : Traits<Out>::kDtype == LORA_F16 ? 2 : 1;
// The kernels of many rows, which the matrix cores bound, have fp16 tiles for an fp16
// q, which then enters as it is, and so do its weights.
template <typename Out> struct Tiles {
  using Elem = bf16_t;
  static constexpr int NT = kTerms<Out>;
};
template <> struct Tiles<half_t> {
  using Elem = half_t;
  static constexpr int NT = 1;
};

// A product of a weight (up to 2^8), a byte's number (below 2^9) and a power of two
// of up to 2^kRoom stays finite in sums of 2^31 of them.  Where a value has a larger
// one (up to 2^121), m is kept kRaise above the scores of its tile, and the weights so
// much lower.  Finding how far each tile needs cost a branch a tile: 66.2 us for
// 65.0 on 64 nodes over 32768 keys.
constexpr int kRoom = 72;
constexpr float kRaise = 49.f;

// A byte to a dword of LDS for each lane.
__device__ inline void byte_to_lds(const char* g, uint32_t lds) {
  lds = __builtin_amdgcn_readfirstlane(lds);
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %1\n\t"
      "s_nop 0\n\t"
      "global_load_lds_ubyte %2, off\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "s"(lds), "v"(g)
      : "memory");
}

// The address of a key's exponent; strides below 2^32 (the host checks).
struct ExpAt {
  uint64_t base;
  uint32_t page;
  __device__ __forceinline__ uint64_t at(uint32_t id, uint32_t block) const { return base + (uint64_t)id * page + block; }
};
__device__ inline ExpAt exp_at(const AttendQuantizedParams& p, int h, bool is_v) {
  return ExpAt{reinterpret_cast<uint64_t>(is_v ? p.v_exp : p.k_exp) + (uint64_t)h * (uint64_t)(is_v ? p.v_exp_head : p.k_exp_head),
               (uint32_t)(is_v ? p.v_exp_page : p.k_exp_page)};
}

// ---- up to 32 rows ----------------------------------------------------------

// A tile of a wave: 4 KB of keys and 4 KB of values (rows of 256 bytes: 8 and 8, as a
// matrix block has 32 keys), rows of DP bytes in pieces of 16, piece c of row r at
// c ^ swz(r): 16 consecutive rows at one piece (the keys'
// reads) and rows 4 i .. 4 i + 3 and 4 i + 8 .. 4 i + 11 at two neighbouring
// pieces (the values' transposing reads) lie in different banks.
template <int DP> struct Tile8 {
  static constexpr int kBytes = DP == 256 ? 8192 : 4096;
  static constexpr int kKeys = kBytes / DP, kBlocks = kKeys / kBlock;
  static constexpr int kPieces = DP / 16;
  static constexpr int kPerLoad = 1024 / DP;  // rows of one 64-lane load
  static constexpr int NL = kBytes / 1024;    // loads of the keys or values
  static constexpr int kGroups = DP == 256 ? 1 : 2;  // workgroups of a compute unit
  static constexpr int NI = (kKeys + 63) / 64;    // loads of page numbers
  static constexpr int NE = kKeys / 32;           // loads of exponents, keys and values
  __device__ static inline int swz(int r) {
    if (DP == 64) return (r >> 2) & 3;
    if (DP == 128) return (((r >> 3) & 1) << 2) | (((r >> 1) & 1) << 1) | ((r >> 2) & 1);
    return (((r >> 3) & 1) << 3) | (((r >> 1) & 1) << 2) | ((r & 1) << 1) | ((r >> 2) & 1);
  }
};

// ---- the work of a workgroup ---------------------------------------------------

// A unit is one (sequence, key/value head, tile of ROWS rows).  Where there are fewer
// units than workgroups at once (p.cuts of them), the keys are cut by the lengths that
// the sequences have, which the host does not know: into chunks of the least number
// of stages (KEYS keys) with which all chunks of all units run at once, and of which
// no sequence has more than p.splits.  Lane b of every wave counts for sequence b; a
// scan over the lanes finds a workgroup's own chunk, and workgroup 0 leaves the
// chunks' length for the join.  Against even chunks of the bounds: 195 -> 142 us for
// 16 sequences of 256 to 8192 keys and 23 to 45 nodes (fp16, INT8), 42 -> 37 for one
// node each, 55.5 -> 32 for 64 nodes over 4096 keys under a bound of 32768; where
// lengths reach the bounds finding the chunk costs 63.7 -> 64.8 (64 nodes over 32768
// keys) and 26.2 -> 27.3 (one node).
// With more units than that, cutting the long ones loses (143 -> 166 us for 32
// sequences of 128 to 4096 keys, 256 units): work_of's even chunks, most often one.
constexpr int64_t kMinChunk = 256;
constexpr int kCutSeqs = 64;  // sequences that this is done for: a lane each
// Over a wave's lanes, by shifts and broadcasts of the vector unit: the sums of the
// lanes up to each, the sum, the largest.
#define LORA_WAVE_STEPS(OP)                                                 \
  OP(0x111, 0xf) OP(0x112, 0xf) OP(0x114, 0xf) OP(0x118, 0xf) /* row_shr */ \
      OP(0x142, 0xa) OP(0x143, 0xc)                           /* row_bcast */
__device__ __forceinline__ int wave_scan(int x) {
#define LORA_ADD(dpp, rows) x += __builtin_amdgcn_update_dpp(0, x, dpp, rows, 0xf, false);
  LORA_WAVE_STEPS(LORA_ADD)
#undef LORA_ADD
  return x;
}
__device__ __forceinline__ uint32_t wave_sum(int x) { return (uint32_t)__builtin_amdgcn_readlane(wave_scan(x), 63); }
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
#define LORA_MAX(dpp, rows) x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, dpp, rows, 0xf, false));
  LORA_WAVE_STEPS(LORA_MAX)
#undef LORA_MAX
  return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}
#undef LORA_WAVE_STEPS
__device__ __forceinline__ uint32_t up(uint32_t a, uint32_t b) { return (a + b - 1) / b; }
template <int ROWS, int KEYS> __device__ __forceinline__ Work work_by_lengths(const AttendQuantizedParams& p) {
  Work w;
  const int lane = threadIdx.x & 63;
  int64_t start = 0;
  int n = 0, ctx = 0;
  if (lane < p.B) sequence_of(p, lane, start, n, ctx);
  const int tiles = (int)(((uint32_t)n * p.group.d + ROWS - 1) / ROWS), per = tiles * p.hk;
  const uint32_t stages = ((uint32_t)ctx + (uint32_t)n + KEYS - 1) / KEYS;
  // ceil(x / c) lies between x / c and x / c + 1, so the sum of all chunks tells where
  // to look: in one place where the units are few
  const uint32_t longest = wave_max(per ? stages : 0), all = wave_sum(per * stages), units = wave_sum(per);
  uint32_t lo = max((uint32_t)(kMinChunk + KEYS - 1) / KEYS, max(up(longest, p.splits), up(all, p.cuts)));
  uint32_t hi = max(lo, min(longest, up(all, p.cuts - units)));
  while (lo < hi) {
    const uint32_t mid = (lo + hi) / 2;
    if (wave_sum(per * up(stages, mid)) <= (uint32_t)p.cuts) hi = mid;
    else lo = mid + 1;
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  if (p.splits > 1 && blockIdx.x == 0 && threadIdx.x == 0) *chunk_of_parts(p) = lo * KEYS;
  const int splits = max(1u, up(stages, lo)), mine = per * splits, ends = wave_scan(mine);
  // neighbouring chunks on one XCD: they read the same pages
  const int total = __builtin_amdgcn_readlane(ends, 63), of_xcd = (total + kXcds - 1) / kXcds;
  const int j = (int)(blockIdx.x / kXcds), rank = (int)(blockIdx.x % kXcds) * of_xcd + j;
  w.none = j >= of_xcd || rank >= total;
  if (w.none) return w;
  w.b = __builtin_ctzll(__ballot(ends > rank));
  const auto of_b = [&](int x) { return __builtin_amdgcn_readlane(x, w.b); };
  const uint32_t r = rank - of_b(ends - mine), nt = of_b(tiles), ns = of_b(splits);
  w.start = (int64_t)(((uint64_t)(uint32_t)of_b((int)(start >> 32)) << 32) | (uint32_t)of_b((int)start));
  w.n = of_b(n);
  w.ctx = of_b(ctx);
  const uint32_t u = __builtin_amdgcn_readfirstlane(r / nt);
  w.h = __builtin_amdgcn_readfirstlane(u / ns);
  w.split = (int)(u - w.h * ns);
  w.row0 = (int)(r - u * nt) * ROWS;
  w.rows = w.n * (int)p.group.d;
  w.whole = ns == 1;
  const int last = min(w.row0 + ROWS, w.rows) - 1;
  const int end = w.ctx + (p.mask ? w.n : min(w.n, (int)p.group.div((uint32_t)last) + 1));
  const int64_t k0 = (int64_t)w.split * lo * KEYS;
  w.k0 = (int)k0;
  w.k1 = (int)min(k0 + (int64_t)lo * KEYS, (int64_t)end);
  return w;
}
template <int ROWS, bool SPREAD, int KEYS> __device__ __forceinline__ Work quantized_work(const AttendQuantizedParams& p) {
  return p.cuts ? work_by_lengths<ROWS, KEYS>(p) : work_of<ROWS, SPREAD>(p);
}

// Up to 32 rows: four waves hold the same rows and take the chunk's tiles in turn,
// each through LDS of its own: a wave waits for no other until their outputs meet
// at the end.  Two tiles are in flight a wave (16 KB): after a tile's scores the keys
// of the tile after the next take its keys' place, after its products with the
// values their values.  Page numbers come four tiles ahead.  Loads past the chunk's
// end go to a row of zeros, so that the number of loads in flight is the same in
// every turn.
// Bound by memory: 256 sequences of 128 to 4096 keys, 32 + 8 bf16 heads of 128, e4m3
// (1.1 GB): 197 us, 5.5 TB/s; 64 sequences of 4096 (0.54 GB): 92 us, 5.9 TB/s.  Two
// workgroups a compute unit, one of which is at its first loads while the other
// reads (260 us on the first with one of twice the tiles, 300 with one of these).
// e4m3 has two forms of the products with the values, of which a tile takes one.  With
// heads of 128 and an fp16 or fp32 query, and with heads of 256, 30 to 190 registers
// then lie in memory; INT8 has one form, and none but with fp32 (4 and 62).
template <typename Out, typename F, int DP>
__global__ __launch_bounds__(256, Tile8<DP>::kGroups) void attend_narrow_quantized_kernel(AttendQuantizedParams p) {
  using L8 = Tile8<DP>;
  constexpr int NT = kTerms<Out>, NW = 4, KT = L8::kKeys, NB = L8::kBlocks, NL = L8::NL, NI = L8::NI, NE = L8::NE;
  using Block = RowBlock<bf16_t, DP, Out, NT>;
  constexpr int kDB = DP / kBlock;
  // Whether the keys' powers of two are taken to the scores: the conversion of a byte
  // takes one for e4m3, for int8 it costs a product an element (226 us for 213 on 256
  // sequences of 128 to 4096 keys).
  constexpr bool kScores = !F::kHasNan;
  __shared__ __attribute__((aligned(1024))) char s_kv[NW][2][2][L8::kBytes];
  __shared__ __attribute__((aligned(16))) const char* s_row[NW][2 * KT];
  __shared__ __attribute__((aligned(16))) int s_exp[NW][2][2 * KT < 64 ? 64 : 2 * KT];
  __shared__ int s_id[NW][4][NI * 64];
  __shared__ float s_ml[NW][2][kBlock];
  warm_args(p);
  const Work w = quantized_work<kBlock, true, 4 * Tile8<DP>::kKeys>(p);
  if (w.none) return;
  Block rb;
  rb.template init<true>(p, w, w.row0);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = rb.lane, r32 = rb.r32, hi = rb.hi;
  const float c = p.scale == 0.f ? 1.0f : fabsf(p.scale) * kLog2e;
  // this wave's tiles, the first nf of them wholly inside the context
  const auto tiles = [&](int keys, bool whole) {
    const int all = keys <= 0 ? 0 : whole ? keys / KT : (keys + KT - 1) / KT;
    return all > wave ? (all - wave + NW - 1) / NW : 0;
  };
  const int nt = tiles(w.k1 - w.k0, false), nf = tiles(min(w.ctx, w.k1) - w.k0, true);
  const auto first_key = [&](int t) { return (int64_t)w.k0 + ((int64_t)wave + (int64_t)NW * t) * KT; };
  const HeadAt hk = head_at<uint8_t>(p, w.h, false), hv = head_at<uint8_t>(p, w.h, true);
  const ExpAt ek = exp_at(p, w.h, false), ev = exp_at(p, w.h, true);

  const auto fetch_ids = [&](int t) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      int col;
      const PageAt a = page_at(p, first_key(t) + 64 * i + lane % KT, w.k1, col);
      word_to_lds(entry_of(p, w.b, a, col), (uint32_t)(uintptr_t)&s_id[wave][t & 3][64 * i]);
    }
  };
  // The rows' addresses to LDS, the exponents on their way; returns which rows are keys.
  const char* exps[NE];
  struct Valid {
    uint32_t of[NB];
  };
  const auto find_rows = [&](int t) {
    Valid v;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      int col;
      const PageAt a = page_at(p, first_key(t) + 64 * i + lane % KT, w.k1, col);
      const uint32_t id = (uint32_t)s_id[wave][t & 3][64 * i + lane];
      const bool valid = a.in_table && id < (uint64_t)p.cache.n_pages && (int)id >= 0;
      const uint32_t block = p.block.div((uint32_t)a.place);
      const char* none = reinterpret_cast<const char*>(g_zero_row);
      const char* k = valid ? reinterpret_cast<const char*>(hk.row_at(id, a.place)) : none;
      const char* v_row = valid ? reinterpret_cast<const char*>(hv.row_at(id, a.place)) : none;
      const char* ke = valid ? reinterpret_cast<const char*>(ek.at(id, block)) : none;
      const char* ve = valid ? reinterpret_cast<const char*>(ev.at(id, block)) : none;
      if constexpr (KT >= 64) {
        s_row[wave][64 * i + lane] = k;
        s_row[wave][KT + 64 * i + lane] = v_row;
        exps[2 * i] = ke;
        exps[2 * i + 1] = ve;
      } else {
        s_row[wave][lane] = hi ? v_row : k;
        exps[0] = hi ? ve : ke;
      }
      const uint64_t all = __ballot(valid);
      v.of[(2 * i) % NB] = (uint32_t)all;
      if constexpr (NB > 1) v.of[2 * i + 1] = (uint32_t)(all >> 32);
    }
    return v;
  };
  const auto load = [&](int which, int t) __attribute__((always_inline)) {
    const uint32_t lds = (uint32_t)(uintptr_t)s_kv[wave][t & 1][which];
    const char* a[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int r = i * L8::kPerLoad + lane / L8::kPieces;
      const int piece = (lane % L8::kPieces) ^ L8::swz(r);
      const char* row = s_row[wave][which * KT + r];
      if (p.d != DP && piece * 16 >= p.d) row = reinterpret_cast<const char*>(g_zero_row);
      a[i] = row + 16 * piece;
    }
#pragma unroll
    for (int i = 0; i < NL; i += 2) two_rows_to_lds<true>(a[i], a[i + 1], lds + 1024 * i);
  };
  // s_exp: of the keys at [key], of the values at [KT + key]
  const auto load_exps = [&](int t) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NE; ++i)
      byte_to_lds(exps[i], (uint32_t)(uintptr_t)&s_exp[wave][t & 1][KT >= 64 ? (i % 2) * KT + (i / 2) * 64 : 0]);
  };

  Valid valid[2];  // of this tile and the next
  if (nt > 0) {
    fetch_ids(0);
    fetch_ids(1);
    wait_loads<0>();
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      valid[t] = find_rows(t);
      load(0, t);
      load_exps(t);
      fetch_ids(t + 2);
      load(1, t);
    }
  }
  const auto tile = [&](int t, auto tail) __attribute__((always_inline)) {
    constexpr bool kTail = decltype(tail)::value;
    // in flight, in order: K E (t), I (t + 2), V (t), K E (t + 1), I (t + 3), V (t + 1)
    wait_loads<3 * NL + NE + 2 * NI>();
    const uint32_t keys = (uint32_t)(uintptr_t)s_kv[wave][t & 1][0];
    const char* const values = s_kv[wave][t & 1][1];
    const uint32_t exp_lds = (uint32_t)(uintptr_t)s_exp[wave][t & 1];
    f32x16 s[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int key = 32 * b + r32;
      const float ks =
          kScores ? 1.0f : power_of_two(exponent_of<F>((int8_t)*(lds_int*)(lds_byte*)(uintptr_t)(exp_lds + 4 * key)));
      u32x4 raw[DP / 32];
#pragma unroll
      for (int j = 0; j < DP / 32; ++j)
        raw[j] = *(lds_u32x4*)(lds_byte*)(uintptr_t)(keys + key * DP + (((2 * j + hi) ^ L8::swz(key)) << 4));
#pragma unroll
      for (int i = 0; i < 16; ++i) s[b][i] = 0.f;
#pragma unroll
      for (int j = 0; j < DP / 32; ++j) {
        const uint32_t w0 = raw[j][0], w1 = raw[j][1], w2 = raw[j][2], w3 = raw[j][3];
        const u32x4 a0 = to_bf16<F>(w0, w1, ks), a1 = to_bf16<F>(w2, w3, ks);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          s[b] = Mma32<bf16_t>::mma(a0, rb.q[n][2 * j], s[b]);
          s[b] = Mma32<bf16_t>::mma(a1, rb.q[n][2 * j + 1], s[b]);
        }
      }
    }
    // the exponents (bf16 keys: the values') become factors
    bool over = false;  // a value's exponent is over kRoom
#pragma unroll
    for (int i = 0; i < (KT >= 64 ? 2 * KT / 64 : 1); ++i) {
      if (!kScores && KT >= 64 && i < KT / 64) continue;
      int* at = &s_exp[wave][t & 1][64 * i + lane];
      if (kScores || KT >= 64 || hi) {
        const int e = exponent_of<F>((int8_t)*at);
        if (KT >= 64 ? i >= KT / 64 : hi != 0) over = e > kRoom;
        *reinterpret_cast<float*>(at) = power_of_two(e);
      }
    }
    const float above = __any(over) ? kRaise : 0.f;
    const auto times = [&](f32x16& x, int first) __attribute__((always_inline)) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4 f = *(lds_f32x4*)(lds_byte*)(uintptr_t)(exp_lds + 4 * (first + 8 * g + 4 * hi));
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * g + e] *= f[e];
      }
    };
    if constexpr (kScores)
#pragma unroll
      for (int b = 0; b < NB; ++b) times(s[b], 32 * b);
    wait_lds();
    wait_loads<3 * NL + NE + NI>();  // page numbers of t + 2
    Valid now = valid[0];
    valid[0] = valid[1];
    valid[1] = find_rows(t + 2);
    load(0, t + 2);
    // exponents of t + 2 would take the place of the factors: they wait in registers for their turn

    uint32_t seen[NB];
    bool uneven = false;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      seen[b] = now.of[b];
      if constexpr (kTail) {
        seen[b] &= rb.sees(p, w, (int)(first_key(t) + 32 * b));
        uneven |= __any(seen[b] != now.of[b]);
      }
      if (__any(seen[b] != ~0u)) rb.mask_scores(s[b], seen[b]);
    }
    rb.template weigh<true>(s, c, above);
    typename Block::Weights weights[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      times(s[b], KT + 32 * b);
      weights[b] = rb.pack(s[b]);
    }
    wait_lds();
    load_exps(t + 2);
    wait_loads<3 * NL + 2 * NE + NI>();  // values of t
    bool odd = false;
    if constexpr (kTail && F::kHasNan) {
      if (uneven) {
        uint32_t any = 0;
        for (int i = lane; i < L8::kBytes / 4; i += 64) any |= nan_bytes<F>(reinterpret_cast<const uint32_t*>(values)[i]);
        odd = __any(any != 0);
      }
    }
    const auto add_values = [&](auto leave_out) __attribute__((always_inline)) {
      const int j = lane & 15, g1 = (lane >> 4) & 1, i = j >> 1;
      const int row = (i < 4 ? i : i + 4) + 4 * hi;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int key = 32 * b + 16 * u + row;
          i32x2 v[kDB];
#pragma unroll
          for (int db = 0; db < kDB; ++db)
            v[db] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                (lds_i32x2*)(lds_byte*)(uintptr_t)((uint32_t)(uintptr_t)values + key * DP +
                                                   (((2 * db + g1) ^ L8::swz(key)) << 4) + 8 * (j & 1)));
#pragma unroll
          for (int db = 0; db < kDB; ++db) {
            uint32_t w0 = (uint32_t)v[db][0], w1 = (uint32_t)v[db][1];
            if constexpr (decltype(leave_out)::value) {
              w0 &= ~((nan_bytes<F>(w0) >> 7) * 0xffu);
              w1 &= ~((nan_bytes<F>(w1) >> 7) * 0xffu);
            }
            const u32x4 a = to_bf16<F>(w0, w1, 1.0f);
#pragma unroll
            for (int n = 0; n < NT; ++n) rb.o[db] = Mma32<bf16_t>::mma(a, weights[b].w[n][u], rb.o[db]);
          }
        }
    };
    if (kTail && odd) {
      add_values(Yes{});
      // NaN reaches the rows that see its key; in the product it would have met a masked weight of 0
#pragma unroll 1
      for (int k = 0; k < KT; ++k) {
        uint32_t seen_k = 0;
#pragma unroll
        for (int b = 0; b < NB; ++b)
          if (k / 32 == b) seen_k = seen[b];
        const bool mine = (seen_k >> (k % 32)) & 1;
#pragma unroll
        for (int db = 0; db < kDB; ++db)
#pragma unroll
          for (int qd = 0; qd < 4; ++qd) {
            const int at = rb.element(db, qd);
            const uint32_t nan = nan_bytes<F>(
                *reinterpret_cast<const uint32_t*>(values + k * DP + (((at >> 4) ^ L8::swz(k)) << 4) + (at & 15)));
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (mine && (nan >> (8 * e + 7)) & 1) rb.o[db][4 * qd + e] = NAN;
          }
      }
    } else {
      add_values(No{});
    }
    wait_lds();
    fetch_ids(t + 4);
    load(1, t + 2);
  };
  int t = 0;
  for (; t < nf; ++t) tile(t, No{});
  for (; t < nt; ++t) tile(t, Yes{});
  wait_loads<0>();

  // the waves' outputs meet: weights to their common maximum, then block db of
  // the output is summed and stored by wave db % NW
  const float l = half_sum(rb.l);
  if (hi == 0) {
    s_ml[wave][0][r32] = rb.m;
    s_ml[wave][1][r32] = l;
  }
  f32x4* red = reinterpret_cast<f32x4*>(&s_kv[wave][0][0][0]);
#pragma unroll
  for (int db = 0; db < kDB; ++db)
#pragma unroll
    for (int qd = 0; qd < 4; ++qd)
      red[(db * 4 + qd) * 64 + lane] =
          f32x4{rb.o[db][4 * qd], rb.o[db][4 * qd + 1], rb.o[db][4 * qd + 2], rb.o[db][4 * qd + 3]};
  __syncthreads();
  float M = -INFINITY, L = 0.f, f[NW];
#pragma unroll
  for (int i = 0; i < NW; ++i) M = fmaxf(M, s_ml[i][0][r32]);
  const float ms = M == -INFINITY ? 0.f : M;
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    f[i] = __builtin_amdgcn_exp2f(s_ml[i][0][r32] - ms);
    L += s_ml[i][1][r32] * f[i];
  }
  if (rb.row < 0) return;
  const bool whole = w.whole;
  const float inv = whole ? inverse(L) : 1.0f;
  for (int db = wave; db < kDB; db += NW) {
#pragma unroll
    for (int qd = 0; qd < 4; ++qd) {
      const int at = rb.element(db, qd);
      if (at >= p.d) continue;
      f32x4 sum = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        const f32x4 x = reinterpret_cast<const f32x4*>(&s_kv[i][0][0][0])[(db * 4 + qd) * 64 + lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] = __builtin_fmaf(x[e], f[i], sum[e]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] *= inv;
      if (whole) rb.store4(p, rb.row, rb.head, at, sum);
      else *reinterpret_cast<f32x4*>(part_o(p, w.split, part_row(p, w.b, w.start, rb.node), rb.head) + at) = sum;
    }
  }
  if (wave == 0 && hi == 0) {
    if (!whole) {
      float* ml = part_ml(p, w.split, part_row(p, w.b, w.start, rb.node), rb.head);
      ml[0] = M;
      ml[1] = L;
    } else if (p.lse) {
      p.lse[rb.row * p.hq + rb.head] = (M + __builtin_amdgcn_logf(L)) * kLn2;
    }
  }
}

// ---- more rows --------------------------------------------------------------

// The bytes of stages of KT keys and values on their way from memory through
// registers to 16-bit tiles in LDS.  Each of the KT / 8 waves brings 8 rows of the
// keys and 8 of the values of a stage.  Where the rows and exponents of four stages
// lie is found together: lane 16 i + 8 v + r finds row r of the i-th stage, of the
// keys (v = 0) or the values, three calls apart: ask() requests page numbers, find()
// turns them into addresses and requests exponents, settle() makes factors of them.
// Both requests go to LDS, and each call says how many loads of the wave may be newer
// than the request it needs: held in registers they were waited for where the steps
// that make them meet those that do not, with every load in flight (216 us for 165,
// 16 sequences of 256 to 8192 keys and 23 to 45 nodes in chunks of 4096 keys).
// fp16 tiles hold the numbers without their powers of two, which have no room in
// fp16; a stage's `factors` are then, of row k, [k] the key's times c, [KT + k] the
// value's exponent, [2 KT + k] 2^-exponent.  bf16 tiles hold the values.
template <typename Elem, typename F, int DP, int KT> struct Staging {
  using R = Rows<Elem, DP>;
  static constexpr bool kFactors = Traits<Elem>::kDtype == LORA_F16;
  static constexpr int kWaves = KT / 8, kPieces = DP / 16;  // pieces: of a row of bytes
  static constexpr int NP = kPieces < 8 ? 1 : kPieces / 4;  // pieces of a lane: of K, then of V (DP = 64: of either)
  // in LDS
  struct Shared {
    const char* row[kWaves][64];
    int id[kWaves][64], exponent[kWaves][64];
    float scale[kWaves][2][kFactors ? 1 : 64];
    float factors[kFactorRing][kFactors ? 3 * KT : 1];
    // of a stage, of each wave's rows: which are keys, and whether an exponent of their
    // values is over kRoom (read together, as 32-bit words)
    struct About {
      uint8_t valid[kWaves], over[kFactors ? 0 : kWaves];
    };
    __attribute__((aligned(16))) About about[kValidRing];
  };
  static constexpr int kWords = kWaves / 4;
  Shared* sh;
  int wave, lane;
  int64_t k0;
  u32x4 data[NP];

  __device__ __forceinline__ void init(Shared& shared, const Work& w) {
    sh = &shared;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    lane = threadIdx.x & 63;
    k0 = w.k0;
  }
  __device__ __forceinline__ PageAt place(const AttendQuantizedParams& p, const Work& w, int four, int& col) const {
    return page_at(p, k0 + ((int64_t)four * 4 + (lane >> 4)) * KT + wave * 8 + (lane & 7), w.k1, col);
  }
  __device__ __forceinline__ void ask(const AttendQuantizedParams& p, const Work& w, int four) {
    int col;
    const PageAt a = place(p, w, four, col);
    word_to_lds(entry_of(p, w.b, a, col), (uint32_t)(uintptr_t)sh->id[wave]);
  }
  template <int NEWER> __device__ __forceinline__ void find(const AttendQuantizedParams& p, const Work& w, int four) {
    int col;
    const PageAt a = place(p, w, four, col);
    wait_loads<NEWER>();
    const int id = sh->id[wave][lane];
    const bool is_v = (lane >> 3) & 1;
    const HeadAt h = head_at<uint8_t>(p, w.h, is_v);
    const ExpAt e = exp_at(p, w.h, is_v);
    const bool ok = a.in_table && (uint32_t)id < (uint64_t)p.cache.n_pages && id >= 0;
    const char* none = reinterpret_cast<const char*>(g_zero_row);
    sh->row[wave][lane] = ok ? reinterpret_cast<const char*>(h.row_at((uint32_t)id, a.place)) : none;
    byte_to_lds(ok ? reinterpret_cast<const char*>(e.at((uint32_t)id, p.block.div((uint32_t)a.place))) : none,
                (uint32_t)(uintptr_t)sh->exponent[wave]);
    const uint64_t all = __ballot(ok);
    if ((lane & 15) == 0) sh->about[(four * 4 + (lane >> 4)) % kValidRing].valid[wave] = (uint8_t)(all >> lane);
  }
  template <int NEWER> __device__ __forceinline__ void settle(int four, float c) {
    wait_loads<NEWER>();
    const int e = exponent_of<F>((int8_t)sh->exponent[wave][lane]);
    if constexpr (kFactors) {
      float* f = sh->factors[(four * 4 + (lane >> 4)) % kFactorRing] + wave * 8 + (lane & 7);
      if ((lane >> 3) & 1) {
        // Smaller exponents than -60 are taken for it: what they stand for is far below
        // the smallest fp16 output either way, and the last factor stays finite in sums.
        const int ev = max(e, -60);
        f[KT] = (float)ev;
        f[2 * KT] = power_of_two(-ev);
      } else {
        f[0] = fminf(power_of_two(e) * c, 3.0e38f);  // (finite: a score may be 0)
      }
    } else {
      sh->scale[wave][four & 1][lane] = power_of_two(e);
      const uint64_t over = __ballot(e > kRoom) >> (lane & 48);  // (from bit 8 on: the values')
      if ((lane & 15) == 0) sh->about[(four * 4 + (lane >> 4)) % kValidRing].over[wave] = (uint8_t)(over >> 8);
    }
  }
  // Which rows of stage t are keys, and how far m is to stay above their scores.
  __device__ __forceinline__ float read_about(int t, uint32_t (&valid)[kWords]) const {
    const uint32_t* at = reinterpret_cast<const uint32_t*>(&sh->about[t % kValidRing]);
    uint32_t over = 0;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      valid[i] = at[i];
      if constexpr (!kFactors) over |= at[kWords + i];
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) valid[i] = __builtin_amdgcn_readfirstlane(valid[i]);
    return over ? kRaise : 0.f;
  }
  // Row and piece of the lane's i-th 16 bytes among the wave's 8 rows of K and 8 of V.
  struct Mine {
    int row, piece, is_v;
  };
  __device__ __forceinline__ Mine mine(int i) const {
    constexpr int kLanes = 8 * kPieces;  // pieces of the wave's rows of K
    const int q = i * 64 + lane;
    const int v = q >= kLanes, x = v ? q - kLanes : q;
    return Mine{x / kPieces, x % kPieces, v};
  }
  __device__ __forceinline__ void load(const AttendQuantizedParams& p, int t) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const Mine m = mine(i);
      const char* at = sh->row[wave][16 * (t & 3) + 8 * m.is_v + m.row] + 16 * m.piece;
      if (p.d != DP && 16 * m.piece >= p.d) at = reinterpret_cast<const char*>(g_zero_row);
      data[i] = *(global_u32x4*)at;
    }
  }
  // To the tiles: keys at `to`, values behind them.
  __device__ __forceinline__ void store(char* to, int t) const {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const Mine m = mine(i);
      const int r = wave * 8 + m.row;
      const uint32_t w0 = data[i][0], w1 = data[i][1], w2 = data[i][2], w3 = data[i][3];
      u32x4 x0, x1;
      if constexpr (kFactors) {
        x0 = to_f16<F>(w0, w1);
        x1 = to_f16<F>(w2, w3);
      } else {
        const float scale = sh->scale[wave][(t >> 2) & 1][16 * (t & 3) + 8 * m.is_v + m.row];
        x0 = to_bf16<F>(w0, w1, scale);
        x1 = to_bf16<F>(w2, w3, scale);
      }
      char* at = to + (m.is_v * KT + r) * R::kBytes;
      const int c = 2 * m.piece, sw = R::swz(r);
      *reinterpret_cast<u32x4*>(at + ((c ^ sw) << 4)) = x0;
      *reinterpret_cast<u32x4*>(at + (((c + 1) ^ sw) << 4)) = x1;
    }
  }
};

// Heads up to 128 elements (fp32: 64): eight waves in two groups of four that take
// turns on the matrix cores and the vector unit, over a ring of four stages of 64
// keys, as the kernel for 16-bit caches does; here a stage's bytes pass through
// registers, are converted once for all waves, and lie in LDS as bf16.  In step t
// stage t + 2, loaded in step t - 1, is converted into the place that stage t - 2
// left, and stage t + 3 is loaded.  A step is 2.1 to 2.2 us, the issue of its products
// (2100 cycles), of the conversion (1200) and of the weights (1230) one after the
// other at the barriers; a workgroup's start, first stages and output are some 18 us.
// 64 nodes over 32768 keys, 32 + 8 bf16 heads of 128, e4m3: 61 us and the join 8, 34
// GFLOP; 16 sequences of 256 to 8192 keys and 23 to 45 nodes, fp16, INT8: 139 and 11.
// With e4m3, heads of 128 and more than 128 rows 4 registers (fp16: 12) lie in memory.
template <typename Out, typename F, int DP, int KG>
__global__ __launch_bounds__(512, 2) void attend_turns_quantized_kernel(AttendQuantizedParams p) {
  using Elem = typename Tiles<Out>::Elem;
  using R = Rows<Elem, DP>;
  using Block = RowBlock<Elem, DP, Out, Tiles<Out>::NT>;
  using Stage = Staging<Elem, F, DP, 64>;
  constexpr int KT = 64, NS = 2 / KG, kRing = kTurnsRing;
  constexpr int kTile = KT * R::kBytes, kStage = 2 * kTile;
  // (aligned to its size, so that an XOR changes stages)
  __shared__ __attribute__((aligned(kRing * kStage))) char s_kv[kRing][kStage];
  __shared__ __attribute__((aligned(16))) typename Stage::Shared s_stage;
  warm_args(p);
  const Work w = quantized_work<32 * 8 / KG, false, 64>(p);
  if (w.none) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int late = wave >> 2;  // the group that runs behind
  const int block = KG == 1 ? wave : wave & 3, part = KG == 1 ? 0 : late;
  Block rb;
  rb.init(p, w, w.row0 + block * kBlock);
  const bool idle = w.row0 + block * kBlock >= w.rows;  // a wave without rows only fetches
  const int lane = rb.lane;
  const float c = p.scale == 0.f ? 1.0f : fabsf(p.scale) * kLog2e;
  const int keys = w.k1 - w.k0, inside = min(w.ctx, w.k1) - w.k0;
  const int nt = keys > 0 ? (keys + KT - 1) / KT : 0, nf = inside > 0 ? inside / KT : 0;
  Stage stage;
  stage.init(s_stage, w);
  const auto first_key = [&](int t) { return (int64_t)w.k0 + (int64_t)t * KT; };

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
    uint32_t all[Stage::kWords];
    const float above = stage.read_about(t, all);
    bool uneven = false;
#pragma unroll
    for (int b = 0; b < NS; ++b) {
      const uint32_t valid = all[part + b];
      seen[b] = valid;
      if constexpr (decltype(tail)::value) {
        seen[b] &= rb.sees(p, w, (int)first_key(t) + (part + b) * kBlock);
        uneven |= __any(seen[b] != valid);
      }
      if (!Stage::kFactors && __any(seen[b] != ~0u)) rb.mask_scores(s[b], seen[b]);
    }
    if constexpr (Stage::kFactors) {
      const uint32_t at = (uint32_t)(uintptr_t)s_stage.factors[t % kFactorRing] + 4 * part * kBlock;
      rb.weigh_scaled(s, seen, at, at + 4 * KT, at + 8 * KT);
    } else {
      rb.template weigh<true>(s, c, above);
    }
#pragma unroll
    for (int b = 0; b < NS; ++b) weights[b] = rb.pack(s[b]);
    if constexpr (decltype(tail)::value && F::kHasNan)
      odd = uneven && rb.any_odd(s_kv[t % kRing] + kTile + part * kBlock * R::kBytes, NS * kBlock);
  };
  // Short heads bring and convert a stage among the end of the products, longer ones
  // after the barrier: 43 us for 49 with heads of 64 (8 sequences of 4096 keys and 48
  // nodes), 194 for 165 the other way with heads of 128 (16 of up to 8192 keys, in chunks of 4096).
  constexpr bool kEarly = DP <= 64;
  auto fetch = [&](int t) __attribute__((always_inline)) {
    if (t + 2 < nt) {
      stage.store(s_kv[(t + 2) % kRing], t + 2);
      if (t + 3 < nt) {
        stage.load(p, t + 3);
        // the rows of stages 4 k + 4 .. 4 k + 7 in step 4 k, once those of the four before are on their way
        if ((t & 3) == kTurnsFind) stage.template find<Stage::NP>(p, w, (t >> 2) + 1);
        if ((t & 3) == kTurnsSettle) stage.template settle<Stage::NP>((t >> 2) + 1, c);
        if ((t & 3) == kTurnsAsk) stage.ask(p, w, (t >> 2) + 2);
      }
    }
  };
  auto step = [&](int t, auto tail) __attribute__((always_inline)) {
    __builtin_amdgcn_s_setprio(1);
    multiply(t, t > 0, true, tail);
    __builtin_amdgcn_s_setprio(0);
    if (kEarly) fetch(t);
    lds_barrier();
    if (!kEarly) fetch(t);
    soften(t, tail);
    lds_barrier();
  };

  if (nt > 0) {
    stage.ask(p, w, 0);
    stage.template find<0>(p, w, 0);
    stage.template settle<0>(0, c);
    stage.ask(p, w, 1);
#pragma unroll 1
    for (int t = 0; t < 3; ++t) {
      if (t > 0) stage.store(s_kv[t - 1], t - 1);
      stage.load(p, t);
    }
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
    // the second group's outputs pass through LDS
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
  if constexpr (KG == 1) __syncthreads();
  store_rows<DP>(p, w, rb, l, w.row0 + block * kBlock, &s_kv[0][0] + block * (KG == 1 ? kStoreBytes<DP> : kOut));
}

// The heads that leave the kernel above no registers: four waves of 32 rows share
// stages of 32 keys, double buffered.  A stage's bytes are in registers during the
// stage before it and converted into the other place at its end.  4 sequences of 8192
// keys and 32 nodes, 16 + 4 bf16 heads of 256, e4m3: 82 us; the output and the query
// fill the registers, with fp32 ones 90 (INT8) to 114 lie in memory.
template <typename Out, typename F, int DP>
__global__ __launch_bounds__(kThreads, 1) void attend_wide_quantized_kernel(AttendQuantizedParams p) {
  using Elem = typename Tiles<Out>::Elem;
  using R = Rows<Elem, DP>;
  constexpr int KT = kBlock;
  using Stage = Staging<Elem, F, DP, KT>;
  constexpr int kTile = KT * R::kBytes;
  constexpr int kLds = kTile < kStoreBytes<DP> ? 4 * kStoreBytes<DP> : 4 * kTile;
  // (aligned to its two stages, so that an XOR changes them)
  __shared__ __attribute__((aligned(4 * kTile))) char s_kv[kLds];
  const auto place = [&](int t) { return s_kv + t % kWideRing * 2 * kTile; };
  static_assert(kWideRing == 2, "an XOR changes places");
  __shared__ __attribute__((aligned(16))) typename Stage::Shared s_stage;
  warm_args(p);
  const Work w = quantized_work<4 * kBlock, true, 64>(p);
  if (w.none) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  RowBlock<Elem, DP, Out, Tiles<Out>::NT> rb;
  rb.init(p, w, w.row0 + wave * kBlock);
  const bool idle = w.row0 + wave * kBlock >= w.rows;  // a wave without rows only fetches
  const float c = p.scale == 0.f ? 1.0f : fabsf(p.scale) * kLog2e;
  const int keys = w.k1 - w.k0, inside = min(w.ctx, w.k1) - w.k0;
  const int nt = keys > 0 ? (keys + KT - 1) / KT : 0, nf = inside > 0 ? inside / KT : 0;
  Stage stage;
  stage.init(s_stage, w);
  const auto first_key = [&](int t) { return (int64_t)w.k0 + (int64_t)t * KT; };
  if (nt > 0) {
    stage.ask(p, w, 0);
    stage.template find<0>(p, w, 0);
    stage.template settle<0>(0, c);
    stage.ask(p, w, 1);
    stage.load(p, 0);
    stage.store(place(0), 0);
    stage.load(p, 1);
  }
  auto tile = [&](int t, auto tail) __attribute__((always_inline)) {
    constexpr bool kTail = decltype(tail)::value;
    lds_barrier();  // everyone's part of stage t is there, and everyone is done with stage t - 1
    if (t + 1 < nt) {
      stage.store(place(t + 1), t + 1);
      if (t + 2 < nt) {
        stage.load(p, t + 2);
        // the rows of stages 4 k + 4 .. 4 k + 7 in step 4 k + 1, once those of the four before are on their way
        if ((t & 3) == kWideFind) stage.template find<Stage::NP>(p, w, (t >> 2) + 1);
        if ((t & 3) == kWideSettle) stage.template settle<Stage::NP>((t >> 2) + 1, c);
        if ((t & 3) == kWideAsk) stage.ask(p, w, (t >> 2) + 2);
      }
    }
    if (!idle) {
      f32x16 s[1] = {rb.template scores<0>()};
      uint32_t seen[1];
      const float above = stage.read_about(t, seen);
      if constexpr (kTail) seen[0] &= rb.sees(p, w, (int)first_key(t));
      if constexpr (Stage::kFactors) {
        const uint32_t at = (uint32_t)(uintptr_t)s_stage.factors[t % kFactorRing];
        rb.weigh_scaled(s, seen, at, at + 4 * KT, at + 8 * KT);
      } else {
        if (__any(seen[0] != ~0u)) rb.mask_scores(s[0], seen[0]);
        rb.template weigh<true>(s, c, above);
      }
      const char* vb = place(t) + kTile;
      // One form of the products a loop: choosing between two by what a tile holds, as the
      // kernel above does, left 94 registers in memory (124 us for 84 at 4 x 32 nodes over
      // 8224 keys of 16 + 4 bf16 heads of 256).
      if constexpr (kTail && F::kHasNan) {
        rb.template add_values<true, 0>(rb.pack(s[0]));
        if (rb.any_odd(vb, KT)) rb.add_odd(vb, seen[0]);
      } else {
        rb.template add_values<false, 0>(rb.pack(s[0]));
      }
    }
    rb.move_keys(2 * kTile);
    rb.move_values(2 * kTile);
  };
  rb.place((uint32_t)(uintptr_t)s_kv, (uint32_t)(uintptr_t)s_kv + kTile);
  int t = 0;
  for (; t < nf; ++t) tile(t, No{});
  for (; t < nt; ++t) tile(t, Yes{});

  __syncthreads();
  store_rows<DP>(p, w, rb, half_sum(rb.l), w.row0 + wave * kBlock, s_kv + wave * kStoreBytes<DP>);
}

// ---- host -------------------------------------------------------------------

// Which kernel takes a call, by the rows of a (sequence, key/value head): up to 32
// the narrow one; else the one whose waves take turns, or the wide one where a
// head (fp32: more than 64 elements, else more than 128) leaves it no registers.
enum class Kind { kNarrow, kTurns128, kTurns256, kWide };
struct Plan {
  Kind kind;
  int32_t chunk, splits, row_tiles;
  int32_t block;   // threads of a workgroup
  int64_t groups;  // workgroups to be had from cutting the keys
  int64_t unit;    // keys that a chunk is a multiple of
  int64_t grid;
  int32_t cuts;    // chunks by the lengths, up to so many in all; 0: even chunks of the bounds
};
int padded(int32_t d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }
Plan plan_kind(bool fp32, int32_t nodes, int32_t group, int32_t d) {
  Plan a{};
  const int64_t rows = (int64_t)nodes * group;
  const int dp = padded(d);
  int64_t tile = kBlock;
  a.groups = dp == 256 ? 256 : 512;
  a.kind = Kind::kNarrow;
  a.block = kThreads;
  a.unit = 4 * (dp == 256 ? 8192 : 4096) / dp;
  if (rows > kBlock) {
    a.kind = dp > (fp32 ? 64 : 128) ? Kind::kWide : rows > 4 * kBlock ? Kind::kTurns256 : Kind::kTurns128;
    tile = a.kind == Kind::kTurns256 ? 8 * kBlock : 4 * kBlock;
    a.groups = a.kind == Kind::kWide ? 512 : 256;
    a.block = a.kind == Kind::kWide ? kThreads : 512;
    a.unit = 64;
  }
  a.row_tiles = (int32_t)ceil_div(rows, tile);
  return a;
}

// How the keys are cut: by their lengths where a lane can count for each sequence,
// else into even chunks, so long that about `groups` workgroups run in all where
// every sequence is as long as its bound; no shorter than kMinChunk.  groups: as many
// as the chip holds at once.  More cost their first loads and parts: 64 sequences of
// 4096 keys, 32 + 8 bf16 heads of 128, 92 us with 512 workgroups, 99 with 1024, 104
// with 2048; one of 32768: 27, 31 and 37.  The wide kernel is given twice as many as
// its registers leave room for (one a compute unit), and that costs it too: 4
// sequences of 8192 keys and 32 nodes, 16 + 4 bf16 heads of 256, take 82 us with 512
// and 66 with 256; 16 unlike ones of up to 8192 keys and 45 nodes 182 and 165.
constexpr int64_t kMaxChunk = (int64_t)1 << 30;

// The most chunks of a sequence; even: if all are as long.  Where others may be short
// a long one gets up to twice as many, at that many parts.
int64_t most_cuts(int64_t B, int64_t even) { return B > 1 ? 2 * even : even; }

Plan plan_of(bool fp32, int32_t B, int32_t max_nodes, int32_t max_context, int32_t hq, int32_t hk, int32_t d) {
  Plan a = plan_kind(fp32, max_nodes, hq / hk, d);
  const int64_t keys = (int64_t)max_context + max_nodes;
  const int64_t units = (int64_t)B * hk * a.row_tiles;
  if (B <= kCutSeqs && units < a.groups && units * ceil_div(keys, 64) < (int64_t)1 << 31) {  // (sums in 32 bits)
    a.cuts = (int32_t)a.groups;
    a.chunk = 1;
    a.splits = (int32_t)std::min(ceil_div(keys, kMinChunk), most_cuts(B, ceil_div(a.groups, units)));
    a.grid = a.groups;
    return a;
  }
  int64_t chunk = units < a.groups ? ceil_div(keys * units, a.groups) : keys;
  if (chunk < kMinChunk) chunk = kMinChunk;
  chunk = ceil_div(ceil_div(keys, ceil_div(keys, chunk)), a.unit) * a.unit;
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

template <typename Out, typename F, int DP>
hipError_t launch_d(const AttendQuantizedParams& p, const Plan& a, hipStream_t stream) {
  const dim3 g((unsigned)a.grid), b((unsigned)a.block);
  if (a.kind == Kind::kNarrow) {
    hipLaunchKernelGGL((attend_narrow_quantized_kernel<Out, F, DP>), g, b, 0, stream, p);
  } else if constexpr (DP > (sizeof(Out) == 4 ? 64 : 128)) {
    hipLaunchKernelGGL((attend_wide_quantized_kernel<Out, F, DP>), g, b, 0, stream, p);
  } else if (a.kind == Kind::kTurns256) {
    hipLaunchKernelGGL((attend_turns_quantized_kernel<Out, F, DP, 1>), g, b, 0, stream, p);
  } else {
    hipLaunchKernelGGL((attend_turns_quantized_kernel<Out, F, DP, 2>), g, b, 0, stream, p);
  }
  return hipGetLastError();
}

template <typename Out, typename F>
hipError_t launch(AttendQuantizedParams p, hipStream_t stream) {
  const Plan a = plan_of(sizeof(Out) == 4, p.B, p.max_nodes, p.max_context, p.hq, p.hk, p.d);
  p.chunk = a.chunk;
  p.splits = a.splits;
  p.cuts = a.cuts;
  if (a.cuts && a.splits > 1) p.part += kChunkBytes / 4;
  p.row_tiles = a.row_tiles;
  p.part_rows = part_rows_of(p.B, p.T, p.max_nodes);
  p.by_tiles = fast_div((uint32_t)a.row_tiles);
  p.by_splits = fast_div((uint32_t)a.splits);
  p.by_sequences = fast_div((uint32_t)p.B);
  p.by_heads = fast_div((uint32_t)p.hk);
  p.by_chunk = fast_div((uint32_t)a.chunk);
  const int dp = padded(p.d);
  const hipError_t e = dp == 64    ? launch_d<Out, F, 64>(p, a, stream)
                       : dp == 128 ? launch_d<Out, F, 128>(p, a, stream)
                                   : launch_d<Out, F, 256>(p, a, stream);
  if (e != hipSuccess || p.splits == 1) return e;
  const dim3 g((unsigned)join_grid(p.max_nodes, p.hq), (unsigned)p.B);
  if (p.cuts) {
    hipLaunchKernelGGL((attend_join_kernel<Out, true>), g, dim3(kThreads), 0, stream, static_cast<const AttendParams&>(p));
  } else {
    hipLaunchKernelGGL((attend_join_kernel<Out, false>), g, dim3(kThreads), 0, stream, static_cast<const AttendParams&>(p));
  }
  return hipGetLastError();
}

}  // namespace

bool attend_quantized_fits(lora_dtype dt, int32_t B, int32_t max_nodes, int32_t max_context, int32_t hq, int32_t hk,
                           int32_t d) {
  const Plan a = plan_of(dt == LORA_F32, B, max_nodes, max_context, hq, hk, d);
  const int64_t most = ((int64_t)1 << 32) - 1;  // threads in a dimension of a grid
  return a.grid <= most / a.block && (a.splits == 1 || join_grid(max_nodes, hq) <= most / kThreads);
}

int64_t attend_quantized_need_bytes(lora_dtype dt, int32_t B, int32_t T, int32_t max_nodes, int32_t max_context,
                                    int32_t hq, int32_t hk, int32_t d) {
  const Plan a = plan_of(dt == LORA_F32, B, max_nodes, max_context, hq, hk, d);
  if (a.splits == 1) return 0;
  return (a.cuts ? kChunkBytes : 0) + part_bytes(a.splits * (int64_t)part_rows_of(B, T, max_nodes), hq, d);
}

// Fewer sequences or nodes are cut into more chunks, so the bytes of a call do not
// grow with its sizes; these are the most of any call up to them.  With G workgroups
// to be had and u = sequences * kv_heads * row tiles a call has at most ceil(keys /
// kMinChunk) and most_cuts of ceil(G / u) chunks (2^30 keys at most an even chunk),
// both largest at the most keys; rows only grow.  What is left is to try the numbers
// of sequences and, of the nodes, those that fill their row tiles.
int64_t attend_quantized_most_bytes(int32_t B, int32_t T, int32_t max_nodes, int32_t max_context, int32_t hq, int32_t hk,
                                    int32_t d) {
  const int32_t group = hq / hk;
  const int64_t keys = (int64_t)max_context + max_nodes, by_keys = ceil_div(keys, kMinChunk);
  const int64_t uncut = ceil_div(keys, kMaxChunk);
  int64_t most = uncut > 1 ? uncut * part_rows_of(B, T, max_nodes) : 0;
  const auto nodes_up_to = [&](bool fp32, int64_t nodes) {
    if (nodes < 1) return;
    nodes = std::min<int64_t>(nodes, max_nodes);
    const Plan a = plan_kind(fp32, (int32_t)nodes, group, d);
    const int64_t per = (int64_t)hk * a.row_tiles;
    for (int64_t b = 1; b <= B && b * per < a.groups; ++b) {
      const int64_t splits = std::max(std::min(by_keys, most_cuts(b, ceil_div(a.groups, b * per))), uncut);
      if (splits > 1) most = std::max(most, splits * part_rows_of((int32_t)b, T, (int32_t)nodes));
    }
  };
  for (const bool fp32 : {false, true}) {
    nodes_up_to(fp32, kBlock / group);
    for (int64_t tiles = 1; tiles * hk < 512; ++tiles) {
      nodes_up_to(fp32, tiles * 4 * kBlock / group);
      nodes_up_to(fp32, tiles * 8 * kBlock / group);
      if (tiles * 4 * kBlock / group >= max_nodes) break;
    }
    nodes_up_to(fp32, max_nodes);
  }
  return most ? kChunkBytes + part_bytes(most, hq, d) : 0;
}

template <typename Out> static hipError_t launch_format(int format, const AttendQuantizedParams& p, hipStream_t stream) {
  return format == LORA_CACHE_E4M3 ? launch<Out, E4m3>(p, stream) : launch<Out, Int8>(p, stream);
}

hipError_t launch_attend_quantized(lora_dtype dt, int format, AttendQuantizedParams p, hipStream_t stream) {
  switch (dt) {
    case LORA_F32: return launch_format<float>(format, p, stream);
    case LORA_F16: return launch_format<half_t>(format, p, stream);
    case LORA_BF16: return launch_format<bf16_t>(format, p, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace lora
