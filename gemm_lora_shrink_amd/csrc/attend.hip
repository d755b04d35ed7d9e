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

#include "attend_unit.h"

namespace lora {

namespace {

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
  store_rows<DP>(p, w, rb, half_sum(rb.l), w.row0 + wave * kBlock, &s_kv[0][0] + wave * kStoreBytes<DP>);
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
  store_rows<DP>(p, w, rb, l, w.row0 + block * kBlock, &s_kv[0][0] + block * (KG == 1 ? kStoreBytes<DP> : kOut));
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
