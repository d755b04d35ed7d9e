// The store that fills a quantized cache, and the move of an accepted path in it.
#include <type_traits>

#include "cache.h"

namespace lora {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// The least exponent e with a <= largest 2^e, from the bits of a.
template <typename F> __device__ inline int least_exponent(float a) {
  const uint32_t bits = __float_as_uint(a);
  const int e = (int)(bits >> 23) - 127 - F::kLargestExp + ((bits & 0x7fffffu) > F::kLargestMantissa ? 1 : 0);
  return e < kExpLow ? kExpLow : (e > F::kTop ? F::kTop : e);
}

// Eight bytes with another exponent: numbers times `down` (a power of two <= 1).
template <typename F> __device__ inline u32x2 lowered(u32x2 w, float down) {
  float x[8];
  const uint32_t w0 = w[0], w1 = w[1];
  F::numbers(w0, x);
  F::numbers(w1, x + 4);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] *= down;
  return u32x2{F::bytes(x), F::bytes(x + 4)};
}

// Eight elements as fp32.
template <typename Elem> __device__ inline void load8(const Elem* p, float* x) {
  const u32x4* w = reinterpret_cast<const u32x4*>(p);
  Traits<Elem>::to_float(w[0], x);
  if constexpr (sizeof(Elem) == 4) Traits<Elem>::to_float(w[1], x + 4);
}

// The largest of the wave's 64 whole numbers, by lane shifts and broadcasts of the vector
// unit: a row of 16 lanes in four steps, then the rows.
__device__ inline uint32_t wave_max(uint32_t x) {
  const auto step = [](uint32_t y, auto dpp) __attribute__((always_inline)) {
    return max(y, (uint32_t)__builtin_amdgcn_update_dpp((int)y, (int)y, decltype(dpp)::value, 0xf, 0xf, false));
  };
  x = step(x, std::integral_constant<int, 0x111>{});  // row_shr 1, 2, 4, 8
  x = step(x, std::integral_constant<int, 0x112>{});
  x = step(x, std::integral_constant<int, 0x114>{});
  x = step(x, std::integral_constant<int, 0x118>{});
  x = step(x, std::integral_constant<int, 0x142>{});  // row_bcast 15, 31
  x = step(x, std::integral_constant<int, 0x143>{});
  return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

// Magnitudes are compared as whole numbers, which their bits without the sign are in
// order, two at a time where they have 16 bits.
template <typename Elem> struct Magnitude {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  static constexpr bool k16 = sizeof(Elem) == 2;
  static constexpr uint32_t kNotFinite = !k16 ? 0x7f800000u : Traits<Elem>::kDtype == LORA_F16 ? 0x7c00u : 0x7f80u;
  uint32_t most = 0;
  __device__ __forceinline__ void take(u32x4 w) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = w[i];
      if constexpr (k16)
        most = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, most),
                                                                     __builtin_bit_cast(u16x2, x & 0x7fff7fffu)));
      else most = max(most, x & 0x7fffffffu);
    }
  }
  // the bits of the largest over the wave
  __device__ __forceinline__ uint32_t of_wave() const {
    return wave_max(k16 ? max(most & 0xffffu, most >> 16) : most);
  }
};

// A wave takes one head, and of that head one block of K and V at a time: the run of
// tokens that starts with a token whose predecessor is not in the row before it in
// the same block.  A row lies over 2^lane_shift lanes, 8 elements each.  The largest
// magnitude of all rows is needed before the first byte can be written; kHeld rows a
// lane stay in registers until then, more are read twice, the second time from L2.
// Bound by the chain row numbers, rows, exponent (256 tokens of 8 heads of 128: 5.4
// us) and, in prompts, by that chain and memory (6144 tokens, 38 MB: 10.4 us, 9.9
// among others, 3.8 TB/s; 14.8 with magnitudes and roundings taken one by one in
// fp32, as they still are where there are infinities or NaN).
template <typename Elem, typename F>
__global__ __launch_bounds__(kThreads) void store_quantized_kernel(StoreParams p) {
  warm_args(p);
  constexpr int kHeld = 4, kPer8 = sizeof(Elem) / 2;  // 16-byte loads of 8 elements
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = (int)blockIdx.y * kWaves + wave;
  if (h >= p.hk) return;
  const QuantizedView& c = p.cache;
  const int t0 = (int)blockIdx.x * p.chunk;
  const int block = (int)c.block.d;

  const int row = t0 + lane < p.T ? p.rows[t0 + lane] : -1;
  int before = __shfl_up(row, 1);
  if (lane == 0) before = t0 ? p.rows[t0 - 1] : -1;
  bool leads = false, follows = false;
  if (row >= 0 && row < p.n_rows) {
    const int place = row - (int)c.page.div((uint32_t)row) * (int)c.page.d;
    follows = before == row - 1 && place - (int)c.block.div((uint32_t)place) * block != 0;
    leads = !follows && lane < p.chunk;
  }
  uint64_t todo = __ballot(leads);
  const uint64_t runs = __ballot(follows);
  const int per = 64 >> p.lane_shift, r = lane >> p.lane_shift, col = 8 * (lane & ((1 << p.lane_shift) - 1));
  const bool in_row = col < p.d;
  for (; todo; todo &= todo - 1) {
    const int i = __builtin_ctzll(todo);
    const int64_t t = t0 + i;
    const int first_row = __builtin_amdgcn_readlane(row, i);
    const int64_t page = c.page.div((uint32_t)first_row);
    const int place = first_row - (int)page * (int)c.page.d, of = (int)c.block.div((uint32_t)place);
    const int first = place - of * block;
    // the run's length: as far as the lanes know, then by looking on
    const uint64_t ends = i == 63 ? 1 : (~runs >> (i + 1)) | (1ull << (63 - i));
    int n = 1 + __builtin_ctzll(ends);
    if (i + n == 64) {
      const int most = block - first;
      for (bool on = true; on && n < most;) {
        const int j = n + lane;
        const uint64_t stop = __ballot(j >= most || t + j >= p.T || p.rows[t + j] != first_row + j);
        n += stop ? __builtin_ctzll(stop) : 64;
        on = !stop;
      }
    }
    const Elem* x[2];
    char* to[2];
    int8_t* exps[2];
    int old[2];
    u32x4 raw[2][kHeld][kPer8];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      x[v] = static_cast<const Elem*>(v ? p.v : p.k) + t * (v ? p.ldv : p.ldk) + (int64_t)h * p.d + col;
      to[v] = static_cast<char*>(v ? c.v : c.k) + page * (v ? c.v_page : c.k_page) + h * (v ? c.v_head : c.k_head) + col;
      exps[v] = (v ? c.v_exp + page * c.v_exp_page + h * c.v_exp_head : c.k_exp + page * c.k_exp_page + h * c.k_exp_head) + of;
#pragma unroll
      for (int u = 0; u < kHeld; ++u) {
        const int j = u * per + r;
#pragma unroll
        for (int q = 0; q < kPer8; ++q)
          raw[v][u][q] = ld16_or0(reinterpret_cast<const u32x4*>(x[v] + j * (v ? p.ldv : p.ldk)) + q, in_row && j < n);
      }
      old[v] = *exps[v];
    }
    const auto eight = [](const u32x4(&w)[kPer8], float* y) __attribute__((always_inline)) {
      Traits<Elem>::to_float(w[0], y);
      if constexpr (kPer8 == 2) Traits<Elem>::to_float(w[1], y + 4);
    };
    uint32_t largest[2];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      Magnitude<Elem> most;
#pragma unroll
      for (int u = 0; u < kHeld; ++u)
#pragma unroll
        for (int q = 0; q < kPer8; ++q) most.take(raw[v][u][q]);
      if (in_row)
        for (int j = kHeld * per + r; j < n; j += per)
#pragma unroll
          for (int q = 0; q < kPer8; ++q)
            most.take(reinterpret_cast<const u32x4*>(x[v] + j * (v ? p.ldv : p.ldk))[q]);
      largest[v] = most.of_wave();
    }
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const int64_t row_b = v ? c.v_row : c.k_row;
      float top = Traits<Elem>::elem_to_float(largest[v]);
      // infinities and NaN have no part in the exponent, and where there are some, or the
      // largest is beyond the format's, numbers are looked at one by one
      bool within = largest[v] < Magnitude<Elem>::kNotFinite;
      if (!within) {
        top = 0.f;
        if (in_row)
          for (int j = r; j < n; j += per) {
            float y[8];
            load8(x[v] + j * (v ? p.ldv : p.ldk), y);
#pragma unroll
            for (int k = 0; k < 8; ++k) top = fabsf(y[k]) < INFINITY ? fmaxf(top, fabsf(y[k])) : top;
          }
        top = __uint_as_float(wave_max(__float_as_uint(top)));
      }
      int e = least_exponent<F>(top);
      within = within && e < F::kTop;
      if (first > 0) {
        const int was = exponent_of<F>((int8_t)old[v]);
        if (e > was) {
          const float down = power_of_two(was - e < kExpLow ? kExpLow : was - e);
          if (in_row)
            for (int j = r; j < first; j += per) {
              u32x2* at = reinterpret_cast<u32x2*>(to[v] + (place - first + j) * row_b);
              *at = lowered<F>(*at, down);
            }
        } else {
          e = was;
        }
      }
      if (lane == 0) *exps[v] = (int8_t)e;
      const float up = power_of_two(-e);
      const auto put = [&](int j, float* y) __attribute__((always_inline)) {
        u32x2 w;
        if (within) {
          w = u32x2{F::bytes_within(y, up), F::bytes_within(y + 4, up)};
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) y[k] *= up;
          w = u32x2{F::bytes(y), F::bytes(y + 4)};
        }
        *reinterpret_cast<u32x2*>(to[v] + (place + j) * row_b) = w;
      };
#pragma unroll
      for (int u = 0; u < kHeld; ++u) {
        const int j = u * per + r;
        if (!in_row || j >= n) continue;
        float y[8];
        eight(raw[v][u], y);
        put(j, y);
      }
      if (in_row)
        for (int j = kHeld * per + r; j < n; j += per) {
          float y[8];
          load8(x[v] + j * (v ? p.ldv : p.ldk), y);
          put(j, y);
        }
    }
  }
}

// Paths of up to 64 nodes: lane j looks up where kept row j comes from and goes to,
// and its exponent, for all rows at once, so that the chain of loads (path, page
// table, exponent and bytes) is walked once and not for every block.  64 sequences,
// up to 8 rows each, 8 layers of 8 heads of 128: 10.2 us (16.1 block after block).
template <typename F>
__global__ __launch_bounds__(kThreads) void keep_short_kernel(KeepQuantizedParams p) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int b = blockIdx.x, h = (int)blockIdx.y * kWaves + wave, layer = (int)blockIdx.z >> 1;
  if (h >= p.kv_heads) return;
  const bool is_v = blockIdx.z & 1;
  const QuantizedView& c = p.cache;
  char* base = static_cast<char*>(is_v ? p.v[layer] : p.k[layer]) + h * (is_v ? c.v_head : c.k_head);
  int8_t* exps = is_v ? p.v_exp[layer] + h * c.v_exp_head : p.k_exp[layer] + h * c.k_exp_head;
  const int64_t page_b = is_v ? c.v_page : c.k_page, row_b = is_v ? c.v_row : c.k_row;
  const int64_t exp_b = is_v ? c.v_exp_page : c.k_exp_page;
  const int64_t ctx = p.context[b];
  int n = p.n_kept[b];
  const int node = lane < p.n_path ? p.path[b * p.ld_path + lane] : -1;
  n = n > p.n_path ? p.n_path : n;
  if (ctx < 0 || n <= 0) return;
  // the path ends before the first entry that does not ascend
  const int before = __shfl_up(node, 1);
  const uint64_t stop = __ballot(lane >= n || node <= (lane ? before : -1));
  n = stop ? __builtin_ctzll(stop) : 64;
  if (n == 0) return;
  const int block = (int)c.block.d;
  const bool there = lane < n;
  const auto page_of = [&](int64_t pos, int& row) {
    row = 0;
    if (!there || pos >= (int64_t)1 << 31) return -1;
    const int col = (int)c.page.div((uint32_t)pos);
    row = (int)((uint32_t)pos - (uint32_t)col * c.page.d);
    if (col >= p.n_table) return -1;
    const int page = p.page_table[b * p.ld_table + col];
    return page >= 0 && page < c.n_pages ? page : -1;
  };
  int of_row, to_row;
  const int of_page = page_of(ctx + node, of_row), to_page = page_of(ctx + lane, to_row);
  const bool moves = of_page >= 0 && to_page >= 0;
  int8_t* mine = exps + (moves ? to_page * exp_b + (int)c.block.div((uint32_t)to_row) : 0);
  const int was = moves ? exponent_of<F>(exps[of_page * exp_b + (int)c.block.div((uint32_t)of_row)]) : kExpLow - 1;
  const int old = moves ? exponent_of<F>(*mine) : kExpLow - 1;
  // the largest exponent of the rows that go to one block: the lanes from `low` to `high`
  const int in_block = (int)((uint32_t)(ctx + lane) % (uint32_t)block);  // (of lanes that are there)
  const int low = max(0, lane - in_block), high = min(n - 1, lane - in_block + block - 1);
  int e = there ? was : kExpLow - 1;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(e, o);
    if (lane - o >= low) e = max(e, y);
  }
  e = __shfl(e, there ? high : lane);
  // earlier rows live in the first block only; where its first row moves nothing, a later one's page is the same
  const int first = (int)((uint32_t)ctx % (uint32_t)block);
  const bool shared = first > 0 && low == 0;
  const bool grows = shared && moves && e > old;
  if (shared && moves) e = max(e, old);
  const int pieces = p.d / 8, per = 64 / pieces;  // (pieces <= 32)
  const int r = lane / pieces, at = 8 * (lane - r * pieces);
  const bool in_row = r < per;
  const uint64_t growing = __ballot(grows);
  if (growing) {
    const int i = __builtin_ctzll(growing);
    const int64_t page = __builtin_amdgcn_readlane(to_page, i);
    const int row0 = __builtin_amdgcn_readlane(to_row - in_block, i);
    const int by = __builtin_amdgcn_readlane(old - e, i);
    char* rows = base + page * page_b + row0 * row_b + at;
    const float down = power_of_two(max(by, kExpLow));
    if (in_row)
      for (int j = r; j < first; j += per) {
        u32x2* q = reinterpret_cast<u32x2*>(rows + j * row_b);
        *q = lowered<F>(*q, down);
      }
  }
  // kept rows, `per` a load; rounds are read whole before they are written, and what a
  // later round reads lies behind everything that this one writes
  constexpr int kAtOnce = 4;
  for (int j0 = 0; j0 < n; j0 += kAtOnce * per) {
    u32x2 w[kAtOnce];
    bool put[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int j = j0 + u * per + r, from = j & 63;
      const int page = __shfl(of_page, from), row = __shfl(of_row, from);
      const bool stays = __shfl(node == lane && was == e, from), goes = __shfl(moves, from);
      put[u] = in_row && j < n && goes && !stays;
      if (put[u]) w[u] = *reinterpret_cast<const u32x2*>(base + page * page_b + row * row_b + at);
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int from = (j0 + u * per + r) & 63;
      const int page = __shfl(to_page, from), row = __shfl(to_row, from), by = __shfl(was - e, from);
      if (put[u])
        *reinterpret_cast<u32x2*>(base + page * page_b + row * row_b + at) =
            by == 0 ? w[u] : lowered<F>(w[u], power_of_two(max(by, kExpLow)));
    }
  }
  // a block's exponent, by the first of its lanes that moves
  const uint64_t movers = __ballot(moves);
  if (moves && (movers & (~0ull << low)) != 0 && __builtin_ctzll(movers & (~0ull << low)) == lane) *mine = (int8_t)e;
}

// Longer paths: a wave takes one head of a layer's K or V of one sequence, block after block of
// the rows that the path moves to, in ascending order.  A source never lies
// before its destination and the sources ascend, so what a block's rows come
// from lies in that block or behind it: no earlier block's write has changed it,
// neither its bytes nor its exponent, which is written when the block is done.
template <typename F>
__global__ __launch_bounds__(kThreads) void keep_quantized_kernel(KeepQuantizedParams p) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int b = blockIdx.x, h = (int)blockIdx.y * kWaves + wave, layer = (int)blockIdx.z >> 1;
  if (h >= p.kv_heads) return;
  const bool is_v = blockIdx.z & 1;
  const QuantizedView& c = p.cache;
  char* base = static_cast<char*>(is_v ? p.v[layer] : p.k[layer]) + h * (is_v ? c.v_head : c.k_head);
  int8_t* exps = is_v ? p.v_exp[layer] + h * c.v_exp_head : p.k_exp[layer] + h * c.k_exp_head;
  const int64_t page_b = is_v ? c.v_page : c.k_page, row_b = is_v ? c.v_row : c.k_row;
  const int64_t exp_b = is_v ? c.v_exp_page : c.k_exp_page;
  const int64_t ctx = p.context[b];
  int n = p.n_kept[b];
  n = n > p.n_path ? p.n_path : n;
  if (ctx < 0 || n <= 0) return;
  const int32_t* path = p.path + b * p.ld_path;
  for (int j0 = 0; j0 < n; j0 += 64) {  // the path ends before the first entry that does not ascend
    const int j = j0 + lane;
    const bool bad = j < n && path[j] <= (j ? path[j - 1] : -1);
    const uint64_t any = __ballot(bad);
    if (any) {
      n = j0 + __builtin_ctzll(any);
      break;
    }
  }
  struct Place {
    int64_t page;  // -1: none
    int row, block;
  };
  const auto place_of = [&](int64_t pos) {
    Place a{-1, 0, 0};
    if (pos >= (int64_t)1 << 31) return a;
    const int64_t col = c.page.div((uint32_t)pos);
    if (col >= p.n_table) return a;
    const int64_t page = p.page_table[b * p.ld_table + col];
    if (page < 0 || page >= c.n_pages) return a;
    a.page = page;
    a.row = (int)(pos - col * c.page.d);
    a.block = (int)c.block.div((uint32_t)a.row);
    return a;
  };
  const int block = (int)c.block.d, pieces = p.d / 8, per = pieces >= 64 ? 1 : 64 / pieces;
  const int r = lane / pieces, at = 8 * (lane - r * pieces);
  const bool in_row = r < per;
  for (int j0 = 0; j0 < n;) {
    const Place to = place_of(ctx + j0);
    const int first = (int)((uint32_t)(ctx + j0) % (uint32_t)block);  // row of the block that j0 moves to
    const int j1 = min(n, j0 + block - first);
    if (to.page >= 0) {
      // the exponents that the rows come with
      int8_t* mine = exps + to.page * exp_b + to.block;
      const int old = exponent_of<F>(*mine);
      int e = kExpLow;
      bool any = false;
      for (int j = j0 + lane; j < j1; j += 64) {
        const Place of = place_of(ctx + path[j]);
        if (of.page < 0) continue;
        any = true;
        e = max(e, exponent_of<F>(exps[of.page * exp_b + of.block]));
      }
#pragma unroll
      for (int o = 32; o; o >>= 1) e = max(e, __shfl_xor(e, o));
      if (__any(any)) {
        char* rows = base + to.page * page_b + (to.row - first) * row_b + at;
        if (first > 0) {
          e = max(e, old);
          if (e > old) {
            const float down = power_of_two(max(old - e, kExpLow));
            for (int i = r; i < first; i += per)
              if (in_row) {
                u32x2* q = reinterpret_cast<u32x2*>(rows + i * row_b);
                *q = lowered<F>(*q, down);
              }
          }
        }
        for (int i0 = j0; i0 < j1; i0 += per) {
          const int j = i0 + r;
          if (!in_row || j >= j1) continue;
          const Place of = place_of(ctx + path[j]);
          if (of.page < 0) continue;
          const int was = exponent_of<F>(exps[of.page * exp_b + of.block]);
          if (path[j] == j && was == e) continue;
          const u32x2 w = *reinterpret_cast<const u32x2*>(base + of.page * page_b + of.row * row_b + at);
          *reinterpret_cast<u32x2*>(rows + (first + j - j0) * row_b) =
              was == e ? w : lowered<F>(w, power_of_two(max(was - e, kExpLow)));
        }
        if (lane == 0) *mine = (int8_t)e;
      }
    }
    j0 = j1;
  }
}

// Tokens of a workgroup: a decode step's are mostly blocks of their own; of a prompt's
// (6144 tokens, blocks of 8) 8, 16 and 32 took 10.8, 9.9 and 12.1 us.  Which a call
// is the host cannot tell, but by its size.  A call with 2 and with 16, host's part
// included: 256 and 1024 single tokens 12 and 22 us, prompts of 512 and 1024 tokens 12
// either way, of 6144 in blocks of 8 19 and 12, of 8192 in blocks of 128 77 and 51;
// 4096 single tokens, and 2048 tokens in blocks of one row, lose: 22 and 13 for 29 and 23.
int store_chunk(int32_t T) { return T <= 1024 ? 2 : 16; }

template <typename Elem>
hipError_t launch_store(int format, const StoreParams& p, dim3 grid, hipStream_t stream) {
  if (format == LORA_CACHE_E4M3)
    hipLaunchKernelGGL((store_quantized_kernel<Elem, E4m3>), grid, dim3(kThreads), 0, stream, p);
  else
    hipLaunchKernelGGL((store_quantized_kernel<Elem, Int8>), grid, dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

bool store_quantized_fits(int32_t T) {
  return ceil_div(T, store_chunk(T)) <= (((int64_t)1 << 32) - 1) / kThreads;  // threads in a dimension of a grid
}

hipError_t launch_store_quantized(lora_dtype dt, int format, StoreParams p, hipStream_t stream) {
  p.chunk = store_chunk(p.T);
  p.lane_shift = 1;
  while ((8 << p.lane_shift) < p.d) ++p.lane_shift;
  const dim3 grid((unsigned)ceil_div(p.T, p.chunk), (unsigned)ceil_div(p.hk, kWaves));
  switch (dt) {
    case LORA_F32: return launch_store<float>(format, p, grid, stream);
    case LORA_F16: return launch_store<half_t>(format, p, grid, stream);
    case LORA_BF16: return launch_store<bf16_t>(format, p, grid, stream);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_keep_quantized(int format, const KeepQuantizedParams& p, int32_t n_layers, int32_t B,
                                 hipStream_t stream) {
  const dim3 grid((unsigned)B, (unsigned)ceil_div(p.kv_heads, kWaves), (unsigned)(2 * n_layers));
  const bool e4m3 = format == LORA_CACHE_E4M3;
  if (p.n_path <= 64) {
    if (e4m3) hipLaunchKernelGGL(keep_short_kernel<E4m3>, grid, dim3(kThreads), 0, stream, p);
    else hipLaunchKernelGGL(keep_short_kernel<Int8>, grid, dim3(kThreads), 0, stream, p);
  } else if (e4m3) {
    hipLaunchKernelGGL(keep_quantized_kernel<E4m3>, grid, dim3(kThreads), 0, stream, p);
  } else {
    hipLaunchKernelGGL(keep_quantized_kernel<Int8>, grid, dim3(kThreads), 0, stream, p);
  }
  return hipGetLastError();
}

}  // namespace lora
