// The store that fills a quantized cache, and the move of an accepted path in it.
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

// A wave takes one block of one head of K or V at a time: the run of tokens that
// starts with a token whose predecessor is not in the row before it in the same
// block.  A row lies over 2^lane_shift lanes, 8 elements each.  The largest
// magnitude of all rows is needed before the first byte can be written, so the
// rows are read twice where they are more than the registers hold (kHeld rows a
// lane), the second time from L2.
template <typename Elem, typename F>
__global__ __launch_bounds__(kThreads) void store_quantized_kernel(StoreParams p) {
  warm_args(p);
  constexpr int kHeld = 4;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = (int)blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  const Elem* x = static_cast<const Elem*>(is_v ? p.v : p.k) + (int64_t)h * p.d;
  const int64_t ld = is_v ? p.ldv : p.ldk;
  const QuantizedView& c = p.cache;
  const int t0 = (int)blockIdx.x * p.chunk;
  const int block = (int)c.block.d;

  int row = -1;
  bool leads = false;
  if (lane < p.chunk && t0 + lane < p.T) {
    row = p.rows[t0 + lane];
    const int before = t0 + lane ? p.rows[t0 + lane - 1] : -1;
    if (row >= 0 && row < p.n_rows) {
      const int place = row - (int)c.page.div((uint32_t)row) * (int)c.page.d;
      leads = before != row - 1 || place % block == 0;
    }
  }
  uint64_t todo = __ballot(leads);
  const int per = 64 >> p.lane_shift, r = lane >> p.lane_shift, col = 8 * (lane & ((1 << p.lane_shift) - 1));
  const bool in_row = col < p.d;
  for (int turn = 0; todo; ++turn, todo &= todo - 1) {
    if (turn % kWaves != wave) continue;
    const int i = __builtin_ctzll(todo);
    const int64_t t = t0 + i;
    const int first_row = __builtin_amdgcn_readlane(row, i);
    const int64_t page = c.page.div((uint32_t)first_row);
    const int place = first_row - (int)page * (int)c.page.d, of = (int)c.block.div((uint32_t)place);
    const int first = place - of * block;
    // the run's length
    int n = block - first;
    for (int j0 = 0; j0 < n; j0 += 64) {
      const int j = j0 + lane;
      const bool ends = j < n && (t + j >= p.T || p.rows[t + j] != first_row + j);
      const uint64_t any = __ballot(ends);
      if (any) {
        n = j0 + __builtin_ctzll(any);
        break;
      }
    }
    const Elem* xt = x + t * ld + col;
    float held[kHeld][8];
    float most = 0.f;
    for (int j0 = 0; j0 < n; j0 += kHeld * per) {
#pragma unroll
      for (int u = 0; u < kHeld; ++u) {
        const int j = j0 + u * per + r;
        if (in_row && j < n) load8(xt + j * ld, held[u]);
        else
#pragma unroll
          for (int e = 0; e < 8; ++e) held[u][e] = 0.f;
      }
#pragma unroll
      for (int u = 0; u < kHeld; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float a = fabsf(held[u][e]);
          most = a < INFINITY && a > most ? a : most;
        }
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) most = fmaxf(most, __shfl_xor(most, o));
    int8_t* exps = (is_v ? c.v_exp + page * c.v_exp_page + h * c.v_exp_head : c.k_exp + page * c.k_exp_page + h * c.k_exp_head);
    char* to = static_cast<char*>(is_v ? c.v : c.k) + page * (is_v ? c.v_page : c.k_page) + h * (is_v ? c.v_head : c.k_head) + col;
    const int64_t row_b = is_v ? c.v_row : c.k_row;
    int e = least_exponent<F>(most);
    if (first > 0) {
      const int old = exponent_of<F>(exps[of]);
      if (e > old) {
        const float down = power_of_two(old - e < kExpLow ? kExpLow : old - e);
        for (int j = r; j < first; j += per)
          if (in_row) {
            u32x2* at = reinterpret_cast<u32x2*>(to + (place - first + j) * row_b);
            *at = lowered<F>(*at, down);
          }
      } else {
        e = old;
      }
    }
    if (lane == 0) exps[of] = (int8_t)e;
    const float up = power_of_two(-e);
    for (int j0 = 0; j0 < n; j0 += kHeld * per)
#pragma unroll
      for (int u = 0; u < kHeld; ++u) {
        const int j = j0 + u * per + r;
        if (!in_row || j >= n) continue;
        if (n > kHeld * per) load8(xt + j * ld, held[u]);
        float y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = held[u][k] * up;
        *reinterpret_cast<u32x2*>(to + (place + j) * row_b) = u32x2{F::bytes(y), F::bytes(y + 4)};
      }
  }
}

// A wave takes one head of a layer's K or V of one sequence, block after block of
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

int store_chunk(int32_t T) { return T <= 1024 ? 8 : 32; }

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
  const dim3 grid((unsigned)ceil_div(p.T, p.chunk), (unsigned)(2 * p.hk));
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
  if (format == LORA_CACHE_E4M3)
    hipLaunchKernelGGL(keep_quantized_kernel<E4m3>, grid, dim3(kThreads), 0, stream, p);
  else
    hipLaunchKernelGGL(keep_quantized_kernel<Int8>, grid, dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace lora
